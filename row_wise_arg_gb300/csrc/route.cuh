// A router's choice: for each row of expert logits the k largest, their weights,
// the row's log-sum-exp, how many rows chose each expert and the balance loss, and
// the gradient of weights, log-sum-exp and loss.
//
// With m = max x, s = sum exp(x - m), p = exp(x - m) / s, N rows that take part, counts_e
// choices of expert e:
//     weights = exp(x_i - m) / (s, or the sum over the chosen ones),
//     balance = E sum_e counts_e / (k N) * (sum over rows of p_e) / N,
// and with c_e = g_balance E counts_e / (k N^2), g the weights' gradients, h the log-sum-exp's
//     dx_e = p_e (c_e - sum_j c_j p_j + h [- sum_i g_i w_i where not normalised])
//            + [e is chosen i] w_i (g_i [- sum_j g_j w_j where normalised]).
//
// A warp per row, its elements in registers; warps go over the rows in turns and keep
// the sums of p of their elements in registers. A CTA leaves its sums and
// counts in scratch, a second kernel joins them in a fixed order: no atomics between CTAs.
#pragma once

#include "logits_common.cuh"
#include "select.h"

namespace argr {

// order32() of an element that can be chosen, 0 for -inf, NaN and what is past the row.
__device__ __forceinline__ unsigned choice_key(float x) { return x > neg_inf() ? order32(x) : 0u; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <class Tag, int NV>
__global__ void __launch_bounds__(kRouteBlock) route_kernel(const RouteProblem pr) {
    using R = typename Tag::raw;
    extern __shared__ __align__(16) unsigned char dyn[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kRouteBlock / 32;
    const int E = pr.experts, k = pr.k;
    int* hist = reinterpret_cast<int*>(dyn);  // [E + 1]
    float* acc = reinterpret_cast<float*>(hist + E + 1);  // [warps][E]
    if (pr.counts)
        for (int i = threadIdx.x; i <= E; i += kRouteBlock) hist[i] = 0;
    float sum_p[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) sum_p[j] = 0.0f;
    allow_dependents();
    grid_dependency_wait();
    __syncthreads();
    int taken = 0;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * warps + warp; r < pr.rows;
         r += static_cast<int64_t>(gridDim.x) * warps) {
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        const bool valid = !pr.valid || pr.valid[r];
        float x[NV];
        float m = neg_inf();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = lane + 32 * j;
            x[j] = valid && e < E ? widen_elem<Tag>(ld_scalar(row + e)) : neg_inf();
            m = fmaxf(m, x[j]);
        }
        m = order_value(__reduce_max_sync(0xffffffffu, order32(m)));
        const float ref = m == neg_inf() ? 0.0f : m;
        float p[NV], s = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            p[j] = ex2((x[j] - ref) * kLog2E);
            s += p[j];
        }
        s = warp_sum(s);
        const bool live = s != 0.0f;  // (a NaN is live)
        // the choices: lane i keeps the i-th
        unsigned key[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = choice_key(x[j]);
        int my_id = -1;
        float my_x = neg_inf();
        for (int i = 0; i < k; ++i) {
            unsigned best = 0;
            int at = 0;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (key[j] > best) {
                    best = key[j];
                    at = j;
                }
            const unsigned top = __reduce_max_sync(0xffffffffu, best);
            if (top == 0u) break;
            const unsigned e = __reduce_min_sync(0xffffffffu, best == top ? static_cast<unsigned>(lane + 32 * at) : ~0u);
            if (lane == i) {
                my_id = static_cast<int>(e);
                my_x = order_value(top);
            }
            if (lane == static_cast<int>(e & 31u)) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (j == static_cast<int>(e >> 5)) key[j] = 0u;
            }
        }
        float w = my_id >= 0 ? ex2((my_x - ref) * kLog2E) : 0.0f;
        float of = s;
        if (pr.normalize) of = warp_sum(w);
        if (live) w = s != s ? quiet_nan() : w / of;
        if (lane < k) {
            pr.weights[r * k + lane] = w;
            pr.ids[r * k + lane] = my_id;
        }
        if (lane == 0 && pr.lse) pr.lse[r] = live ? m + logf(s) : neg_inf();
        if (pr.counts && live) {
            ++taken;
            if (my_id >= 0) atomicAdd(&hist[my_id], 1);
            if (pr.balance) {
                const float inv = 1.0f / s;
#pragma unroll
                for (int j = 0; j < NV; ++j) sum_p[j] += p[j] * inv;
            }
        }
    }
    if (!pr.counts) return;
    if (lane == 0 && taken) atomicAdd(&hist[E], taken);
    if (pr.balance) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (lane + 32 * j < E) acc[warp * E + lane + 32 * j] = sum_p[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= E; i += kRouteBlock) {
        pr.part_counts[static_cast<int64_t>(blockIdx.x) * (E + 1) + i] = hist[i];
        if (pr.balance && i < E) {
            float v = 0.0f;
            for (int q = 0; q < warps; ++q) v += acc[q * E + i];
            pr.part_sums[static_cast<int64_t>(blockIdx.x) * E + i] = v;
        }
    }
}

template <class Tag, int NV>
__global__ void __launch_bounds__(kRouteBlock) route_grad_kernel(const RouteProblem pr) {
    using R = typename Tag::raw;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kRouteBlock / 32;
    const int E = pr.experts, k = pr.k;
    allow_dependents();
    grid_dependency_wait();
    float c[NV];
    {
        float per = 0.0f;
        if (pr.grad_balance) {
            const int64_t taken = *pr.taken;
            const float n = static_cast<float>(taken > 0 ? taken : 1);
            per = *pr.grad_balance * (static_cast<float>(E) / (static_cast<float>(k) * n)) / n;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = lane + 32 * j;
            c[j] = pr.grad_balance && e < E ? per * static_cast<float>(pr.counts[e]) : 0.0f;
        }
    }
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * warps + warp; r < pr.rows;
         r += static_cast<int64_t>(gridDim.x) * warps) {
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        R* out = static_cast<R*>(pr.grad) + r * pr.grad_stride;
        const float lse = pr.lse[r];
        if (lse == neg_inf()) {  // (alike in every lane) padding, or nothing above -inf: not read
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (lane + 32 * j < E) out[lane + 32 * j] = narrow_elem<Tag>(0.0f);
            continue;
        }
        float p[NV], dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = lane + 32 * j;
            p[j] = e < E ? ex2((widen_elem<Tag>(row[e]) - lse) * kLog2E) : 0.0f;
            dot += p[j] * c[j];
        }
        const float h = pr.grad_lse ? pr.grad_lse[r] : 0.0f;
        int id = -1;
        float g = 0.0f, w = 0.0f;
        if (lane < k && pr.grad_weights) {
            const int64_t e = pr.ids[r * k + lane];
            id = e >= 0 && e < E ? static_cast<int>(e) : -1;
            if (id >= 0) {
                g = pr.grad_weights[r * k + lane];
                w = pr.weights[r * k + lane];
            }
        }
        dot = warp_sum(dot);
        const float along = warp_sum(g * w);
        const float rest = h - dot - (pr.normalize ? 0.0f : along);
        const float at_id = w * (pr.normalize ? g - along : g);
        float d[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) d[j] = p[j] * (c[j] + rest);
        if (pr.grad_weights) {
            for (int i = 0; i < k; ++i) {
                const int e = __shfl_sync(0xffffffffu, id, i);
                const float v = __shfl_sync(0xffffffffu, at_id, i);
                if (e >= 0 && lane == (e & 31)) {
#pragma unroll
                    for (int j = 0; j < NV; ++j)
                        if (j == (e >> 5)) d[j] += v;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (lane + 32 * j < E) out[lane + 32 * j] = narrow_elem<Tag>(d[j]);
    }
}

template <class Tag, int NV>
cudaError_t launch_route_nv(const RouteProblem& pr) {
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    const size_t smem = 4 * (static_cast<size_t>(pr.experts) * (1 + kRouteBlock / 32) + 1);
    return launch_ex_smem(route_kernel<Tag, NV>, dim3(static_cast<unsigned>(pr.ctas)), dim3(kRouteBlock), 1, smem, p,
                          pr.stream, pr);
}
template <class Tag, int NV>
cudaError_t launch_route_grad_nv(const RouteProblem& pr) {
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    return launch_ex_smem(route_grad_kernel<Tag, NV>, dim3(static_cast<unsigned>(pr.ctas)), dim3(kRouteBlock), 1, 0, p,
                          pr.stream, pr);
}

#define ARGR_ROUTE_NV(fn, Tag, pr)               \
    ((pr).experts <= 32    ? fn<Tag, 1>(pr)      \
     : (pr).experts <= 64  ? fn<Tag, 2>(pr)      \
     : (pr).experts <= 128 ? fn<Tag, 4>(pr)      \
     : (pr).experts <= 256 ? fn<Tag, 8>(pr)      \
     : (pr).experts <= 512 ? fn<Tag, 16>(pr)     \
                           : fn<Tag, 32>(pr))

template <class Tag>
cudaError_t launch_route_t(const RouteProblem& pr, const argr_caps&) {
    const cudaError_t e = ARGR_ROUTE_NV(launch_route_nv, Tag, pr);
    return e == cudaSuccess && pr.counts ? launch_route_finish(pr) : e;
}
template <class Tag>
cudaError_t launch_route_grad_t(const RouteProblem& pr, const argr_caps&) {
    return ARGR_ROUTE_NV(launch_route_grad_nv, Tag, pr);
}

#define ARGR_DEFINE_SELECT(sfx, Tag)                                                          \
    namespace argr {                                                                          \
    cudaError_t launch_beam_select_##sfx(const BeamProblem& pr, const argr_caps& caps) {      \
        return launch_beam_select_t<Tag>(pr, caps);                                           \
    }                                                                                         \
    cudaError_t launch_route_##sfx(const RouteProblem& pr, const argr_caps& caps) {           \
        return launch_route_t<Tag>(pr, caps);                                                 \
    }                                                                                         \
    cudaError_t launch_route_grad_##sfx(const RouteProblem& pr, const argr_caps& caps) {      \
        return launch_route_grad_t<Tag>(pr, caps);                                            \
    }                                                                                         \
    }

}  // namespace argr
