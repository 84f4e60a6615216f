// Vocabulary-row kernels, templated on the element type: log probabilities
// with entropy and top alternatives, the distillation loss from a teacher's
// top logits, and the gradients of both.
//
// Softmax statistics of a set of elements are held as (m, s, t): m the largest
// element, s = sum exp((x - m) / T) and t = sum exp((x - m) / T) y with
// y = log2(exp((x - m) / T)). Two such triples join by moving both to the larger
// m, in a fixed order, so results repeat exactly. From the row's triple
//     ln s            gives log p_j = (x_j - m) / T - ln s,
//     entropy       = ln 2 (log2 s - t / s).
// Differences are taken before the scaling by 1 / T, so that rows at the lowest
// finite value do not overflow; y is held above kYMin, where exp2 is zero, so
// that an element of -inf adds 0 * kYMin = 0 to t. NaN passes through both.
#pragma once

#include <cuda_bf16.h>

#include <cfloat>

#include "kernels_impl.cuh"
#include "logits.h"

namespace argr {

constexpr float kYMin = -200.0f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2E = 1.44269504088896341f;

__device__ __forceinline__ float ex2(float y) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
    return e;
}
// max that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

__device__ __forceinline__ float widen(float v) { return v; }
template <class Tag>
__device__ __forceinline__ float widen_elem(typename Tag::raw v) {
    if constexpr (std::is_same<Tag, TagF32>::value) return v;
    else return Tag::widen(v);
}
template <class Tag>
__device__ __forceinline__ typename Tag::raw narrow_elem(float v) {
    if constexpr (std::is_same<Tag, TagF32>::value) return v;
    else if constexpr (std::is_same<Tag, TagF16>::value) return __half_as_ushort(__float2half_rn(v));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// ---------------------------------------------------------------------------
// Softmax statistics.
// ---------------------------------------------------------------------------
struct SoftSum {
    float m = -FLT_MAX;
    float s = 0.0f;
    float t = 0.0f;

    // Move the sums to another reference element.
    __device__ __forceinline__ void rebase(float to, float scale2) {
        const float y = max_nan((m - to) * scale2, kYMin);
        const float r = ex2(y);
        t = r * (t + y * s);
        s *= r;
        m = to;
    }
    __device__ __forceinline__ void add(float x, float scale2) {
        if (x > m) rebase(x, scale2);
        const float y = max_nan((x - m) * scale2, kYMin);
        const float e = ex2(y);
        s += e;
        t += e * y;
    }
    __device__ __forceinline__ void join(SoftSum o, float scale2) {
        const float to = fmaxf(m, o.m);
        rebase(to, scale2);
        o.rebase(to, scale2);
        s += o.s;
        t += o.t;
    }
    __device__ __forceinline__ bool empty() const { return s == 0.0f; }
};

// The CTA's triple, in every thread. `smem` holds 3 * 32 floats.
__device__ __forceinline__ SoftSum block_softsum(SoftSum c, float scale2, float* smem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        SoftSum d;
        d.m = __shfl_xor_sync(0xffffffffu, c.m, o);
        d.s = __shfl_xor_sync(0xffffffffu, c.s, o);
        d.t = __shfl_xor_sync(0xffffffffu, c.t, o);
        c.join(d, scale2);
    }
    __syncthreads();
    if (lane == 0) {
        smem[warp] = c.m;
        smem[32 + warp] = c.s;
        smem[64 + warp] = c.t;
    }
    __syncthreads();
    SoftSum r;
    for (int w = 0; w < nwarps; ++w) {
        SoftSum d;
        d.m = smem[w];
        d.s = smem[32 + w];
        d.t = smem[64 + w];
        r.join(d, scale2);
    }
    return r;
}

// Sum and maximum over the CTA, in every thread and in a fixed order. `smem`
// holds 32 values.
__device__ __forceinline__ float block_sum(float v, float* smem) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = 0.0f;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) r += smem[w];
    return r;
}
__device__ __forceinline__ float block_max(float v, float* smem) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = neg_inf();
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) r = fmaxf(r, smem[w]);
    return r;
}

// ---------------------------------------------------------------------------
// Order of the alternatives: larger values first, equal ones (both zeros are
// equal) by index, NaNs after every number. A key is larger for an earlier
// alternative; 0 is below every key of an element.
// ---------------------------------------------------------------------------
__device__ __forceinline__ unsigned order32(float v) {
    const unsigned b = __float_as_uint(v + 0.0f);
    const unsigned u = b ^ (static_cast<unsigned>(static_cast<int>(b) >> 31) | 0x80000000u);
    return v != v ? 0u : u;
}
__device__ __forceinline__ unsigned long long order_key(float v, int index) {
    return static_cast<unsigned long long>(order32(v)) << 32 | (0xffffffffu - static_cast<unsigned>(index));
}
__device__ __forceinline__ int key_index(unsigned long long k) {
    return static_cast<int>(0xffffffffu - static_cast<unsigned>(k));
}

// The CTA's largest key, in every thread. `smem` holds 32 keys.
__device__ __forceinline__ unsigned long long block_max_key(unsigned long long k, unsigned long long* smem) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const unsigned long long d = __shfl_xor_sync(0xffffffffu, k, o);
        k = d > k ? d : k;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = k;
    __syncthreads();
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) k = smem[w] > k ? smem[w] : k;
    return k;
}

constexpr int kRun = 2048;

// ---------------------------------------------------------------------------
// Log probabilities: a CTA per row.
// ---------------------------------------------------------------------------
template <class Tag>
__global__ void __launch_bounds__(512) logprobs_kernel(const LogitsProblem pr, float scale2) {
    using R = typename Tag::raw;
    __shared__ float red[96];
    __shared__ unsigned long long kred[32];
    grid_dependency_wait();
    allow_dependents();
    const int t = threadIdx.x;
    for (int64_t r = blockIdx.x; r < pr.rows; r += gridDim.x) {
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        SoftSum c;  // joined from runs of at most kRun elements, so that long rows' sums keep their digits
        for (int64_t j = t; j < pr.cols;) {
            SoftSum d;
            for (int n = 0; n < kRun && j < pr.cols; ++n, j += blockDim.x) d.add(widen_elem<Tag>(row[j]), scale2);
            c.join(d, scale2);
        }
        c = block_softsum(c, scale2, red);
        const float ln_s = c.empty() ? neg_inf() : logf(c.s);
        if (t == 0) {
            const float h = kLn2 * (log2f(c.s) - c.t / c.s);
            const float entropy = c.empty() ? 0.0f : (h < 0.0f ? 0.0f : h);
            if (pr.logprob) {
                const int64_t tok = pr.tokens[r];
                float lp = 0.0f;
                if (tok >= pr.cols) lp = quiet_nan();
                else if (tok >= 0)
                    lp = c.empty() ? neg_inf() : (widen_elem<Tag>(row[tok]) - c.m) / pr.temperature - ln_s;
                pr.logprob[r] = lp;
            }
            if (pr.entropy) pr.entropy[r] = entropy;
            if (pr.lse) pr.lse[r] = c.empty() ? neg_inf() : c.m / pr.temperature + ln_s;
            if (pr.stats) pr.stats[r] = make_float4(c.empty() ? neg_inf() : c.m, ln_s, entropy, 0.0f);
        }
        unsigned long long last = ~0ull;
        for (int i = 0; i < pr.top_k; ++i) {
            unsigned long long best = 0;
            for (int64_t j = t; j < pr.cols; j += blockDim.x) {
                const unsigned long long k = order_key(widen_elem<Tag>(row[j]), static_cast<int>(j));
                if (k < last && k > best) best = k;
            }
            last = block_max_key(best, kred);
            if (t == 0) {
                const int id = key_index(last);
                const float lp = c.empty() ? neg_inf() : (widen_elem<Tag>(row[id]) - c.m) / pr.temperature - ln_s;
                if (pr.top_ids) pr.top_ids[r * pr.top_k + i] = id;
                if (pr.top_logprobs) pr.top_logprobs[r * pr.top_k + i] = lp;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The teacher's side of a row. A filled slot has 0 <= id < cols.
// ---------------------------------------------------------------------------
struct Teacher {
    float shift;  // ln q = v - shift (v = teacher / T without the tail, teacher with it)
    float total;  // sum of q over the filled slots
    float rest;   // what the tail holds
    bool any;     // a slot holds something
    bool bad;     // a slot names an index past the row
    float inv_t;

    __device__ __forceinline__ float lnq(float teacher) const { return teacher * inv_t - shift; }
};

__device__ __forceinline__ Teacher read_teacher(const LogitsProblem& pr, int64_t r, float* red) {
    const int64_t* ids = pr.ids + r * pr.slots;
    const float* val = pr.teacher + r * pr.slots;
    Teacher q;
    q.inv_t = pr.tail ? 1.0f : 1.0f / pr.temperature;
    q.shift = 0.0f;
    bool any = false, bad = false;
    float top = -FLT_MAX;
    for (int i = threadIdx.x; i < pr.slots; i += blockDim.x) {
        const int64_t id = ids[i];
        any = any || (id >= 0 && (pr.tail || val[i] != neg_inf()));
        bad = bad || id >= pr.cols;
        if (id >= 0) top = fmaxf(top, val[i] * q.inv_t);
    }
    q.any = __syncthreads_or(any);
    q.bad = __syncthreads_or(bad);
    if (!pr.tail) q.shift = block_max(top, red);
    float sum = 0.0f;
    for (int i = threadIdx.x; i < pr.slots; i += blockDim.x)
        if (ids[i] >= 0) sum += expf(q.lnq(val[i]));
    sum = block_sum(sum, red);
    if (pr.tail) {
        q.total = sum;
        q.rest = q.any ? fmaxf(0.0f, 1.0f - sum) : 0.0f;
    } else {
        q.shift = q.any ? q.shift + logf(sum) : 0.0f;
        q.total = q.any ? 1.0f : 0.0f;
        q.rest = 0.0f;
    }
    return q;
}

// Elements of a segment of the row that slots name, as a bit map.
constexpr int kSegElems = 1 << 18;

template <class Tag>
__global__ void __launch_bounds__(512) distill_kernel(const LogitsProblem pr, float scale2) {
    using R = typename Tag::raw;
    __shared__ float red[96];
    __shared__ unsigned named[kSegElems / 32];
    grid_dependency_wait();
    allow_dependents();
    const int t = threadIdx.x;
    for (int64_t r = blockIdx.x; r < pr.rows; r += gridDim.x) {
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        const int64_t* ids = pr.ids + r * pr.slots;
        const float* val = pr.teacher + r * pr.slots;
        const Teacher q = read_teacher(pr, r, red);
        SoftSum c;  // without the tail: the row; with it: the indices that no slot names
        for (int64_t lo = 0; lo < pr.cols; lo += kSegElems) {
            const int64_t hi = pr.cols - lo > kSegElems ? lo + kSegElems : pr.cols;
            if (pr.tail) {
                __syncthreads();
                for (int i = t; i < kSegElems / 32; i += blockDim.x) named[i] = 0u;
                __syncthreads();
                for (int i = t; i < pr.slots; i += blockDim.x) {
                    const int64_t id = ids[i];
                    if (id >= lo && id < hi) atomicOr(&named[(id - lo) >> 5], 1u << ((id - lo) & 31));
                }
                __syncthreads();
            }
            SoftSum d;
            for (int64_t j = lo + t; j < hi; j += blockDim.x) {
                const int o = static_cast<int>(j - lo);
                if (!pr.tail || !(named[o >> 5] >> (o & 31) & 1u)) d.add(widen_elem<Tag>(row[j]), scale2);
            }
            c.join(d, scale2);
        }
        c = block_softsum(c, scale2, red);
        SoftSum all = c;
        if (pr.tail) {
            SoftSum d;
            for (int i = t; i < pr.slots; i += blockDim.x) {
                const int64_t id = ids[i];
                if (id >= 0 && id < pr.cols) d.add(widen_elem<Tag>(row[id]), scale2);
            }
            all.join(block_softsum(d, scale2, red), scale2);
            c.rebase(all.m, scale2);
        }
        const float ln_s = all.empty() ? neg_inf() : logf(all.s);
        const float ln_rest = c.empty() ? neg_inf() : logf(c.s);
        float loss = 0.0f;
        for (int i = t; i < pr.slots; i += blockDim.x) {
            const int64_t id = ids[i];
            if (id < 0 || id >= pr.cols) continue;
            const float lnq = q.lnq(val[i]);
            const float p = expf(lnq);
            const float lp = all.empty() ? neg_inf() : (widen_elem<Tag>(row[id]) - all.m) / pr.temperature - ln_s;
            if (!(p == 0.0f)) loss += p * (lnq - lp);
        }
        loss = block_sum(loss, red);
        if (t == 0) {
            if (q.rest > 0.0f && !c.empty()) loss += q.rest * (logf(q.rest) - (ln_rest - ln_s));
            if (all.s != all.s && q.any) loss = quiet_nan();
            if (q.bad) loss = quiet_nan();
            if (pr.loss) pr.loss[r] = loss;
            if (pr.stats) pr.stats[r] = make_float4(all.empty() ? neg_inf() : all.m, ln_s, ln_rest, 0.0f);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Gradients: a row in blocks_per_row chunks, a CTA each. grad may be x itself:
// every element is read by the thread that writes it, and the single entries
// (the token, the slots) are read by all before any is written.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void chunk_of(int cols, int nb, int b, int64_t* lo, int64_t* hi) {
    const int64_t n = (static_cast<int64_t>(cols) + nb - 1) / nb;
    *lo = n * b < cols ? n * b : cols;
    *hi = *lo + n < cols ? *lo + n : cols;
}

template <class Tag>
__global__ void __launch_bounds__(512) logprobs_grad_kernel(const LogitsProblem pr, float scale2) {
    using R = typename Tag::raw;
    grid_dependency_wait();
    allow_dependents();
    int64_t lo, hi;
    chunk_of(pr.cols, gridDim.x, blockIdx.x, &lo, &hi);
    const float inv_t = 1.0f / pr.temperature;
    for (int64_t r = blockIdx.y; r < pr.rows; r += gridDim.y) {
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        R* out = static_cast<R*>(pr.grad) + r * pr.grad_stride;
        const float4 st = pr.stats[r];
        const int64_t tok = pr.tokens ? pr.tokens[r] : -1;
        float g = pr.grad_logprob && tok >= 0 ? pr.grad_logprob[r] : 0.0f;
        if (tok >= pr.cols && pr.grad_logprob) g = quiet_nan();
        const float h = pr.grad_entropy ? pr.grad_entropy[r] : 0.0f;
        const float c = pr.grad_lse ? pr.grad_lse[r] : 0.0f;
        const float a = (c - g - h * st.z) * inv_t, b = -h * kLn2 * inv_t;
        const float ls2 = st.y * kLog2E;
        const bool empty = st.x == neg_inf();
        for (int64_t j = lo + threadIdx.x; j < hi; j += blockDim.x) {
            const float y = max_nan((widen_elem<Tag>(row[j]) - st.x) * scale2 - ls2, kYMin);
            float d = ex2(y) * (a + b * y);
            if (j == tok) d += g * inv_t;
            out[j] = narrow_elem<Tag>(empty ? 0.0f : d);
        }
    }
}

template <class Tag>
__global__ void __launch_bounds__(512) distill_grad_kernel(const LogitsProblem pr, float scale2) {
    using R = typename Tag::raw;
    __shared__ float red[32];
    __shared__ float named_x[ARGR_LOGITS_MAX_SLOTS];
    grid_dependency_wait();
    allow_dependents();
    int64_t lo, hi;
    chunk_of(pr.cols, gridDim.x, blockIdx.x, &lo, &hi);
    const int t = threadIdx.x;
    for (int64_t r = blockIdx.y; r < pr.rows; r += gridDim.y) {
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        R* out = static_cast<R*>(pr.grad) + r * pr.grad_stride;
        const int64_t* ids = pr.ids + r * pr.slots;
        const float* val = pr.teacher + r * pr.slots;
        const float4 st = pr.stats[r];
        for (int i = t; i < pr.slots; i += blockDim.x)
            if (ids[i] >= lo && ids[i] < hi) named_x[i] = widen_elem<Tag>(row[ids[i]]);
        const Teacher q = read_teacher(pr, r, red);  // its barriers order the reads above before the stores below
        __syncthreads();
        const float rest = st.z > neg_inf() ? q.rest : 0.0f;
        float g = pr.grad_logprob[r] / pr.temperature;
        if (q.bad || (st.y != st.y && q.any)) g = quiet_nan();
        const float ls2 = st.y * kLog2E;
        const float total = q.total + rest;
        const float dense = g * (rest > 0.0f ? total - rest * expf(st.y - st.z) : total);
        const bool none = st.x == neg_inf() || !q.any;
        for (int64_t j = lo + t; j < hi; j += blockDim.x) {
            const float y = (widen_elem<Tag>(row[j]) - st.x) * scale2 - ls2;
            out[j] = narrow_elem<Tag>(none ? (q.bad ? g : 0.0f) : dense * ex2(y));
        }
        __syncthreads();
        for (int i = t; i < pr.slots; i += blockDim.x)
            if (ids[i] >= lo && ids[i] < hi && !none)
                out[ids[i]] = narrow_elem<Tag>(
                    g * (total * ex2((named_x[i] - st.x) * scale2 - ls2) - expf(q.lnq(val[i]))));
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Launchers.
// ---------------------------------------------------------------------------
inline float scale2_of(const LogitsProblem& pr) { return kLog2E / pr.temperature; }

template <class Tag>
cudaError_t launch_logprobs_t(const argr_plan& p, const LogitsProblem& pr) {
    return launch_ex(logprobs_kernel<Tag>, dim3(static_cast<unsigned>(p.grid_rows)), dim3(p.block), 1, p, pr.stream,
                     pr, scale2_of(pr));
}
template <class Tag>
cudaError_t launch_distill_t(const argr_plan& p, const LogitsProblem& pr) {
    return launch_ex(distill_kernel<Tag>, dim3(static_cast<unsigned>(p.grid_rows)), dim3(p.block), 1, p, pr.stream,
                     pr, scale2_of(pr));
}
inline dim3 grad_grid(const argr_plan& p) {
    return dim3(static_cast<unsigned>(p.blocks_per_row), static_cast<unsigned>(p.grid_rows < 65535 ? p.grid_rows : 65535));
}
template <class Tag>
cudaError_t launch_logprobs_grad_t(const argr_plan& p, const LogitsProblem& pr) {
    return launch_ex(logprobs_grad_kernel<Tag>, grad_grid(p), dim3(p.block), 1, p, pr.stream, pr, scale2_of(pr));
}
template <class Tag>
cudaError_t launch_distill_grad_t(const argr_plan& p, const LogitsProblem& pr) {
    return launch_ex(distill_grad_kernel<Tag>, grad_grid(p), dim3(p.block), 1, p, pr.stream, pr, scale2_of(pr));
}

#define ARGR_DEFINE_LOGITS(sfx, Tag)                                                                                 \
    namespace argr {                                                                                                 \
    cudaError_t launch_logprobs_##sfx(const argr_plan& p, const LogitsProblem& pr) {                                 \
        return launch_logprobs_t<Tag>(p, pr);                                                                        \
    }                                                                                                                \
    cudaError_t launch_distill_##sfx(const argr_plan& p, const LogitsProblem& pr) {                                  \
        return launch_distill_t<Tag>(p, pr);                                                                         \
    }                                                                                                                \
    cudaError_t launch_logprobs_grad_##sfx(const argr_plan& p, const LogitsProblem& pr) {                            \
        return launch_logprobs_grad_t<Tag>(p, pr);                                                                   \
    }                                                                                                                \
    cudaError_t launch_distill_grad_##sfx(const argr_plan& p, const LogitsProblem& pr) {                             \
        return launch_distill_grad_t<Tag>(p, pr);                                                                    \
    }                                                                                                                \
    }

}  // namespace argr
