// Gradients of the vocabulary-row operators: a row in blocks_per_row chunks, a
// CTA each, one exponential per element against the row's saved statistics.
//
// Where the gradient's row lies as x's does within 32 bytes (always when both are
// whole tensors, or one is the other) a thread handles 64-byte groups, two in flight;
// otherwise element by element. The few single entries (the token, the slots'
// indices) are written a second time after the dense pass, by the same thread
// or behind a barrier. grad may be x itself: every element is read by the thread that writes it,
// and the single entries are read before the dense pass writes any.
#pragma once

#include "logits_common.cuh"

namespace argr {

constexpr int kGradMaxBlock = 256;

// A CTA's chunk of a row: f(y) gives the gradient of an element with log2 p = y.
// x and out may be the same memory. entry(lo, n): called before the elements
// [lo, lo + n) are written by this thread, then after(lo, n).
template <class Tag, class F, class B, class A>
__device__ __forceinline__ void grad_chunk(const typename Tag::raw* row, typename Tag::raw* out, int cols, int b,
                                           int nb, float m, float ls2, float scale2, F f, B before, A after) {
    using R = typename Tag::raw;
    constexpr int E = kGroupElems<Tag>;
    const int t = threadIdx.x, nt = blockDim.x;
    const Part<Tag> part(row, cols, b, nb);
    const int lo = part.align + part.first * E;
    const int begin = part.is_first ? 0 : lo, end = part.is_last ? cols : lo + part.count * E;
    const auto one = [&](int j) {
        before(j, 1);
        out[j] = narrow_elem<Tag>(f((widen_elem<Tag>(row[j]) - m) * scale2 - ls2));
        after(j, 1);
    };
    if (((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 31u) != 0) {
        for (unsigned i = t; i < static_cast<unsigned>(end - begin); i += nt) one(begin + static_cast<int>(i));
        return;
    }
    const f32x2 minus = pack2(-m, -m), scale = pack2(scale2, scale2), shift = pack2(-ls2, -ls2);
    const auto group = [&](Group<Tag>& v, int g) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            float p, q;
            v.pair(i, p, q);
            unpack2(fma2(add2(pack2(p, q), minus), scale, shift), p, q);
            v.set_pair(i, f(p), f(q));
        }
        const int at = lo + g * E;
        before(at, E);
        v.store(out + at);
        after(at, E);
    };
    for (int g = t; g < part.count; g += 2 * nt) {
        Group<Tag> u, v;
        u.template load<false>(row + lo + static_cast<int64_t>(g) * E);
        const bool two = part.count - g > nt;
        if (two) v.template load<false>(row + lo + static_cast<int64_t>(g + nt) * E);
        group(u, g);
        if (two) group(v, g + nt);
    }
    if (t < lo - begin) one(begin + t);
    if (t < end - (lo + part.count * E)) one(lo + part.count * E + t);
}

template <class Tag, bool ENT>
__global__ void __launch_bounds__(kGradMaxBlock, 4) logprobs_grad_kernel(const LogitsProblem pr, float scale2) {
    using R = typename Tag::raw;
    grid_dependency_wait();
    allow_dependents();
    const float inv_t = 1.0f / pr.temperature;
    for (int64_t r = blockIdx.y; r < pr.rows; r += gridDim.y) {
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        R* out = static_cast<R*>(pr.grad) + r * pr.grad_stride;
        const float4 st = pr.stats[r];
        const int64_t tok = pr.grad_logprob ? pr.tokens[r] : -1;
        float g = tok >= 0 ? pr.grad_logprob[r] : 0.0f;
        if (tok >= pr.cols) g = quiet_nan();
        const float h = ENT ? pr.grad_entropy[r] : 0.0f;
        const float c = pr.grad_lse ? pr.grad_lse[r] : 0.0f;
        const bool empty = st.x == neg_inf();
        const float a = empty ? 0.0f : (c - g - h * st.z) * inv_t, b = empty ? 0.0f : -h * kLn2 * inv_t;
        const float m = empty ? 0.0f : st.x, ls2 = empty ? 0.0f : st.y * kLog2E;
        const int at = tok >= 0 && tok < pr.cols && !empty ? static_cast<int>(tok) : -1;
        const auto f = [&](float y) {
            if constexpr (ENT) {
                y = max_nan(y, kYMin);
                return ex2(y) * (a + b * y);
            } else {
                return ex2(y) * a;
            }
        };
        float x_at = 0.0f;
        grad_chunk<Tag>(
            row, out, pr.cols, blockIdx.x, gridDim.x, m, ls2, scale2, f,
            [&](int lo, int n) {
                if (at >= lo && at - lo < n) x_at = widen_elem<Tag>(row[at]);
            },
            [&](int lo, int n) {
                if (at >= lo && at - lo < n)
                    out[at] = narrow_elem<Tag>(f((x_at - m) * scale2 - ls2) + g * inv_t);
            });
    }
}

template <class Tag>
__global__ void __launch_bounds__(kGradMaxBlock, 4) distill_grad_kernel(const LogitsProblem pr, float scale2) {
    using R = typename Tag::raw;
    __shared__ Slots sl;
    grid_dependency_wait();
    allow_dependents();
    const int t = threadIdx.x;
    for (int64_t r = blockIdx.y; r < pr.rows; r += gridDim.y) {
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        R* out = static_cast<R*>(pr.grad) + r * pr.grad_stride;
        const Part<Tag> part(row, pr.cols, blockIdx.x, gridDim.x);
        const int lo = part.is_first ? 0 : part.align + part.first * kGroupElems<Tag>;
        const int hi = part.is_last ? pr.cols : part.align + (part.first + part.count) * kGroupElems<Tag>;
        load_slots<Tag>(pr, r, row, lo, hi, sl);
        const float4 st = pr.stats[r];
        const Teacher q = teacher_of(pr, sl);  // its barriers order the reads above before the stores below
        const float rest = st.z > neg_inf() ? q.rest : 0.0f;
        float g = pr.grad_logprob[r] / pr.temperature;
        if (q.bad || (st.y != st.y && q.any)) g = quiet_nan();
        const bool none = st.x == neg_inf() || !q.any;  // nothing is taught, or nothing can be
        const float total = q.total + rest;
        float dense = g * (rest > 0.0f ? total - rest * expf(st.y - st.z) : total);
        if (none) dense = q.bad ? g : 0.0f;
        const float m = none ? 0.0f : st.x, ls2 = none ? 0.0f : st.y * kLog2E;
        const auto nothing = [](int, int) {};
        if (none) {
            const R fill = narrow_elem<Tag>(dense);
            for (unsigned i = t; i < static_cast<unsigned>(hi - lo); i += blockDim.x) out[lo + i] = fill;
        } else {
            grad_chunk<Tag>(row, out, pr.cols, blockIdx.x, gridDim.x, m, ls2, scale2,
                            [&](float y) { return dense * ex2(y); }, nothing, nothing);
            __syncthreads();
            for (int i = t; i < pr.slots; i += blockDim.x) {
                const int j = sl.id[i];
                if (j >= lo && j < hi)
                    out[j] = narrow_elem<Tag>(g * (total * ex2((sl.x[i] - m) * scale2 - ls2) - expf(sl.v[i] - q.shift)));
            }
        }
        __syncthreads();
    }
}

}  // namespace argr
