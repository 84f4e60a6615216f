// Gradients of the vocabulary-row operators: a row in blocks_per_row chunks, a
// CTA each, one exponential per element against the row's saved statistics.
//
// Where the gradient's row lies as x's does within 32 bytes (always when both are
// whole tensors, or one is the other) a thread handles 64-byte groups, two in flight;
// otherwise words of the size that both allow. The few single entries (the token, the slots'
// indices) are written a second time after the dense pass, by the same thread
// or behind a barrier. grad may be x itself: every element is read by the thread that writes it,
// and the single entries are read before the dense pass writes any.
//
//   log probabilities: dx_j = ((g_lse - g_lp) p_j - g_H p_j (log p_j + H) + [j = token] g_lp) / T
//   distillation:      dx_j = g (w p_j - q_j) / T at a slot's index, g w p_j / T elsewhere, with a tail
//                      g (w p_rest - rest) (p_j / p_rest) / T there
//
// Bound by the memory: [2048, 202048] bf16 239 us, 6.9 TB/s read and written; [1024, 262144]
// bf16, 64 slots, 157 us, 6.9 TB/s; [1024, 100000] f32 121 us, 6.8 TB/s (a copy: 6.8). By words of 2 to 8
// bytes it is not: [1024, 50257] bf16, 64 slots and a tail, 39 us, with rows 50304 apart and the gradient's 50257 97 us.
#pragma once

#include "logits_common.cuh"

namespace argr {

constexpr int kGradMaxBlock = 256;

// Elements [begin, end) of a row whose gradient lies otherwise than x within 32
// bytes: words of W bytes, W the most that both allow, consecutive threads on
// consecutive words, kWords loads in flight.
constexpr int kWords = 4;
template <class Tag, int W, class F>
__device__ __forceinline__ void grad_words(const typename Tag::raw* row, typename Tag::raw* out, int begin, int end,
                                           float m, float ls2, float scale2, F f) {
    using R = typename Tag::raw;
    using Word = std::conditional_t<W == 8, uint2, std::conditional_t<W == 4, uint32_t, uint16_t>>;
    constexpr int N = W / static_cast<int>(sizeof(R));
    const int t = threadIdx.x, nt = blockDim.x;
    const auto one = [&](int j) { out[j] = narrow_elem<Tag>(f((widen_elem<Tag>(row[j]) - m) * scale2 - ls2)); };
    int head = static_cast<int>(((W - (reinterpret_cast<uintptr_t>(row + begin) & (W - 1))) & (W - 1)) / sizeof(R));
    if (head > end - begin) head = end - begin;
    const int words = (end - begin - head) / N, done = begin + head + words * N;
    const R* src = row + begin + head;
    R* dst = out + begin + head;
    for (int w0 = 0; w0 < words;) {
        Word v[kWords];
        const int left = words - w0;
#pragma unroll
        for (int u = 0; u < kWords; ++u)
            if (t + u * nt < left) v[u] = reinterpret_cast<const Word*>(src)[static_cast<int64_t>(w0) + t + u * nt];
#pragma unroll
        for (int u = 0; u < kWords; ++u) {
            if (t + u * nt >= left) continue;
            R* e = reinterpret_cast<R*>(&v[u]);
#pragma unroll
            for (int i = 0; i < N; ++i) e[i] = narrow_elem<Tag>(f((widen_elem<Tag>(e[i]) - m) * scale2 - ls2));
            reinterpret_cast<Word*>(dst)[static_cast<int64_t>(w0) + t + u * nt] = v[u];
        }
        if (left <= kWords * nt) break;
        w0 += kWords * nt;
    }
    if (t < head) one(begin + t);
    if (t < end - done) one(done + t);
}

// A CTA's chunk of a row: f(y) gives the gradient of an element with log2 p = y.
// x and out may be the same memory. before(lo, n) is called before the elements
// [lo, lo + n) are written by this thread, then after(lo, n); where x and out
// are not the same memory, they may be called by any thread, after a barrier, for the whole
// chunk instead.
template <class Tag, class F, class B, class A>
__device__ __forceinline__ void grad_chunk(const typename Tag::raw* row, typename Tag::raw* out, int cols, int b,
                                           int nb, float m, float ls2, float scale2, F f, B before, A after) {
    constexpr int E = kGroupElems<Tag>;
    const int t = threadIdx.x, nt = blockDim.x;
    const Part<Tag> part(row, cols, b, nb);
    const int lo = part.align + part.first * E;
    const int begin = part.begin(), end = part.end();
    const unsigned apart = static_cast<unsigned>((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 31u);
    if (apart != 0) {
        if ((apart & 7u) == 0) grad_words<Tag, 8>(row, out, begin, end, m, ls2, scale2, f);
        else if (sizeof(typename Tag::raw) == 4 || (apart & 3u) == 0) grad_words<Tag, 4>(row, out, begin, end, m, ls2, scale2, f);
        else if constexpr (sizeof(typename Tag::raw) == 2) grad_words<Tag, 2>(row, out, begin, end, m, ls2, scale2, f);
        __syncthreads();
        if (t == 0) {
            before(begin, end - begin);
            after(begin, end - begin);
        }
        return;
    }
    const auto one = [&](int j) {
        before(j, 1);
        out[j] = narrow_elem<Tag>(f((widen_elem<Tag>(row[j]) - m) * scale2 - ls2));
        after(j, 1);
    };
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
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ GradWeights weights;
    const Slots sl(dyn, pr.slots);
    grid_dependency_wait();
    allow_dependents();
    const int t = threadIdx.x;
    for (int64_t r = blockIdx.y; r < pr.rows; r += gridDim.y) {
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        R* out = static_cast<R*>(pr.grad) + r * pr.grad_stride;
        const Part<Tag> part(row, pr.cols, blockIdx.x, gridDim.x);
        const int lo = part.begin(), hi = part.end();
        load_slots<Tag>(pr, r, row, lo, hi, sl);
        // its barriers order the reads above before the stores below
        const Teacher q = teacher_of(pr, sl, [&](const Teacher& sums) {
            const float4 st = pr.stats[r];
            if (t == 0) weights = GradWeights(pr, sums, pr.grad_logprob[r], st.x, st.y, st.z, st.x, st.z);
        });
        const GradWeights w = weights;
        if (w.none) {
            const R fill = narrow_elem<Tag>(w.dense);
            for (unsigned i = t; i < static_cast<unsigned>(hi - lo); i += blockDim.x) out[lo + i] = fill;
        } else {
            const auto nothing = [](int, int) {};
            grad_chunk<Tag>(row, out, pr.cols, blockIdx.x, gridDim.x, w.dense_m, w.dense_ls2, scale2,
                            [&](float y) { return w.dense * ex2(y); }, nothing, nothing);
            __syncthreads();
            for (int i = t; i < pr.slots; i += blockDim.x) {
                const int j = sl.id[i];
                if (j >= lo && j < hi) out[j] = narrow_elem<Tag>(w.named(sl.x[i], teacher_log(pr, q, sl.v[i]), scale2));
            }
        }
        __syncthreads();
    }
}

}  // namespace argr
