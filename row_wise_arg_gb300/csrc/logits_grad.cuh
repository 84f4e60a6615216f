// Gradients of the vocabulary-row operators.
#pragma once

#include "logits_common.cuh"

namespace argr {

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

}  // namespace argr
