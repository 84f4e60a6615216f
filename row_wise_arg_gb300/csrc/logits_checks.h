// Argument checks that the entry points over rows of logits share.
#pragma once

#include <climits>
#include <cmath>

#include "logits.h"

namespace argr {

inline bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// Bytes from the first to past the last element of `rows` rows of cols
// elements, stride apart; false when that does not fit 63 bits.
inline bool extent(int64_t rows, int64_t cols, int64_t stride, int64_t es, int64_t* bytes) {
    const int64_t most = INT64_MAX / es - cols;
    if (rows > 1 && stride > most / (rows - 1)) return false;
    *bytes = ((rows - 1) * stride + cols) * es;
    return true;
}

inline argr_status check_rows(const void* x, int dtype, int64_t rows, int64_t cols, int64_t row_stride, float temperature) {
    if (dtype == ARGR_F64 || dtype == ARGR_I32 || dtype == ARGR_I64) return ARGR_EUNSUPPORTED;
    if (dtype != ARGR_F32 && dtype != ARGR_F16 && dtype != ARGR_BF16) return ARGR_EINVAL;
    if (rows < 0 || cols < 1 || cols > INT_MAX || row_stride < 0) return ARGR_EINVAL;
    // the kernels scale by log2(e) / T
    if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(1.44269504f / temperature)) return ARGR_EINVAL;
    if (rows == 0) return ARGR_OK;
    int64_t bytes;
    if (!extent(rows, cols, row_stride, elem_size(dtype), &bytes)) return ARGR_EINVAL;
    if (!x || misaligned(x, static_cast<uintptr_t>(elem_size(dtype)))) return ARGR_EINVAL;
    return ARGR_OK;
}

// The gradient is x itself or does not touch it.
inline argr_status check_grad(const void* x, int dtype, int64_t rows, int64_t cols, int64_t row_stride, const void* grad,
                       int64_t grad_stride) {
    const int64_t es = elem_size(dtype);
    int64_t nx, ng;
    if (!grad || misaligned(grad, static_cast<uintptr_t>(es))) return ARGR_EINVAL;
    if (grad_stride < 0 || (rows > 1 && grad_stride < cols)) return ARGR_EINVAL;
    if (!extent(rows, cols, row_stride, es, &nx) || !extent(rows, cols, grad_stride, es, &ng)) return ARGR_EINVAL;
    if (grad == x && (rows == 1 || grad_stride == row_stride)) return ARGR_OK;
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), g = reinterpret_cast<uintptr_t>(grad);
    return a < g + static_cast<uintptr_t>(ng) && g < a + static_cast<uintptr_t>(nx) ? ARGR_EINVAL : ARGR_OK;
}

inline argr_status launched(cudaError_t e) {
    if (e == cudaSuccess) return ARGR_OK;
    cudaGetLastError();  // clear a non-sticky launch error
    return e == cudaErrorInvalidClusterSize ? ARGR_EUNSUPPORTED : ARGR_ECUDA;
}

}  // namespace argr
