// Building blocks of the vocabulary-row kernels: softmax statistics, the order
// of alternatives, CTA-wide reductions, packed arithmetic and the teacher's side
// of a distillation row.
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

// The warp's triple, in every lane: one common reference, then plain sums.
__device__ __forceinline__ SoftSum warp_softsum(SoftSum c, float scale2) {
    float to = c.m;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
    c.rebase(to, scale2);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        c.s += __shfl_xor_sync(0xffffffffu, c.s, o);
        c.t += __shfl_xor_sync(0xffffffffu, c.t, o);
    }
    return c;
}

// The CTA's triple, in every thread of warp 0. `smem` holds 3 * 32 floats.
// Contains __syncthreads().
__device__ __forceinline__ SoftSum block_softsum(SoftSum c, float scale2, float* smem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    c = warp_softsum(c, scale2);
    __syncthreads();
    if (lane == 0) {
        smem[warp] = c.m;
        smem[32 + warp] = c.s;
        smem[64 + warp] = c.t;
    }
    __syncthreads();
    if (warp != 0) return c;
    SoftSum r;
    if (lane < nwarps) {
        r.m = smem[lane];
        r.s = smem[32 + lane];
        r.t = smem[64 + lane];
    }
    return warp_softsum(r, scale2);
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
// equal) by index, NaNs after every number. order32() is larger for an earlier
// value, at least 1; a key adds the index and is larger for an earlier
// alternative. order_value() undoes order32() (a zero comes back as +0).
// ---------------------------------------------------------------------------
__device__ __forceinline__ unsigned order32(float v) {
    const unsigned b = __float_as_uint(v + 0.0f);
    const unsigned u = b ^ (static_cast<unsigned>(static_cast<int>(b) >> 31) | 0x80000000u);
    return v != v ? 1u : u;
}
__device__ __forceinline__ float order_value(unsigned u) {
    const unsigned b = u ^ ((u & 0x80000000u) ? 0x80000000u : 0xffffffffu);
    return u == 1u ? quiet_nan() : __uint_as_float(b);
}
__device__ __forceinline__ unsigned long long order_key(float v, int index) {
    return static_cast<unsigned long long>(order32(v)) << 32 | (0xffffffffu - static_cast<unsigned>(index));
}
__device__ __forceinline__ int key_index(unsigned long long k) {
    return static_cast<int>(0xffffffffu - static_cast<unsigned>(k));
}

// ---------------------------------------------------------------------------
// Packed arithmetic on two binary32 values (each half rounds as the single
// instruction does).
// ---------------------------------------------------------------------------
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
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

// The loss of a row from its softmax statistics `c` (in warp 0; with the tail:
// those of the indices that no slot names), and its entry of stats. All threads
// of the CTA take part.
template <class Tag, bool TAIL>
__device__ __forceinline__ void finish_distill(const LogitsProblem& pr, int64_t r, const typename Tag::raw* row,
                                               const int64_t* ids, const float* val, SoftSum c, float scale2,
                                               float* red) {
    __shared__ float m_ln_s[3];
    const int t = threadIdx.x;
    const Teacher q = read_teacher(pr, r, red);
    SoftSum all = c;
    if constexpr (TAIL) {
        SoftSum d;
        for (int i = t; i < pr.slots; i += blockDim.x) {
            const int64_t id = ids[i];
            if (id >= 0 && id < pr.cols) d.add(widen_elem<Tag>(row[id]), scale2);
        }
        d = block_softsum(d, scale2, red);
        if (t < 32) {
            all.join(d, scale2);
            c.rebase(all.m, scale2);
        }
    }
    if (t == 0) {
        m_ln_s[0] = all.m;
        m_ln_s[1] = all.empty() ? neg_inf() : logf(all.s);
        m_ln_s[2] = c.empty() ? neg_inf() : logf(c.s);
    }
    __syncthreads();
    const float m = m_ln_s[0], ln_s = m_ln_s[1], ln_rest = m_ln_s[2];
    float loss = 0.0f;
    for (int i = t; i < pr.slots; i += blockDim.x) {
        const int64_t id = ids[i];
        if (id < 0 || id >= pr.cols) continue;
        const float lnq = q.lnq(val[i]);
        const float p = expf(lnq);
        const float lp = ln_s == neg_inf() ? neg_inf() : (widen_elem<Tag>(row[id]) - m) / pr.temperature - ln_s;
        if (!(p == 0.0f)) loss += p * (lnq - lp);
    }
    loss = block_sum(loss, red);
    if (t == 0) {
        if (q.rest > 0.0f && ln_rest != neg_inf()) loss += q.rest * (logf(q.rest) - (ln_rest - ln_s));
        if ((ln_s != ln_s && q.any) || q.bad) loss = quiet_nan();
        if (pr.loss) pr.loss[r] = loss;
        if (pr.stats) pr.stats[r] = make_float4(ln_s == neg_inf() ? neg_inf() : m, ln_s, ln_rest, 0.0f);
    }
    __syncthreads();
}

}  // namespace argr
