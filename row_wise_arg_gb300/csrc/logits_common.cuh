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
constexpr unsigned kOrderNegInf = 0x007fffffu;  // order32 of -inf, the least number
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
    c.rebase(order_value(__reduce_max_sync(0xffffffffu, order32(c.m))), scale2);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        c.s += __shfl_xor_sync(0xffffffffu, c.s, o);
        c.t += __shfl_xor_sync(0xffffffffu, c.t, o);
    }
    return c;
}

// The CTA's triple in two steps with a barrier between them: every warp's to `smem`
// (3 * 32 floats), and the whole in every thread of the warp that asks.
__device__ __forceinline__ void softsum_to(SoftSum c, float scale2, float* smem) {
    c = warp_softsum(c, scale2);
    if ((threadIdx.x & 31) == 0) {
        smem[threadIdx.x >> 5] = c.m;
        smem[32 + (threadIdx.x >> 5)] = c.s;
        smem[64 + (threadIdx.x >> 5)] = c.t;
    }
}
__device__ __forceinline__ SoftSum softsum_from(float scale2, const float* smem) {
    const int lane = threadIdx.x & 31;
    SoftSum r;
    if (lane < static_cast<int>(blockDim.x >> 5)) {
        r.m = smem[lane];
        r.s = smem[32 + lane];
        r.t = smem[64 + lane];
    }
    return warp_softsum(r, scale2);
}

// Both, in every thread of warp 0. Contains __syncthreads().
__device__ __forceinline__ SoftSum block_softsum(SoftSum c, float scale2, float* smem) {
    __syncthreads();
    softsum_to(c, scale2, smem);
    __syncthreads();
    if (threadIdx.x < 32) c = softsum_from(scale2, smem);
    return c;
}

// Sum over the CTA, in every thread and in a fixed order. `smem` holds 32 values.
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
// Groups: 64 bytes of a row, a thread's unit of work.
// ---------------------------------------------------------------------------
constexpr int kGroupBytes = 64;
constexpr int kSegGroups = 8192;  // groups of a CTA's range that the forward passes handle at a time
template <class Tag> constexpr int kGroupElems = kGroupBytes / static_cast<int>(sizeof(typename Tag::raw));

template <class Tag>
struct Group {
    uint32_t w[16];
    // 64 bytes at a 32-byte boundary, through the read-only path or, where this
    // kernel may write them, the plain one.
    template <bool READ_ONLY = true>
    __device__ __forceinline__ void load(const typename Tag::raw* p) {
#define ARGR_LOAD32(OP)                                                                            \
    asm volatile(OP " {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"                                     \
                 : "=r"(w[8 * h]), "=r"(w[8 * h + 1]), "=r"(w[8 * h + 2]), "=r"(w[8 * h + 3]),     \
                   "=r"(w[8 * h + 4]), "=r"(w[8 * h + 5]), "=r"(w[8 * h + 6]), "=r"(w[8 * h + 7])  \
                 : "l"(reinterpret_cast<const char*>(p) + 32 * h)                                  \
                 : "memory")
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (READ_ONLY) ARGR_LOAD32("ld.global.nc.L1::no_allocate.v8.b32");
            else ARGR_LOAD32("ld.global.L1::no_allocate.v8.b32");
        }
#undef ARGR_LOAD32
    }
    // Elements 2i and 2i + 1 of a word pair (binary32) or of word i (16 bits).
    __device__ __forceinline__ void pair(int i, float& lo, float& hi) const {
        if constexpr (std::is_same<Tag, TagF32>::value) {
            lo = __uint_as_float(w[2 * i]);
            hi = __uint_as_float(w[2 * i + 1]);
        } else if constexpr (std::is_same<Tag, TagBF16>::value) {
            lo = __uint_as_float(w[i] << 16);
            hi = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            lo = f.x;
            hi = f.y;
        }
    }
    __device__ __forceinline__ void store(typename Tag::raw* p) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[8 * h]),
                         "r"(w[8 * h + 1]), "r"(w[8 * h + 2]), "r"(w[8 * h + 3]), "r"(w[8 * h + 4]),
                         "r"(w[8 * h + 5]), "r"(w[8 * h + 6]), "r"(w[8 * h + 7]),
                         "l"(reinterpret_cast<char*>(p) + 32 * h)
                         : "memory");
    }
    __device__ __forceinline__ void set_pair(int i, float lo, float hi) {
        if constexpr (std::is_same<Tag, TagF32>::value) {
            w[2 * i] = __float_as_uint(lo);
            w[2 * i + 1] = __float_as_uint(hi);
        } else if constexpr (std::is_same<Tag, TagBF16>::value) {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
        } else {
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
        }
    }
    // The largest element, NaN if there is no other.
    __device__ __forceinline__ float largest() const {
        if constexpr (std::is_same<Tag, TagF32>::value) {
            float m = __uint_as_float(w[0]);
#pragma unroll
            for (int i = 1; i < 16; ++i) m = fmaxf(m, __uint_as_float(w[i]));
            return m;
        } else {
            uint32_t m = w[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) {
                if constexpr (std::is_same<Tag, TagBF16>::value) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
                else asm("max.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
            }
            return fmaxf(Tag::widen(static_cast<uint16_t>(m & 0xffffu)), Tag::widen(static_cast<uint16_t>(m >> 16)));
        }
    }
    // Put -inf in the place of the elements whose bits are set.
    __device__ __forceinline__ void drop(unsigned bits) {
        if constexpr (std::is_same<Tag, TagF32>::value) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (bits >> i & 1u) w[i] = 0xff800000u;
        } else {
            constexpr uint32_t ninf = std::is_same<Tag, TagBF16>::value ? 0xff80u : 0xfc00u;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (bits >> (2 * i) & 1u) w[i] = (w[i] & 0xffff0000u) | ninf;
                if (bits >> (2 * i + 1) & 1u) w[i] = (w[i] & 0xffffu) | ninf << 16;
            }
        }
    }
};

// ---------------------------------------------------------------------------
// A CTA's part of a row, and a segment of it. Slot i of a segment's groups is its
// head (i = 0, may be empty), group i - 1 of its body, or its tail (i = body + 1,
// may be empty); positions are elements of the row.
// ---------------------------------------------------------------------------
template <class Tag>
struct Segment {
    int head_lo, body_lo, body, tail_lo, tail_hi;  // [head_lo, body_lo) head, [tail_lo, tail_hi) tail
    __device__ __forceinline__ int slots() const { return body + 2; }
    __device__ __forceinline__ void range(int i, int& lo, int& n) const {
        lo = i == 0 ? head_lo : body_lo + (i - 1) * kGroupElems<Tag>;
        n = i == 0 ? body_lo - head_lo : i <= body ? kGroupElems<Tag> : tail_hi - tail_lo;
    }
};

template <class Tag>
struct Part {
    int align;         // elements before the first 32-byte boundary
    int first, count;  // body groups of this CTA
    int cols;
    bool is_first, is_last;

    __device__ __forceinline__ Part(const typename Tag::raw* row, int n, int rank, int ranks) {
        const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(row) & 31u);
        align = static_cast<int>(((32u - off) & 31u) / sizeof(typename Tag::raw));
        if (align > n) align = n;
        // 32-bit division: a 64-bit one costs a thread as much as 30 elements
        const unsigned groups = static_cast<unsigned>(n - align) / kGroupElems<Tag>;
        const unsigned each = groups / static_cast<unsigned>(ranks), more = groups - each * ranks;
        first = static_cast<int>(each * rank + min(static_cast<unsigned>(rank), more));
        count = static_cast<int>(each + (static_cast<unsigned>(rank) < more));
        cols = n;
        is_first = rank == 0;
        is_last = rank == ranks - 1;
    }
    // The elements of this part, ragged ends included.
    __device__ __forceinline__ int begin() const { return is_first ? 0 : align + first * kGroupElems<Tag>; }
    __device__ __forceinline__ int end() const { return is_last ? cols : align + (first + count) * kGroupElems<Tag>; }
    __device__ __forceinline__ Segment<Tag> segment(int at) const {
        Segment<Tag> s;
        s.body = count - at < kSegGroups ? count - at : kSegGroups;
        s.body_lo = align + (first + at) * kGroupElems<Tag>;
        s.head_lo = is_first && at == 0 ? 0 : s.body_lo;
        s.tail_lo = s.body_lo + s.body * kGroupElems<Tag>;
        s.tail_hi = is_last && at + s.body == count ? cols : s.tail_lo;
        return s;
    }
};

// ---------------------------------------------------------------------------
// The teacher's side of a row, in shared memory.
// ---------------------------------------------------------------------------
struct Teacher {
    float top;    // without the tail: ln q = (v - top) / T - ln_sum, so that what the values have in common
    float ln_sum; // costs no digits, and the largest differences overflow to q = 0 alone
    float total;  // sum of q over the filled slots
    float rest;   // what the tail holds
    bool any;     // a slot holds something
    bool bad;     // a slot names an index past the row
};

struct Slots {
    int* id;   // the index named, kNoId or kBadId
    float* v;  // teacher
    float* x;  // the row's element, where it was asked for
    Teacher* sums;

    // In `bytes(n)` bytes of shared memory at p (16-byte aligned).
    __device__ __forceinline__ Slots(unsigned char* p, int n)
        : id(reinterpret_cast<int*>(p + sizeof(Teacher) + 12)),
          v(reinterpret_cast<float*>(id + n)),
          x(v + n),
          sums(reinterpret_cast<Teacher*>(p)) {}
    static __host__ __device__ size_t bytes(int n) {
        return (sizeof(Teacher) + 12 + 12 * static_cast<size_t>(n) + 15) / 16 * 16;
    }
};
constexpr int kNoId = -1;
constexpr int kBadId = -2;  // past the row

// Fill a row's slots, with the row's elements for those of [lo, hi). A barrier
// must follow (and come between earlier uses and this).
template <class Tag>
__device__ __forceinline__ void load_slots(const LogitsProblem& pr, int64_t r, const typename Tag::raw* row, int lo,
                                           int hi, const Slots& sl) {
    const int64_t* ids = pr.ids + r * pr.slots;
    const float* val = pr.teacher + r * pr.slots;
    for (int i = threadIdx.x; i < pr.slots; i += blockDim.x) {
        const int64_t id = ids[i];
        const int j = id < 0 ? kNoId : id >= pr.cols ? kBadId : static_cast<int>(id);
        sl.id[i] = j;
        sl.v[i] = val[i];
        if (j >= lo && j < hi) sl.x[i] = widen_elem<Tag>(row[j]);
    }
}

// The teacher's sums over filled slots, by one warp, in all its lanes; the slots
// are complete for it.
__device__ __forceinline__ Teacher warp_teacher(const LogitsProblem& pr, const Slots& sl) {
    const int lane = threadIdx.x & 31;
    bool any = false, bad = false;
    float top = -FLT_MAX;
    for (int i = lane; i < pr.slots; i += 32) {
        const int id = sl.id[i];
        any = any || (id != kNoId && (pr.tail || sl.v[i] != neg_inf()));
        bad = bad || id == kBadId;
        if (id != kNoId) top = fmaxf(top, sl.v[i]);
    }
    if (!pr.tail) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    float sum = 0.0f;
    for (int i = lane; i < pr.slots; i += 32)
        if (sl.id[i] != kNoId) sum += expf(pr.tail ? sl.v[i] : (sl.v[i] - top) * pr.inv_t);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    Teacher q;
    q.any = __any_sync(0xffffffffu, any);
    q.bad = __any_sync(0xffffffffu, bad);
    q.top = top;
    q.ln_sum = q.any ? logf(sum) : 0.0f;  // (nothing given: every ln q is -inf)
    q.total = pr.tail ? sum : q.any ? 1.0f : 0.0f;
    q.rest = pr.tail && q.any ? fmaxf(0.0f, 1.0f - sum) : 0.0f;
    return q;
}

// The same by warp 0, for every thread of the CTA. Contains barriers, the first of
// them after which the slots are complete; `also`, given the sums, runs in warp 0
// before the second.
template <class F>
__device__ __forceinline__ Teacher teacher_of(const LogitsProblem& pr, const Slots& sl, F also) {
    __syncthreads();
    if (threadIdx.x < 32) {
        const Teacher q = warp_teacher(pr, sl);
        if (threadIdx.x == 0) *sl.sums = q;
        also(q);
    }
    __syncthreads();
    return *sl.sums;
}
__device__ __forceinline__ Teacher teacher_of(const LogitsProblem& pr, const Slots& sl) {
    return teacher_of(pr, sl, [](const Teacher&) {});
}

// The tail's share of a row, p_rest, may be far below what binary32 holds, so the
// tail's sum stays relative to the tail's own largest element and p_rest a logarithm. Below
// kLeastTail it is 0 in binary64 as well: tails masked by finite values (an f16 row's
// lowest, say) count as masked.
constexpr float kLeastTail = -745.0f;

// ln s_rest of a tail, against the row's largest element m; -inf where there is none.
__device__ __forceinline__ float tail_log(const LogitsProblem& pr, const SoftSum& rest, float m, float ln_s) {
    if (rest.empty()) return neg_inf();
    const float ln_rest = logf(rest.s) + (rest.m - m) * pr.inv_t;
    return ln_rest - ln_s < kLeastTail ? neg_inf() : ln_rest;
}

// ln q of a slot with this value.
__device__ __forceinline__ float teacher_log(const LogitsProblem& pr, const Teacher& q, float v) {
    return pr.tail ? v : (v - q.top) * pr.inv_t - q.ln_sum;
}

// What a slot adds to the loss of a row with largest element m.
__device__ __forceinline__ float slot_loss(const LogitsProblem& pr, const Teacher& q, const Slots& sl, int i, float m,
                                           float ln_s) {
    if (sl.id[i] < 0) return 0.0f;
    const float lnq = teacher_log(pr, q, sl.v[i]);
    const float p = expf(lnq);
    const float lp = ln_s == neg_inf() ? neg_inf() : (sl.x[i] - m) / pr.temperature - ln_s;
    return p == 0.0f ? 0.0f : p * (lnq - lp);
}
__device__ __forceinline__ float whole_loss(const Teacher& q, float loss, float ln_s, float ln_rest) {
    if (q.rest > 0.0f && ln_rest != neg_inf()) loss += q.rest * (logf(q.rest) - (ln_rest - ln_s));
    return (ln_s != ln_s && q.any) || q.bad ? quiet_nan() : loss;
}

// The loss of a row, in thread 0, from its largest element, ln s and ln s_rest.
// All threads of the CTA take part; the slots hold every element that they name.
__device__ __forceinline__ float row_loss(const LogitsProblem& pr, const Teacher& q, const Slots& sl, float m,
                                          float ln_s, float ln_rest, float* red) {
    float loss = 0.0f;
    for (int i = threadIdx.x; i < pr.slots; i += blockDim.x) loss += slot_loss(pr, q, sl, i, m, ln_s);
    return whole_loss(q, block_sum(loss, red), ln_s, ln_rest);
}

// The weights of a row's gradient. Named elements: g (total p - q). Others: without a
// tail g total p; with one g (total p_rest - rest) p / p_rest, the last factor (at most 1) one
// exponential against the tail's own sum, so that neither factor leaves binary32's range
// where p and p_rest do. ln_rest is against the row's largest element, own_ln_rest the same against
// own_m (the tail's largest where it is known, else the row's).
// `none`: every element is `dense`.
struct GradWeights {
    float g, total, m, ls2;
    float dense, dense_m, dense_ls2;
    bool none;

    GradWeights() = default;
    __device__ __forceinline__ GradWeights(const LogitsProblem& pr, const Teacher& q, float grad_loss, float row_m,
                                           float ln_s, float ln_rest, float own_m, float own_ln_rest) {
        const float rest = ln_rest > neg_inf() ? q.rest : 0.0f;
        g = grad_loss * pr.inv_t;
        if (q.bad || (ln_s != ln_s && q.any)) g = quiet_nan();
        none = ln_s == neg_inf() || !q.any;  // nothing is taught, or nothing can be
        total = q.total + rest;
        dense = g * total;
        m = none ? 0.0f : row_m;
        ls2 = none ? 0.0f : ln_s * kLog2E;
        dense_m = m;
        dense_ls2 = ls2;
        if (none) dense = q.bad ? g : 0.0f;
        else if (rest > 0.0f) {
            dense = g * (total * expf(ln_rest - ln_s) - rest);
            dense_m = own_m;
            dense_ls2 = own_ln_rest * kLog2E;
        }
    }
    __device__ __forceinline__ float named(float x, float lnq, float scale2) const {
        return g * (total * ex2((x - m) * scale2 - ls2) - expf(lnq));
    }
};

// The loss of a row from its softmax statistics `c` (in warp 0; with the tail:
// those of the indices that no slot names), and its entry of stats.
template <class Tag, bool TAIL>
__device__ __forceinline__ void finish_distill(const LogitsProblem& pr, int64_t r, SoftSum c, float scale2,
                                               float* red, const Slots& sl) {
    __shared__ float m_ln_s[3];
    const int t = threadIdx.x;
    const Teacher q = teacher_of(pr, sl);
    SoftSum all = c;
    if constexpr (TAIL) {
        SoftSum d;
        for (int i = t; i < pr.slots; i += blockDim.x)
            if (sl.id[i] >= 0) d.add(sl.x[i], scale2);
        d = block_softsum(d, scale2, red);
        if (t < 32) all.join(d, scale2);
    }
    if (t == 0) {
        m_ln_s[0] = all.empty() ? neg_inf() : all.m;
        m_ln_s[1] = all.empty() ? neg_inf() : logf(all.s);
        m_ln_s[2] = TAIL ? tail_log(pr, c, all.m, m_ln_s[1]) : m_ln_s[1];
    }
    __syncthreads();
    const float m = m_ln_s[0], ln_s = m_ln_s[1], ln_rest = m_ln_s[2];
    const float loss = row_loss(pr, q, sl, m, ln_s, ln_rest, red);
    if (t == 0) {
        if (pr.loss) pr.loss[r] = loss;
        if (pr.stats) pr.stats[r] = make_float4(m, ln_s, ln_rest, 0.0f);
    }
    __syncthreads();
}

}  // namespace argr
