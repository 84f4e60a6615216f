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
// The gradient sums e = exp(x - lse) of a row again and takes p = e / sum e. With a binary32 lse, e itself is off by |lse| 2^-24, and by a
// factor of E where a row is the type's lowest value throughout (lse = m + ln s has lost ln s); what lse is off by is
// common to a row's e, and at most about ln s, so the quotient is as exact far from zero as near it.
//
// Two phases. A row is read once, by G lanes of a warp, in blocks of 8 elements dealt to the lanes in turns, the warp's
// 32 / G rows side by side: sums, p, and the largest element of each block, which goes to shared memory. Then, for
// up to 32 such rows, a lane to a row: it takes the block of the largest head, reads that block again, finds the
// element and the block's next head, k times over. A choice so costs a handful of instructions of one lane and none of
// them crosses lanes; with a warp, or 8 lanes, to a row a choice took most of 540 or 280 instructions a
// row ([65536, 256], top 8), in chains of votes and shuffles. Warps own evenly dealt, contiguous rows
// and keep the sums of p of their elements in registers. Sums over CTAs are joined in a fixed order, without
// atomics: where one cluster suffices by it, through distributed shared memory;
// else every CTA leaves its sums and counts in scratch and a second kernel joins them
// (route_finish.cu).
//
// [65536, 256] f32, top 8, a tenth of it padding, counts and loss, in a graph of calls: 25 us (2.7 TB/s, 151 instructions a row; 16
// warps an SM, each with one batch: read, then eight dependent looks into blocks; 3.5 us are the second kernel's). [65536, 8] bf16,
// top 2, 6.9 us. The gradient, 32 lanes to a row of 256 experts: 28.9 us, 4.7 TB/s, 298 instructions a row in 55% of the
// issue slots (with exp(x - lse) as it is 28.4 and 271); [20001, 60] bf16, top 4, 7.6 us.
#pragma once

#include "logits_forward.cuh"
#include "select.h"

namespace argr {

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Both sums in every lane: each half of the group takes on one of them, so that two cost one exchange more than one does.
template <int G>
__device__ __forceinline__ void group_sums(float& a, float& b) {
    if constexpr (G > 1) {
        const bool upper = threadIdx.x & (G / 2);
        const float away = upper ? a : b, stays = upper ? b : a;
        float v = stays + __shfl_xor_sync(0xffffffffu, away, G / 2);
#pragma unroll
        for (int o = G / 4; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const float w = __shfl_xor_sync(0xffffffffu, v, G / 2);
        a = upper ? w : v;
        b = upper ? v : w;
    }
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
    if constexpr (G == 32) {
        return order_value(__reduce_max_sync(0xffffffffu, order32(v)));
    } else {
#pragma unroll
        for (int o = G / 2; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}

// N contiguous elements [lo, lo + N) of a row of E, as they lie in memory; -inf past the row's end.
template <class Tag, int N>
struct LaneRow {
    using R = typename Tag::raw;
    static constexpr int P = 16 / static_cast<int>(sizeof(R));  // elements of 16 bytes
    uint32_t w[N * sizeof(R) / 4];

    // `align`: rows begin at boundaries of so many bytes. (Eight binary32 elements come in one load where they may: in two,
    // 32 bytes from lane to lane, they take the L1 twice as long.)
    __device__ __forceinline__ void load(const R* row, int lo, int E, int align) {
        if (sizeof(R) == 4 && N == 8 && align == 32 && lo + N <= E) {
            if constexpr (sizeof(R) == 4 && N == 8)
                asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                             : "l"(row + lo)
                             : "memory");
        } else if (align >= 16 && lo + N <= E) {
#pragma unroll
            for (int i = 0; i < N / P; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(row + lo + i * P);
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const R v = lo + j < E ? row[lo + j] : none();
                if constexpr (sizeof(R) == 4) w[j] = __float_as_uint(v);
                else if (j & 1) w[j >> 1] |= static_cast<uint32_t>(v) << 16;
                else w[j >> 1] = v;
            }
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < N * static_cast<int>(sizeof(R)) / 4; ++i)
            w[i] = sizeof(R) == 4 ? 0xff800000u : std::is_same<Tag, TagBF16>::value ? 0xff80ff80u : 0xfc00fc00u;
    }
    static __device__ __forceinline__ R none() {
        if constexpr (sizeof(R) == 4) return neg_inf();
        else return std::is_same<Tag, TagBF16>::value ? 0xff80 : 0xfc00;
    }
    __device__ __forceinline__ void widen(float* x) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if constexpr (sizeof(R) == 4) x[j] = __uint_as_float(w[j]);
            else x[j] = Tag::widen(static_cast<uint16_t>(j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu));
        }
    }
};

// The boundaries that rows begin at: 32 bytes, 16, or less (0).
template <class R>
__device__ __forceinline__ int rows_aligned(const void* x, int64_t stride) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(x) | static_cast<uintptr_t>(stride) * sizeof(R);
    return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 0;
}

// Gradient: rows of a warp at a time, one after the other, where a row takes all its lanes (by the registers of a lane and the
// shared memory).
template <int G, int V> constexpr int kTurns = G < 32 ? 1 : V <= 8 ? 4 : V <= 16 ? 2 : 1;

// This warp's units [lo, hi) of `units`, dealt evenly over all warps.
struct WarpShare {
    int64_t lo, hi;
    __device__ __forceinline__ explicit WarpShare(int64_t units) {
        const int64_t w = static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x;  // (what is over, an SM after the other)
        const int64_t all = static_cast<int64_t>(gridDim.x) * kRouteWarps, each = units / all, more = units - each * all;
        lo = w * each + (w < more ? w : more);
        hi = lo + each + (w < more);
    }
};

// Shared memory of the forward kernel: the CTA's choices and rows [E + 1], its sums of p [E]; per warp the rows' maxima and
// sums, the heads of their blocks, from which element on a block's elements equal to its head are left, and
// their choices (weights, then ids); at the end the warps' sums.
template <int G, int V>
struct RouteLayout {
    static constexpr int BLOCKS = G * V / 8;                          // of a row
    static constexpr int ROWS = BLOCKS <= 32 ? 32 : 1024 / BLOCKS;    // of a batch
    static constexpr int PITCH = ROWS + 1;                            // of a block's heads: lanes and blocks in different banks
    size_t hist, acc, warp, sums, heads, after, weights, ids, each, total;
    __host__ __device__ RouteLayout(int E, int k) {
        hist = 0;
        acc = 4 * static_cast<size_t>((E + 1 + 3) / 4 * 4);
        warp = acc + 4 * static_cast<size_t>((E + 3) / 4 * 4);
        sums = 0;  // (in a warp's part)
        heads = 8 * ROWS;
        after = heads + 4 * static_cast<size_t>(BLOCKS) * PITCH;
        weights = (after + static_cast<size_t>(BLOCKS) * PITCH + 15) / 16 * 16;
        ids = weights + 4 * static_cast<size_t>(ROWS) * k;
        each = (ids + 4 * static_cast<size_t>(ROWS) * k + 15) / 16 * 16;
        const size_t a = kRouteWarps * each, b = 4 * static_cast<size_t>(kRouteWarps) * G * V;
        total = warp + (a > b ? a : b);
    }
};

// The k choices of this lane's row, in order. Its heads are at heads[block * PITCH], with after[...] as above (0 at first).
// Of the blocks' heads the largest of every 8 are kept in registers. A block's elements are taken in order, so what is left
// of it is what is below the element taken last, or equals it further on.
template <class Tag, int G, int V, class Put>
__device__ __forceinline__ void choose(const typename Tag::raw* row, int E, int align, float* heads, unsigned char* after, int k,
                                       Put put) {
    constexpr int BLOCKS = RouteLayout<G, V>::BLOCKS, PITCH = RouteLayout<G, V>::PITCH;
    constexpr int S = BLOCKS < 8 ? BLOCKS : 8, M = BLOCKS / S;  // M sets of S blocks
    float most[M];
#pragma unroll
    for (int q = 0; q < M; ++q) {
        most[q] = heads[q * S * PITCH];
#pragma unroll
        for (int i = 1; i < S; ++i) most[q] = fmaxf(most[q], heads[(q * S + i) * PITCH]);
    }
    int n = 0;
    for (; n < k; ++n) {
        float g = most[0];
#pragma unroll
        for (int q = 1; q < M; ++q) g = fmaxf(g, most[q]);
        if (!(g > neg_inf())) break;  // (NaN: blocks of NaNs alone, which are never chosen)
        int set = 0;
#pragma unroll
        for (int q = M - 1; q >= 0; --q)
            if (most[q] == g) set = q;
        float h[S];
        int at = 0;
#pragma unroll
        for (int i = S - 1; i >= 0; --i) {
            h[i] = heads[(set * S + i) * PITCH];
            if (h[i] == g) at = i;
        }
        const int block = set * S + at, from = after[block * PITCH];
        LaneRow<Tag, 8> raw;
        raw.load(row, block * 8, E, align);
        float x[8];
        raw.widen(x);
        int j = 8, again = 8;
        float below = neg_inf();
#pragma unroll
        for (int i = 7; i >= 0; --i) {
            const bool same = x[i] == g && i >= from;
            if (same) {
                again = j;
                j = i;
            }
            if (x[i] < g) below = fmaxf(below, x[i]);
        }
        const float next = again < 8 ? g : below;
        heads[block * PITCH] = next;
        after[block * PITCH] = static_cast<unsigned char>(again < 8 ? again : 0);
        float best = neg_inf();
#pragma unroll
        for (int i = 0; i < S; ++i) best = fmaxf(best, i == at ? next : h[i]);
#pragma unroll
        for (int q = 0; q < M; ++q)
            if (q == set) most[q] = best;
        put(n, block * 8 + j, g);
    }
    for (; n < k; ++n) put(n, -1, neg_inf());
}

__device__ __forceinline__ int ld_cluster(unsigned addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <class Tag, int G, int V>
__global__ void __launch_bounds__(kRouteBlock, V <= 8 ? 2 : 1) route_kernel(const RouteProblem pr, int cluster) {
    using R = typename Tag::raw;
    using Layout = RouteLayout<G, V>;
    constexpr int U = 32 / G, B = V / 8, ROWS = Layout::ROWS, PITCH = Layout::PITCH;  // U: rows of a unit; B: blocks of a lane
    extern __shared__ __align__(16) unsigned char dyn[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lg = lane & (G - 1), sub = lane / G;
    const int E = pr.experts, k = pr.k;
    const Layout lay(E, k);
    int* hist = reinterpret_cast<int*>(dyn + lay.hist);
    float* acc = reinterpret_cast<float*>(dyn + lay.acc);
    unsigned char* part = dyn + lay.warp + warp * lay.each;
    float2* row_sums = reinterpret_cast<float2*>(part + lay.sums);
    float* heads = reinterpret_cast<float*>(part + lay.heads);
    unsigned char* after = part + lay.after;
    float* weights = reinterpret_cast<float*>(part + lay.weights);  // [ROWS][k]
    int* ids = reinterpret_cast<int*>(part + lay.ids);
    const R* base = static_cast<const R*>(pr.x);
    const int align = rows_aligned<R>(pr.x, pr.row_stride);
    const WarpShare share((pr.rows + U - 1) / U);
    const int64_t end = share.hi * U < pr.rows ? share.hi * U : pr.rows;
    allow_dependents();
    if (pr.counts)
        for (int i = threadIdx.x; i <= E; i += kRouteBlock) hist[i] = 0;
    float sum_p[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum_p[j] = 0.0f;
    grid_dependency_wait();
    __syncthreads();
    int taken = 0;
    for (int64_t r0 = share.lo * U; r0 < end; r0 += ROWS) {
        const int rows = end - r0 < ROWS ? static_cast<int>(end - r0) : ROWS;
        const bool here = lane < rows && (!pr.valid || pr.valid[r0 + lane]);
        const unsigned valid = __ballot_sync(0xffffffffu, here);
        if (lane < ROWS) {
#pragma unroll 4
            for (int b = 0; b < Layout::BLOCKS; ++b) after[b * PITCH + lane] = 0;
        }
        for (int q0 = 0; q0 < rows; q0 += U) {
            const int q = q0 + sub;  // row of the batch
            const bool on = valid >> q & 1u;
            const R* row = base + (r0 + q) * pr.row_stride;
            float x[V], top = neg_inf();
#pragma unroll
            for (int b = 0; b < B; ++b) {
                LaneRow<Tag, 8> raw;
                raw.clear();
                if (on) raw.load(row, (b * G + lg) * 8, E, align);
                raw.widen(x + 8 * b);
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const float* y = x + 8 * b;
                const float h = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
                heads[(b * G + lg) * PITCH + q] = h;
                top = fmaxf(top, h);
            }
            const float m = group_max<G>(top), ref = m == neg_inf() ? 0.0f : m;
            const f32x2 minus = pack2(-ref, -ref), scale = pack2(kLog2E, kLog2E);
            f32x2 sums = 0;
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                unpack2(mul2(add2(pack2(x[j], x[j + 1]), minus), scale), x[j], x[j + 1]);
                x[j] = ex2(x[j]);
                x[j + 1] = ex2(x[j + 1]);
                sums = add2(sums, pack2(x[j], x[j + 1]));
            }
            float lo, hi;
            unpack2(sums, lo, hi);
            const float s = group_sum<G>(lo + hi);
            if (lg == 0) row_sums[q] = make_float2(m, s);
            if (pr.balance && s != 0.0f) {
                const float inv = __frcp_rn(s);
                const f32x2 of = pack2(inv, inv);
#pragma unroll
                for (int j = 0; j < V; j += 2)
                    unpack2(fma2(pack2(x[j], x[j + 1]), of, pack2(sum_p[j], sum_p[j + 1])), sum_p[j], sum_p[j + 1]);
            }
        }
        __syncwarp();
        float inv = 0.0f;
        if (lane < rows) {
            const float2 v = row_sums[lane];
            const float m = v.x, s = v.y, ref = m == neg_inf() ? 0.0f : m;
            const bool live = s != 0.0f;  // (a NaN is live)
            float all = 0.0f;
            choose<Tag, G, V>(base + (r0 + lane) * pr.row_stride, E, align, heads + lane, after + lane, k, [&](int i, int e, float x) {
                const float w = ex2((x - ref) * kLog2E);  // (0 where nothing was chosen)
                all += w;
                weights[lane * k + i] = w;
                ids[lane * k + i] = e;
            });
            inv = !live ? 0.0f : s != s ? quiet_nan() : 1.0f / (pr.normalize ? all : s);
            pr.lse[r0 + lane] = live ? m + logf(s) : neg_inf();
            taken += live;
        }
        __syncwarp();
        for (int i0 = 0; i0 < rows * k; i0 += 32) {
            const int i = i0 + lane, q = i < rows * k ? i / k : 0;
            const float scale = __shfl_sync(0xffffffffu, inv, q);
            if (i < rows * k) {
                const int id = ids[i];
                pr.weights[r0 * k + i] = weights[i] * scale;
                pr.ids[r0 * k + i] = id;
                if (pr.counts && id >= 0) atomicAdd(&hist[id], 1);
            }
        }
        __syncwarp();
    }
    if (!pr.counts) return;
    if (taken) atomicAdd(&hist[E], taken);
    if (pr.balance) {
        // over the warp's rows, then over the warps, in order
        float* lanes = reinterpret_cast<float*>(dyn + lay.warp);  // [warps][G * V]
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int o = 16; o >= G; o >>= 1) sum_p[j] += __shfl_xor_sync(0xffffffffu, sum_p[j], o);
            if (sub == 0) lanes[warp * G * V + (j / 8 * G + lg) * 8 + j % 8] = sum_p[j];
        }
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += kRouteBlock) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kRouteWarps; ++w) v += lanes[w * G * V + e];
            acc[e] = v;
        }
    }
    __syncthreads();
    if (cluster == 0) {
        for (int i = threadIdx.x; i <= E; i += kRouteBlock) {
            pr.part_counts[static_cast<int64_t>(blockIdx.x) * (E + 1) + i] = hist[i];
            if (pr.balance && i < E) pr.part_sums[static_cast<int64_t>(blockIdx.x) * E + i] = acc[i];
        }
        return;
    }
    // the grid is one cluster: every CTA joins its share of the experts
    __shared__ double red[kRouteWarps], shares[8];
    if (cluster > 1) {
        cluster_arrive();
        cluster_wait();
    }
    const int cta = static_cast<int>(blockIdx.x);
    double sum = 0.0;
    for (int e = threadIdx.x * cluster + cta; e < E; e += kRouteBlock * cluster) {
        long long n = 0;
        float t = 0.0f;
        for (int q = 0; q < cluster; ++q) {
            n += cluster > 1 ? ld_cluster(cluster_addr(smem_u32(hist + e), q)) : hist[e];
            if (pr.balance) t += cluster > 1 ? __int_as_float(ld_cluster(cluster_addr(smem_u32(acc + e), q))) : acc[e];
        }
        pr.counts[e] = n;
        sum += static_cast<double>(n) * t;
    }
    if (pr.balance) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) red[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            double all = 0.0;
            for (int w = 0; w < kRouteWarps; ++w) all += red[w];
            if (cluster > 1) {
                const unsigned to = cluster_addr(smem_u32(&shares[cta]), 0);
                st_cluster(to, static_cast<unsigned long long>(__double_as_longlong(all)));
            } else {
                shares[0] = all;
            }
        }
    }
    long long rows = 0;
    if (cta == 0 && threadIdx.x == 0)
        for (int q = 0; q < cluster; ++q) rows += cluster > 1 ? ld_cluster(cluster_addr(smem_u32(hist + E), q)) : hist[E];
    if (cluster > 1) {  // (nobody leaves while its shared memory is read)
        cluster_arrive();
        cluster_wait();
    }
    if (cta == 0 && threadIdx.x == 0) {
        *pr.taken = rows;
        if (pr.balance) {
            double all = 0.0;
            for (int q = 0; q < cluster; ++q) all += shares[q];
            *pr.balance = route_balance(all, rows, E, k);
        }
    }
}

// A lane's elements in the gradient's kernel: chunks of 16 bytes, dealt to the lanes in turns, so that a warp's loads and
// stores are of contiguous memory. (32 contiguous bytes to a lane took 30 us for [65536, 256] f32, the L1 66% busy.)
template <class Tag, int G>
struct Dealt {
    static constexpr int P = 16 / static_cast<int>(sizeof(typename Tag::raw));
    static __device__ __forceinline__ int first(int chunk, int lg) { return (chunk * G + lg) * P; }
    // The place of element e of a row of `elems` in shared memory: a lane reads 4 at a time, next to its neighbours'.
    static __device__ __forceinline__ int place(int e, int elems) {
        return P == 4 ? e : (e >> 3) * 4 + (e & 3) + (e >> 2 & 1) * (elems / 2);
    }
};

// Shared memory of the gradient's kernel, per warp: what the chosen elements of its RW rows get, 0 elsewhere, and the
// products of their weights and gradients [RW][k].
template <int G, int V>
struct RouteGradLayout {
    static constexpr int RW = 32 / G * kTurns<G, V>;
    size_t prods, each;
    __host__ __device__ explicit RouteGradLayout(int k) {
        prods = 4 * static_cast<size_t>(RW) * G * V;
        each = (prods + 4 * static_cast<size_t>(RW) * k + 15) / 16 * 16;
    }
};

template <class Tag, int G, int V>
__global__ void __launch_bounds__(kRouteBlock, V <= 8 ? 2 : 1) route_grad_kernel(const RouteProblem pr) {
    using R = typename Tag::raw;
    using D = Dealt<Tag, G>;
    constexpr int T = kTurns<G, V>, RW = 32 / G * T, LG = 32 / RW, P = D::P, C = V / P;  // C: chunks of a lane
    extern __shared__ __align__(16) unsigned char dyn[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lg = lane & (G - 1), sub = lane / G;
    const int E = pr.experts, k = pr.k;
    const RouteGradLayout<G, V> lay(k);
    float* at = reinterpret_cast<float*>(dyn + warp * lay.each);  // [RW][G * V]
    float* prods = reinterpret_cast<float*>(dyn + warp * lay.each + lay.prods);
    const R* base = static_cast<const R*>(pr.x);
    constexpr int U = G < 32 ? 32 / G : 1;
    const WarpShare share((pr.rows + U - 1) / U);
    const int64_t end = share.hi * U < pr.rows ? share.hi * U : pr.rows;
    allow_dependents();
    for (int i = lane; i < RW * G * V; i += 32) at[i] = 0.0f;
    grid_dependency_wait();
    __syncwarp();
    const int align = rows_aligned<R>(pr.x, pr.row_stride), align_out = rows_aligned<R>(pr.grad, pr.grad_stride);
    // lane q: of row q of the next pass, loaded a pass ahead. lse -inf: padding, or nothing above -inf: not read
    float next_lse = neg_inf(), next_h = 0.0f;
    const auto look_ahead = [&](int64_t r) {
        const bool in = lane < RW && r + lane < end;
        next_lse = in ? pr.lse[r + lane] : neg_inf();
        next_h = in && pr.grad_lse ? pr.grad_lse[r + lane] : 0.0f;
    };
    look_ahead(share.lo * U);
    float c[V];
    {
        float per = 0.0f;
        if (pr.grad_balance) {
            const int64_t taken = *pr.taken;
            const float n = static_cast<float>(taken > 0 ? taken : 1);
            per = *pr.grad_balance * (static_cast<float>(E) / (static_cast<float>(k) * n)) / n;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = D::first(j / P, lg) + j % P;
            c[j] = pr.grad_balance && e < E ? per * static_cast<float>(pr.counts[e]) : 0.0f;
        }
    }
    LaneRow<Tag, P> raw[C];
    const auto load = [&](int64_t row, bool on) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            raw[i].clear();
            if (on) raw[i].load(base + row * pr.row_stride, D::first(i, lg), E, align);
        }
    };
    for (int64_t r0 = share.lo * U; r0 < end; r0 += RW) {
        const int rows = end - r0 < RW ? static_cast<int>(end - r0) : RW;
        const float my_lse = next_lse, my_h = next_h;
        const unsigned live = __ballot_sync(0xffffffffu, my_lse != neg_inf());
        load(r0 + sub, live >> sub & 1u);
        look_ahead(r0 + RW);
        // the chosen elements: g w of each, their sums over a row, and what each gets
        float along = 0.0f;  // of row lane / LG
        if (pr.grad_weights) {
            for (int i = lane; i < rows * k; i += 32) {
                const bool in = pr.ids[r0 * k + i] >= 0;
                prods[i] = in ? pr.grad_weights[r0 * k + i] * pr.weights[r0 * k + i] : 0.0f;
            }
            __syncwarp();
            if (lane / LG < rows)
                for (int i = lane % LG; i < k; i += LG) along += prods[lane / LG * k + i];
            along = group_sum<LG>(along);
            for (int i0 = 0; i0 < rows * k; i0 += 32) {
                const int i = i0 + lane, q = i < rows * k ? i / k : 0;
                const float a = __shfl_sync(0xffffffffu, along, q * LG);
                if (i < rows * k && (live >> q & 1u)) {
                    const int64_t e = pr.ids[r0 * k + i];
                    if (e >= 0 && e < E)
                        at[q * G * V + D::place(static_cast<int>(e), G * V)] = pr.normalize ? prods[i] - pr.weights[r0 * k + i] * a : prods[i];
                }
            }
            __syncwarp();
        }
#pragma unroll 1
        for (int q = 0; q < T; ++q) {
            const int row = G < 32 ? sub : q;
            if (G == 32 && q >= rows) break;
            float d[V];
#pragma unroll
            for (int i = 0; i < C; ++i) raw[i].widen(d + P * i);
            if (G == 32 && q + 1 < T) load(r0 + q + 1, live >> 1 >> q & 1u);
            const float lse = __shfl_sync(0xffffffffu, my_lse, row), h = __shfl_sync(0xffffffffu, my_h, row);
            const float a = __shfl_sync(0xffffffffu, along, row * LG);
            const bool on = live >> row & 1u;
            float s = 0.0f, dot = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                d[j] = on ? ex2((d[j] - lse) * kLog2E) : 0.0f;
                s += d[j];
                dot += d[j] * c[j];
            }
            group_sums<G>(s, dot);
            const float inv = on ? __fdividef(1.0f, s) : 0.0f;  // (s is near 1, or E; off by two units at most)
            const float rest = (h - dot * inv - (pr.normalize ? 0.0f : a)) * inv;
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (pr.grad_weights && on) {
                    float4* mine = reinterpret_cast<float4*>(at + row * G * V + D::place(D::first(j / P, lg) + j % P, G * V));
                    v = *mine;
                    *mine = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                d[j] = d[j] * fmaf(c[j], inv, rest) + v.x;
                d[j + 1] = d[j + 1] * fmaf(c[j + 1], inv, rest) + v.y;
                d[j + 2] = d[j + 2] * fmaf(c[j + 2], inv, rest) + v.z;
                d[j + 3] = d[j + 3] * fmaf(c[j + 3], inv, rest) + v.w;
            }
            if (!on) {
#pragma unroll
                for (int j = 0; j < V; ++j) d[j] = 0.0f;
            }
            if (row >= rows) continue;  // (the last pass)
            R* out = static_cast<R*>(pr.grad) + (r0 + row) * pr.grad_stride;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int e = D::first(i, lg);
                if (align_out >= 16 && e + P <= E) {
                    uint32_t w[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if constexpr (P == 4) w[u] = __float_as_uint(d[4 * i + u]);
                        else
                            w[u] = static_cast<uint32_t>(narrow_elem<Tag>(d[8 * i + 2 * u])) |
                                   static_cast<uint32_t>(narrow_elem<Tag>(d[8 * i + 2 * u + 1])) << 16;
                    }
                    *reinterpret_cast<uint4*>(out + e) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        if (e + j < E) out[e + j] = narrow_elem<Tag>(d[P * i + j]);
                }
            }
        }
        __syncwarp();
    }
}

template <class Tag, int G, int V>
cudaError_t launch_route_gv(RouteProblem pr, const argr_caps& caps) {
    static KernelLaunchCache cache;
    auto kern = route_kernel<Tag, G, V>;
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    const size_t smem = RouteLayout<G, V>(pr.experts, pr.k).total;
    cudaError_t e = ensure_smem_limit(kern, smem + 1024, cache);  // with the static part
    if (e != cudaSuccess) return e;
    const RouteGrid grid = route_grid(pr.rows, pr.experts, pr.counts != nullptr, caps);
    pr.ctas = grid.ctas;
    e = launch_ex_smem(kern, dim3(static_cast<unsigned>(grid.ctas)), dim3(kRouteBlock), grid.cluster, smem, p, pr.stream, pr,
                       grid.cluster);
    return e == cudaSuccess && pr.counts && !grid.cluster ? launch_route_finish(pr) : e;
}
template <class Tag, int G, int V>
cudaError_t launch_route_grad_gv(const RouteProblem& pr, const argr_caps& caps) {
    static KernelLaunchCache cache;
    auto kern = route_grad_kernel<Tag, G, V>;
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    const size_t smem = kRouteWarps * RouteGradLayout<G, V>(pr.k).each;
    const cudaError_t e = ensure_smem_limit(kern, smem, cache);
    if (e != cudaSuccess) return e;
    const int64_t each = 32 / G * kRouteWarps, want = (pr.rows + each - 1) / each, most = (V <= 8 ? 2 : 1) * caps.sm_count;
    return launch_ex_smem(kern, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kRouteBlock), 1, smem, p,
                          pr.stream, pr);
}

#define ARGR_ROUTE_GV(fn, Tag, pr, caps)                \
    ((pr).experts <= 8     ? fn<Tag, 1, 8>(pr, caps)    \
     : (pr).experts <= 16  ? fn<Tag, 2, 8>(pr, caps)    \
     : (pr).experts <= 32  ? fn<Tag, 4, 8>(pr, caps)    \
     : (pr).experts <= 64  ? fn<Tag, 8, 8>(pr, caps)    \
     : (pr).experts <= 128 ? fn<Tag, 16, 8>(pr, caps)   \
     : (pr).experts <= 256 ? fn<Tag, 32, 8>(pr, caps)   \
     : (pr).experts <= 512 ? fn<Tag, 32, 16>(pr, caps)  \
                           : fn<Tag, 32, 32>(pr, caps))

template <class Tag>
cudaError_t launch_route_t(const RouteProblem& pr, const argr_caps& caps) {
    const RouteShape s = route_shape(pr.experts);
    switch (s.lanes) {
        case 1: return launch_route_gv<Tag, 1, 8>(pr, caps);
        case 2: return launch_route_gv<Tag, 2, 8>(pr, caps);
        case 4: return launch_route_gv<Tag, 4, 8>(pr, caps);
        case 8:
            return s.elems == 8    ? launch_route_gv<Tag, 8, 8>(pr, caps)
                   : s.elems == 16 ? launch_route_gv<Tag, 8, 16>(pr, caps)
                                   : launch_route_gv<Tag, 8, 32>(pr, caps);
        case 16: return launch_route_gv<Tag, 16, 32>(pr, caps);
        default: return launch_route_gv<Tag, 32, 32>(pr, caps);
    }
}
template <class Tag>
cudaError_t launch_route_grad_t(const RouteProblem& pr, const argr_caps& caps) {
    return ARGR_ROUTE_GV(launch_route_grad_gv, Tag, pr, caps);
}

#define ARGR_DEFINE_SELECT(sfx, Tag, dtype)                                                                           \
    namespace argr {                                                                                                  \
    cudaError_t beam_plan_##sfx(int64_t items, int beams, int64_t cols, int k, const argr_caps& caps, BeamPlan* p) {  \
        return beam_plan_t<Tag>(items, beams, cols, dtype, k, caps, p);                                               \
    }                                                                                                                 \
    cudaError_t launch_beam_select_##sfx(const BeamProblem& pr, const BeamPlan& b, const argr_caps& caps) {           \
        return launch_beam_select_t<Tag>(pr, b, caps);                                                                \
    }                                                                                                                 \
    cudaError_t launch_route_##sfx(const RouteProblem& pr, const argr_caps& caps) {                                   \
        return launch_route_t<Tag>(pr, caps);                                                                         \
    }                                                                                                                 \
    cudaError_t launch_route_grad_##sfx(const RouteProblem& pr, const argr_caps& caps) {                              \
        return launch_route_grad_t<Tag>(pr, caps);                                                                    \
    }                                                                                                                 \
    }

}  // namespace argr
