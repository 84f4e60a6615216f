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
// A row is held by G lanes of a warp, V contiguous elements to a lane, and every element is read
// once. A warp takes RW rows at a time (32 / G side by side, or some one after the other where a row
// takes all lanes), so that what is done once per row or per choice (logarithm,
// quotients, ranks, stores) is done by different lanes for different rows. Warps own evenly dealt, contiguous rows
// and keep the sums of p of their elements in registers. Sums over CTAs are joined in a fixed order, without
// atomics: where one cluster suffices by it, through distributed shared memory;
// else every CTA leaves its sums and counts in scratch and a second kernel joins them
// (route_finish.cu).
#pragma once

#include "logits_forward.cuh"
#include "select.h"

namespace argr {

constexpr int kRouteWarps = kRouteBlock / 32;

// order32() of an element that can be chosen, 0 for -inf, NaN and what is past the row.
__device__ __forceinline__ unsigned choice_key(float x) { return x > neg_inf() ? order32(x) : 0u; }

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
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

// A lane's V elements [lo, lo + V) of a row of E, as they lie in memory; -inf past the row's end.
template <class Tag, int V>
struct LaneRow {
    using R = typename Tag::raw;
    static constexpr int P = 16 / static_cast<int>(sizeof(R));  // elements of 16 bytes
    uint32_t w[V * sizeof(R) / 4];

    // `wide`: rows begin at 16-byte boundaries.
    __device__ __forceinline__ void load(const R* row, int lo, int E, bool wide) {
        if (wide && lo + V <= E) {
#pragma unroll
            for (int i = 0; i < V / P; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(row + lo + i * P);
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const R v = lo + j < E ? row[lo + j] : none();
                if constexpr (sizeof(R) == 4) w[j] = __float_as_uint(v);
                else if (j & 1) w[j >> 1] |= static_cast<uint32_t>(v) << 16;
                else w[j >> 1] = v;
            }
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < V * static_cast<int>(sizeof(R)) / 4; ++i)
            w[i] = sizeof(R) == 4 ? 0xff800000u : std::is_same<Tag, TagBF16>::value ? 0xff80ff80u : 0xfc00fc00u;
    }
    static __device__ __forceinline__ R none() {
        if constexpr (sizeof(R) == 4) return neg_inf();
        else return std::is_same<Tag, TagBF16>::value ? 0xff80 : 0xfc00;
    }
    __device__ __forceinline__ void widen(float (&x)[V]) const {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (sizeof(R) == 4) x[j] = __uint_as_float(w[j]);
            else x[j] = Tag::widen(static_cast<uint16_t>(j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu));
        }
    }
};

// Rows of a warp at a time, one after the other, where a row takes all its lanes (by the registers of a lane and the gradient's
// shared memory).
template <int G, int V> constexpr int kTurns = G < 32 ? 1 : V <= 8 ? 4 : V <= 16 ? 2 : 1;

// This warp's units [lo, hi) of `units`, dealt evenly over all warps.
struct WarpShare {
    int64_t lo, hi;
    __device__ __forceinline__ explicit WarpShare(int64_t units) {
        const int64_t w = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
        const int64_t all = static_cast<int64_t>(gridDim.x) * kRouteWarps, each = units / all, more = units - each * all;
        lo = w * each + (w < more ? w : more);
        hi = lo + each + (w < more);
    }
};

// What a lane's rows choose, in order: G lanes find the largest of what is left k times. Lane 0 of the
// group hands each choice to `put(i, e, x)`.
template <int G, int V, class Put>
__device__ __forceinline__ void choose_in_turns(const float (&x)[V], int lg, int k, Put put) {
    unsigned key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = choice_key(x[j]);
    for (int i = 0; i < k; ++i) {
        unsigned best = 0;
        int e = 0;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (key[j] > best) {
                best = key[j];
                e = lg * V + j;
            }
        if constexpr (G == 32) {
            const unsigned top = __reduce_max_sync(0xffffffffu, best);
            e = static_cast<int>(__reduce_min_sync(0xffffffffu, best == top ? static_cast<unsigned>(e) : ~0u));
            best = top;
        } else {
#pragma unroll
            for (int o = G / 2; o >= 1; o >>= 1) {
                const unsigned b = __shfl_xor_sync(0xffffffffu, best, o);
                const int f = __shfl_xor_sync(0xffffffffu, e, o);
                if (b > best || (b == best && f < e)) {
                    best = b;
                    e = f;
                }
            }
        }
        put(i, best ? e : -1, best ? order_value(best) : neg_inf());
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e == lg * V + j) key[j] = 0u;
    }
}

// What reaches the threshold of a row over a whole warp, collected in `cand` (32 keys, any order); returns how many, or -1
// where they are more. The k-th largest of the lanes' own largest elements is reached by at
// least k elements, seldom by many more.
template <class Tag, int V>
__device__ __forceinline__ int collect(const float (&x)[V], int lane, int k, unsigned long long* cand) {
    float big = x[0];
#pragma unroll
    for (int j = 1; j < V; ++j) big = fmaxf(big, x[j]);
    unsigned left = choice_key(big), at = 0;
#pragma unroll 4
    for (int i = 0; i < k; ++i) {
        at = __reduce_max_sync(0xffffffffu, left);
        if (left == at) left = 0u;
    }
    // fewer lanes than k have one: every element that can be chosen
    const float least = at == 0u ? -FLT_MAX : order_value(at);
    unsigned hits = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) hits |= static_cast<unsigned>(x[j] >= least) << j;
    const unsigned below = (1u << lane) - 1u;
    int n = 0;
    for (;;) {
        const unsigned has = __ballot_sync(0xffffffffu, hits != 0);
        if (has == 0) return n;
        const int p = n + __popc(has & below);
        n += __popc(has);
        if (n > 32) return -1;
        if (hits) {
            const int j = __ffs(hits) - 1;
            hits &= hits - 1;
            float v = x[0];
#pragma unroll
            for (int i = 1; i < V; ++i)
                if (i == j) v = x[i];
            cand[p] = order_key(v, lane * V + j);
        }
    }
}

// Shared memory of the forward kernel: the CTA's choices and rows [E + 1], its sums of p [E] and half its warps'
// on the way there, and per warp its rows' choices (weights, then ids) and, where a row takes all lanes, 32 keys for each.
template <int G, int V>
struct RouteLayout {
    static constexpr int RW = 32 / G * kTurns<G, V>;
    size_t hist, acc, half, stage, keys, each, total;
    __host__ __device__ RouteLayout(int E, int k) {
        hist = 0;
        acc = 4 * static_cast<size_t>((E + 1 + 3) / 4 * 4);
        half = acc + 4 * static_cast<size_t>((E + 3) / 4 * 4);
        stage = half + 4 * static_cast<size_t>(kRouteWarps / 2) * G * V;
        keys = 8 * static_cast<size_t>(RW) * k;  // (in a warp's part)
        each = (keys + (G == 32 ? 8 * 32 * static_cast<size_t>(RW) : 0) + 15) / 16 * 16;
        total = stage + kRouteWarps * each;
    }
};

__device__ __forceinline__ int ld_cluster(unsigned addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <class Tag, int G, int V>
__global__ void __launch_bounds__(kRouteBlock, V <= 8 ? 2 : 1) route_kernel(const RouteProblem pr, int cluster) {
    using R = typename Tag::raw;
    constexpr int T = kTurns<G, V>, RW = 32 / G * T, LG = 32 / RW;  // rows at a time, and lanes to each where they are finished
    extern __shared__ __align__(16) unsigned char dyn[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lg = lane & (G - 1), sub = lane / G;
    const int E = pr.experts, k = pr.k;
    const RouteLayout<G, V> lay(E, k);
    int* hist = reinterpret_cast<int*>(dyn + lay.hist);
    float* acc = reinterpret_cast<float*>(dyn + lay.acc);
    unsigned char* stage = dyn + lay.stage + warp * lay.each;
    float* weights = reinterpret_cast<float*>(stage);  // [RW][k]
    int* ids = reinterpret_cast<int*>(weights + RW * k);
    allow_dependents();
    if (pr.counts)
        for (int i = threadIdx.x; i <= E; i += kRouteBlock) hist[i] = 0;
    float sum_p[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum_p[j] = 0.0f;
    grid_dependency_wait();
    __syncthreads();
    const bool wide = (reinterpret_cast<uintptr_t>(pr.x) | static_cast<uintptr_t>(pr.row_stride) * sizeof(R)) % 16 == 0;
    const R* base = static_cast<const R*>(pr.x);
    int taken = 0;
    // units: passes of 32 / G rows, or rows
    constexpr int U = G < 32 ? 32 / G : 1;
    const WarpShare share((pr.rows + U - 1) / U);
    const int64_t end = share.hi * U < pr.rows ? share.hi * U : pr.rows;
    for (int64_t r0 = share.lo * U; r0 < end; r0 += RW) {
        const int rows = end - r0 < RW ? static_cast<int>(end - r0) : RW;  // of this pass
        const bool mine = lane < rows && (!pr.valid || pr.valid[r0 + lane]);
        const unsigned valid = __ballot_sync(0xffffffffu, mine);
        // of row lane / LG, for what is done once a row
        float ref = 0.0f, m = neg_inf(), s = 0.0f, all = 0.0f;
        if constexpr (G < 32) {
            LaneRow<Tag, V> raw;
            raw.clear();
            if (valid >> sub & 1u) raw.load(base + (r0 + sub) * pr.row_stride, lg * V, E, wide);
            float x[V], p[V];
            raw.widen(x);
            m = x[0];
#pragma unroll
            for (int j = 1; j < V; ++j) m = fmaxf(m, x[j]);
            m = group_max<G>(m);
            if (m != m) m = neg_inf();  // (NaN alone)
            ref = m == neg_inf() ? 0.0f : m;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                p[j] = ex2((x[j] - ref) * kLog2E);
                s += p[j];
            }
            s = group_sum<G>(s);
            if (pr.balance && s != 0.0f) {
                const float inv = 1.0f / s;
#pragma unroll
                for (int j = 0; j < V; ++j) sum_p[j] += p[j] * inv;
            }
            choose_in_turns<G, V>(x, lg, k, [&](int i, int e, float v) {
                const float w = ex2((v - ref) * kLog2E);  // (0 where nothing was chosen)
                all += w;
                if (lg == 0) {
                    weights[sub * k + i] = w;
                    ids[sub * k + i] = e;
                }
            });
        } else {
            unsigned long long* cand = reinterpret_cast<unsigned long long*>(stage + lay.keys);  // [RW][32]
            int found = 0;
            LaneRow<Tag, V> raw;
            raw.clear();
            if (valid & 1u) raw.load(base + r0 * pr.row_stride, lane * V, E, wide);
            for (int q = 0; q < rows; ++q) {
                float x[V], p[V];
                raw.widen(x);
                raw.clear();
                if (valid >> 1 >> q & 1u) raw.load(base + (r0 + q + 1) * pr.row_stride, lane * V, E, wide);
                if (!(valid >> q & 1u)) continue;
                float big = x[0];
#pragma unroll
                for (int j = 1; j < V; ++j) big = fmaxf(big, x[j]);
                big = group_max<32>(big);
                if (big != big) big = neg_inf();  // (NaN alone)
                const float r = big == neg_inf() ? 0.0f : big;
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    p[j] = ex2((x[j] - r) * kLog2E);
                    sum += p[j];
                }
                sum = group_sum<32>(sum);
                if (pr.balance && sum != 0.0f) {
                    const float inv = 1.0f / sum;
#pragma unroll
                    for (int j = 0; j < V; ++j) sum_p[j] += p[j] * inv;
                }
                int n = collect<Tag, V>(x, lane, k, cand + 32 * q);
                if (n < 0) {
                    n = 0;
                    choose_in_turns<G, V>(x, lane, k, [&](int i, int e, float v) {
                        if (e >= 0) {
                            if (lane == 0) cand[32 * q + i] = order_key(v, e);
                            n = i + 1;
                        }
                    });
                }
                if (lane / LG == q) {
                    m = big;
                    ref = r;
                    s = sum;
                    found = n;
                }
            }
            __syncwarp();
            // ranks by counting, LG lanes to a row
            const int q = lane / LG;
            const unsigned long long* mine = cand + 32 * q;
            for (int c = lane % LG; c < found; c += LG) {
                const unsigned long long key = mine[c];
                int rank = 0;
#pragma unroll 4
                for (int i = 0; i < found; ++i) rank += mine[i] > key;
                if (rank < k) {
                    const float w = ex2((order_value(static_cast<unsigned>(key >> 32)) - ref) * kLog2E);
                    all += w;
                    weights[q * k + rank] = w;
                    ids[q * k + rank] = key_index(key);
                }
            }
            for (int i = found + lane % LG; i < k; i += LG) {
                weights[q * k + i] = 0.0f;
                ids[q * k + i] = -1;
            }
            all = group_sum<LG>(all);
        }
        const bool live = s != 0.0f;  // (a NaN is live)
        const float inv = !live ? 0.0f : s != s ? quiet_nan() : 1.0f / (pr.normalize ? all : s);
        if (lane % LG == 0 && lane / LG < rows) {
            pr.lse[r0 + lane / LG] = live ? m + logf(s) : neg_inf();
            taken += live;
        }
        __syncwarp();
        for (int i0 = 0; i0 < rows * k; i0 += 32) {
            const int i = i0 + lane, q = i < rows * k ? i / k : 0;  // row of the pass
            const float scale = __shfl_sync(0xffffffffu, inv, q * LG);
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
        // over the warp's rows, then half of the warps hand theirs to the other half
        float* half = reinterpret_cast<float*>(dyn + lay.half);
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int o = 16; o >= G; o >>= 1) sum_p[j] += __shfl_xor_sync(0xffffffffu, sum_p[j], o);
        }
        for (int h = kRouteWarps / 2; h >= 1; h >>= 1) {
            if (warp >= h && warp < 2 * h && sub == 0) {
#pragma unroll
                for (int j = 0; j < V; ++j) half[((warp - h) * V + j) * G + lg] = sum_p[j];
            }
            __syncthreads();
            if (warp < h) {
#pragma unroll
                for (int j = 0; j < V; ++j) sum_p[j] += half[(warp * V + j) * G + lg];
            }
            __syncthreads();
        }
        if (warp == 0 && sub == 0) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (lg * V + j < E) acc[lg * V + j] = sum_p[j];
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
    constexpr int T = kTurns<G, V>, RW = 32 / G * T, LG = 32 / RW, P = 16 / static_cast<int>(sizeof(R));
    extern __shared__ __align__(16) unsigned char dyn[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lg = lane & (G - 1), sub = lane / G;
    const int E = pr.experts, k = pr.k;
    const RouteGradLayout<G, V> lay(k);
    float* at = reinterpret_cast<float*>(dyn + warp * lay.each);  // [RW][G * V]
    float* prods = reinterpret_cast<float*>(dyn + warp * lay.each + lay.prods);
    allow_dependents();
    for (int i = lane; i < RW * G * V; i += 32) at[i] = 0.0f;
    grid_dependency_wait();
    __syncwarp();
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
            const int e = lg * V + j;
            c[j] = pr.grad_balance && e < E ? per * static_cast<float>(pr.counts[e]) : 0.0f;
        }
    }
    const bool wide = (reinterpret_cast<uintptr_t>(pr.x) | static_cast<uintptr_t>(pr.row_stride) * sizeof(R)) % 16 == 0;
    const bool wide_out = (reinterpret_cast<uintptr_t>(pr.grad) | static_cast<uintptr_t>(pr.grad_stride) * sizeof(R)) % 16 == 0;
    const R* base = static_cast<const R*>(pr.x);
    constexpr int U = G < 32 ? 32 / G : 1;
    const WarpShare share((pr.rows + U - 1) / U);
    const int64_t end = share.hi * U < pr.rows ? share.hi * U : pr.rows;
    for (int64_t r0 = share.lo * U; r0 < end; r0 += RW) {
        const int rows = end - r0 < RW ? static_cast<int>(end - r0) : RW;
        // lane q: of row q. lse -inf: padding, or nothing above -inf: not read
        const float my_lse = lane < rows ? pr.lse[r0 + lane] : neg_inf();
        const float my_h = lane < rows && pr.grad_lse ? pr.grad_lse[r0 + lane] : 0.0f;
        const unsigned live = __ballot_sync(0xffffffffu, my_lse != neg_inf());
        LaneRow<Tag, V> raw;
        raw.clear();
        if (live >> sub & 1u) raw.load(base + (r0 + sub) * pr.row_stride, lg * V, E, wide);
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
                        at[q * G * V + e] = pr.normalize ? prods[i] - pr.weights[r0 * k + i] * a : prods[i];
                }
            }
            __syncwarp();
        }
#pragma unroll 1
        for (int q = 0; q < T; ++q) {
            const int row = G < 32 ? sub : q;
            if (G == 32 && q >= rows) break;
            float d[V];
            raw.widen(d);
            if (G == 32 && q + 1 < T) {
                raw.clear();
                if (live >> 1 >> q & 1u) raw.load(base + (r0 + q + 1) * pr.row_stride, lg * V, E, wide);
            }
            const float lse = __shfl_sync(0xffffffffu, my_lse, row), h = __shfl_sync(0xffffffffu, my_h, row);
            const float a = __shfl_sync(0xffffffffu, along, row * LG);
            const bool on = live >> row & 1u;
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                d[j] = on ? ex2((d[j] - lse) * kLog2E) : 0.0f;
                dot += d[j] * c[j];
            }
            dot = pr.grad_balance ? group_sum<G>(dot) : 0.0f;
            const float rest = h - dot - (pr.normalize ? 0.0f : a);
            float4* mine = reinterpret_cast<float4*>(at + row * G * V + lg * V);
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (pr.grad_weights && on) {
                    v = mine[j / 4];
                    mine[j / 4] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                d[j] = d[j] * (c[j] + rest) + v.x;
                d[j + 1] = d[j + 1] * (c[j + 1] + rest) + v.y;
                d[j + 2] = d[j + 2] * (c[j + 2] + rest) + v.z;
                d[j + 3] = d[j + 3] * (c[j + 3] + rest) + v.w;
            }
            if (!on) {
#pragma unroll
                for (int j = 0; j < V; ++j) d[j] = 0.0f;
            }
            if (row >= rows) continue;  // (the last pass)
            R* out = static_cast<R*>(pr.grad) + (r0 + row) * pr.grad_stride + lg * V;
            if (wide_out && lg * V + V <= E) {
#pragma unroll
                for (int i = 0; i < V / P; ++i) {
                    uint32_t w[4];
                    if constexpr (P == 4) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) w[u] = __float_as_uint(d[4 * i + u]);
                    } else {
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            w[u] = static_cast<uint32_t>(narrow_elem<Tag>(d[8 * i + 2 * u])) |
                                   static_cast<uint32_t>(narrow_elem<Tag>(d[8 * i + 2 * u + 1])) << 16;
                    }
                    *reinterpret_cast<uint4*>(out + i * P) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (lg * V + j < E) out[j] = narrow_elem<Tag>(d[j]);
            }
        }
        __syncwarp();
    }
}

// CTAs of a problem: enough for a unit (32 / G rows) per warp, `per_sm` to an SM at most.
inline int route_grid(int64_t rows, int unit, int per_sm, const argr_caps& caps) {
    const int64_t each = static_cast<int64_t>(unit) * kRouteWarps;
    const int64_t want = (rows + each - 1) / each, most = static_cast<int64_t>(per_sm) * caps.sm_count;
    return static_cast<int>(want < most ? want : most);
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
    pr.ctas = route_grid(pr.rows, 32 / G, V <= 8 ? 2 : 1, caps);
    if (pr.ctas > kRouteMaxCtas) pr.ctas = kRouteMaxCtas;
    // one cluster, without a second kernel, while its warps take few units each
    int cluster = 0;
    if (pr.counts && pr.ctas <= kRouteOneTurns * 8) {
        cluster = 1;
        while (cluster < 8 && cluster < pr.ctas) cluster *= 2;
        if (cluster > caps.max_cluster) cluster = 0;
    }
    if (cluster) pr.ctas = cluster;
    e = launch_ex_smem(kern, dim3(static_cast<unsigned>(pr.ctas)), dim3(kRouteBlock), cluster, smem, p, pr.stream, pr, cluster);
    return e == cudaSuccess && pr.counts && !cluster ? launch_route_finish(pr) : e;
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
    return launch_ex_smem(kern, dim3(static_cast<unsigned>(route_grid(pr.rows, 32 / G, V <= 8 ? 2 : 1, caps))),
                          dim3(kRouteBlock), 1, smem, p, pr.stream, pr);
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
    return ARGR_ROUTE_GV(launch_route_gv, Tag, pr, caps);
}
template <class Tag>
cudaError_t launch_route_grad_t(const RouteProblem& pr, const argr_caps& caps) {
    return ARGR_ROUTE_GV(launch_route_grad_gv, Tag, pr, caps);
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
