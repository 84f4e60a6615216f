// A beam search's step: the continuations (beam, token) of the largest totals of
// each item, over all its beams and the vocabulary.
//
// With a beam's total s_b and its logits x, m = max x and S = sum exp((x - m) / T),
//     total_bv = s_b + (x_v - m) / T - ln S.
// Within a beam the totals come in the logits' order, so the `count` first of an
// item are among the `count` first of each of its beams: a beam's logits are read
// once, for S and for its first alternatives (logits_forward.cuh), and the
// lists of all beams are merged. Totals of different beams lie close together,
// and what decides between them is the difference of their ln S: the merge works
// in 64 bits (a handful of operations per list entry; the 64-bit unit is slow), S is the
// binary32 sum of the pass.
//
// Few rows: one cluster per item, `ranks` CTAs to a beam. Every CTA hands
// its sums and its list to CTA 0 through distributed shared memory, which merges: no
// scratch, one launch. Many rows: a CTA per row, or the persistent kernel of long rows
// (logits_stream.cuh), leaves lists and sums in scratch, and a second kernel merges them.
//
// Bound by latency for few rows: in a graph of calls whose inputs rotate past L2, [1, 4, 32000] f32, 8 continuations, 7.6 us: read
// 1.5, threshold and alternatives 2.2, hand-over 0.6, merge 2 (sums and logarithms 0.5, ranks 0.7, threshold and places
// 1); [16, 4, 202048] bf16 14.6 us. [64, 16, 202048] bf16, 32 continuations, 92 us, 4.3 TB/s: 1024 rows in 3.4 rounds.
#pragma once

#include "logits_stream.cuh"
#include "select.h"

namespace argr {

constexpr int kMaxBeams = ARGR_BEAM_MAX_BEAMS;
constexpr int kMergeBlock = 512;
constexpr int kMergeMax = 256;  // entries ranked by counting, at most
constexpr int kMergeEntries = kMaxBeams * ARGR_LOGITS_MAX_TOP;  // of all lists

// What the merge knows of a beam.
struct BeamSum {
    double base;   // s_b - ln S
    double scale;  // of the rank
    double m;
    int state;     // kBeamGone, kBeamEnded or kBeamLive
};
constexpr int kBeamGone = 0, kBeamEnded = 1, kBeamLive = 2;

// A key that orders ranks: 0 for -inf and NaN, at least 1 for numbers; both zeros alike.
__device__ __forceinline__ unsigned long long rank_key(double rank) {
    const unsigned hi = static_cast<unsigned>(__double2hiint(rank)), lo = static_cast<unsigned>(__double2loint(rank));
    if ((hi & 0x7ff00000u) == 0x7ff00000u) return 0ull;
    const unsigned long long b = static_cast<unsigned long long>(hi) << 32 | lo;
    return (hi >> 31) ? 0ull - b : b | 0x8000000000000000ull;  // (-0, 1 << 63, maps to itself, as +0 does)
}
__device__ __forceinline__ double key_rank(unsigned long long key) {
    return __longlong_as_double(static_cast<long long>((key >> 63) ? key & 0x7fffffffffffffffull : 0ull - key));
}

// base - ln s for a binary32 s >= 1/2, off by less than 3e-9: with s = 2^e f, f in [2/3, 4/3), ln f = 2 artanh u,
// u = (f - 1) / (f + 1), |u| <= 1/5. u is held as a sum of two binary32 numbers, the series past its first term as one
// (at most 0.0055, so its rounding is below 4e-10; it ends where u^13 / 13 < 1e-10). 64-bit arithmetic only joins the
// parts: log() in 64 bits took 0.3 us of a merge.
__device__ __forceinline__ double minus_log(double base, float s) {
    const int bits = __float_as_int(s);
    const int e = (bits - 0x3f2aaaab) >> 23;  // 0x3f2aaaab: 2/3
    const float f = __int_as_float(bits - (e << 23));
    const float a = f - 1.0f, b = f + 1.0f;  // (b is off by up to half a unit: b + c is exact)
    const float c = f - (b - 1.0f);
    const float u = a / b;
    const float v = (fmaf(-u, b, a) - u * c) / b;  // what u lacks
    const float q = u * u;
    float tail = 2.0f / 11.0f;
    tail = fmaf(tail, q, 2.0f / 9.0f);
    tail = fmaf(tail, q, 2.0f / 7.0f);
    tail = fmaf(tail, q, 2.0f / 5.0f);
    tail = fmaf(tail, q, 2.0f / 3.0f);
    tail = fmaf(tail * q, u, 2.0f * v);
    return (base - static_cast<double>(2.0f * u)) - static_cast<double>(tail) - e * 0.69314718055994530942;
}

struct MergeShared {
    BeamSum beam[kMaxBeams];
    unsigned long long key[kMergeMax];
    unsigned long long place[kMergeMax];
    int win[ARGR_LOGITS_MAX_TOP];
    unsigned low[32], high[32];
    int poisoned, n;
};

// A beam's total and scale, before its row has been read. Returns whether they are what they may be.
__device__ __forceinline__ bool load_beam(const BeamProblem& pr, int64_t r, BeamSum& v) {
    const float s = pr.rows.beam_scores[r];
    const float w = pr.scale ? pr.scale[r] : 1.0f;
    v.base = s;
    v.scale = w;
    v.m = 0.0;
    v.state = s == neg_inf() ? kBeamGone : pr.rows.beam_ended && pr.rows.beam_ended[r] ? kBeamEnded : kBeamLive;
    return v.state == kBeamGone || (fabsf(s) <= FLT_MAX && w > 0.0f && w <= FLT_MAX);
}
__device__ __forceinline__ void load_beams(const BeamProblem& pr, int64_t item, MergeShared& sh) {
    if (threadIdx.x >= 32) return;
    bool bad = false;
    for (int b = threadIdx.x; b < pr.beams; b += 32)
        if (!load_beam(pr, item * pr.beams + b, sh.beam[b])) bad = true;
    bad = __any_sync(0xffffffffu, bad);
    if (threadIdx.x == 0) {
        sh.poisoned = bad;
        sh.n = 0;
    }
}

// The merge of an item's lists, ranks (a power of two, 1 << shift) of k keys to a beam, each in order and filled up
// with 0; load_beams() has been called. `keys` and `totals` (where there are scales): room for as many. The entries become ranks in 64 bits; a
// value that at least `count` of them reach, and not many more, is found bit by bit in their
// upper 32 bits, a barrier each, from the first bit on in which they differ; what reaches it is ranked by counting.
// Where too many do (ties), one warp takes the best of the lists' heads `count` times.
__device__ __forceinline__ void merge_beams(const BeamProblem& pr, int64_t item, int k, int shift,
                                            const unsigned long long* gathered, unsigned long long* keys, float* totals,
                                            const float2* sums, float scale2, MergeShared& sh) {
    const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5, warps = nt >> 5;
    const int beams = pr.beams, lists = beams << shift, count = pr.count, ranks = 1 << shift;
    if (warp == 0) {
        // a lane to a list (two, past 32 of them, which are then of as many beams)
        bool bad = false;
        for (int l0 = 0; l0 < lists; l0 += 32) {
            const int l = l0 + lane, b = l >> shift;
            const bool live = l < lists && sh.beam[b].state == kBeamLive;
            const float2 v = live ? sums[l] : make_float2(-FLT_MAX, 0.0f);
            SoftSum c;
            c.m = v.x;
            c.s = v.y;
            for (int o = 1; o < ranks; o <<= 1) {
                SoftSum d;
                d.m = __shfl_xor_sync(0xffffffffu, c.m, o);
                d.s = __shfl_xor_sync(0xffffffffu, c.s, o);
                c.join(d, scale2);
            }
            if (live && (l & (ranks - 1)) == 0) {
                BeamSum& to = sh.beam[b];
                to.m = c.m;
                if (c.s != c.s) bad = true;
                else if (c.empty()) to.state = kBeamGone;
                else to.base = minus_log(to.base, c.s);
            }
        }
        if (bad) sh.poisoned = 1;
    }
    __syncthreads();
    const bool poisoned = sh.poisoned != 0;
    unsigned low = ~0u, high = 0u;  // of the upper halves of this thread's keys
    for (int l = warp; l < lists; l += warps) {
        const BeamSum v = sh.beam[l >> shift];
        for (int i = lane; i < k; i += 32) {
            unsigned long long key = 0;
            double total = v.base;
            if (v.state == kBeamLive) {
                const unsigned long long g = gathered[l * k + i];
                if (g) {
                    total = v.base + (static_cast<double>(order_value(static_cast<unsigned>(g >> 32))) - v.m) * pr.inv_t;
                    key = rank_key(pr.scale ? total * v.scale : total);
                }
            } else if (v.state == kBeamEnded && (l & (ranks - 1)) == 0 && i == 0) {
                key = rank_key(pr.scale ? total * v.scale : total);
            }
            if (poisoned) key = 0;
            keys[l * k + i] = key;
            if (pr.scale) totals[l * k + i] = static_cast<float>(total);
            const unsigned hi = static_cast<unsigned>(key >> 32);
            if (key) low = min(low, hi);
            high = max(high, hi);
        }
    }
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) {
        sh.low[warp] = low;
        sh.high[warp] = high;
    }
    __syncthreads();
    low = lane < warps ? sh.low[lane] : ~0u;
    high = lane < warps ? sh.high[lane] : 0u;
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    const int all = lists * k;
    unsigned at = high ? low : 1u;  // every entry reaches it
    if (all > kMergeMax / 2 && high > low) {
        const int slack = count + count / 2 + 16;
        int bit = 31 - __clz(high ^ low);
        at = high & ~((2u << bit) - 1u);
        for (; bit >= 0; --bit) {
            const unsigned trial = at | 1u << bit;
            int n = 0;
            for (int i0 = 0; i0 < all; i0 += nt) {
                const bool in = i0 + t < all && static_cast<unsigned>(keys[i0 + t < all ? i0 + t : 0] >> 32) >= trial;
                n += __syncthreads_count(in);
            }
            if (n < count) continue;
            at = trial;
            if (n <= slack) break;
        }
    }
    // Which of two entries of the same rank is first: the lower beam's, within a beam the larger logit, then the lower index. A list
    // is in this order (and there are kMergeEntries at most); the parts of a beam's row are lists of their own, in which
    // different logits may have totals that round to one binary64 value.
    const auto place_of = [&](int i) {
        if (shift == 0) return static_cast<unsigned long long>(i);
        const unsigned later = ~static_cast<unsigned>(gathered[i] >> 32);
        return (static_cast<unsigned long long>(i / (k << shift)) << 32 | later) * kMergeEntries + i;
    };
    for (int i = t; i < all; i += nt) {
        const unsigned long long key = keys[i];
        if (key == 0 || static_cast<unsigned>(key >> 32) < at) continue;
        const int p = atomicAdd(&sh.n, 1);
        if (p < kMergeMax) {
            sh.key[p] = key;
            sh.place[p] = place_of(i);
        }
    }
    __syncthreads();
    const int n = sh.n;
    const auto put = [&](int r, int i, unsigned long long key) {
        const int parent = i / k >> shift;
        pr.tokens[item * count + r] = sh.beam[parent].state == kBeamEnded ? pr.end_token : key_index(gathered[i]);
        pr.parents[item * count + r] = parent;
        pr.out_scores[item * count + r] = pr.scale ? totals[i] : static_cast<float>(key_rank(key));
    };
    if (n <= kMergeMax) {
        // four lanes to an entry
        for (int q0 = 0; q0 < n; q0 += nt / 4) {
            const int q = q0 + (t >> 2);
            const unsigned long long key = q < n ? sh.key[q] : 0ull;
            const unsigned long long place = q < n ? sh.place[q] : 0ull;
            int r = 0;
#pragma unroll 4
            for (int j = t & 3; j < n; j += 4) {
                const unsigned long long other = sh.key[j];
                r += other > key || (other == key && sh.place[j] < place);
            }
            r += __shfl_xor_sync(0xffffffffu, r, 1);
            r += __shfl_xor_sync(0xffffffffu, r, 2);
            if (q < n && (t & 3) == 0 && r < count) put(r, static_cast<int>(place % kMergeEntries), key);
        }
        for (int r = n + t; r < count; r += nt) {
            pr.tokens[item * count + r] = -1;
            pr.parents[item * count + r] = -1;
            pr.out_scores[item * count + r] = poisoned ? quiet_nan() : neg_inf();
        }
        return;
    }
    if (warp == 0) {
        // lane l holds the lists 2 l and 2 l + 1
        int p[2] = {0, 0};
        unsigned long long head[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) head[j] = 2 * lane + j < lists ? keys[(2 * lane + j) * k] : 0ull;
        for (int r = 0; r < count; ++r) {  // (more than kMergeMax entries are there)
            int j = head[1] > head[0];
            if (shift > 0 && head[1] == head[0] && head[1] != 0)  // two lists of one beam
                j = gathered[(2 * lane + 1) * k + p[1]] > gathered[2 * lane * k + p[0]];
            const unsigned long long h = j ? head[1] : head[0];
            const unsigned hi = static_cast<unsigned>(h >> 32), top = __reduce_max_sync(0xffffffffu, hi);
            const unsigned lo = hi == top ? static_cast<unsigned>(h) : 0u;
            const unsigned least = __reduce_max_sync(0xffffffffu, lo);
            const bool best = hi == top && lo == least;
            unsigned holds = __ballot_sync(0xffffffffu, best);
            if (shift > 0) {
                // of the lowest of these beams, the largest logit
                const int l = 2 * lane + j, beam = 2 * (__ffs(holds) - 1) >> shift;
                const bool in = best && l >> shift == beam;
                const unsigned long long g = in ? gathered[l * k + (j ? p[1] : p[0])] : 0ull;
                const unsigned g_hi = static_cast<unsigned>(g >> 32), g_top = __reduce_max_sync(0xffffffffu, g_hi);
                const unsigned g_lo = g_hi == g_top ? static_cast<unsigned>(g) : 0u;
                const unsigned g_least = __reduce_max_sync(0xffffffffu, g_lo);
                const bool first = in && g_hi == g_top && g_lo == g_least;
                holds = __ballot_sync(0xffffffffu, first);
            }
            if (lane == __ffs(holds) - 1) {
                const int l = 2 * lane + j, i = j ? p[1] : p[0];
                sh.win[r] = l * k + i;
                const unsigned long long next = i + 1 < k ? keys[l * k + i + 1] : 0ull;
                if (j) {
                    head[1] = next;
                    p[1] = i + 1;
                } else {
                    head[0] = next;
                    p[0] = i + 1;
                }
            }
        }
    }
    __syncthreads();
    for (int r = t; r < count; r += nt) put(r, sh.win[r], keys[sh.win[r]]);
}

// Shared memory of a CTA that reads rows: a segment's slots, the list so far, and, where it merges too, `lists` lists.
struct BeamLayout {
    size_t big, cand, best, list, gathered, keys, totals, sums, total;  // offsets
    __host__ __device__ BeamLayout(int k, int lists, int seg_slots, int group_elems) {
        size_t at = 0;
        big = at;
        at += 4 * static_cast<size_t>(seg_slots);
        cand = at;
        at += 8 * static_cast<size_t>(cand_room(k, group_elems));
        best = at;
        at += 8 * 2 * ARGR_LOGITS_MAX_TOP;
        gathered = at;
        at += 8 * static_cast<size_t>(lists) * k;
        keys = at;
        at += 8 * static_cast<size_t>(lists) * k;
        sums = at;
        at += 8 * static_cast<size_t>(lists);
        totals = at;
        at += 4 * static_cast<size_t>(lists) * k;
        list = at;
        at += 2 * kListGroups;
        total = (at + 15) / 16 * 16;
    }
};

// One part of a row: its list to sh.best (returns its length), its sums to warp 0. `red`: 96 floats.
template <class Tag>
__device__ __forceinline__ int scan_beam(const typename Tag::raw* row, const Part<Tag>& part, int k, float scale2,
                                         const TopShared& sh, float* red, SoftSum& c) {
    int have = 0;
    for (int at = 0;;) {
        const Segment<Tag> sg = part.segment(at);
        SoftSum d;
        unsigned most = 0;
        scan_segment<Tag, false, true, false>(d, row, sg, scale2, sh.big, nullptr, most, row + part.end());
        d.t = 0.0f;
        c.join(d, scale2);
        if (at + sg.body >= part.count) softsum_to(c, scale2, red);
        have = take_segment<Tag>(row, sg, k, have, most, sh);
        at += sg.body;
        if (at >= part.count) break;
    }
    if (threadIdx.x < 32) c = softsum_from(scale2, red);
    return have;
}

template <class Tag>
__device__ __forceinline__ TopShared beam_shared(unsigned char* dyn, const BeamLayout& lay, int k, int* count) {
    TopShared sh;
    sh.room = cand_room(k, kGroupElems<Tag>);
    sh.big = reinterpret_cast<unsigned*>(dyn + lay.big);
    sh.cand = reinterpret_cast<unsigned long long*>(dyn + lay.cand);
    sh.best = reinterpret_cast<unsigned long long*>(dyn + lay.best);
    sh.list = reinterpret_cast<unsigned short*>(dyn + lay.list);
    sh.count = count;
    return sh;
}

template <class Tag, int BLOCK, int PER_SM>
__global__ void __launch_bounds__(BLOCK, PER_SM) beam_select_kernel(const BeamProblem pr, float scale2, int cluster,
                                                                    int shift, int seg_slots) {
    using R = typename Tag::raw;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ float red[96];
    __shared__ int count[3];
    __shared__ MergeShared merge;
    const int t = threadIdx.x;
    const int cta = static_cast<int>(blockIdx.x % cluster), ranks = 1 << shift, rank = cta & (ranks - 1);
    const int b = cta >> shift;
    const int64_t item = blockIdx.x / cluster;
    const int k = pr.rows.top_k;
    const BeamLayout lay(k, pr.beams << shift, seg_slots, kGroupElems<Tag>);
    const TopShared sh = beam_shared<Tag>(dyn, lay, k, count);
    unsigned long long* gathered = reinterpret_cast<unsigned long long*>(dyn + lay.gathered);
    float2* sums = reinterpret_cast<float2*>(dyn + lay.sums);
    allow_dependents();
    if (cluster > 1) cluster_ready();
    const int64_t r = item * pr.beams + b;
    prefetch_part<Tag>(pr.rows, r, rank, ranks);
    grid_dependency_wait();
    if (cta == 0) load_beams(pr, item, merge);
    if (cluster > 1) cluster_wait();
    const unsigned to_lists = cluster > 1 ? cluster_addr(smem_u32(gathered), 0) : 0;
    const unsigned to_sums = cluster > 1 ? cluster_addr(smem_u32(sums), 0) : 0;
    if (beam_looks(pr.rows, r)) {  // (alike in every thread)
        const R* row = static_cast<const R*>(pr.rows.x) + r * pr.rows.row_stride;
        SoftSum c;
        const int have = scan_beam<Tag>(row, Part<Tag>(row, pr.rows.cols, rank, ranks), k, scale2, sh, red, c);
        if (cluster > 1) {
            if (t == 0) {
                st_cluster(to_sums + 8 * cta, c.m);
                st_cluster(to_sums + 8 * cta + 4, c.s);
            }
            for (int i = t; i < k; i += blockDim.x) st_cluster(to_lists + 8 * (cta * k + i), i < have ? sh.best[i] : 0ull);
        } else {
            if (t == 0) sums[0] = make_float2(c.m, c.s);
            for (int i = t; i < k; i += blockDim.x) gathered[i] = i < have ? sh.best[i] : 0ull;
        }
    }
    if (cluster > 1) {
        cluster_arrive();
        cluster_wait();
        if (cta != 0) return;
    } else {
        __syncthreads();
    }
    merge_beams(pr, item, k, shift, gathered, reinterpret_cast<unsigned long long*>(dyn + lay.keys),
                reinterpret_cast<float*>(dyn + lay.totals), sums, scale2, merge);
}

// Many rows: a CTA per row, and the merge of an item's lists by a CTA.
template <class Tag, int BLOCK, int PER_SM>
__global__ void __launch_bounds__(BLOCK, PER_SM) beam_rows_kernel(const LogitsProblem pr, float scale2, int seg_slots) {
    using R = typename Tag::raw;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ float red[96];
    __shared__ int count[3];
    const int t = threadIdx.x, k = pr.top_k;
    const TopShared sh = beam_shared<Tag>(dyn, BeamLayout(k, 0, seg_slots, kGroupElems<Tag>), k, count);
    const int64_t r = blockIdx.x;
    allow_dependents();
    prefetch_part<Tag>(pr, r, 0, 1);
    grid_dependency_wait();
    if (!beam_looks(pr, r)) return;
    const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
    SoftSum c;
    const int have = scan_beam<Tag>(row, Part<Tag>(row, pr.cols, 0, 1), k, scale2, sh, red, c);
    if (t == 0) pr.beam_sums[r] = make_float2(c.m, c.s);
    for (int i = t; i < k; i += blockDim.x) pr.beam_keys[r * k + i] = i < have ? sh.best[i] : 0ull;
}

// (beam_merge.cu)
cudaError_t launch_beam_merge(const BeamProblem& pr);

template <class Tag>
int beam_seg_slots(int cols, int shift) {
    const int64_t parts = (cols / kGroupElems<Tag> >> shift) + 1;
    return static_cast<int>((parts < kSegGroups ? parts : kSegGroups) + 2 + 3) / 4 * 4;
}

// The kernel of a cluster per item: its launch's cache and shared memory.
template <class Tag>
struct BeamCluster {
    static constexpr auto kernel() { return beam_select_kernel<Tag, 512, 1>; }
    static KernelLaunchCache& cache() {
        static KernelLaunchCache c;
        return c;
    }
    int seg_slots;
    size_t smem;
    BeamCluster(int beams, int cols, int k, const BeamPlan& b)
        : seg_slots(beam_seg_slots<Tag>(cols, b.shift)), smem(BeamLayout(k, beams << b.shift, seg_slots, kGroupElems<Tag>).total) {}

    cudaError_t allow(const BeamPlan& b) const {
        const cudaError_t e = ensure_smem_limit(kernel(), smem + sizeof(MergeShared) + 1024, cache());  // with the static part
        return e == cudaSuccess && b.cluster > 8 ? allow_big_cluster(kernel(), cache()) : e;
    }
    // Whether the current device places such clusters.
    cudaError_t fits(const BeamPlan& b, bool* ok) const {
        cudaError_t e = allow(b);
        if (e == cudaSuccess)
            e = cluster_fits(kernel(), dim3(static_cast<unsigned>(b.cluster)), b.block, b.cluster, smem, cache(), ok);
        if (e != cudaErrorInvalidClusterSize) return e;
        cudaGetLastError();
        *ok = false;
        return cudaSuccess;
    }
};

template <class Tag>
cudaError_t beam_plan_t(int64_t items, int beams, int64_t cols, int dtype, int k, const argr_caps& caps, BeamPlan* p) {
    const auto fits = [&](const BeamPlan& b, bool* ok) { return BeamCluster<Tag>(beams, static_cast<int>(cols), k, b).fits(b, ok); };
    return fitting_beam_plan(items, beams, cols, dtype, k, caps, fits, p);
}

template <class Tag>
cudaError_t launch_beam_cluster(const BeamProblem& pr, const BeamPlan& b) {
    const BeamCluster<Tag> c(pr.beams, pr.rows.cols, pr.rows.top_k, b);
    const cudaError_t e = c.allow(b);
    if (e != cudaSuccess) return e;
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    return launch_ex_smem(c.kernel(), dim3(static_cast<unsigned>(pr.items * b.cluster)), dim3(b.block), b.cluster, c.smem, p,
                          pr.rows.stream, pr, kLog2E / pr.rows.temperature, b.cluster, b.shift, c.seg_slots);
}

template <class Tag, int BLOCK, int PER_SM>
cudaError_t launch_beam_rows(const BeamProblem& pr, const BeamPlan& b) {
    auto kern = beam_rows_kernel<Tag, BLOCK, PER_SM>;
    static KernelLaunchCache cache;
    const int seg_slots = beam_seg_slots<Tag>(pr.rows.cols, 0);
    const size_t smem = BeamLayout(pr.rows.top_k, 0, seg_slots, kGroupElems<Tag>).total;
    const cudaError_t e = ensure_smem_limit(kern, smem + 1024, cache);
    if (e != cudaSuccess) return e;
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    return launch_ex_smem(kern, dim3(static_cast<unsigned>(pr.rows.rows)), dim3(b.block), 1, smem, p, pr.rows.stream, pr.rows,
                          kLog2E / pr.rows.temperature, seg_slots);
}

template <class Tag>
cudaError_t launch_beam_stream(const BeamProblem& pr, const argr_caps& caps) {
    auto kern = logits_stream_kernel<Tag, kStreamBeam>;
    static KernelLaunchCache cache;
    argr_plan p;
    if (!beam_stream_plan(pr.rows.rows, pr.rows.cols, pr.rows.dtype, pr.rows.top_k, caps, &p)) return cudaErrorInvalidValue;
    const size_t smem = StreamLayout(kStreamBeam, p.block / 32 - p.group, p.group, kWideElems<Tag>, pr.rows.cols, 0).total;
    const cudaError_t e = ensure_smem_limit(kern, smem, cache);
    if (e != cudaSuccess) return e;
    return launch_ex_smem(kern, dim3(static_cast<unsigned>(p.grid_rows)), dim3(p.block), 1, smem, p, pr.rows.stream, pr.rows,
                          kLog2E / pr.rows.temperature, p.group);
}

template <class Tag>
cudaError_t launch_beam_select_t(const BeamProblem& pr, const BeamPlan& b, const argr_caps& caps) {
    if (b.cluster) return launch_beam_cluster<Tag>(pr, b);
    const cudaError_t e = b.stream        ? launch_beam_stream<Tag>(pr, caps)
                          : b.block > 128 ? launch_beam_rows<Tag, 256, 3>(pr, b)
                                          : launch_beam_rows<Tag, 128, 5>(pr, b);
    return e == cudaSuccess ? launch_beam_merge(pr) : e;
}

}  // namespace argr
