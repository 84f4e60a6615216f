// Forward passes over vocabulary rows: log probabilities with entropy and top
// alternatives, and the distillation loss. One cluster of C CTAs (C = 1: one
// CTA) per row reads the row once.
//
// A row is cut into groups of 64 bytes: the 32-byte aligned body, with a head
// and a tail of less than a group around it. Thread t of a CTA takes the groups t,
// t + blockDim, ... of its CTA's range, loads the next one (two 32-byte loads)
// while it adds up the current one, and keeps (m, s, t) in registers: the
// group's largest element first, then one pass of packed binary32 arithmetic
// against a reference that only a larger group maximum moves.
//
// Top alternatives cost the pass one shared-memory word per group, its largest
// element. Groups are contiguous, so in the order (largest element, position)
// the k first groups hold the k first elements: an element of any other group
// comes after the largest elements of k groups. A threshold that k of the
// threads' own largest elements reach (found among 32 of them, or bit by bit with barrier counts)
// picks the groups, usually hardly more than k of them; their elements are read
// again (from L2) and the few that reach the threshold are ranked by counting. Where ties
// make more groups reach it, the k first groups are found exactly.
//
// Bound by latency for few rows: [32, 202048] bf16, in a graph of calls whose inputs rotate past
// L2: 6.1 us (13 MB, 2.1 TB/s), 12 us with the top 20 (the threshold, the second read, the merge over
// the cluster; most of it is code that runs once, so short loops beat unrolled ones; how many ties the
// threshold meets moves it by 3 us). For many rows by instruction issue and the barriers between
// a CTA's phases: [8192, 32000] bf16 92 us, 5.7 TB/s, with the top 20 123 us, 4.2 TB/s; [4096, 50257]
// bf16, top 20, 99 us, 4.2 TB/s; [512, 100003] f16, 32 slots and a tail, 24.6 us, 4.2 TB/s (one wave:
// all CTAs read at first and all finish at last).
#pragma once

#include "logits_common.cuh"

namespace argr {

constexpr int kFwdMaxBlock = 512;
constexpr int kListGroups = 1024; // groups picked by a threshold, at most
// Alternatives that 32 values find a threshold for; more of them bit by bit. Crossing, 32 values / bit by bit,
// us: [128, 50257] f32 9.9 / 10.2 for the top 8, 10.1 / 10.4 16, 10.9 / 10.5 20, 12.0 / 10.8 28; [4096, 50257]
// bf16 89 / 91, 102 / 101, 99 / 102, 105 / 109, and 119 / 109 for 32; [32, 202048] bf16 12.9 / 19.3 for 20, 15.6 / 17.9 for 32.
constexpr int kFewTop = 20;
constexpr int kRankMax = 512;     // candidates ranked by counting, at most

// Add a group whose largest element is `big`. Without ENT, t is left alone (and
// elements of -inf need no bound: exp2 of -inf is 0).
template <class Tag, bool ENT>
__device__ __forceinline__ void add_group(SoftSum& c, const Group<Tag>& g, float big, float scale2) {
    if (big > c.m) {
        if constexpr (ENT) c.rebase(big, scale2);
        else {
            c.s *= ex2((c.m - big) * scale2);
            c.m = big;
        }
    }
    const f32x2 minus = pack2(-c.m, -c.m), scale = pack2(scale2, scale2);
    f32x2 s = 0, t = 0;
#pragma unroll
    for (int i = 0; i < kGroupElems<Tag> / 2; ++i) {
        float lo, hi;
        g.pair(i, lo, hi);
        unpack2(mul2(add2(pack2(lo, hi), minus), scale), lo, hi);
        if constexpr (ENT) {
            lo = max_nan(lo, kYMin);
            hi = max_nan(hi, kYMin);
        }
        const f32x2 e = pack2(ex2(lo), ex2(hi));
        s = add2(s, e);
        if constexpr (ENT) t = fma2(e, pack2(lo, hi), t);
    }
    float a, b;
    unpack2(s, a, b);
    c.s += a + b;
    if constexpr (ENT) {
        unpack2(t, a, b);
        c.t += a + b;
    }
}

// L2 prefetch of a CTA's part: the first kAheadBytes before anything else (also
// before the wait for the previous grid), then, while the part is read, the bytes kAheadBytes ahead of
// the loads. DRAM latency is then hidden without registers for loads in flight. (A caller's plan
// may have more row slots than there are rows.)
constexpr int kAheadBytes = 128 * 1024;
template <class Tag>
__device__ __forceinline__ void prefetch_part(const LogitsProblem& pr, int64_t r, int rank, int ranks) {
    using R = typename Tag::raw;
    if (r >= pr.rows) return;
    const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
    const Part<Tag> part(row, pr.cols, rank, ranks);
    prefetch_l2_range(row + part.begin(), row + part.end(), kAheadBytes);
}

// One pass over a segment. TOP: each slot's largest element goes to big[slot]
// (order32, 0 for an empty slot), the thread's to `most`. DROP: the elements whose
// bits are set in named[] (kGroupElems bits per slot) are left out.
template <class Tag, bool ENT, bool TOP, bool DROP>
__device__ __forceinline__ void scan_segment(SoftSum& c, const typename Tag::raw* row, const Segment<Tag>& sg,
                                             float scale2, unsigned* big, const void* named, unsigned& most,
                                             const typename Tag::raw* part_end) {
    using Bits = std::conditional_t<kGroupElems<Tag> == 32, uint32_t, uint16_t>;
    const Bits* bits = static_cast<const Bits*>(named);
    const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5;
    const typename Tag::raw* body = row + sg.body_lo;
    Group<Tag> a, b;
    int g = t;
    if (g < sg.body) a.load(body + static_cast<int64_t>(g) * kGroupElems<Tag>);
    // the ragged ends, an element per lane: the head by the first warp, the tail by the last
    if (warp == 0 || warp == (nt >> 5) - 1) {
#pragma unroll
        for (int end = 0; end < 2; ++end) {
            if (warp != (end ? (nt >> 5) - 1 : 0)) continue;
            const int slot = end ? sg.body + 1 : 0;
            const int lo = end ? sg.tail_lo : sg.head_lo, n = end ? sg.tail_hi - sg.tail_lo : sg.body_lo - sg.head_lo;
            unsigned o = 0;
            if (lane < n) {
                const float x = widen_elem<Tag>(ld_scalar(row + lo + lane));
                bool in = true;
                if constexpr (DROP) in = !(bits[slot] >> lane & 1u);
                if (in) c.add(x, scale2);
                o = order32(x);
            }
            if constexpr (TOP) {
                o = __reduce_max_sync(0xffffffffu, o);
                if (lane == 0) {
                    big[slot] = o;
                    if (o > most) most = o;
                }
            }
        }
    }
    const auto use = [&](Group<Tag>& v, int at) {
        if constexpr (DROP) {
            const unsigned d = bits[at + 1];
            if (d) v.drop(d);
        }
        const float m = v.largest();
        if constexpr (TOP) {
            const unsigned o = order32(m);
            big[at + 1] = o;
            if (o > most) most = o;
        }
        add_group<Tag, ENT>(c, v, m, scale2);
    };
    const auto ahead = [&](int at) {  // one thread, for the CTA's next pass over nt groups
        if (t != 0) return;
        const char* p = reinterpret_cast<const char*>(body) + static_cast<int64_t>(at) * kGroupBytes + kAheadBytes;
        const int64_t left = (reinterpret_cast<const char*>(part_end) - p) & ~static_cast<int64_t>(15);
        if (left > 0)
            prefetch_l2_bulk(reinterpret_cast<uintptr_t>(p),
                             static_cast<unsigned>(left < nt * kGroupBytes ? left : nt * kGroupBytes));
    };
    while (g < sg.body) {
        ahead(g);
        int next = g + nt;
        if (next < sg.body) b.load(body + static_cast<int64_t>(next) * kGroupElems<Tag>);
        use(a, g);
        g = next;
        if (g >= sg.body) break;
        ahead(g);
        next = g + nt;
        if (next < sg.body) a.load(body + static_cast<int64_t>(next) * kGroupElems<Tag>);
        use(b, g);
        g = next;
    }
}

// ---------------------------------------------------------------------------
// Top alternatives.
// ---------------------------------------------------------------------------
struct TopShared {
    unsigned* big;              // a segment's slots
    unsigned short* list;       // kListGroups slots picked
    unsigned long long* cand;   // room candidates
    unsigned long long* best;   // 2 * ARGR_LOGITS_MAX_TOP keys: the best so far, in order, and a spare
    int* count;                 // 3 counters
    int room;
};

// Sum of an int over the CTA, in every thread.
__device__ __forceinline__ int block_count(int v, int* slot) {
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if (threadIdx.x == 0) *slot = 0;
    __syncthreads();
    if ((threadIdx.x & 31) == 0 && v) atomicAdd(slot, v);
    __syncthreads();
    return *slot;
}

// The k largest of n distinct keys (0: none), in order, into out[0, min(k, n)).
// Contains barriers; src is complete for every thread beforehand.
__device__ __forceinline__ void rank_keys(const unsigned long long* src, int n, int k, unsigned long long* out,
                                          unsigned long long* spare, int* count) {
    const int t = threadIdx.x, nt = blockDim.x;
    if (n > k && (n > kRankMax || n > 4 * nt)) {
        // the k-th largest key, bit by bit; then only the keys that reach it
        unsigned long long at = 0;
        for (int b = 63; b >= 0; --b) {
            const unsigned long long trial = at | 1ull << b;
            int mine = 0;
            for (int i = t; i < n; i += nt) mine += src[i] >= trial;
            const int m = block_count(mine, count);
            if (m >= k) at = trial;
            if (m == k) break;
        }
        __syncthreads();
        if (t == 0) *count = 0;
        __syncthreads();
        for (int i = t; i < n; i += nt)
            if (src[i] >= at && src[i] != 0) {
                const int p = atomicAdd(count, 1);
                if (p < k) spare[p] = src[i];
            }
        __syncthreads();
        src = spare;
        n = *count < k ? *count : k;
    }
    for (int i = t; i < n; i += nt) {
        const unsigned long long key = src[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += src[j] > key;
        if (r < k && key != 0) out[r] = key;
    }
    __syncthreads();
}

// The k largest of `lists` lists (at most 32) of k distinct keys each, every list in
// order and filled up with 0. A list's key at place ceil(k / lists) has that many keys of
// its list before or at it, so at least k keys reach the least of these: only they are
// ranked.
__device__ __forceinline__ void merge_keys(const unsigned long long* src, int lists, int k, unsigned long long* cand,
                                           unsigned long long* out, unsigned long long* spare, int* count) {
    const int lane = threadIdx.x & 31;
    unsigned long long least = lane < lists ? src[lane * k + (k + lists - 1) / lists - 1] : ~0ull;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const unsigned long long d = __shfl_xor_sync(0xffffffffu, least, o);
        if (d < least) least = d;
    }
    __syncthreads();
    if (threadIdx.x == 0) *count = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < lists * k; i += blockDim.x)
        if (src[i] >= least && src[i] != 0) cand[atomicAdd(count, 1)] = src[i];
    __syncthreads();
    const int n = *count;
    __syncthreads();
    rank_keys(cand, n, k, out, spare, count);
}

// Take a scanned segment into the best keys so far; returns their number. `most`
// is the thread's largest element of the segment (order32). Begins with a barrier
// that completes the segment's slots, and ends with one.
template <class Tag>
__device__ __forceinline__ int take_segment(const typename Tag::raw* row, const Segment<Tag>& sg, int k, int have,
                                            unsigned most, const TopShared& sh) {
    using R = typename Tag::raw;
    constexpr int E = kGroupElems<Tag>, P = 16 / static_cast<int>(sizeof(R));
    const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5, warps = nt >> 5;
    const int slots = sg.slots();
    const auto usable = [&](unsigned v) {  // as a threshold
        if (have == k) v = max(v, static_cast<unsigned>(sh.best[k - 1] >> 32));
        return v > 1 && v < kOrderNegInf ? kOrderNegInf : max(v, 1u);  // (nothing lies between a NaN and -inf)
    };
    // A value that at least k elements reach (or 1: every element does). Few alternatives: the k-th
    // largest of 32 values, each the largest of a 32nd of the threads (1.5 k elements or fewer reach it,
    // as a rule); one barrier, and every warp ranks them itself. More: the k-th largest of the threads'
    // values or near it, bit by bit, a barrier each.
    if (t < 3) sh.count[t] = 0;
    unsigned at = 0;
    if (k <= kFewTop) {
        unsigned* tops = reinterpret_cast<unsigned*>(sh.cand);  // (all have read it, a barrier ago)
        const int share = warps > 1 ? 1 << (32 - __clz(warps - 1)) : 1;  // threads, a power of two
        unsigned v = most;
        for (int o = share >> 1; o >= 1; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        if ((lane & (share - 1)) == 0) tops[t / share] = v;
        if (t < 32 && t >= nt / share) tops[t] = 0u;
        __syncthreads();
        v = tops[lane];
        int over = 0;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const uint4 o = *reinterpret_cast<const uint4*>(tops + j);
            over += (o.x > v) + (o.y > v) + (o.z > v) + (o.w > v);
        }
        at = __reduce_min_sync(0xffffffffu, over < k ? v : ~0u);
    } else {
        for (int b = 31; b >= 0; --b) {
            const unsigned trial = at | 1u << b;
            const int n = __syncthreads_count(most >= trial);
            if (n < k) continue;
            at = trial;
            if (n <= k + k / 4 + 2) break;
        }
    }
    at = usable(at);
    bool exact = false, again = false;
    // Mode 0 looks into every slot that reaches `at`, or exceeds it where many equal
    // it and k exceed it. Mode 1, where fewer than k slots exceed it and many equal it (a masked row, whose -inf fill the places that its
    // few numbers leave): into those that exceed it, and takes the first elements that equal it in
    // order. Mode 2, where still too many reach it: into the k first by (largest element,
    // position), found exactly.
    int mode = 0, cut = slots;  // cut: of the slots whose largest element equals `at`, those up to here
    for (;; again = true) {
        if (mode == 2) {
            at = 0;
            for (int b = 31; b >= 0; --b) {
                const unsigned trial = at | 1u << b;
                int mine = 0;
                for (int i = t; i < slots; i += nt) mine += sh.big[i] >= trial;
                if (block_count(mine, sh.count) >= k) at = trial;
            }
            int lo = 0, hi = slots - 1;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                int mine = 0;
                for (int i = t; i < slots; i += nt) mine += sh.big[i] > at || (sh.big[i] == at && i <= mid);
                if (block_count(mine, sh.count) >= k) hi = mid;
                else lo = mid + 1;
            }
            cut = lo;
        }
        if (again) {
            __syncthreads();
            if (t < 3) sh.count[t] = 0;
            __syncthreads();
        }
        int equal = 0;
        if (most >= at) {  // a thread looks at the slots that it wrote
            const auto picks = [&](int i) {
                const unsigned o = sh.big[i];
                equal += o == at;
                return o > at || (o == at && i <= cut && mode != 1);
            };
            for (int g = t; g < sg.body;) {
                unsigned in = 0;
                const int first = g;
#pragma unroll 4
                for (int u = 0; u < 32 && g < sg.body; ++u, g += nt) in |= static_cast<unsigned>(picks(g + 1)) << u;
                if (in == 0) continue;
                int p = atomicAdd(&sh.count[0], __popc(in));
                for (; in; in &= in - 1, ++p)
                    if (p < kListGroups) sh.list[p] = static_cast<unsigned short>(first + (__ffs(in) - 1) * nt + 1);
            }
            // the ragged ends: lane 0 of the first warp and of the last
            for (int end = 0; end < 2; ++end) {
                if (t != (end ? nt - 32 : 0) || !picks(end ? sg.body + 1 : 0)) continue;
                const int p = atomicAdd(&sh.count[0], 1);
                if (p < kListGroups) sh.list[p] = static_cast<unsigned short>(end ? sg.body + 1 : 0);
            }
        }
        if (mode == 0 && equal) atomicAdd(&sh.count[2], equal);
        __syncthreads();
        const int picked = sh.count[0];
        if (mode == 0) {
            const int over = picked - sh.count[2];  // slots that exceed it
            if (over < picked && (picked > 2 * k + 32 || picked * E > sh.room)) {
                if (over < k) mode = 1;
                else ++at;
                continue;
            }
        }
        const auto too_many = [&]() {  // first a better threshold, then the exact way
            if (exact) {
                mode = 2;
            } else {
                unsigned v = 0;  // the k-th largest of the threads' values
                for (int b = 31; b >= 0; --b)
                    if (__syncthreads_count(most >= (v | 1u << b)) >= k) v |= 1u << b;
                at = usable(v);
                exact = true;
                mode = 0;
            }
        };
        if (picked > kListGroups && mode != 2) {
            too_many();
            continue;
        }
        // the best so far that reach `at`: k elements do, so the others are out, and must not stand in for
        // elements that equal it
        for (int i = t; i < have; i += nt)
            if (static_cast<unsigned>(sh.best[i] >> 32) >= at) sh.cand[atomicAdd(&sh.count[1], 1)] = sh.best[i];
        // the picked slots' elements that reach `floor`, 16 bytes per lane, 8 slots per warp at a time
        const unsigned floor = at + (mode == 1);
        for (int p0 = 8 * warp; p0 < picked; p0 += 8 * warps) {
            const int p = p0 + (lane >> 2);
            if (p >= picked) continue;
            const int slot = sh.list[p];
            if (slot < 1 || slot > sg.body) {  // a ragged end, element by element
                int first, n;
                sg.range(slot, first, n);
                for (int i = lane & 3; i < n; i += 4) {
                    const unsigned long long key = order_key(widen_elem<Tag>(ld_scalar(row + first + i)), first + i);
                    if (static_cast<unsigned>(key >> 32) < floor) continue;
                    const int q = atomicAdd(&sh.count[1], 1);
                    if (q < sh.room) sh.cand[q] = key;
                }
                continue;
            }
            const int lo = sg.body_lo + (slot - 1) * E + (lane & 3) * P;
            const uint4 w = ld_stream16(row + lo);
            const auto elem = [&](int e) {
                if constexpr (P == 4) {
                    return __uint_as_float(e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w);
                } else {
                    const uint32_t v = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
                    return Tag::widen(static_cast<uint16_t>(e & 1 ? v >> 16 : v & 0xffffu));
                }
            };
            unsigned hits = 0;
#pragma unroll
            for (int e = 0; e < P; ++e) hits |= static_cast<unsigned>(order32(elem(e)) >= floor) << e;
            if (hits == 0) continue;
            int q = atomicAdd(&sh.count[1], __popc(hits));
            for (; hits; hits &= hits - 1, ++q) {
                const int e = __ffs(hits) - 1;
                if (q < sh.room) sh.cand[q] = order_key(elem(e), lo + e);
            }
        }
        __syncthreads();
        if (sh.count[1] > sh.room && mode != 2) {
            too_many();
            continue;
        }
        if (mode == 1 && sh.count[1] < k && t < 32) {
            // the first warp fills up to k, in order, from the slots that reach `at` (a warp that still
            // reads the count above sees at most k, which fits)
            int n = sh.count[1];
            for (int s0 = 0; s0 < slots && n < k; s0 += 32) {
                unsigned hit = __ballot_sync(0xffffffffu, s0 + lane < slots && sh.big[s0 + lane] >= at);
                while (hit && n < k) {
                    int lo, size;
                    sg.range(s0 + __ffs(hit) - 1, lo, size);
                    hit &= hit - 1;
                    const float x = lane < size ? widen_elem<Tag>(ld_scalar(row + lo + lane)) : 0.0f;
                    const bool in = lane < size && order32(x) == at;
                    const unsigned got = __ballot_sync(0xffffffffu, in);
                    const int q = n + __popc(got & ((1u << lane) - 1u));
                    if (in && q < k) sh.cand[q] = order_key(x, lo + lane);
                    n += __popc(got);
                }
            }
            if (lane == 0) sh.count[1] = n < k ? n : k;
        }
        if (mode == 1) __syncthreads();
        break;
    }
    const int n = sh.count[1] < sh.room ? sh.count[1] : sh.room;
    rank_keys(sh.cand, n, k, sh.best, sh.best + ARGR_LOGITS_MAX_TOP, sh.count);
    return n < k ? n : k;
}

// ---------------------------------------------------------------------------
// Clusters: CTAs hand what they have to CTA 0.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void st_cluster(unsigned addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(unsigned addr, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
// Before the first write into another CTA: that it runs, and has consumed what
// was written for the row before. Orders nothing, so it waits for no memory operation.
__device__ __forceinline__ void cluster_ready() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

constexpr int kMaxRanks = 16;

// Shared memory of the forward kernels past their static part.
inline __host__ __device__ int cand_room(int k, int group_elems) {
    const int n = k * group_elems + k;
    return n < kRankMax ? kRankMax : n;
}

template <class Tag, bool TOP, int BLOCK, int PER_SM>
__global__ void __launch_bounds__(BLOCK, PER_SM) logprobs_kernel(const LogitsProblem pr, float scale2, int ranks,
                                                                   int seg_slots) {
    using R = typename Tag::raw;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ float red[96];
    __shared__ float parts[3 * kMaxRanks];
    __shared__ float row_m, row_ln_s;
    __shared__ int count[3];
    const int t = threadIdx.x;
    const int rank = static_cast<int>(blockIdx.x % ranks);
    const int k = pr.top_k;
    TopShared sh;
    unsigned long long* gathered = nullptr;  // CTA 0: every CTA's best
    if constexpr (TOP) {
        sh.room = cand_room(k, kGroupElems<Tag>);
        sh.big = reinterpret_cast<unsigned*>(dyn);  // (seg_slots is a multiple of 4: `cand` is aligned to 16 bytes)
        sh.cand = reinterpret_cast<unsigned long long*>(sh.big + seg_slots);
        sh.best = sh.cand + sh.room;
        gathered = sh.best + 2 * ARGR_LOGITS_MAX_TOP;
        sh.list = reinterpret_cast<unsigned short*>(gathered + (ranks > 1 ? ranks * k : 0));
        sh.count = count;
    }
    allow_dependents();
    prefetch_part<Tag>(pr, blockIdx.x / ranks, rank, ranks);
    grid_dependency_wait();
    const int64_t slots = gridDim.x / ranks;
    for (int64_t r = blockIdx.x / ranks; r < pr.rows; r += slots) {
        if (ranks > 1) cluster_ready();
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        int64_t tok = -1;
        float tok_x = 0.0f;
        if (rank == 0 && t == 0 && pr.logprob) {
            tok = pr.tokens[r];
            if (tok >= 0 && tok < pr.cols) tok_x = widen_elem<Tag>(ld_scalar(row + tok));
        }
        const Part<Tag> part(row, pr.cols, rank, ranks);
        SoftSum c;
        int have = 0;
        for (int at = 0;;) {
            const Segment<Tag> sg = part.segment(at);
            SoftSum d;
            unsigned most = 0;
            scan_segment<Tag, true, TOP, false>(d, row, sg, scale2, sh.big, nullptr, most, row + part.end());
            c.join(d, scale2);
            if constexpr (TOP) {
                if (at + sg.body >= part.count) softsum_to(c, scale2, red);
                have = take_segment<Tag>(row, sg, k, have, most, sh);
            }
            at += sg.body;
            if (at >= part.count) break;
        }
        if constexpr (!TOP) {
            softsum_to(c, scale2, red);
            __syncthreads();
        }
        if (t < 32) c = softsum_from(scale2, red);
        if (ranks > 1) {
            cluster_wait();
            if (t == 0) {
                const unsigned at = cluster_addr(smem_u32(parts), 0);
                st_cluster(at + 4 * rank, c.m);
                st_cluster(at + 4 * (kMaxRanks + rank), c.s);
                st_cluster(at + 4 * (2 * kMaxRanks + rank), c.t);
            }
            if constexpr (TOP) {
                const unsigned at = cluster_addr(smem_u32(gathered), 0) + 8 * rank * k;
                for (int i = t; i < k; i += blockDim.x) st_cluster(at + 8 * i, i < have ? sh.best[i] : 0ull);
            }
            cluster_arrive();
            cluster_wait();
            if (rank != 0) continue;
            if (t < 32) {
                SoftSum d;
                if (t < ranks) {
                    d.m = parts[t];
                    d.s = parts[kMaxRanks + t];
                    d.t = parts[2 * kMaxRanks + t];
                }
                c = warp_softsum(d, scale2);
            }
            if constexpr (TOP) {
                merge_keys(gathered, ranks, k, sh.cand, sh.best, sh.best + ARGR_LOGITS_MAX_TOP, count);
            }
        }
        if (t == 0) {
            const float ln_s = c.empty() ? neg_inf() : logf(c.s);
            const float h = kLn2 * (log2f(c.s) - c.t / c.s);
            const float entropy = c.empty() ? 0.0f : (h < 0.0f ? 0.0f : h);
            if (pr.logprob) {
                float lp = 0.0f;
                if (tok >= pr.cols) lp = quiet_nan();
                else if (tok >= 0) lp = c.empty() ? neg_inf() : (tok_x - c.m) / pr.temperature - ln_s;
                pr.logprob[r] = lp;
            }
            if (pr.entropy) pr.entropy[r] = entropy;
            if (pr.lse) pr.lse[r] = c.empty() ? neg_inf() : c.m / pr.temperature + ln_s;
            if (pr.stats) pr.stats[r] = make_float4(c.empty() ? neg_inf() : c.m, ln_s, entropy, 0.0f);
            row_m = c.m;
            row_ln_s = ln_s;
        }
        if constexpr (TOP) {
            __syncthreads();
            for (int i = t; i < k; i += blockDim.x) {
                const unsigned long long key = sh.best[i];
                const float v = order_value(static_cast<unsigned>(key >> 32));
                if (pr.top_ids) pr.top_ids[r * k + i] = key_index(key);
                if (pr.top_logprobs)
                    pr.top_logprobs[r * k + i] =
                        row_ln_s == neg_inf() ? neg_inf() : (v - row_m) / pr.temperature - row_ln_s;
            }
            __syncthreads();
        } else if (ranks == 1 && r + slots < pr.rows) {
            __syncthreads();  // `red` has been read
        }
    }
}

// ---------------------------------------------------------------------------
// Distillation. With the tail, the elements that slots name are left out of the
// pass (a bit per element in shared memory) and added once from the slots, so
// that the tail's sum is a sum of its own.
// ---------------------------------------------------------------------------
// The bits of a segment's elements that slots name (the slots are complete after
// the first barrier).
template <class Tag>
__device__ __forceinline__ void name_segment(const Segment<Tag>& sg, const Slots& sl, int slots, unsigned* named) {
    constexpr int E = kGroupElems<Tag>;
    const int t = threadIdx.x, nt = blockDim.x;
    __syncthreads();
    for (int i = t; i < (sg.slots() * E + 31) / 32; i += nt) named[i] = 0u;
    __syncthreads();
    for (int i = t; i < slots; i += nt) {
        const int j = sl.id[i];
        if (j < sg.head_lo || j >= sg.tail_hi) continue;
        const int bit = j < sg.body_lo    ? j - sg.head_lo
                        : j >= sg.tail_lo ? (sg.body + 1) * E + (j - sg.tail_lo)
                                          : E + (j - sg.body_lo);
        atomicOr(&named[bit >> 5], 1u << (bit & 31));
    }
    __syncthreads();
}

template <class Tag, bool TAIL>
__global__ void __launch_bounds__(kFwdMaxBlock, 2) distill_kernel(const LogitsProblem pr, float scale2, int ranks,
                                                                  int seg_slots) {
    using R = typename Tag::raw;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ float red[96];
    __shared__ float parts[2 * kMaxRanks];
    const int t = threadIdx.x;
    const int rank = static_cast<int>(blockIdx.x % ranks);
    const Slots sl(dyn, pr.slots);
    unsigned* named = reinterpret_cast<unsigned*>(dyn + Slots::bytes(pr.slots));
    allow_dependents();
    prefetch_part<Tag>(pr, blockIdx.x / ranks, rank, ranks);
    grid_dependency_wait();
    const int64_t row_slots = gridDim.x / ranks;
    for (int64_t r = blockIdx.x / ranks; r < pr.rows; r += row_slots) {
        if (ranks > 1) cluster_ready();
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        if (TAIL || rank == 0) load_slots<Tag>(pr, r, row, 0, rank == 0 ? pr.cols : 0, sl);
        const Part<Tag> part(row, pr.cols, rank, ranks);
        SoftSum c;  // without the tail: the row; with it: the indices that no slot names
        for (int at = 0;;) {
            const Segment<Tag> sg = part.segment(at);
            if constexpr (TAIL) {
                name_segment<Tag>(sg, sl, pr.slots, named);
            }
            SoftSum d;
            unsigned most = 0;
            scan_segment<Tag, false, false, TAIL>(d, row, sg, scale2, nullptr, named, most, row + part.end());
            d.t = 0.0f;
            c.join(d, scale2);
            at += sg.body;
            if (at >= part.count) break;
        }
        c = block_softsum(c, scale2, red);
        if (ranks > 1) {
            cluster_wait();
            if (t == 0) {
                const unsigned at = cluster_addr(smem_u32(parts), 0);
                st_cluster(at + 4 * rank, c.m);
                st_cluster(at + 4 * (kMaxRanks + rank), c.s);
            }
            cluster_arrive();
            cluster_wait();
            if (rank != 0) continue;
            if (t < 32) {
                SoftSum d;
                if (t < ranks) {
                    d.m = parts[t];
                    d.s = parts[kMaxRanks + t];
                }
                c = warp_softsum(d, scale2);
            }
        }
        finish_distill<Tag, TAIL>(pr, r, c, scale2, red, sl);
    }
}

}  // namespace argr
