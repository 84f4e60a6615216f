// Forward passes over many vocabulary rows: persistent CTAs that never stop
// reading.
//
// Most warps of a CTA stream its rows, one after the other: 128-byte groups, a
// warp 4 KB at a time, the next 4 KB (of this row or the next) prefetched into
// L2. At the end of a row each warp leaves its softmax sums (and, for
// alternatives, the groups' largest elements) in a buffer and goes on with the next row.
// The last F warps finish rows in turn: join the sums, pick the alternatives or
// take the loss, and prepare the buffer for the row that will use it next. Row i
// uses buffer i mod (F + 1) and finisher i mod F; a pair of named barriers per
// buffer hands it over ("full" from the streamers, "free" back), so that no
// streaming warp waits as long as a finish takes less than F rows' time. A named barrier
// counts warps, whoever they are, and successive rows of a buffer belong to different finishers: each
// waits for its row only after the finisher of the row before has met the streamers there ("turn", a barrier per
// pair of neighbours). Rows become complete in this order, so it delays nobody. The 4 KB
// tiles of successive rows are dealt to the warps in one sequence, so that rows of few tiles keep
// all warps equally busy.
//
// The streaming loop is bound by instruction issue before it is by memory for
// 16-bit types (5.5 thread instructions per element at best, 11 elements per SM
// and cycle at the copy rate), hence: wide groups, packed arithmetic, and a
// reference for the exponentials that moves only when a group exceeds it by more
// than 2^kSlack.
//
// [2048, 202048] bf16: 134 us in a graph of calls, 6.2 TB/s; 143, 151, 160 us with the top 1, 20, 64 (the finishing warps
// take issue slots, and the last rows' finish is not hidden); distillation, 64 slots and a tail,
// 145 us. [2048, 100000] f32 138 us, 6.0 TB/s; [1500, 65537] f32, top 1, 70 us, 5.6 TB/s. A CTA of 256
// threads and twice as many of them, and picked groups staged in shared memory for the finisher,
// were slower.
#pragma once

#include "logits_forward.cuh"

namespace argr {

constexpr float kSlack = 8.0f;        // in powers of two; sums stay far below overflow
constexpr int kStreamCands = 1024;    // candidates for alternatives, at most
constexpr int kStreamList = 640;      // slots looked into at a time, at most
constexpr int kRankKeys = 192;        // keys that the finisher ranks by counting, at most (and its spare keys)
enum StreamMode { kStreamSums = 0, kStreamTop = 1, kStreamLoss = 2, kStreamLossTail = 3, kStreamBeam = 4 };
inline __host__ __device__ constexpr bool stream_top(int mode) { return mode == kStreamTop || mode == kStreamBeam; }

template <class Tag> constexpr int kWideElems = 2 * kGroupElems<Tag>;

// Barriers of a buffer: one warp on the finishers' side; of a finisher: it waits, the one before it arrives.
constexpr int kMaxFinishers = 3;
static_assert(1 + 2 * (kMaxFinishers + 1) + kMaxFinishers <= 16, "named barriers of a CTA");
__device__ __forceinline__ int full_bar(int buffer) { return 1 + 2 * buffer; }
__device__ __forceinline__ int free_bar(int buffer) { return 2 + 2 * buffer; }
__device__ __forceinline__ int turn_bar(int finisher) { return 1 + 2 * (kMaxFinishers + 1) + finisher; }
__device__ __forceinline__ void bar_sync(int id, int threads) {
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
    __syncwarp();
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Whether a beam's row is looked at (argreduce_beam_select).
__device__ __forceinline__ bool beam_looks(const LogitsProblem& pr, int64_t r) {
    return pr.beam_scores[r] != neg_inf() && !(pr.beam_ended && pr.beam_ended[r]);
}

// A row in wide groups. Slot 0 is its head, slots 1 .. body the groups, slot body + 1 its tail.
template <class Tag>
struct WideRow {
    const typename Tag::raw* p;
    int align, body, cols;
    __device__ __forceinline__ WideRow(const LogitsProblem& pr, int64_t r) {
        p = static_cast<const typename Tag::raw*>(pr.x) + r * pr.row_stride;
        cols = pr.cols;
        const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) & 31u);
        align = static_cast<int>(((32u - off) & 31u) / sizeof(typename Tag::raw));
        if (align > cols) align = cols;
        body = (cols - align) / kWideElems<Tag>;
    }
    __device__ __forceinline__ int tail() const { return align + body * kWideElems<Tag>; }
    __device__ __forceinline__ int slots() const { return body + 2; }
    __device__ __forceinline__ int slot_begin(int s) const { return s == 0 ? 0 : align + (s - 1) * kWideElems<Tag>; }
    __device__ __forceinline__ int slot_size(int s) const {
        return s == 0 ? align : s <= body ? kWideElems<Tag> : cols - tail();
    }
    // the bit of an element: slots of kWideElems bits
    __device__ __forceinline__ int bit(int j) const {
        return j < align ? j : kWideElems<Tag> + (j - align);
    }
};

// Layout of a CTA's shared memory.
struct StreamLayout {
    int streamers;  // streaming warps
    int finishers;  // finishing warps; one buffer more
    int slots;      // room for a row's slots
    int k;          // distillation slots
    size_t sums, most, tile, big, named, teacher, buffer;  // offsets in a buffer, and its size
    size_t cand, list, total;
    __host__ __device__ StreamLayout(int mode, int warps, int fin, int wide_elems, int cols, int n) {
        streamers = warps;
        finishers = fin;
        k = n;
        slots = (cols / wide_elems + 2 + 3) / 4 * 4;
        size_t at = 0;
        sums = at;
        at += 4 * sizeof(float) * static_cast<size_t>(warps);
        most = at;
        if (stream_top(mode)) at += 4 * 32 * static_cast<size_t>(warps);
        tile = at;
        if (stream_top(mode)) at += 4 * static_cast<size_t>((slots / 32 + 1 + 3) / 4 * 4);
        big = at;
        if (stream_top(mode)) at += 4 * static_cast<size_t>(slots);
        named = at;
        if (mode == kStreamLossTail) at += (static_cast<size_t>(slots) * wide_elems / 8 + 15) / 16 * 16;
        teacher = at;
        if (mode == kStreamLoss || mode == kStreamLossTail) at += Slots::bytes(n);
        buffer = (at + 15) / 16 * 16;
        cand = (fin + 1) * buffer;
        list = cand + (stream_top(mode) ? 8 * static_cast<size_t>(fin) * (kStreamCands + kRankKeys) : 0);
        total = list + (stream_top(mode) ? 2 * static_cast<size_t>(fin) * kStreamList : 0);
    }
};

// ---------------------------------------------------------------------------
// Streaming warps.
// ---------------------------------------------------------------------------
// A wide group against the thread's sums; top is the largest element so far,
// c.m the reference.
template <class Tag, bool ENT>
__device__ __forceinline__ void add_wide(SoftSum& c, const Group<Tag>& a, const Group<Tag>& b, float big,
                                         float scale2) {
    if ((big - c.m) * scale2 > kSlack) {
        if constexpr (ENT) c.rebase(big, scale2);
        else {
            c.s *= ex2((c.m - big) * scale2);
            c.m = big;
        }
    }
    const f32x2 minus = pack2(-c.m, -c.m), scale = pack2(scale2, scale2);
    f32x2 s = 0, t = 0;
#pragma unroll
    for (int i = 0; i < kGroupElems<Tag>; ++i) {
        float lo, hi;
        (i < kGroupElems<Tag> / 2 ? a : b).pair(i % (kGroupElems<Tag> / 2), lo, hi);
        unpack2(mul2(add2(pack2(lo, hi), minus), scale), lo, hi);
        if constexpr (ENT) {
            lo = max_nan(lo, kYMin);
            hi = max_nan(hi, kYMin);
        }
        const f32x2 e = pack2(ex2(lo), ex2(hi));
        s = add2(s, e);
        if constexpr (ENT) t = fma2(e, pack2(lo, hi), t);
    }
    float p, q;
    unpack2(s, p, q);
    c.s += p + q;
    if constexpr (ENT) {
        unpack2(t, p, q);
        c.t += p + q;
    }
}

template <class Tag, int MODE>
__device__ __forceinline__ void stream_rows(const LogitsProblem& pr, float scale2, const StreamLayout& lay,
                                            unsigned char* dyn) {
    using R = typename Tag::raw;
    constexpr bool ENT = MODE == kStreamSums || MODE == kStreamTop;
    constexpr bool TOP = stream_top(MODE), DROP = MODE == kStreamLossTail;
    constexpr int E = kWideElems<Tag>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = (lay.streamers + 1) * 32;
    int at = 0;        // the row's buffer
    int mine = warp;   // this warp's next tile (32 groups), counted from the row's first
    for (int64_t r = blockIdx.x; r < pr.rows; r += gridDim.x, at = at < lay.finishers ? at + 1 : 0) {
        unsigned char* buf = dyn + at * lay.buffer;
        unsigned* big_at = reinterpret_cast<unsigned*>(buf + lay.big);
        const WideRow<Tag> row(pr, r);
        const R* body = row.p + row.align;
        const bool look = MODE != kStreamBeam || beam_looks(pr, r);
        const int tiles = look ? (row.body + 31) >> 5 : 0;
        bar_sync(free_bar(at), threads);  // the buffer is free (and holds this row's bits)
        SoftSum c;
        float top = neg_inf();
        unsigned most = 0;
        for (; mine < tiles; mine += lay.streamers) {
            const int g = mine * 32 + lane;
            unsigned o = 0;
            if (g < row.body) {
            Group<Tag> a, b;
            const R* p = body + static_cast<int64_t>(g) * E;
            a.load(p);
            b.load(p + kGroupElems<Tag>);
            if (lane == 0) {
                // this warp's next tile: in this row, or in the next
                int tile = mine + lay.streamers;
                const R* q = body;
                int64_t elems = row.cols - row.align;
                if (tile >= tiles && r + gridDim.x < pr.rows) {
                    const WideRow<Tag> next(pr, r + gridDim.x);
                    tile -= tiles;
                    q = next.p + next.align;
                    elems = next.cols - next.align;
                }
                const int64_t first = static_cast<int64_t>(tile) * (32 * E);
                const int64_t left = (elems - first) * static_cast<int64_t>(sizeof(R)) & ~static_cast<int64_t>(15);
                if (left > 0)
                    prefetch_l2_bulk(reinterpret_cast<uintptr_t>(q + first), static_cast<unsigned>(left < 4096 ? left : 4096));
            }
            if constexpr (DROP) {
                if constexpr (E == 64) {
                    const uint2 bits = reinterpret_cast<const uint2*>(buf + lay.named)[g + 1];
                    if (bits.x) a.drop(bits.x);
                    if (bits.y) b.drop(bits.y);
                } else {
                    const unsigned bits = reinterpret_cast<const unsigned*>(buf + lay.named)[g + 1];
                    if (bits) {
                        a.drop(bits & 0xffffu);
                        b.drop(bits >> 16);
                    }
                }
            }
            const float big = fmaxf(a.largest(), b.largest());
            top = fmaxf(top, big);
            if constexpr (TOP) {
                o = order32(big);
                big_at[g + 1] = o;
                if (o > most) most = o;
            }
            add_wide<Tag, ENT>(c, a, b, big, scale2);
            }
            if constexpr (TOP) {
                o = __reduce_max_sync(0xffffffffu, o);
                if (lane == 0) reinterpret_cast<unsigned*>(buf + lay.tile)[mine] = o;
            }
        }
        mine -= tiles;
        // the ragged ends: the head with the first warp, the tail with the last
        if (look && (warp == 0 || warp == lay.streamers - 1)) {
#pragma unroll
            for (int end = 0; end < 2; ++end) {
                if (warp != (end ? lay.streamers - 1 : 0)) continue;
                const int slot = end ? row.body + 1 : 0;
                const int lo = row.slot_begin(slot), n = row.slot_size(slot);
                unsigned o = 0;
                for (int j = lane; j < n; j += 32) {
                    const float x = widen_elem<Tag>(ld_scalar(row.p + lo + j));
                    if constexpr (DROP) {
                        const int bit = slot * E + j;
                        if (reinterpret_cast<const unsigned*>(buf + lay.named)[bit >> 5] >> (bit & 31) & 1u) continue;
                    }
                    c.add(x, scale2);
                    top = fmaxf(top, x);
                    const unsigned ox = order32(x);
                    if (ox > o) o = ox;
                }
                if constexpr (TOP) {
                    o = __reduce_max_sync(0xffffffffu, o);
                    if (lane == 0) {
                        big_at[slot] = o;
                        if (o > most) most = o;
                    }
                }
            }
        }
        // the warp's sums, against its largest element
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (top == neg_inf()) top = -FLT_MAX;
        if constexpr (!ENT) c.t = 0.0f;
        c.rebase(top, scale2);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            c.s += __shfl_xor_sync(0xffffffffu, c.s, o);
            if constexpr (ENT) c.t += __shfl_xor_sync(0xffffffffu, c.t, o);
        }
        if (lane == 0) reinterpret_cast<float4*>(buf + lay.sums)[warp] = make_float4(c.m, c.s, c.t, 0.0f);
        if constexpr (TOP) reinterpret_cast<unsigned*>(buf + lay.most)[threadIdx.x] = most;
        bar_arrive(full_bar(at), threads);  // the row is complete
    }
}

// ---------------------------------------------------------------------------
// The finishing warp.
// ---------------------------------------------------------------------------
__device__ __forceinline__ SoftSum joined_sums(const unsigned char* sums, int n, float scale2) {
    const int lane = threadIdx.x & 31;
    SoftSum c;
    if (lane < n) {
        const float4 v = reinterpret_cast<const float4*>(sums)[lane];
        c.m = v.x;
        c.s = v.y;
        c.t = v.z;
    }
    return warp_softsum(c, scale2);
}

// The k largest of n distinct keys to the front of `keys` (any order), by a bitwise search
// for the k-th; the k-th key is returned. n > k.
__device__ __forceinline__ unsigned long long warp_prune(unsigned long long* keys, int n, int k,
                                                         unsigned long long* spare) {
    const int lane = threadIdx.x & 31;
    unsigned long long at = 0;
    for (int b = 63; b >= 0; --b) {
        const unsigned long long trial = at | 1ull << b;
        int mine = 0;
        for (int i = lane; i < n; i += 32) mine += keys[i] >= trial;
        const int m = __reduce_add_sync(0xffffffffu, mine);
        if (m >= k) at = trial;
        if (m == k) break;
    }
    int kept = 0;
    unsigned long long least = ~0ull;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const unsigned long long key = i0 + lane < n ? keys[i0 + lane] : 0;
        const bool keep = key >= at && key != 0;
        const unsigned got = __ballot_sync(0xffffffffu, keep);
        const int p = kept + __popc(got & ((1u << lane) - 1u));
        if (keep && p < k) {
            spare[p] = key;
            if (key < least) least = key;
        }
        kept += __popc(got);
    }
    __syncwarp();
    for (int i = lane; i < k; i += 32) keys[i] = spare[i];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const unsigned long long d = __shfl_xor_sync(0xffffffffu, least, o);
        if (d < least) least = d;
    }
    __syncwarp();
    return least;
}

__device__ __forceinline__ uint32_t at4(const uint4& w, int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }

// A value (order32) that at least k of a warp's V * 32 values reach, or 0.
template <int V>
__device__ __forceinline__ unsigned warp_threshold(const unsigned (&v)[V], int k) {
    const auto reach = [&](unsigned trial) {
        int mine = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) mine += v[i] >= trial;
        return __reduce_add_sync(0xffffffffu, mine);
    };
    // from the first bit on in which those that are not 0 differ
    unsigned low = ~0u, high = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        low = min(low, v[i] - 1u);
        high = max(high, v[i]);
    }
    low = __reduce_min_sync(0xffffffffu, low) + 1u;
    high = __reduce_max_sync(0xffffffffu, high);
    int b = 31 - __clz(low ^ high);  // -1: none
    unsigned at = b < 0 ? high : b < 31 ? high & ~((2u << b) - 1u) : 0u;
    if (high == 0 || reach(at > 1u ? at : 1u) < k) return 0;
    for (; b >= 0; --b) {
        const unsigned trial = at | 1u << b;
        const int n = reach(trial);
        if (n >= k) {
            at = trial;
            if (n <= k + k / 8 + 2) break;
        }
    }
    return at;
}

// The position of each lane's first of `mine` items among all lanes', from *n on,
// which moves past them.
__device__ __forceinline__ int warp_places(int mine, int* n) {
    const int lane = threadIdx.x & 31;
    const unsigned one = __ballot_sync(0xffffffffu, mine != 0), more = __ballot_sync(0xffffffffu, mine > 1);
    int first = *n + __popc(one & ((1u << lane) - 1u)), all = __popc(one);
    if (more) {  // rarely: whole sums
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int d = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += d;
        }
        first = *n + sum - mine;
        all = __shfl_sync(0xffffffffu, sum, 31);
    }
    *n += all;
    return first;
}

// The k largest of n <= 32 R keys (0: none) to their places in `out`, by counting; every lane holds R.
template <int R>
__device__ __forceinline__ void rank_lane_keys(const unsigned long long* keys, int n, int k, unsigned long long* out) {
    const int lane = threadIdx.x & 31;
    unsigned long long mine[R];
    int rank[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
        mine[u] = lane + 32 * u < n ? keys[lane + 32 * u] : 0ull;
        rank[u] = 0;
    }
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
        const unsigned long long other = keys[j];
#pragma unroll
        for (int u = 0; u < R; ++u) rank[u] += other > mine[u];
    }
#pragma unroll
    for (int u = 0; u < R; ++u)
        if (mine[u] != 0 && rank[u] < k) out[rank[u]] = mine[u];
}

// The row's k first alternatives, in order, as keys in cand[kStreamCands, + k),
// from the largest elements of its slots (big), of its tiles of 32 groups (tile)
// and of the streaming threads (most). The finisher shares its scheduler with
// streaming warps and works alone, so its chains of dependent instructions count, and branches, whose code is
// mostly not at hand: a tile's 32 slots are compared by one lane without any, 128 units of 16 bytes are looked at
// side by side, and their hits get places together. A last row's finish, 36 slots picked for the top 32 of
// [., 202048]: threshold 1.0 us, slots 2.8, units 3.7, order 0.7. (128 slots at a time, with a ballot for each, and
// units of 32 lanes with places of their own took 4.9 and 4.1, 7.7 and 18 for the top 128, now 4 and 15; picked slots
// prefetched in bulk, each by its lane, 9 in place of 2.8.)
template <class Tag>
__device__ __forceinline__ void warp_top(const WideRow<Tag>& row, int k, const unsigned* big, const unsigned* tile,
                                         const unsigned* most, int streamers, unsigned long long* cand,
                                         unsigned short* list) {
    constexpr int P = 16 / static_cast<int>(sizeof(typename Tag::raw));  // elements of a unit
    constexpr int V = kFwdMaxBlock / 32, U = 4;
    const int lane = threadIdx.x & 31;
    unsigned long long* spare = cand + kStreamCands;
    unsigned at;
    if (k > 64) {
        unsigned v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < streamers ? most[32 * i + lane] : 0u;
        at = warp_threshold(v, k);
    } else {  // pairs of threads do
        unsigned v[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            v[i] = max(2 * i < streamers ? most[64 * i + lane] : 0u, 2 * i + 1 < streamers ? most[64 * i + 32 + lane] : 0u);
        at = warp_threshold(v, k);
    }
    // Only keys above `above` matter: at first every element that reaches the
    // value, then, whenever the candidates are cut to k, those before the k-th.
    unsigned long long above = static_cast<unsigned long long>(at) << 32;
    float least = at > kOrderNegInf ? order_value(at) : neg_inf();  // numbers below it are out
    bool nans = at <= 1;
    int n = 0;
    const auto room_for = [&](int more) {
        if (n <= kStreamCands - more) return;
        above = warp_prune(cand, n, k, spare);
        n = k;
        at = static_cast<unsigned>(above >> 32);
        least = at > kOrderNegInf ? order_value(at) : neg_inf();
        nans = at <= 1;
    };
    const auto take = [&](float x, int j, bool in) {
        const unsigned long long key = order_key(x, j);
        const bool hit = in && key > above;
        const int p = warp_places(hit, &n);
        if (hit) cand[p] = key;
    };
    // the ragged ends
    for (int end = 0; end < 2; ++end) {
        const int s = end ? row.body + 1 : 0, lo = row.slot_begin(s), size = row.slot_size(s);
        if (big[s] < at) continue;
        for (int j0 = 0; j0 < size; j0 += 32) {
            const int j = j0 + lane;
            take(j < size ? widen_elem<Tag>(ld_scalar(row.p + lo + j)) : 0.0f, lo + j, j < size);
        }
    }
    int picked = 0;
    const auto look = [&]() {
        __syncwarp();
        for (int i0 = 0; i0 < 8 * picked; i0 += 32 * U) {
            uint4 w[U];
            int lo[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + 32 * u + lane;
                lo[u] = i < 8 * picked ? row.slot_begin(list[i >> 3]) + (i & 7) * P : -1;
                w[u] = lo[u] >= 0 ? ld_stream16(row.p + lo[u]) : make_uint4(0, 0, 0, 0);
            }
            // bit u * P + e: element e of unit u may matter
            unsigned hits = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t word[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    float x;
                    if constexpr (P == 4) x = __uint_as_float(word[e]);
                    else x = Tag::widen(static_cast<uint16_t>(e & 1 ? word[e >> 1] >> 16 : word[e >> 1] & 0xffffu));
                    if ((x >= least || nans) && lo[u] >= 0) hits |= 1u << (u * P + e);
                }
            }
            const auto put = [&](unsigned in, int p) {
                for (; in; in &= in - 1) {
                    const int b = __ffs(in) - 1, i = b / (P / 4), u = b / P;  // the word, the unit
                    uint32_t v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = i & 8 ? (i & 4 ? at4(w[3], q) : at4(w[2], q)) : (i & 4 ? at4(w[1], q) : at4(w[0], q));
                    v[0] = i & 2 ? (i & 1 ? v[3] : v[2]) : (i & 1 ? v[1] : v[0]);
                    const int j = (u & 2 ? (u & 1 ? lo[3] : lo[2]) : (u & 1 ? lo[1] : lo[0])) + b % P;
                    float x;
                    if constexpr (P == 4) x = __uint_as_float(v[0]);
                    else x = Tag::widen(static_cast<uint16_t>(b & 1 ? v[0] >> 16 : v[0] & 0xffffu));
                    const unsigned long long key = order_key(x, j);
                    cand[p++] = key > above ? key : 0;
                }
            };
            const int more = __reduce_add_sync(0xffffffffu, __popc(hits));
            if (n + more <= kStreamCands) {
                put(hits, warp_places(__popc(hits), &n));
            } else {
#pragma unroll 1
                for (int u = 0; u < U; ++u) {
                    __syncwarp();
                    room_for(32 * P);
                    const unsigned in = hits & ((1u << P) - 1u) << (u * P);
                    put(in, warp_places(__popc(in), &n));
                }
            }
            __syncwarp();
        }
        picked = 0;
    };
    const int tiles = (row.body + 31) / 32;
    for (int t0 = 0; t0 < tiles; t0 += 32) {
        // a lane to a tile, each from another slot on: 32 banks
        const int s0 = 1 + (t0 + lane) * 32;
        const unsigned big_tile = t0 + lane < tiles ? tile[t0 + lane] : 0u;
        const auto scan = [&]() {
            unsigned in = 0;
            if (big_tile == 0 || big_tile < at) return in;
            const unsigned least_big = at > 0 ? at : 1u;
#pragma unroll 8
            for (int i = 0; i < 32; ++i) {
                const unsigned o = big[min(s0 + ((i + lane) & 31), row.body)];
                in |= static_cast<unsigned>(o >= least_big) << i;
            }
            in = __funnelshift_l(in, in, lane);
            if (row.body - s0 < 31) in &= (2u << (row.body - s0)) - 1u;
            if (const unsigned kept = static_cast<unsigned>(above)) {
                // a largest element that equals `at` has to come before the last of those that were kept
                for (unsigned rest = in; rest; rest &= rest - 1) {
                    const int q = __ffs(rest) - 1;
                    if (big[s0 + q] == at && 0xffffffffu - static_cast<unsigned>(row.slot_begin(s0 + q)) <= kept) in ^= 1u << q;
                }
            }
            return in;
        };
        const auto pick = [&](unsigned in) {
            int p = warp_places(__popc(in), &picked);
            for (; in; in &= in - 1) list[p++] = static_cast<unsigned short>(s0 + __ffs(in) - 1);
        };
        const bool any = __any_sync(0xffffffffu, big_tile != 0 && big_tile >= at);
        if (!any) continue;  // (of the whole warp)
        const unsigned in = scan();
        const int more = __reduce_add_sync(0xffffffffu, __popc(in));
        if (picked + more > kStreamList) look();
        if (more <= kStreamList) {
            pick(in);
        } else {  // (ties) a quarter at a time, as what was kept by then allows
#pragma unroll 1
            for (int part = 0; part < 32; part += 8) {
                if (picked > kStreamList - 8 * 32) look();
                __syncwarp();
                pick(scan() & 255u << part);
            }
        }
    }
    look();
    __syncwarp();
    if (n > kRankKeys) {
        warp_prune(cand, n, k, spare);
        n = k;
    }
    // in order, by counting
    const int per_lane = (n + 31) / 32;
    if (per_lane <= 1) rank_lane_keys<1>(cand, n, k, spare);
    else if (per_lane == 2) rank_lane_keys<2>(cand, n, k, spare);
    else if (per_lane == 3) rank_lane_keys<3>(cand, n, k, spare);
    else rank_lane_keys<kRankKeys / 32>(cand, n, k, spare);
    __syncwarp();
}

// Prepare a buffer for the distillation row r: its slots, and the bits of the
// elements that they name.
template <class Tag, int MODE>
__device__ __forceinline__ void prepare_loss(const LogitsProblem& pr, const WideRow<Tag>& row, int64_t r,
                                             const Slots& sl, unsigned* named) {
    const int lane = threadIdx.x & 31;
    const int64_t* ids = pr.ids + r * pr.slots;
    const float* val = pr.teacher + r * pr.slots;
    constexpr int U = 4;  // slots per lane at a time
    for (int i0 = lane; i0 < pr.slots; i0 += 32 * U) {
        int id[U];
        float v[U], x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 32 * u;
            const int64_t j = i < pr.slots ? ids[i] : -1;
            id[u] = j < 0 ? kNoId : j >= pr.cols ? kBadId : static_cast<int>(j);
            v[u] = i < pr.slots ? val[i] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = id[u] >= 0 ? widen_elem<Tag>(ld_scalar(row.p + id[u])) : 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 32 * u;
            if (i >= pr.slots) continue;
            sl.id[i] = id[u];
            sl.v[i] = v[u];
            sl.x[i] = x[u];
            if constexpr (MODE == kStreamLossTail) {
                if (id[u] < 0) continue;
                const int bit = row.bit(id[u]);
                atomicOr(&named[bit >> 5], 1u << (bit & 31));
            }
        }
    }
    __syncwarp();
}

template <class Tag, int MODE>
__device__ __forceinline__ void finish_rows(const LogitsProblem& pr, float scale2, const StreamLayout& lay,
                                            unsigned char* dyn, int finisher) {
    constexpr bool LOSS = MODE == kStreamLoss || MODE == kStreamLossTail;
    const int lane = threadIdx.x & 31, threads = (lay.streamers + 1) * 32;
    const int buffers = lay.finishers + 1;
    const int64_t cta = blockIdx.x, ctas = gridDim.x;
    // Hand a buffer out for this CTA's row i.
    const auto hand_out = [&](int64_t i) {
        const int64_t r = cta + i * ctas;
        if (r >= pr.rows) return;
        const int at = static_cast<int>(i % buffers);
        unsigned char* buf = dyn + at * lay.buffer;
        if constexpr (LOSS)
            prepare_loss<Tag, MODE>(pr, WideRow<Tag>(pr, r), r, Slots(buf + lay.teacher, pr.slots),
                                    reinterpret_cast<unsigned*>(buf + lay.named));
        bar_arrive(free_bar(at), threads);
    };
    // the first row of each buffer: one per finisher, and one more of the first's
    for (int at = finisher; at < buffers; at += lay.finishers) {
        if constexpr (MODE == kStreamLossTail) {
            unsigned* named = reinterpret_cast<unsigned*>(dyn + at * lay.buffer + lay.named);
            for (int i = lane; i < static_cast<int>((lay.teacher - lay.named) / 4); i += 32) named[i] = 0u;
            __syncwarp();
        }
        hand_out(at);
    }
    // a row's token and its logit, loaded while the row before is finished
    int64_t tok = -1;
    float tok_x = 0.0f;
    const auto load_token = [&](int64_t r) { return !LOSS && MODE != kStreamBeam && pr.logprob && r < pr.rows ? pr.tokens[r] : -1; };
    const auto load_logit = [&](int64_t r, int64_t t) {
        return t >= 0 && t < pr.cols ? widen_elem<Tag>(ld_scalar(WideRow<Tag>(pr, r).p + t)) : 0.0f;
    };
    tok = load_token(cta + finisher * ctas);
    tok_x = load_logit(cta + finisher * ctas, tok);
    for (int64_t i = finisher;; i += lay.finishers) {
        const int64_t r = cta + i * ctas;
        if (r >= pr.rows) break;
        const int64_t next = r + lay.finishers * ctas;
        const int at = static_cast<int>(i % buffers);
        unsigned char* buf = dyn + at * lay.buffer;
        const WideRow<Tag> row(pr, r);
        if (lay.finishers > 1 && i > 0) bar_sync(turn_bar(finisher), 64);
        bar_sync(full_bar(at), threads);
        if (lay.finishers > 1 && r + ctas < pr.rows)
            bar_arrive(turn_bar(finisher + 1 < lay.finishers ? finisher + 1 : 0), 64);
        SoftSum c = joined_sums(buf + lay.sums, lay.streamers, scale2);
        if constexpr (MODE == kStreamBeam) {
            if (beam_looks(pr, r)) {
                unsigned long long* cand = reinterpret_cast<unsigned long long*>(dyn + lay.cand) +
                                           finisher * (kStreamCands + kRankKeys);
                const int k = pr.top_k;
                warp_top<Tag>(row, k, reinterpret_cast<const unsigned*>(buf + lay.big),
                              reinterpret_cast<const unsigned*>(buf + lay.tile),
                              reinterpret_cast<const unsigned*>(buf + lay.most), lay.streamers, cand,
                              reinterpret_cast<unsigned short*>(dyn + lay.list) + finisher * kStreamList);
                for (int i = lane; i < k; i += 32) pr.beam_keys[r * k + i] = cand[kStreamCands + i];
                if (lane == 0) pr.beam_sums[r] = make_float2(c.m, c.s);
                __syncwarp();
            }
        } else if constexpr (!LOSS) {
            const float ln_s = c.empty() ? neg_inf() : logf(c.s);
            if (lane == 0) {
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
            }
            tok = load_token(next);
            if constexpr (MODE == kStreamTop) {
                unsigned long long* cand = reinterpret_cast<unsigned long long*>(dyn + lay.cand) +
                                           finisher * (kStreamCands + kRankKeys);
                const int k = pr.top_k;
                warp_top<Tag>(row, k, reinterpret_cast<const unsigned*>(buf + lay.big),
                              reinterpret_cast<const unsigned*>(buf + lay.tile),
                              reinterpret_cast<const unsigned*>(buf + lay.most), lay.streamers, cand,
                              reinterpret_cast<unsigned short*>(dyn + lay.list) + finisher * kStreamList);
                for (int i = lane; i < k; i += 32) {
                    const unsigned long long key = cand[kStreamCands + i];
                    const float v = order_value(static_cast<unsigned>(key >> 32));
                    if (pr.top_ids) pr.top_ids[r * k + i] = key_index(key);
                    if (pr.top_logprobs)
                        pr.top_logprobs[r * k + i] = c.empty() ? neg_inf() : (v - c.m) / pr.temperature - ln_s;
                }
                __syncwarp();
            }
            tok_x = load_logit(next, tok);
        } else {
            const Slots sl(buf + lay.teacher, pr.slots);
            const Teacher q = warp_teacher(pr, sl);
            SoftSum all = c;
            if constexpr (MODE == kStreamLossTail) {
                SoftSum d;
                for (int i = lane; i < pr.slots; i += 32)
                    if (sl.id[i] >= 0) d.add(sl.x[i], scale2);
                all.join(warp_softsum(d, scale2), scale2);
            }
            const float m = all.empty() ? neg_inf() : all.m;
            const float ln_s = all.empty() ? neg_inf() : logf(all.s);
            const float ln_rest = MODE == kStreamLossTail ? tail_log(pr, c, all.m, ln_s) : ln_s;
            float loss = 0.0f;
            for (int i = lane; i < pr.slots; i += 32) loss += slot_loss(pr, q, sl, i, m, ln_s);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
            if (lane == 0) {
                if (pr.loss) pr.loss[r] = whole_loss(q, loss, ln_s, ln_rest);
                if (pr.stats) pr.stats[r] = make_float4(m, ln_s, ln_rest, 0.0f);
            }
            __syncwarp();
            if constexpr (MODE == kStreamLossTail) {
                // clear this row's bits
                unsigned* named = reinterpret_cast<unsigned*>(buf + lay.named);
                for (int i = lane; i < pr.slots; i += 32)
                    if (sl.id[i] >= 0) named[row.bit(sl.id[i]) >> 5] = 0u;
                __syncwarp();
            }
        }
        hand_out(i + buffers);
    }
}

template <class Tag, int MODE>
__global__ void __launch_bounds__(kFwdMaxBlock, 2) logits_stream_kernel(const LogitsProblem pr, float scale2,
                                                                        int finishers) {
    extern __shared__ __align__(16) unsigned char dyn[];
    const int streamers = static_cast<int>(blockDim.x / 32) - finishers, warp = threadIdx.x >> 5;
    const StreamLayout lay(MODE, streamers, finishers, kWideElems<Tag>, pr.cols, pr.slots);
    allow_dependents();
    grid_dependency_wait();
    if (warp < streamers) stream_rows<Tag, MODE>(pr, scale2, lay, dyn);
    else finish_rows<Tag, MODE>(pr, scale2, lay, dyn, warp - streamers);
}

}  // namespace argr
