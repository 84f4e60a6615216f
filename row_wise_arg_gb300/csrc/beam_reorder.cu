// The states of an item's beams, in place: beam j takes over what beam parents[j]
// kept.
//
// A thread owns the same word of every beam of its item: it reads the word of each
// moving beam's parent, all of them before it writes any, so that beams may
// exchange states without a copy elsewhere. Beams that keep their own state are neither read
// (but as a parent) nor written. A parent of several beams is read from memory once, its other
// reads hit L1.
//
// The words of an item's live positions are numbered through, segment after segment, and cut into tiles; the tiles of
// all items are dealt to as many CTAs as run at once. (With CTAs for each item, and for segments of the
// longest, items of different lengths left them waiting in waves: 12 states of 9 items, 5 beams, 77 positions took 21 us.)
//
// Bound by memory: each distinct parent read once, each moving beam written once. 32 caches of [16 x 4, 8, 1024, 128] bf16, ragged (1.6 to
// 1.8 GB move, by parents and lengths): 5.9 to 6.1 TB/s of the bytes that move, 264 us for 1612 MB.
#include "kernels_impl.cuh"
#include "select.h"

namespace argr {

constexpr int kReorderBlock = 256;
template <int BEAMS> constexpr int kReorderItems = BEAMS <= 16 ? 32 : 8;  // items at a time
// CTAs of an SM, at least. What is in flight decides (45 KB an SM at the copy rate), words per thread against threads; for
// words of 4 bytes and less it is the instructions (addresses, above all). us:
//   32 bf16 caches of [16, 4, 8, 1024, 128], one draw of ragged lengths, words of 16 bytes: 309, 335, 379 with 2, 4, 1 of them to a thread
//   and 4, 2, 6 CTAs; 16 of [8, 8, 8, 1024, 128]: 208, 246 with 2, 1 and 2, 4 CTAs;
//   words of 4 bytes: 12 states of [9, 5, 3, 77, 129] f32 13.2, 4 of [6, 13, 5, 401, 77] 37; of 2: 8 of [16, 4, 7, 701, 33] 34. Two
//   words to a thread, an address each: 15.6, 55, 59.
// The grid: the CTAs that run at once. Four times as many: the caches 258 in place of 264 us (another draw), but 12 states of [9, 5, 3, 77, 129] f32
// 19.4 in place of 15.1 (every CTA plans its items before its first tile).
template <int BEAMS, int W> constexpr int kReorderCtas = BEAMS <= 4 ? 4 : BEAMS <= 8 ? (W == 16 ? 2 : 3) : BEAMS <= 16 ? 2 : 1;
// Words per thread at a time.
template <int BEAMS, int W>
constexpr int kReorderWords = BEAMS <= 8 ? (W >= 8 ? 2 : 4) : BEAMS <= 16 ? (W >= 8 ? 1 : 4) : BEAMS <= 32 && W <= 4 ? 2 : 1;

template <int W> struct WordOf;
template <> struct WordOf<16> { using type = uint4; };
template <> struct WordOf<8> { using type = uint2; };
template <> struct WordOf<4> { using type = uint32_t; };
template <> struct WordOf<2> { using type = uint16_t; };
template <> struct WordOf<1> { using type = uint8_t; };

// a / b and what is left, in 32 bits where they fit.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b, int64_t* left) {
    int64_t q;
    if (((a | b) >> 32) == 0) q = static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    else q = a / b;
    *left = a - q * b;
    return q;
}

template <int BEAMS>
struct Moves {
    int64_t to[kReorderItems<BEAMS>][BEAMS], from[kReorderItems<BEAMS>][BEAMS];  // bytes from beam 0
    int n[32];
    int64_t bytes[32];  // live in a segment
    int64_t end[32];    // of the item's tiles
};

// U words of type Word at the offsets at[u] of beam 0 (negative: none), for all moves of an item.
template <class Word, int BEAMS, int U>
__device__ __forceinline__ void move_words(unsigned char* base, const int64_t (&at)[U], int n, const int64_t* to,
                                           const int64_t* from) {
    Word v[U][BEAMS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < BEAMS; ++i)
            if (i < n && at[u] >= 0) v[u][i] = *reinterpret_cast<const Word*>(base + at[u] + from[i]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < BEAMS; ++i)
            if (i < n && at[u] >= 0) *reinterpret_cast<Word*>(base + at[u] + to[i]) = v[u][i];
    }
}

// The same for U words kReorderBlock apart from `first` (of beam 0) on: one address to a beam, where the addresses of narrow
// words would cost more than the words do.
template <class Word, int BEAMS, int U>
__device__ __forceinline__ void move_run(unsigned char* first, int n, const int64_t* to, const int64_t* from) {
    Word v[BEAMS][U];
#pragma unroll
    for (int i = 0; i < BEAMS; ++i) {
        if (i < n) {
            const Word* p = reinterpret_cast<const Word*>(first + from[i]);
#pragma unroll
            for (int u = 0; u < U; ++u) v[i][u] = p[u * kReorderBlock];
        }
    }
#pragma unroll
    for (int i = 0; i < BEAMS; ++i) {
        if (i < n) {
            Word* p = reinterpret_cast<Word*>(first + to[i]);
#pragma unroll
            for (int u = 0; u < U; ++u) p[u * kReorderBlock] = v[i][u];
        }
    }
}

// BEAMS: beams at most; a tile is kReorderBlock * U words of a state (or, of what is past the segments' last words, bytes).
template <int W, int BEAMS, int U>
__global__ void __launch_bounds__(kReorderBlock, kReorderCtas<BEAMS, W>) beam_reorder_kernel(const ReorderProblem pr) {
    using Word = typename WordOf<W>::type;
    constexpr int kTile = kReorderBlock * U, kItems = kReorderItems<BEAMS>;
    __shared__ Moves<BEAMS> sh;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    allow_dependents();
    grid_dependency_wait();
    for (int64_t item0 = 0; item0 < pr.items; item0 += kItems) {
        const int items = pr.items - item0 < kItems ? static_cast<int>(pr.items - item0) : kItems;
        __syncthreads();
        for (int q = warp; q < 32; q += kReorderBlock / 32) {
            // the beams of an item that move, in order
            int n = 0;
            for (int j0 = 0; j0 < pr.beams && q < items; j0 += 32) {
                const int j = j0 + lane;
                const int64_t p = j < pr.beams ? pr.parents[(item0 + q) * pr.beams + j] : -1;
                const bool in = p >= 0 && p < pr.beams && p != j;
                const unsigned all = __ballot_sync(0xffffffffu, in);
                if (in) {
                    const int at = n + __popc(all & ((1u << lane) - 1u));
                    sh.to[q][at] = j * pr.beam_stride;
                    sh.from[q][at] = p * pr.beam_stride;
                }
                n += __popc(all);
            }
            if (lane == 0) {
                int64_t live = pr.positions;
                if (pr.lengths && q < items) {
                    const int64_t len = pr.lengths[item0 + q];
                    live = len < 0 ? 0 : len < live ? len : live;
                }
                const int64_t bytes = live * pr.pos_bytes, words = bytes / W, rest = bytes - words * W;
                sh.n[q] = n;
                sh.bytes[q] = bytes;
                sh.end[q] = n ? ((words * pr.outer + kTile - 1) / kTile + (rest * pr.outer + kTile - 1) / kTile) * pr.n : 0;
            }
        }
        __syncthreads();
        if (warp == 0) {
            int64_t end = sh.end[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t d = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += d;
            }
            sh.end[lane] = end;
        }
        __syncthreads();
        int q = 0;
        for (int64_t tile = blockIdx.x; tile < sh.end[31]; tile += gridDim.x) {
            while (tile >= sh.end[q]) ++q;
            const int64_t bytes = sh.bytes[q], words = bytes / W, rest = bytes - words * W;
            const int64_t word_tiles = (words * pr.outer + kTile - 1) / kTile;
            const int64_t tiles = word_tiles + (rest * pr.outer + kTile - 1) / kTile;
            int64_t in_state;
            const int64_t state = divide(tile - (q ? sh.end[q - 1] : 0), tiles, &in_state);
            unsigned char* base = pr.states[state] + (item0 + q) * pr.item_stride;
            [[maybe_unused]] int64_t at[U];  // (of wide words)
            if (in_state < word_tiles) {
                // the tile's first word, and from it on: one division a tile where segments are longer than tiles
                int64_t first = in_state * kTile, o0 = 0;
                const int64_t left = words * pr.outer - first;
                if (pr.outer > 1) o0 = divide(first, words, &first);
                if constexpr (W >= 8) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        int64_t w = first + (u * kReorderBlock + t), o = o0;
                        if (w >= words) {
                            if (words >= kTile) {
                                w -= words;
                                ++o;
                            } else {
                                o += divide(w, words, &w);
                            }
                        }
                        at[u] = u * kReorderBlock + t < left ? o * pr.outer_stride + w * W : -1;
                    }
                    move_words<Word, BEAMS, U>(base, at, sh.n[q], sh.to[q], sh.from[q]);
                } else if (first + kTile <= words) {
                    move_run<Word, BEAMS, U>(base + o0 * pr.outer_stride + (first + t) * W, sh.n[q], sh.to[q], sh.from[q]);
                } else {  // a tile over several segments, in smaller steps
                    constexpr int A = U < 2 ? 1 : 2;
#pragma unroll 1
                    for (int u0 = 0; u0 < kTile && u0 < left; u0 += kReorderBlock * A) {
                        int64_t some[A];
#pragma unroll
                        for (int u = 0; u < A; ++u) {
                            int64_t w = first + (u0 + u * kReorderBlock + t), o = o0;
                            if (w >= words) {
                                if (words >= kTile) {
                                    w -= words;
                                    ++o;
                                } else {
                                    o += divide(w, words, &w);
                                }
                            }
                            some[u] = u0 + u * kReorderBlock + t < left ? o * pr.outer_stride + w * W : -1;
                        }
                        move_words<Word, BEAMS, A>(base, some, sh.n[q], sh.to[q], sh.from[q]);
                    }
                }
            } else if constexpr (W >= 8) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t b = (in_state - word_tiles) * kTile + u * kReorderBlock + t;
                    at[u] = -1;
                    if (b < rest * pr.outer) {
                        int64_t in_segment;
                        const int64_t o = divide(b, rest, &in_segment);
                        at[u] = o * pr.outer_stride + words * W + in_segment;
                    }
                }
                move_words<uint8_t, BEAMS, U>(base, at, sh.n[q], sh.to[q], sh.from[q]);
            } else {
#pragma unroll 1
                for (int u = 0; u < U; ++u) {
                    const int64_t b = (in_state - word_tiles) * kTile + u * kReorderBlock + t;
                    if (b >= rest * pr.outer) break;
                    int64_t in_segment;
                    const int64_t o = divide(b, rest, &in_segment);
                    const int64_t one[1] = {o * pr.outer_stride + words * W + in_segment};
                    move_words<uint8_t, BEAMS, 1>(base, one, sh.n[q], sh.to[q], sh.from[q]);
                }
            }
        }
    }
}

template <int W, int BEAMS>
cudaError_t launch_reorder_n(const ReorderProblem& pr, const argr_caps& caps) {
    constexpr int U = kReorderWords<BEAMS, W>;
    auto kern = beam_reorder_kernel<W, BEAMS, U>;
    static std::atomic<int> known[kLaunchCacheDevices];  // CTAs of an SM, by device
    int dev = 0, per_sm = 0;
    cudaError_t e = launch_device(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0) per_sm = known[dev].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kReorderBlock, 0)) != cudaSuccess) return e;
        if (dev >= 0) known[dev].store(per_sm, std::memory_order_relaxed);
    }
    const int64_t most = static_cast<int64_t>(per_sm > 0 ? per_sm : 1) * caps.sm_count;
    // tiles, at most: every position of every item
    const double tiles = (static_cast<double>(pr.positions) * pr.pos_bytes * pr.outer / (W * kReorderBlock * U) + 2) * pr.n * pr.items;
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    return launch_ex_smem(kern, dim3(static_cast<unsigned>(tiles < most ? tiles : most)), dim3(kReorderBlock), 1, 0, p,
                          pr.stream, pr);
}

// Words of all moving beams stay in registers, at most 64 of them (128 for 32 beams of 16 bytes), hence narrower
// words from 33 beams on.
template <int W>
cudaError_t launch_reorder_w(const ReorderProblem& pr, const argr_caps& caps) {
    if (pr.beams <= 4) return launch_reorder_n<W, 4>(pr, caps);
    if (pr.beams <= 8) return launch_reorder_n<W, 8>(pr, caps);
    if (pr.beams <= 16) return launch_reorder_n<W, 16>(pr, caps);
    if (pr.beams <= 32) return launch_reorder_n<W, 32>(pr, caps);
    return launch_reorder_n<(W < 8 ? W : 8), 64>(pr, caps);
}

cudaError_t launch_beam_reorder(const ReorderProblem& pr, const argr_caps& caps) {
    switch (pr.word) {
        case 16: return launch_reorder_w<16>(pr, caps);
        case 8: return launch_reorder_w<8>(pr, caps);
        case 4: return launch_reorder_w<4>(pr, caps);
        case 2: return launch_reorder_w<2>(pr, caps);
        default: return launch_reorder_w<1>(pr, caps);
    }
}

}  // namespace argr
