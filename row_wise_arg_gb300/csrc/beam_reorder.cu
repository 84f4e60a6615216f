// The states of an item's beams, in place: beam j takes over what beam parents[j]
// kept.
//
// A thread owns the same word of every beam of its item: it reads the word of each
// moving beam's parent, all of them before it writes any, so that beams may
// exchange states without a copy elsewhere. Beams that keep their own state are neither read
// (but as a parent) nor written. A parent of several beams is read from memory once, its other
// reads hit L1.
//
// Bound by memory: each distinct parent read once, each moving beam written once.
#include "kernels_impl.cuh"
#include "select.h"

namespace argr {

constexpr int kReorderBlock = 256;

template <int W> struct WordOf;
template <> struct WordOf<16> { using type = uint4; };
template <> struct WordOf<8> { using type = uint2; };
template <> struct WordOf<4> { using type = uint32_t; };
template <> struct WordOf<2> { using type = uint16_t; };
template <> struct WordOf<1> { using type = uint8_t; };

// A tile: kReorderBlock words of a segment of one state. BEAMS: beams at most; U words per thread at a time.
template <int W, int BEAMS, int U>
__global__ void __launch_bounds__(kReorderBlock) beam_reorder_kernel(const ReorderProblem pr) {
    using Word = typename WordOf<W>::type;
    __shared__ int move_to[BEAMS], move_from[BEAMS];
    __shared__ int moves;
    const int t = threadIdx.x;
    allow_dependents();
    grid_dependency_wait();
    for (int64_t item = blockIdx.y; item < pr.items; item += gridDim.y) {
        __syncthreads();
        if (t < 32) {
            // the beams that move, in order
            int n = 0;
            for (int j0 = 0; j0 < pr.beams; j0 += 32) {
                const int j = j0 + t;
                int64_t p = j < pr.beams ? pr.parents[item * pr.beams + j] : -1;
                const bool in = p >= 0 && p < pr.beams && p != j;
                const unsigned all = __ballot_sync(0xffffffffu, in);
                if (in) {
                    const int at = n + __popc(all & ((1u << t) - 1u));
                    move_to[at] = j;
                    move_from[at] = static_cast<int>(p);
                }
                n += __popc(all);
            }
            if (t == 0) moves = n;
        }
        __syncthreads();
        const int n = moves;
        if (n == 0) continue;
        int64_t live = pr.positions;
        if (pr.lengths) {
            const int64_t len = pr.lengths[item];
            live = len < 0 ? 0 : len < live ? len : live;
        }
        const int64_t bytes = live * pr.pos_bytes, words = bytes / W;
        const int rest = static_cast<int>(bytes - words * W);  // past the last word, byte by byte
        const int64_t per_tile = static_cast<int64_t>(kReorderBlock) * U;
        const int64_t chunks = (words + per_tile - 1) / per_tile + (rest > 0);
        const int64_t tiles = chunks * pr.outer * pr.n;
        for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int64_t seg = tile / chunks, chunk = tile - seg * chunks;
            const int64_t state = seg / pr.outer, o = seg - state * pr.outer;
            unsigned char* base = pr.states[state] + item * pr.item_stride + o * pr.outer_stride;
            if (rest > 0 && chunk == chunks - 1) {
                if (t < rest) {
                    unsigned char* p = base + words * W + t;
                    unsigned char v[BEAMS];
#pragma unroll
                    for (int i = 0; i < BEAMS; ++i)
                        if (i < n) v[i] = p[move_from[i] * pr.beam_stride];
#pragma unroll
                    for (int i = 0; i < BEAMS; ++i)
                        if (i < n) p[move_to[i] * pr.beam_stride] = v[i];
                }
                continue;
            }
            const int64_t w0 = chunk * per_tile + t;
            Word v[U][BEAMS];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (w0 + u * kReorderBlock >= words) break;
                const unsigned char* p = base + (w0 + u * kReorderBlock) * W;
#pragma unroll
                for (int i = 0; i < BEAMS; ++i)
                    if (i < n) v[u][i] = *reinterpret_cast<const Word*>(p + move_from[i] * pr.beam_stride);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (w0 + u * kReorderBlock >= words) break;
                unsigned char* p = base + (w0 + u * kReorderBlock) * W;
#pragma unroll
                for (int i = 0; i < BEAMS; ++i)
                    if (i < n) *reinterpret_cast<Word*>(p + move_to[i] * pr.beam_stride) = v[u][i];
            }
        }
    }
}

template <int W, int BEAMS, int U>
cudaError_t launch_reorder_n(const ReorderProblem& pr, const argr_caps& caps) {
    // about eight CTAs per SM; past that the tiles come in turns
    const int64_t per_tile = static_cast<int64_t>(kReorderBlock) * U;
    const int64_t words = pr.positions * pr.pos_bytes / W;
    const int64_t tiles = ((words + per_tile - 1) / per_tile + 1) * pr.outer * pr.n;
    const int64_t items = pr.items < 65535 ? pr.items : 65535;
    int64_t x = (32 * static_cast<int64_t>(caps.sm_count) + items - 1) / items;
    x = x < tiles ? x : tiles;
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    return launch_ex_smem(beam_reorder_kernel<W, BEAMS, U>, dim3(static_cast<unsigned>(x), static_cast<unsigned>(items)),
                          dim3(kReorderBlock), 1, 0, p, pr.stream, pr);
}

// Words of all moving beams stay in registers: 64 beams of 16-byte words are 256 of them, so narrower
// words from 33 beams on.
template <int W>
cudaError_t launch_reorder_w(const ReorderProblem& pr, const argr_caps& caps) {
    if (pr.beams <= 4) return launch_reorder_n<W, 4, 4>(pr, caps);
    if (pr.beams <= 8) return launch_reorder_n<W, 8, 2>(pr, caps);
    if (pr.beams <= 16) return launch_reorder_n<W, 16, 1>(pr, caps);
    if (pr.beams <= 32) return launch_reorder_n<W, 32, 1>(pr, caps);
    return launch_reorder_n<(W < 8 ? W : 8), 64, 1>(pr, caps);
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
