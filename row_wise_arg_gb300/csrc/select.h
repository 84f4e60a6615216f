// Host-side declarations of the selections over rows of scores
// (argreduce_beam_select, argreduce_beam_reorder, argreduce_route and its
// gradient): the problems as the launchers see them, and the launchers.
#pragma once

#include "logits.h"

namespace argr {

struct BeamProblem {
    LogitsProblem rows;   // x, cols, row_stride, temperature, beam_*; rows = items * beams
    int64_t items;
    int beams;
    int count;
    const float* scale;           // [items, beams] or null
    int64_t end_token;
    double inv_t;                 // 1 / temperature
    int64_t* tokens;              // [items, count]
    int64_t* parents;
    float* out_scores;
};

// The plan of a step: one cluster per item, 1 << shift CTAs to a beam, or (cluster == 0) rows and merge.
struct BeamPlan {
    int cluster, shift, block;
    bool stream;
};
// By the figures of a device that places clusters of up to caps.max_cluster CTAs (plan_beams.cpp).
BeamPlan plan_beams(int64_t items, int beams, int64_t cols, int dtype, int k, const argr_caps& caps);
// Whether rows are streamed, and their plan.
bool beam_stream_plan(int64_t rows, int64_t cols, int dtype, int k, const argr_caps& caps, argr_plan* p);
// The plan for a device of which fits(plan, &ok) says whether it places a plan's clusters: with smaller ones, or without, where it
// does not (a part of a GPU).
template <class Fits>
cudaError_t fitting_beam_plan(int64_t items, int beams, int64_t cols, int dtype, int k, argr_caps caps, Fits fits, BeamPlan* p) {
    for (;;) {
        *p = plan_beams(items, beams, cols, dtype, k, caps);
        if (p->cluster <= 1) return cudaSuccess;
        bool ok = false;
        const cudaError_t e = fits(*p, &ok);
        if (e != cudaSuccess || ok) return e;
        caps.max_cluster = p->cluster - 1;
    }
}

constexpr int kReorderStates = 128;  // tensors of one launch

struct ReorderProblem {
    unsigned char* states[kReorderStates];
    int n;
    int64_t items;
    int beams;
    int64_t item_stride, beam_stride;  // bytes
    int64_t outer, outer_stride;       // segments of a beam's state, bytes
    int64_t positions, pos_bytes;      // a segment is positions * pos_bytes contiguous bytes
    int word;                          // bytes that every address is a multiple of: 1, 2, 4, 8 or 16
    const int64_t* parents;            // [items, beams]
    const int64_t* lengths;            // [items] or null
    cudaStream_t stream;
};

struct RouteProblem {
    const void* x;
    int dtype;
    int64_t rows;
    int experts;
    int64_t row_stride;  // elements
    int k;
    int normalize;
    const uint8_t* valid;  // [rows] or null
    // forward
    float* weights;  // [rows, k]
    int64_t* ids;
    float* lse;         // [rows]
    int64_t* counts;    // [experts] or null
    int64_t* taken;     // rows that take part
    float* balance;     // or null
    float* part_sums;   // scratch: [ctas, experts] sums of the softmax
    int* part_counts;   // scratch: [ctas, experts + 1] choices, and the rows that take part
    int ctas;
    // gradient
    const float* grad_weights;  // or null
    const float* grad_lse;      // or null
    const float* grad_balance;  // one value, or null
    void* grad;
    int64_t grad_stride;
    cudaStream_t stream;
};

constexpr int kRouteBlock = 512;
constexpr int kRouteWarps = kRouteBlock / 32;
constexpr int kRouteMaxCtas = 512;  // CTAs that leave partial sums, at most
constexpr int kRouteOneTurns = 2;   // units of a warp where one cluster does it all, at most

// How the forward kernel takes rows of so many experts: `lanes` to a row, `elems` elements to a lane. Rows of 8 lanes
// for 33 to 256 experts, then more lanes, as the sums of p take a register per element of a lane.
struct RouteShape {
    int lanes, elems;
};
inline RouteShape route_shape(int64_t experts) {
    if (experts <= 32) return {experts <= 8 ? 1 : experts <= 16 ? 2 : 4, 8};
    if (experts <= 256) return {8, experts <= 64 ? 8 : experts <= 128 ? 16 : 32};
    return {experts <= 512 ? 16 : 32, 32};
}
// The grid of the forward kernel: a unit (32 / lanes rows) per warp, up to two CTAs per SM (one where a lane's elements
// take the registers). cluster: the CTAs are one cluster that joins its sums itself (counts alone need
// that), while its warps take few units each; 0: they leave them in scratch.
struct RouteGrid {
    int ctas, cluster;
};
inline RouteGrid route_grid(int64_t rows, int64_t experts, bool counts, const argr_caps& caps) {
    const RouteShape s = route_shape(experts);
    const int64_t each = static_cast<int64_t>(32 / s.lanes) * kRouteWarps, want = (rows + each - 1) / each;
    if (counts && want <= 8 * kRouteOneTurns) {
        int c = 1;
        while (c < 8 && c < want) c *= 2;
        if (c <= caps.max_cluster) return {c, c};
    }
    int64_t most = static_cast<int64_t>(s.elems <= 8 ? 2 : 1) * caps.sm_count;
    if (most > kRouteMaxCtas) most = kRouteMaxCtas;
    return {static_cast<int>(want < most ? want : most), 0};
}

#ifdef __CUDACC__
// The balance loss from sum_e counts_e (sum over the rows of p_e).
__device__ __forceinline__ float route_balance(double sum, long long rows, int experts, int k) {
    const double n = static_cast<double>(rows > 0 ? rows : 1);
    return static_cast<float>(sum * experts / (k * n * n));
}
#endif

cudaError_t launch_beam_reorder(const ReorderProblem& pr, const argr_caps& caps);
cudaError_t launch_route_finish(const RouteProblem& pr);
#define ARGR_DECLARE_SELECT(sfx)                                                                                    \
    cudaError_t beam_plan_##sfx(int64_t items, int beams, int64_t cols, int k, const argr_caps& caps, BeamPlan* p); \
    cudaError_t launch_beam_select_##sfx(const BeamProblem& pr, const BeamPlan& b, const argr_caps& caps);          \
    cudaError_t launch_route_##sfx(const RouteProblem& pr, const argr_caps& caps);                                  \
    cudaError_t launch_route_grad_##sfx(const RouteProblem& pr, const argr_caps& caps);
ARGR_DECLARE_SELECT(f32)
ARGR_DECLARE_SELECT(f16)
ARGR_DECLARE_SELECT(bf16)
#undef ARGR_DECLARE_SELECT

}  // namespace argr
