// C entry points of beam selection, beam reordering and routing: argument checks
// (all before anything is queued) and dispatch by element type.
#include <algorithm>
#include <climits>
#include <cmath>

#include "logits_checks.h"
#include "select.h"

namespace argr {
namespace {

#define ARGR_SELECT_DISPATCH(fn, dtype, pr, caps)                      \
    ((dtype) == ARGR_F32   ? launched(fn##_f32((pr), (caps)))          \
     : (dtype) == ARGR_F16 ? launched(fn##_f16((pr), (caps)))          \
                           : launched(fn##_bf16((pr), (caps))))

// One dimension of a state: `count` parts, `stride` bytes apart, of `inner` bytes from first to last.
struct Dim {
    int64_t stride, count, inner;
};

// The dimensions of a state, outermost first, and the bytes that it spans; false where they do not nest or overflow.
struct Layout {
    Dim dim[3];
    int n = 0;
    int64_t segment = 0, extent = 0;

    void add(int64_t stride, int64_t count) {
        if (count > 1) dim[n++] = Dim{stride, count, 0};
    }
    bool nest(int64_t bytes) {
        segment = extent = bytes;
        for (int i = 1; i < n; ++i)
            for (int j = i; j > 0 && dim[j].stride > dim[j - 1].stride; --j) std::swap(dim[j], dim[j - 1]);
        for (int i = n - 1; i >= 0; --i) {
            if (dim[i].stride < extent) return false;
            dim[i].inner = extent;
            if (dim[i].stride > (INT64_MAX - extent) / (dim[i].count - 1)) return false;
            extent += dim[i].stride * (dim[i].count - 1);
        }
        return true;
    }
    // Whether two states of this layout, the second `d` bytes after the first, share a byte.
    bool meets(int64_t d, int level = 0) const {
        if (level == n) return d > -segment && d < segment;
        const Dim& m = dim[level];
        int64_t q = 0;
        if (d < 0 || d >= m.stride) {
            q = d / m.stride;
            if (d % m.stride < 0) --q;
        }
        for (int64_t k = q; k <= q + 1; ++k) {
            const int64_t left = d - k * m.stride;
            if (k > -m.count && k < m.count && left > -m.inner && left < m.inner && meets(left, level + 1)) return true;
        }
        return false;
    }
};

bool reorder_layout(int64_t items, int beams, int64_t item_stride, int64_t beam_stride, int64_t outer, int64_t outer_stride,
                    int64_t segment, Layout* lay) {
    lay->add(item_stride, items);
    lay->add(beam_stride, beams);
    lay->add(outer_stride, outer);
    return lay->nest(segment);
}

bool touches(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

argr_status check_route(const void* x, int dtype, int64_t rows, int64_t experts, int64_t row_stride, int top_k) {
    const argr_status s = check_rows(x, dtype, rows, experts, row_stride, 1.0f);
    if (s != ARGR_OK) return s;
    if (experts > ARGR_ROUTE_MAX_EXPERTS || top_k < 1 || top_k > ARGR_ROUTE_MAX_TOP || top_k > experts) return ARGR_EINVAL;
    return ARGR_OK;
}

// Scratch of a route whose CTAs leave their sums and counts: the sums, then the counts.
size_t route_sums_bytes(int64_t ctas, int64_t experts) { return align_up(4 * static_cast<size_t>(ctas) * experts, 16); }
size_t route_scratch(int64_t rows, int64_t experts, const argr_caps& caps) {
    const RouteGrid g = route_grid(rows, experts, true, caps);
    return g.cluster ? 0 : route_sums_bytes(g.ctas, experts) + 4 * static_cast<size_t>(g.ctas) * (experts + 1);
}

// Scratch of a step, 0 where it is one launch: a list and sums for every row.
size_t beam_scratch(const BeamPlan& b, int64_t rows, int k) { return b.cluster ? 0 : 8 * static_cast<size_t>(rows) * (k + 1); }
argr_status beam_plan(int64_t items, int beams, int64_t cols, int dtype, int k, const argr_caps& caps, BeamPlan* b) {
    return launched(dtype == ARGR_F32   ? beam_plan_f32(items, beams, cols, k, caps, b)
                    : dtype == ARGR_F16 ? beam_plan_f16(items, beams, cols, k, caps, b)
                                        : beam_plan_bf16(items, beams, cols, k, caps, b));
}

}  // namespace
}  // namespace argr

using namespace argr;

extern "C" {

argr_status argreduce_beam_select(const void* x, argr_dtype dtype, int64_t items, int32_t beams, int64_t cols,
                                  int64_t row_stride, float temperature, const float* scores, const uint8_t* ended,
                                  int64_t end_token, const float* scale, int32_t count, int64_t* tokens,
                                  int64_t* parents, float* out_scores, void* scratch, size_t scratch_bytes,
                                  argr_stream stream) {
    if (beams < 1 || beams > ARGR_BEAM_MAX_BEAMS || items < 0 || items > INT_MAX / 64) return ARGR_EINVAL;
    argr_status s = check_rows(x, dtype, items * beams, cols, row_stride, temperature);
    if (s != ARGR_OK) return s;
    if (count < 1 || count > ARGR_LOGITS_MAX_TOP) return ARGR_EINVAL;
    if (misaligned(scores, 4) || misaligned(scale, 4) || misaligned(tokens, 8) || misaligned(parents, 8) ||
        misaligned(out_scores, 4))
        return ARGR_EINVAL;
    if (items == 0) return ARGR_OK;
    if (!scores || !tokens || !parents || !out_scores) return ARGR_EINVAL;
    argr_caps caps;
    if ((s = current_caps(&caps)) != ARGR_OK) return s;
    BeamProblem pr = {};
    pr.rows.x = x;
    pr.rows.dtype = dtype;
    pr.rows.rows = items * beams;
    pr.rows.cols = static_cast<int>(cols);
    pr.rows.row_stride = row_stride;
    pr.rows.temperature = temperature;
    pr.rows.top_k = static_cast<int>(std::min<int64_t>(count, cols));
    pr.rows.stream = reinterpret_cast<cudaStream_t>(stream);
    pr.items = items;
    pr.beams = beams;
    pr.count = count;
    pr.rows.beam_scores = scores;
    pr.rows.beam_ended = ended;
    pr.scale = scale;
    pr.end_token = end_token;
    pr.inv_t = 1.0 / static_cast<double>(temperature);
    pr.tokens = tokens;
    pr.parents = parents;
    pr.out_scores = out_scores;
    BeamPlan plan;
    if ((s = beam_plan(items, beams, cols, dtype, pr.rows.top_k, caps, &plan)) != ARGR_OK) return s;
    if (const size_t need = beam_scratch(plan, pr.rows.rows, pr.rows.top_k)) {
        if (!scratch || misaligned(scratch, 16) || scratch_bytes < need) return ARGR_ESCRATCH;
        pr.rows.beam_keys = static_cast<unsigned long long*>(scratch);
        pr.rows.beam_sums = reinterpret_cast<float2*>(pr.rows.beam_keys + pr.rows.rows * pr.rows.top_k);
    }
    return launched(dtype == ARGR_F32   ? launch_beam_select_f32(pr, plan, caps)
                    : dtype == ARGR_F16 ? launch_beam_select_f16(pr, plan, caps)
                                        : launch_beam_select_bf16(pr, plan, caps));
}

size_t argreduce_beam_scratch_bytes(int64_t items, int32_t beams, int64_t cols, argr_dtype dtype, int32_t count) {
    argr_caps caps;
    BeamPlan plan;
    if (items < 1 || beams < 1 || beams > ARGR_BEAM_MAX_BEAMS || items > INT_MAX / 64 || cols < 1 || cols > INT_MAX || count < 1 ||
        count > ARGR_LOGITS_MAX_TOP || (dtype != ARGR_F32 && dtype != ARGR_F16 && dtype != ARGR_BF16) || current_caps(&caps) != ARGR_OK)
        return 0;
    const int k = static_cast<int>(std::min<int64_t>(count, cols));
    if (beam_plan(items, beams, cols, dtype, k, caps, &plan) != ARGR_OK) return 0;
    return beam_scratch(plan, items * beams, k);
}

argr_status argreduce_beam_reorder_check(void* const* states, int32_t n_states, int64_t items, int32_t beams,
                                         int64_t item_stride, int64_t beam_stride, int64_t outer, int64_t outer_stride,
                                         int64_t positions, int64_t position_bytes, const int64_t* parents,
                                         const int64_t* lengths) {
    if (n_states < 0 || n_states > ARGR_REORDER_MAX_STATES || items < 0 || beams < 1 || beams > ARGR_BEAM_MAX_BEAMS ||
        outer < 0 || positions < 0 || position_bytes < 1 || item_stride < 0 || beam_stride < 0 || outer_stride < 0)
        return ARGR_EINVAL;
    if (misaligned(parents, 8) || misaligned(lengths, 8)) return ARGR_EINVAL;
    if (n_states == 0 || items == 0 || outer == 0 || positions == 0) return ARGR_OK;
    if (!states || !parents || positions > INT64_MAX / position_bytes || items > INT64_MAX / 8 / beams) return ARGR_EINVAL;
    Layout lay;
    if (!reorder_layout(items, beams, item_stride, beam_stride, outer, outer_stride, positions * position_bytes, &lay))
        return ARGR_EINVAL;
    uintptr_t at[ARGR_REORDER_MAX_STATES];
    for (int i = 0; i < n_states; ++i) {
        if (!states[i]) return ARGR_EINVAL;
        if (touches(states[i], lay.extent, parents, 8 * items * beams) ||
            (lengths && touches(states[i], lay.extent, lengths, 8 * items)))
            return ARGR_EINVAL;
        at[i] = reinterpret_cast<uintptr_t>(states[i]);
    }
    std::sort(at, at + n_states);
    for (int i = 0; i < n_states; ++i)
        for (int j = i + 1; j < n_states && at[j] - at[i] < static_cast<uintptr_t>(lay.extent); ++j)
            if (lay.meets(static_cast<int64_t>(at[j] - at[i]))) return ARGR_EINVAL;
    return ARGR_OK;
}

argr_status argreduce_beam_reorder(void* const* states, int32_t n_states, int64_t items, int32_t beams,
                                   int64_t item_stride, int64_t beam_stride, int64_t outer, int64_t outer_stride,
                                   int64_t positions, int64_t position_bytes, const int64_t* parents,
                                   const int64_t* lengths, argr_stream stream) {
    argr_status s = argreduce_beam_reorder_check(states, n_states, items, beams, item_stride, beam_stride, outer, outer_stride,
                                                 positions, position_bytes, parents, lengths);
    if (s != ARGR_OK || n_states == 0 || items == 0 || outer == 0 || positions == 0) return s;
    Layout lay;
    reorder_layout(items, beams, item_stride, beam_stride, outer, outer_stride, positions * position_bytes, &lay);
    uintptr_t low = 0;
    for (int i = 0; i < n_states; ++i) low |= reinterpret_cast<uintptr_t>(states[i]);
    if (beams == 1) return ARGR_OK;  // nothing can move
    argr_caps caps;
    if ((s = current_caps(&caps)) != ARGR_OK) return s;
    ReorderProblem pr = {};
    pr.items = items;
    pr.beams = beams;
    pr.item_stride = item_stride;
    pr.beam_stride = beam_stride;
    pr.outer = outer;
    pr.outer_stride = outer_stride;
    pr.positions = positions;
    pr.pos_bytes = position_bytes;
    for (int i = 0; i < lay.n; ++i) low |= static_cast<uintptr_t>(lay.dim[i].stride);
    pr.word = low % 16 == 0 ? 16 : static_cast<int>(low & (~low + 1));
    pr.parents = parents;
    pr.lengths = lengths;
    pr.stream = reinterpret_cast<cudaStream_t>(stream);
    for (int i = 0; i < n_states; i += kReorderStates) {
        pr.n = std::min(kReorderStates, n_states - i);
        for (int j = 0; j < pr.n; ++j) pr.states[j] = static_cast<unsigned char*>(states[i + j]);
        if ((s = launched(launch_beam_reorder(pr, caps))) != ARGR_OK) return s;
    }
    return ARGR_OK;
}

size_t argreduce_route_scratch_bytes(int64_t rows, int64_t experts) {
    argr_caps caps;
    if (rows < 1 || experts < 1 || experts > ARGR_ROUTE_MAX_EXPERTS || current_caps(&caps) != ARGR_OK) return 0;
    return route_scratch(rows, experts, caps);
}

argr_status argreduce_route(const void* x, argr_dtype dtype, int64_t rows, int64_t experts, int64_t row_stride,
                            int32_t top_k, int normalize, const uint8_t* valid, float* weights, int64_t* ids,
                            float* lse, int64_t* counts, int64_t* taken, float* balance, void* scratch,
                            size_t scratch_bytes, argr_stream stream) {
    argr_status s = check_route(x, dtype, rows, experts, row_stride, top_k);
    if (s != ARGR_OK) return s;
    if (misaligned(weights, 4) || misaligned(ids, 8) || misaligned(lse, 4) || misaligned(counts, 8) ||
        misaligned(taken, 8) || misaligned(balance, 4))
        return ARGR_EINVAL;
    if (!counts != !taken || (balance && !counts)) return ARGR_EINVAL;
    if (rows > 0 && (!weights || !ids || !lse)) return ARGR_EINVAL;
    if (rows == 0 && !counts) return ARGR_OK;
    argr_caps caps;
    if ((s = current_caps(&caps)) != ARGR_OK) return s;
    RouteProblem pr = {};
    pr.x = x;
    pr.dtype = dtype;
    pr.rows = rows;
    pr.experts = static_cast<int>(experts);
    pr.row_stride = row_stride;
    pr.k = top_k;
    pr.normalize = normalize != 0;
    pr.valid = valid;
    pr.weights = weights;
    pr.ids = ids;
    pr.lse = lse;
    pr.counts = counts;
    pr.taken = taken;
    pr.balance = balance;
    pr.stream = reinterpret_cast<cudaStream_t>(stream);
    if (const size_t need = counts && rows > 0 ? route_scratch(rows, experts, caps) : 0) {
        if (!scratch || misaligned(scratch, 16) || scratch_bytes < need) return ARGR_ESCRATCH;
        pr.part_sums = static_cast<float*>(scratch);
        pr.part_counts = reinterpret_cast<int*>(static_cast<char*>(scratch) +
                                                route_sums_bytes(route_grid(rows, experts, true, caps).ctas, experts));
    }
    if (rows == 0) return launched(launch_route_finish(pr));
    return ARGR_SELECT_DISPATCH(launch_route, dtype, pr, caps);
}

argr_status argreduce_route_backward(const void* x, argr_dtype dtype, int64_t rows, int64_t experts,
                                     int64_t row_stride, int32_t top_k, int normalize, const float* weights,
                                     const int64_t* ids, const float* lse, const int64_t* counts,
                                     const int64_t* taken, const float* grad_weights, const float* grad_lse,
                                     const float* grad_balance, void* grad, int64_t grad_stride, argr_stream stream) {
    argr_status s = check_route(x, dtype, rows, experts, row_stride, top_k);
    if (s != ARGR_OK) return s;
    if (misaligned(weights, 4) || misaligned(ids, 8) || misaligned(lse, 4) || misaligned(counts, 8) ||
        misaligned(taken, 8) || misaligned(grad_weights, 4) || misaligned(grad_lse, 4) || misaligned(grad_balance, 4))
        return ARGR_EINVAL;
    if (rows == 0) return ARGR_OK;
    if (!lse || (grad_weights && (!weights || !ids)) || (grad_balance && (!counts || !taken))) return ARGR_EINVAL;
    if ((s = check_grad(x, dtype, rows, experts, row_stride, grad, grad_stride)) != ARGR_OK) return s;
    argr_caps caps;
    if ((s = current_caps(&caps)) != ARGR_OK) return s;
    RouteProblem pr = {};
    pr.x = x;
    pr.dtype = dtype;
    pr.rows = rows;
    pr.experts = static_cast<int>(experts);
    pr.row_stride = row_stride;
    pr.k = top_k;
    pr.normalize = normalize != 0;
    pr.weights = const_cast<float*>(weights);
    pr.ids = const_cast<int64_t*>(ids);
    pr.lse = const_cast<float*>(lse);
    pr.counts = const_cast<int64_t*>(counts);
    pr.taken = const_cast<int64_t*>(taken);
    pr.grad_weights = grad_weights;
    pr.grad_lse = grad_lse;
    pr.grad_balance = grad_balance;
    pr.grad = grad;
    pr.grad_stride = grad_stride;
    pr.stream = reinterpret_cast<cudaStream_t>(stream);
    return ARGR_SELECT_DISPATCH(launch_route_grad, dtype, pr, caps);
}

}  // extern "C"
