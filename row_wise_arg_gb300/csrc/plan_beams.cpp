// Planner of beam selection: pure host code.
#include "select.h"

namespace argr {

// Whether rows go to the persistent kernel, and its plan: those that the planner of token_logprobs streams, and last rounds
// that three quarters of the CTAs take part in (it asks for 85%; without entropies a round is shorter).
bool beam_stream_plan(int64_t rows, int64_t cols, int dtype, int k, const argr_caps& caps, argr_plan* p) {
    const int64_t ctas = 2 * static_cast<int64_t>(caps.sm_count), rounds = (rows + ctas - 1) / ctas;
    if (rows * 100 < rounds * ctas * 75) return false;
    return make_logits_plan(ARGR_LOGITS_LOGPROBS, rounds * ctas, cols, dtype, k, caps, p) == ARGR_OK &&
           p->path == ARGR_PATH_LOGITS_STREAM;
}

// A cluster's CTAs start together, wait for one another, and hold their SMs while CTA 0 merges, which costs little while
// the grid leaves room for the next one's clusters. So, for up to 16 beams: a CTA per beam, and several to a beam while
// they are two thirds of the SMs at most and have 64 KB each. Of 4 beams with 1, 2, 4
// CTAs each, 8 continuations, us in a graph of calls: [1, 4, 32000] f32 7.9, 8.0, 9.3; [1, 4, 202048] bf16 13.3, 10.9, 11.0;
// [4, 4, 128000] bf16 11.0, 9.6, 10.3; [16, 4, 202048] bf16 14.8, 20.7, 26.6. Clusters of up to 8 CTAs are kept up to two
// waves, those of 16 up to one (they find few places): cluster against a CTA per row and a merge,
// [64, 4, 128000] bf16 17.5 / 22.3 (streaming 24.6), [60, 4, 32000] 9.8 / 11.7, [30, 8, 32000] 10.7 / 12.7, but [19, 16, 202048], 32
// continuations, 60.6 / 53.3 (streaming 49.2), [19, 16, 32000] 25.8 / 24.6 (21.2 with 128 threads). Past that long rows are
// streamed ([64, 16, 202048], 32: 92, against 107.8 with a CTA per row).
BeamPlan plan_beams(int64_t items, int beams, int64_t cols, int dtype, int k, const argr_caps& caps) {
    BeamPlan p = {};
    const int64_t groups = cols / (dtype == ARGR_F32 ? 16 : 32), rows = items * beams;
    const int most = caps.max_cluster < 16 ? caps.max_cluster : 16;
    int64_t per_cta = groups, n = rows;
    argr_plan q;
    if (beams <= most && rows <= (beams <= 8 ? 2 : 1) * static_cast<int64_t>(caps.sm_count)) {
        p.cluster = beams;
        while (2 * p.cluster <= most && 3 * items * p.cluster <= caps.sm_count && (groups >> (p.shift + 1)) >= 1024) {
            p.cluster *= 2;
            ++p.shift;
        }
        per_cta = groups >> p.shift;
        n = items * p.cluster;
    } else {
        p.stream = beam_stream_plan(rows, cols, dtype, k, caps, &q);
    }
    p.block = p.cluster ? 512 : 256;
    if (n > caps.sm_count) {
        p.block = 256;
        while (p.block > 32 && per_cta <= 8 * p.block &&
               n > (p.block == 256 ? 3 : 640 / p.block) * static_cast<int64_t>(caps.sm_count))
            p.block /= 2;
        while (p.block < 256 && p.block < 2 * k) p.block *= 2;
    } else {
        while (p.block > 32 && p.block / 2 >= per_cta && p.block > 2 * k) p.block /= 2;
    }
    return p;
}

}  // namespace argr
