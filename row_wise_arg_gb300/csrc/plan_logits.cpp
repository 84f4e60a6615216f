// Planner of the vocabulary-row operators: pure host code.
#include <algorithm>
#include <climits>
#include <cstring>

#include "logits.h"

namespace argr {
namespace {

constexpr int64_t kMaxGridRows = 1 << 24;

bool forward(int what) { return what == ARGR_LOGITS_LOGPROBS || what == ARGR_LOGITS_DISTILL || what == ARGR_LOGITS_DISTILL_STEP; }

bool valid_problem(int what, int64_t rows, int64_t cols, int dtype, int k) {
    return what >= ARGR_LOGITS_LOGPROBS && what <= ARGR_LOGITS_DISTILL_STEP && rows >= 0 && cols >= 1 &&
           cols <= INT_MAX && k >= 0 && k <= ARGR_LOGITS_MAX_SLOTS &&
           (dtype == ARGR_F32 || dtype == ARGR_F16 || dtype == ARGR_BF16);
}

}  // namespace

argr_status make_logits_plan(int what, int64_t rows, int64_t cols, int dtype, int k, const argr_caps& caps,
                             argr_plan* out) {
    std::memset(out, 0, sizeof(*out));
    if (dtype == ARGR_F64 || dtype == ARGR_I32 || dtype == ARGR_I64) return ARGR_EUNSUPPORTED;
    if (!valid_problem(what, rows, cols, dtype, k) || caps.sm_count < 1) return ARGR_EINVAL;
    if (rows == 0) return ARGR_OK;
    out->flags = ARGR_PLAN_PDL;
    out->block = 512;
    out->cluster = 1;
    out->blocks_per_row = 1;
    out->path = forward(what) ? ARGR_PATH_LOGITS : ARGR_PATH_LOGITS_GRAD;
    if (out->path == ARGR_PATH_LOGITS_GRAD) {
        // chunks of about 64 KB (four groups per thread)
        out->block = 256;
        out->grid_rows = std::min<int64_t>(rows, 65535);
        const int64_t groups = cols / (dtype == ARGR_F32 ? 16 : 32);
        out->blocks_per_row = std::min<int64_t>(4096, std::max<int64_t>(1, (groups + 1023) / 1024));
        return ARGR_OK;
    }
    const int64_t groups = cols / (dtype == ARGR_F32 ? 16 : 32);
    while (out->cluster < std::min(16, caps.max_cluster) && rows * out->cluster < 4 * caps.sm_count &&
           groups / (2 * out->cluster) >= 128)
        out->cluster *= 2;
    const int64_t per_cta = groups / out->cluster;
    while (out->block > 32 && out->block > per_cta) out->block /= 2;
    out->grid_rows = std::min<int64_t>(rows, kMaxGridRows);
    return ARGR_OK;
}

argr_status check_logits_plan(int what, const argr_plan& p, int64_t rows, int64_t cols, int dtype, int k,
                              const argr_caps& caps) {
    if (!valid_problem(what, rows, cols, dtype, k) || caps.sm_count < 1) return ARGR_EINVAL;
    if (p.path != (forward(what) ? ARGR_PATH_LOGITS : ARGR_PATH_LOGITS_GRAD)) return ARGR_EINVAL;
    if (p.block < 32 || p.block > 512 || p.block % 32) return ARGR_EINVAL;
    if (p.flags & ~ARGR_PLAN_PDL) return ARGR_EINVAL;
    if (p.path == ARGR_PATH_LOGITS_GRAD) {
        if (p.block > 256) return ARGR_EINVAL;
        if (p.grid_rows < 1 || p.grid_rows > 65535 || p.blocks_per_row < 1 || p.blocks_per_row > 4096 || p.cluster != 1)
            return ARGR_EINVAL;
    } else {
        if (p.grid_rows < 1 || p.grid_rows > kMaxGridRows || p.blocks_per_row != 1) return ARGR_EINVAL;
        if (p.cluster < 1 || p.cluster > 16 || (p.cluster & (p.cluster - 1))) return ARGR_EINVAL;
        if (p.cluster > caps.max_cluster) return ARGR_EUNSUPPORTED;
    }
    return ARGR_OK;
}

}  // namespace argr
