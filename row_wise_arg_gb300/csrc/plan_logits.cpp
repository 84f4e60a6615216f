// Planner of the vocabulary-row operators: pure host code. Unless a rule says
// otherwise, its figures come from one call repeated on one input, which up to about 100 MB
// then comes from L2 (both sides of a rule alike).
#include <algorithm>
#include <climits>
#include <cstring>

#include "logits.h"

namespace argr {
namespace {

constexpr int64_t kMaxGridRows = 1 << 24;
constexpr size_t kStreamSmem = 110 * 1024;  // two CTAs per SM
constexpr int64_t kStepPart = 41 * 1024;    // bytes of a row per CTA of the step's kernel

bool forward(int what) { return what == ARGR_LOGITS_LOGPROBS || what == ARGR_LOGITS_DISTILL || what == ARGR_LOGITS_DISTILL_STEP; }

bool valid_problem(int what, int64_t rows, int64_t cols, int dtype, int k) {
    return what >= ARGR_LOGITS_LOGPROBS && what <= ARGR_LOGITS_DISTILL_STEP && rows >= 0 && cols >= 1 &&
           cols <= INT_MAX && k >= 0 && k <= ARGR_LOGITS_MAX_SLOTS &&
           (dtype == ARGR_F32 || dtype == ARGR_F16 || dtype == ARGR_BF16);
}

// Finishing warps that keep up with the streaming ones. Measured (two CTAs per SM): a
// row streams at 22 bytes per ns; a finish takes about 5 us, 0.1 us per slot of a
// distillation, or 0.3 us per alternative and 4 ns per 128-byte group of the row.
// [2048, 202048] bf16, top 20: 164, 152, 154 us with 1, 2, 3 of them; top 64: 222,
// 176, 168 us; [4096, 65536] bf16, 32 slots: 112, 90 us with 1, 2.
int stream_finishers(bool distill, int64_t row_bytes, int k) {
    const double row_us = row_bytes / 22.0e3;
    const double finish_us = 5.0 + (distill ? 0.1 * k : k > 0 ? 0.3 * k + 0.004 * (row_bytes / 128) : 0.0);
    return finish_us <= row_us ? 1 : finish_us <= 2 * row_us ? 2 : 3;
}

}  // namespace

// The most that any mode of the kernel lays out (logits_stream.cuh, StreamLayout).
size_t logits_stream_smem(bool distill, int64_t cols, int dtype, int k, int warps, int finishers) {
    const int64_t elems = dtype == ARGR_F32 ? 32 : 64;
    const size_t slots = static_cast<size_t>(cols / elems + 6);
    size_t buffer = 16 * static_cast<size_t>(warps) + 16;
    if (distill) buffer += slots * elems / 8 + 64 + 12 * static_cast<size_t>(k);
    else if (k > 0) buffer += 4 * slots + slots / 8 + 64 + 128 * static_cast<size_t>(warps);
    return (finishers + 1) * buffer + (!distill && k > 0 ? finishers * (8 * (1024 + 192) + 2 * 640) : 0);
}

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
        // chunks of about 64 KB (four groups per thread); down to one group per thread
        // while that leaves fewer than four CTAs per SM
        out->block = 256;
        out->grid_rows = std::min<int64_t>(rows, 65535);
        const int64_t groups = cols / (dtype == ARGR_F32 ? 16 : 32);
        int64_t chunks = std::max<int64_t>(1, (groups + 1023) / 1024);
        chunks = std::max(chunks, std::min((groups + 255) / 256, (4 * static_cast<int64_t>(caps.sm_count) + rows - 1) / rows));
        out->blocks_per_row = std::min<int64_t>(4096, chunks);
        return ARGR_OK;
    }
    const int64_t groups = cols / (dtype == ARGR_F32 ? 16 : 32);
    out->grid_rows = std::min<int64_t>(rows, kMaxGridRows);
    if (what == ARGR_LOGITS_DISTILL_STEP) {
        // Parts of about 40 KB, five or more CTAs of 128 threads per SM, whose phases
        // overlap; more parts while the rows are few. Clusters of an odd size find fewer places
        // (SMs come in pairs): [1024, 202048] bf16, 64 slots: 175, 195, 168, 183, 156, 169, 197 us with
        // 6, 7, 8, 9, 10, 12, 16 CTAs; [2048, 65536]: 113, 121, 103 with 2, 3, 4. Of 8 CTAs with
        // 256, 192, 128, 96 threads: 180, 176, 168, 177 us.
        const int most = std::min(16, caps.max_cluster);
        int64_t c = std::max<int64_t>(1, (groups * 64 + kStepPart - 1) / kStepPart);
        if (c > 1) c += c % 2;
        while (2 * c <= most && rows * c < 4 * caps.sm_count && groups / (2 * c) >= 128) c *= 2;
        c = std::min<int64_t>(c, most);
        if ((groups + c - 1) / c * 64 <= kStepMaxChunk) {
            out->path = ARGR_PATH_LOGITS_STEP;
            out->cluster = static_cast<int>(c);
            out->block = 128;
            while (out->block > 32 && out->block > groups / c) out->block /= 2;
            return ARGR_OK;
        }
    }
    // Long rows, and enough of them to keep two persistent CTAs per SM busy: the
    // streaming kernel. Rows below the limits finish too often for it ([8192, 32000]
    // bf16: 120 us against 100 us with a CTA of 128 threads per row; [4096, 65536] bf16: 98
    // against 104 us, with 20 alternatives 119 against 116 us); so does a last round that few CTAs
    // take part in. Streaming against a CTA per row, us, inputs rotating past L2, the last round 54, 69, 79,
    // 84, 89, 99% full (330 to 600 rows): [., 202048] bf16 31 / 35, 40 / 39, 41 / 42, 42 / 45, 42 / 48, 43 / 54, with the top
    // 20 43 / 51, 54 / 46, 54 / 54, 55 / 60, 55 / 65, 55 / 71; [., 100003] f16, 32 slots and a tail 22.7 / 21.7, 25.9 / 22.7,
    // 26.6 / 23.7, 27.1 / 24.4, 27.1 / 24.5, 27.4 / 26.1. The limit, 85%, lies between these.
    const int es = dtype == ARGR_F32 ? 4 : 2;
    const bool distill = what != ARGR_LOGITS_LOGPROBS;
    const int64_t ctas = 2 * static_cast<int64_t>(caps.sm_count), row_bytes = cols * es;
    const int64_t rounds = (rows + ctas - 1) / ctas;
    if (row_bytes >= (distill || k == 0 ? 96 : 160) * 1024 && rows * 100 >= rounds * ctas * 85) {
        for (int f = stream_finishers(distill, row_bytes, k); f >= 1; --f) {
            if (logits_stream_smem(distill, cols, dtype, k, 16, f) > kStreamSmem) continue;
            out->path = ARGR_PATH_LOGITS_STREAM;
            out->grid_rows = ctas;
            out->group = f;
            return ARGR_OK;
        }
    }
    if (!distill && k > 0) {
        // With alternatives: clusters while every CTA still has an SM of its own ([32, 202048] bf16, top 20:
        // 10.4, 15.4 us with 4, 8 CTAs of 512, 256 threads; [100, 100000]: 11.0, 17.0 us with 1, 2). Then
        // 512 threads; 256 for two CTAs per SM, and where neither smaller CTAs fit one wave nor 16 groups a
        // thread suffice ([256, 128000] bf16, top 64: 45, 19 us with 512, 256; [700, 65536], top 40: 38, 23, 37
        // us with 256, 128, 64; [4096, 50257], top 20: 118, 98, 110; [8192, 32000]: 182, 138, 122, 146 down to 32;
        // [1000, 131072]: 63, 81 with 256, 128).
        while (out->cluster < std::min(16, caps.max_cluster) && 2 * rows * out->cluster <= caps.sm_count &&
               groups / (2 * out->cluster) >= 128)
            out->cluster *= 2;
        const int64_t per_cta = groups / out->cluster, n = rows * out->cluster;
        if (n > caps.sm_count) {
            out->block = 256;
            while (out->block > 32 && per_cta <= 8 * out->block &&
                   n > (out->block == 256 ? 3 : 640 / out->block) * static_cast<int64_t>(caps.sm_count))
                out->block /= 2;
            // the threshold for alternatives needs more threads than alternatives to be near them
            while (out->block < 256 && out->block < 2 * k) out->block *= 2;
        } else {
            while (out->block > 32 && out->block / 2 >= per_cta && out->block > 2 * k) out->block /= 2;
        }
        return ARGR_OK;
    }
    // Clusters until there are about three CTAs for two SMs, a group per thread, and
    // 256 threads where more than two CTAs per SM would make a second wave ([64, 202048] bf16, 64 slots:
    // 25, 16 us with 16, 8 CTAs). Where the rows alone are three per SM, about eight groups per thread:
    // small CTAs, whose phases overlap ([512, 100003] f16, 32 slots: 29, 25, 34 us with 512, 256, 128 threads).
    while (out->cluster < std::min(16, caps.max_cluster) && 5 * rows * out->cluster < 7 * caps.sm_count &&
           groups / (2 * out->cluster) >= 128)
        out->cluster *= 2;
    const int64_t per_cta = groups / out->cluster;
    if (out->cluster == 1 && rows >= 3 * caps.sm_count) {
        while (out->block > 32 && out->block * 8 > per_cta + per_cta / 8) out->block /= 2;
    } else {
        if (rows * out->cluster > ctas) out->block = 256;
        while (out->block > 32 && out->block / 2 >= per_cta) out->block /= 2;
    }
    return ARGR_OK;
}

argr_status check_logits_plan(int what, const argr_plan& p, int64_t rows, int64_t cols, int dtype, int k,
                              const argr_caps& caps) {
    if (!valid_problem(what, rows, cols, dtype, k) || caps.sm_count < 1) return ARGR_EINVAL;
    const bool step = what == ARGR_LOGITS_DISTILL_STEP && p.path == ARGR_PATH_LOGITS_STEP;
    const bool stream = forward(what) && p.path == ARGR_PATH_LOGITS_STREAM;
    if (!step && !stream && p.path != (forward(what) ? ARGR_PATH_LOGITS : ARGR_PATH_LOGITS_GRAD)) return ARGR_EINVAL;
    if (p.block < 32 || p.block > 512 || p.block % 32) return ARGR_EINVAL;
    if (p.flags & ~(ARGR_PLAN_PDL | (step ? ARGR_PLAN_TEST_EXPIRE : 0))) return ARGR_EINVAL;
    if (p.path == ARGR_PATH_LOGITS_GRAD) {
        if (p.block > 256) return ARGR_EINVAL;
        if (p.grid_rows < 1 || p.grid_rows > 65535 || p.blocks_per_row < 1 || p.blocks_per_row > 4096 || p.cluster != 1)
            return ARGR_EINVAL;
    } else {
        if (p.grid_rows < 1 || p.grid_rows > kMaxGridRows || p.blocks_per_row != 1) return ARGR_EINVAL;
        if (p.cluster < 1 || p.cluster > 16) return ARGR_EINVAL;
        if (stream &&
            (p.cluster != 1 || p.group < 1 || p.group > 3 || p.block < 32 * (p.group + 1) ||
             logits_stream_smem(what != ARGR_LOGITS_LOGPROBS, cols, dtype, k, p.block / 32, p.group) > kStreamSmem))
            return ARGR_EINVAL;
        if (step) {
            const int64_t groups = cols / (dtype == ARGR_F32 ? 16 : 32);
            if (p.block > 256 || (groups + p.cluster - 1) / p.cluster * 64 > kStepMaxChunk) return ARGR_EINVAL;
        }
        if (p.cluster > caps.max_cluster) return ARGR_EUNSUPPORTED;
    }
    return ARGR_OK;
}

}  // namespace argr
