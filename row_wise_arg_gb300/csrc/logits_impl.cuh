// Launchers of the vocabulary-row kernels, templated on the element type.
#pragma once

#include "logits_forward.cuh"
#include "logits_grad.cuh"
#include "logits_step.cuh"
#include "logits_stream.cuh"

namespace argr {

// ---------------------------------------------------------------------------
// Launchers.
// ---------------------------------------------------------------------------
inline float scale2_of(const LogitsProblem& pr) { return kLog2E / pr.temperature; }

// Launch a forward kernel: `ranks` CTAs per row, `smem` bytes of dynamic shared memory.
template <class K, typename... More>
cudaError_t launch_forward(K kern, KernelLaunchCache& cache, const argr_plan& p, const LogitsProblem& pr, size_t smem,
                           More... more) {
    cudaError_t e = ensure_smem_limit(kern, smem + 2048, cache);  // with the static part
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(p.grid_rows * p.cluster));
    if (p.cluster > 1) {
        bool ok = false;
        if (p.cluster > 8 && (e = allow_big_cluster(kern, cache)) != cudaSuccess) return e;
        if ((e = cluster_fits(kern, dim3(static_cast<unsigned>(p.cluster)), p.block, p.cluster, smem, cache, &ok)) !=
            cudaSuccess)
            return e;
        if (!ok) return cudaErrorInvalidClusterSize;
    }
    return launch_ex_smem(kern, grid, dim3(p.block), p.cluster, smem, p, pr.stream, pr, scale2_of(pr), p.cluster,
                          more...);
}

// Slots of the longest segment of a CTA's part of a row (a multiple of 4).
template <class Tag>
int segment_slots(const argr_plan& p, int cols) {
    const int64_t groups = (cols / kGroupElems<Tag> + p.cluster - 1) / p.cluster;
    return static_cast<int>((groups < kSegGroups ? groups : kSegGroups) + 2 + 3) / 4 * 4;
}

// The persistent kernel of one mode: p.group finishers per CTA.
template <class Tag, int MODE>
cudaError_t launch_stream(const argr_plan& p, const LogitsProblem& pr) {
    auto kern = logits_stream_kernel<Tag, MODE>;
    static KernelLaunchCache cache;
    const size_t smem = StreamLayout(MODE, p.block / 32 - p.group, p.group, kWideElems<Tag>, pr.cols, pr.slots).total;
    const cudaError_t e = ensure_smem_limit(kern, smem, cache);
    if (e != cudaSuccess) return e;
    return launch_ex_smem(kern, dim3(static_cast<unsigned>(p.grid_rows)), dim3(p.block), 1, smem, p, pr.stream, pr,
                          scale2_of(pr), p.group);
}

template <class Tag>
cudaError_t launch_logprobs_t(const argr_plan& p, const LogitsProblem& pr) {
    if (p.path == ARGR_PATH_LOGITS_STREAM)
        return pr.top_k ? launch_stream<Tag, kStreamTop>(p, pr) : launch_stream<Tag, kStreamSums>(p, pr);
    const int slots = segment_slots<Tag>(p, pr.cols);
    if (pr.top_k == 0) {
        static KernelLaunchCache cache;
        return launch_forward(logprobs_kernel<Tag, false, kFwdMaxBlock, 2>, cache, p, pr, 0, slots);
    }
    // Alternatives need about 100 registers; with 64, what is spilled costs more than the CTAs that fewer
    // registers leave room for bring ([4096, 50257] bf16, top 20, 256 threads: 127, 99, 111 us with 64,
    // 80, 128 registers; [2048, 32000] f16, top 5, 128 threads: 41, 36, 42 with 64, 96, 128). All of
    // them where the grid then still fits ([32, 202048] bf16, top 20: 15.8 and 10.5 us with 64 and 128).
    static KernelLaunchCache caches[3];
    const size_t keys = cand_room(pr.top_k, kGroupElems<Tag>) + 2 * ARGR_LOGITS_MAX_TOP +
                        (p.cluster > 1 ? p.cluster * pr.top_k : 0);
    const size_t smem = 8 * keys + 4 * slots + 2 * kListGroups;
    argr_caps caps;
    if (current_caps(&caps) != ARGR_OK) return cudaErrorInvalidDevice;
    if (p.block > 256 || p.grid_rows * p.cluster * p.block <= static_cast<int64_t>(caps.sm_count) * kFwdMaxBlock)
        return launch_forward(logprobs_kernel<Tag, true, kFwdMaxBlock, 1>, caches[0], p, pr, smem, slots);
    return p.block > 128 ? launch_forward(logprobs_kernel<Tag, true, 256, 3>, caches[1], p, pr, smem, slots)
                         : launch_forward(logprobs_kernel<Tag, true, 128, 5>, caches[2], p, pr, smem, slots);
}
template <class Tag>
cudaError_t launch_distill_t(const argr_plan& p, const LogitsProblem& pr) {
    if (p.path == ARGR_PATH_LOGITS_STREAM)
        return pr.tail ? launch_stream<Tag, kStreamLossTail>(p, pr) : launch_stream<Tag, kStreamLoss>(p, pr);
    const int slots = segment_slots<Tag>(p, pr.cols);
    const size_t smem = Slots::bytes(pr.slots);
    if (!pr.tail) {
        static KernelLaunchCache cache;
        return launch_forward(distill_kernel<Tag, false>, cache, p, pr, smem, slots);
    }
    static KernelLaunchCache cache;
    return launch_forward(distill_kernel<Tag, true>, cache, p, pr,
                          smem + static_cast<size_t>(slots) * kGroupElems<Tag> / 8 + 16, slots);
}
// The step's kernel holds ceil(groups / C) groups of a row per CTA.
template <class Tag>
cudaError_t launch_distill_step_t(const argr_plan& p, const LogitsProblem& pr) {
    const int groups = (pr.cols / kGroupElems<Tag> + p.cluster - 1) / p.cluster;
    const int units = groups * (kGroupBytes / 16);
    const size_t smem = 16 * static_cast<size_t>(units) + Slots::bytes(pr.slots);
    static KernelLaunchCache caches[2];
    const int flags = static_cast<int>(p.flags);
    return pr.tail ? launch_forward(distill_step_kernel<Tag, true>, caches[1], p, pr, smem, units, flags)
                   : launch_forward(distill_step_kernel<Tag, false>, caches[0], p, pr, smem, units, flags);
}
inline dim3 grad_grid(const argr_plan& p) {
    return dim3(static_cast<unsigned>(p.blocks_per_row), static_cast<unsigned>(p.grid_rows < 65535 ? p.grid_rows : 65535));
}
template <class Tag>
cudaError_t launch_logprobs_grad_t(const argr_plan& p, const LogitsProblem& pr) {
    auto kern = pr.grad_entropy ? logprobs_grad_kernel<Tag, true> : logprobs_grad_kernel<Tag, false>;
    return launch_ex(kern, grad_grid(p), dim3(p.block), 1, p, pr.stream, pr, scale2_of(pr));
}
template <class Tag>
cudaError_t launch_distill_grad_t(const argr_plan& p, const LogitsProblem& pr) {
    return launch_ex_smem(distill_grad_kernel<Tag>, grad_grid(p), dim3(p.block), 1, Slots::bytes(pr.slots), p, pr.stream,
                          pr, scale2_of(pr));
}

#define ARGR_DEFINE_LOGITS(sfx, Tag)                                                                                 \
    namespace argr {                                                                                                 \
    cudaError_t read_and_clear_logits_error_##sfx(unsigned* out) {                                                   \
        return read_and_clear_error_t(out);                                                                             \
    }                                                                                                                \
    cudaError_t launch_logprobs_##sfx(const argr_plan& p, const LogitsProblem& pr) {                                 \
        return launch_logprobs_t<Tag>(p, pr);                                                                        \
    }                                                                                                                \
    cudaError_t launch_distill_##sfx(const argr_plan& p, const LogitsProblem& pr) {                                  \
        return launch_distill_t<Tag>(p, pr);                                                                         \
    }                                                                                                                \
    cudaError_t launch_distill_step_##sfx(const argr_plan& p, const LogitsProblem& pr) {                             \
        return launch_distill_step_t<Tag>(p, pr);                                                                    \
    }                                                                                                                \
    cudaError_t launch_logprobs_grad_##sfx(const argr_plan& p, const LogitsProblem& pr) {                            \
        return launch_logprobs_grad_t<Tag>(p, pr);                                                                   \
    }                                                                                                                \
    cudaError_t launch_distill_grad_##sfx(const argr_plan& p, const LogitsProblem& pr) {                             \
        return launch_distill_grad_t<Tag>(p, pr);                                                                    \
    }                                                                                                                \
    }

}  // namespace argr
