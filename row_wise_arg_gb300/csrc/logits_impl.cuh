// Launchers of the vocabulary-row kernels, templated on the element type.
#pragma once

#include "logits_forward.cuh"
#include "logits_grad.cuh"

namespace argr {

// ---------------------------------------------------------------------------
// Launchers.
// ---------------------------------------------------------------------------
inline float scale2_of(const LogitsProblem& pr) { return kLog2E / pr.temperature; }

// Launch a forward kernel: `ranks` CTAs per row, `smem` bytes of dynamic shared memory.
template <class K>
cudaError_t launch_forward(K kern, KernelLaunchCache& cache, const argr_plan& p, const LogitsProblem& pr, size_t smem,
                           int seg_slots) {
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
                          seg_slots);
}

// Slots of the longest segment of a CTA's part of a row (a multiple of 4).
template <class Tag>
int segment_slots(const argr_plan& p, int cols) {
    const int64_t groups = (cols / kGroupElems<Tag> + p.cluster - 1) / p.cluster;
    return static_cast<int>((groups < kSegGroups ? groups : kSegGroups) + 2 + 3) / 4 * 4;
}

template <class Tag>
cudaError_t launch_logprobs_t(const argr_plan& p, const LogitsProblem& pr) {
    const int slots = segment_slots<Tag>(p, pr.cols);
    if (pr.top_k == 0) {
        static KernelLaunchCache cache;
        return launch_forward(logprobs_kernel<Tag, false>, cache, p, pr, 0, slots);
    }
    static KernelLaunchCache cache;
    const size_t keys = cand_room(pr.top_k, kGroupElems<Tag>) + 2 * ARGR_LOGITS_MAX_TOP +
                        (p.cluster > 1 ? p.cluster * pr.top_k : 0);
    return launch_forward(logprobs_kernel<Tag, true>, cache, p, pr, 8 * keys + 4 * slots + 2 * kListGroups, slots);
}
template <class Tag>
cudaError_t launch_distill_t(const argr_plan& p, const LogitsProblem& pr) {
    const int slots = segment_slots<Tag>(p, pr.cols);
    if (!pr.tail) {
        static KernelLaunchCache cache;
        return launch_forward(distill_kernel<Tag, false>, cache, p, pr, 0, slots);
    }
    static KernelLaunchCache cache;
    return launch_forward(distill_kernel<Tag, true>, cache, p, pr, static_cast<size_t>(slots) * kGroupElems<Tag> / 8 + 16,
                          slots);
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
    return launch_ex(distill_grad_kernel<Tag>, grad_grid(p), dim3(p.block), 1, p, pr.stream, pr, scale2_of(pr));
}

#define ARGR_DEFINE_LOGITS(sfx, Tag)                                                                                 \
    namespace argr {                                                                                                 \
    cudaError_t launch_logprobs_##sfx(const argr_plan& p, const LogitsProblem& pr) {                                 \
        return launch_logprobs_t<Tag>(p, pr);                                                                        \
    }                                                                                                                \
    cudaError_t launch_distill_##sfx(const argr_plan& p, const LogitsProblem& pr) {                                  \
        return launch_distill_t<Tag>(p, pr);                                                                         \
    }                                                                                                                \
    cudaError_t launch_logprobs_grad_##sfx(const argr_plan& p, const LogitsProblem& pr) {                            \
        return launch_logprobs_grad_t<Tag>(p, pr);                                                                   \
    }                                                                                                                \
    cudaError_t launch_distill_grad_##sfx(const argr_plan& p, const LogitsProblem& pr) {                             \
        return launch_distill_grad_t<Tag>(p, pr);                                                                    \
    }                                                                                                                \
    }

}  // namespace argr
