// The merge of lists that a kernel over many rows left in scratch (beam_select.cuh): a CTA per item.
#include "beam_select.cuh"

namespace argr {

__global__ void __launch_bounds__(kMergeBlock) beam_merge_kernel(const BeamProblem pr, float scale2) {
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ MergeShared merge;
    const int64_t item = blockIdx.x, r = item * pr.beams;
    allow_dependents();
    grid_dependency_wait();
    load_beams(pr, item, merge);
    __syncthreads();
    const int k = pr.rows.top_k;
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(dyn);
    merge_beams(pr, item, k, 0, pr.rows.beam_keys + r * k, keys, reinterpret_cast<float*>(keys + pr.beams * k),
                pr.rows.beam_sums + r, scale2, merge);
}

cudaError_t launch_beam_merge(const BeamProblem& pr) {
    static KernelLaunchCache cache;
    const size_t smem = 12 * static_cast<size_t>(pr.beams) * pr.rows.top_k;
    const cudaError_t e = ensure_smem_limit(beam_merge_kernel, smem + sizeof(MergeShared) + 1024, cache);
    if (e != cudaSuccess) return e;
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    return launch_ex_smem(beam_merge_kernel, dim3(static_cast<unsigned>(pr.items)), dim3(kMergeBlock), 1, smem, p,
                          pr.rows.stream, pr, kLog2E / pr.rows.temperature);
}

}  // namespace argr
