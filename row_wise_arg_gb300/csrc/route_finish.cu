// Joins what the CTAs of a router's kernel left: per-expert counts, the number of
// rows that take part, and the balance loss (route.cuh). One cluster: each CTA
// joins a share of the experts, a lane to an expert, its warps the CTAs' parts in turns. About 3.5 us after a route of 256 experts (152 CTAs'
// parts, 314 KB): a launch, two rounds of loads, a cluster's barriers. (One CTA took 150 us for 608 parts, a thread to an expert.)
#include "logits_forward.cuh"
#include "select.h"

namespace argr {

constexpr int kFinishCtas = 8;
constexpr int kFinishWarps = 32;

__global__ void __cluster_dims__(kFinishCtas, 1, 1) __launch_bounds__(32 * kFinishWarps) route_finish_kernel(const RouteProblem pr) {
    __shared__ int parts[kFinishWarps][32];
    __shared__ float sums[kFinishWarps][32];
    __shared__ double shares[kFinishCtas];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = pr.experts, cta = static_cast<int>(blockIdx.x);
    allow_dependents();
    grid_dependency_wait();
    double mine = 0.0;  // of warp 0's lanes
    __shared__ long long rows;
    // 32 experts at a time; the rows that take part follow the last expert
    for (int e0 = 32 * cta; e0 <= E; e0 += 32 * kFinishCtas) {
        const int e = e0 + lane;
        int n = 0;
        float p = 0.0f;
        if (e <= E) {
#pragma unroll 4
            for (int b = warp; b < pr.ctas; b += kFinishWarps) {
                n += pr.part_counts[static_cast<int64_t>(b) * (E + 1) + e];
                if (pr.balance && e < E) p += pr.part_sums[static_cast<int64_t>(b) * E + e];
            }
        }
        parts[warp][lane] = n;
        sums[warp][lane] = p;
        __syncthreads();
        if (warp == 0 && e <= E) {
            long long all = 0;
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < kFinishWarps; ++w) {
                all += parts[w][lane];
                t += sums[w][lane];
            }
            if (e < E) {
                pr.counts[e] = all;
                mine += static_cast<double>(all) * t;
            } else {
                *pr.taken = all;
                rows = all;
            }
        }
        __syncthreads();
    }
    if (!pr.balance) return;
    if (warp == 0) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    }
    // to the CTA that has the number of rows
    const int owner = E / 32 % kFinishCtas;
    cluster_ready();
    cluster_wait();
    if (threadIdx.x == 0)
        st_cluster(cluster_addr(smem_u32(&shares[cta]), owner), static_cast<unsigned long long>(__double_as_longlong(mine)));
    cluster_arrive();
    cluster_wait();
    if (cta == owner && threadIdx.x == 0) {
        double all = 0.0;
        for (int q = 0; q < kFinishCtas; ++q) all += shares[q];
        *pr.balance = route_balance(all, rows, E, pr.k);
    }
}

cudaError_t launch_route_finish(const RouteProblem& pr) {
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    return launch_ex_smem(route_finish_kernel, dim3(kFinishCtas), dim3(32 * kFinishWarps), 1, 0, p, pr.stream, pr);
}

}  // namespace argr
