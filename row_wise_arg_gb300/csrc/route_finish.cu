// Joins what the CTAs of a router's kernel left: per-expert counts, the number of
// rows that take part, and the balance loss (route.cuh).
#include "logits_common.cuh"
#include "select.h"

namespace argr {

constexpr int kFinishBlock = 1024;

__global__ void __launch_bounds__(kFinishBlock) route_finish_kernel(const RouteProblem pr) {
    __shared__ double red[32];
    __shared__ long long rows;
    const int t = threadIdx.x, E = pr.experts;
    allow_dependents();
    grid_dependency_wait();
    double sum = 0.0;
    for (int e = t; e <= E; e += kFinishBlock) {
        long long n = 0;
        double p = 0.0;
        for (int b = 0; b < pr.ctas; ++b) {
            n += pr.part_counts[static_cast<int64_t>(b) * (E + 1) + e];
            if (pr.balance && e < E) p += pr.part_sums[static_cast<int64_t>(b) * E + e];
        }
        if (e < E) pr.counts[e] = n;
        else {
            *pr.taken = n;
            rows = n;
        }
        sum += static_cast<double>(n) * p;
    }
    if (!pr.balance) return;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((t & 31) == 0) red[t >> 5] = sum;
    __syncthreads();
    if (t == 0) {
        double all = 0.0;
        for (int w = 0; w < kFinishBlock / 32; ++w) all += red[w];
        const double n = static_cast<double>(rows > 0 ? rows : 1);
        *pr.balance = static_cast<float>(all * E / (pr.k * n * n));
    }
}

cudaError_t launch_route_finish(const RouteProblem& pr) {
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    return launch_ex_smem(route_finish_kernel, dim3(1), dim3(kFinishBlock), 1, 0, p, pr.stream, pr);
}

int route_ctas(int64_t rows, int experts, const argr_caps& caps) {
    (void)experts;
    const int64_t want = (rows + kRouteBlock / 32 - 1) / (kRouteBlock / 32);
    int64_t most = 4 * static_cast<int64_t>(caps.sm_count);
    if (most > kRouteMaxCtas) most = kRouteMaxCtas;
    return static_cast<int>(want < most ? want : most);
}

}  // namespace argr
