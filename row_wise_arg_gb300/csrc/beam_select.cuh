// A beam search's step: the continuations (beam, token) of the largest totals of
// each item, over all its beams and the vocabulary.
//
// With a beam's total s_b and its logits x, m = max x and S = sum exp((x - m) / T),
//     total_bv = s_b + (x_v - m) / T - ln S.
// Within a beam the totals come in the logits' order, so the `count` first of an
// item are among the `count` first of each of its beams: a beam's logits are read
// once, for S and for its first alternatives (logits_forward.cuh), and the
// lists of all beams are merged. Totals of different beams lie close together,
// and what decides between them is the difference of their ln S: the merge works
// in 64 bits (a handful of operations per list entry; the 64-bit unit is slow), S is the
// binary32 sum of the pass.
//
// One cluster per item: `groups` beams at a time, `ranks` CTAs to a beam. Every CTA hands
// its sums and its list to CTA 0 through distributed shared memory, which merges: no
// scratch, one launch.
#pragma once

#include "logits_forward.cuh"
#include "select.h"

namespace argr {

constexpr int kMaxBeams = ARGR_BEAM_MAX_BEAMS;

// What the merge knows of a beam.
struct BeamSum {
    double base;   // s_b - ln S
    double scale;  // of the rank
    float m;
    int state;     // kBeamGone, kBeamEnded or kBeamLive
};
constexpr int kBeamGone = 0, kBeamEnded = 1, kBeamLive = 2;

// A key that orders ranks: 0 for what is not above -inf (NaN included).
__device__ __forceinline__ unsigned long long rank_key(double rank) {
    const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(rank + 0.0));
    if (!(rank > -static_cast<double>(__int_as_float(0x7f800000)))) return 0ull;
    return b ^ ((b >> 63) ? ~0ull : 0x8000000000000000ull);
}

struct BeamLayout {
    size_t big, cand, best, list, gathered, ranks, sums, total;  // offsets
    __host__ __device__ BeamLayout(int k, int lists, int seg_slots, int group_elems) {
        size_t at = 0;
        big = at;
        at += 4 * static_cast<size_t>(seg_slots);
        cand = at;
        at += 8 * static_cast<size_t>(cand_room(k, group_elems));
        best = at;
        at += 8 * 2 * ARGR_LOGITS_MAX_TOP;
        gathered = at;
        at += 8 * static_cast<size_t>(lists) * k;
        ranks = at;
        at += 8 * static_cast<size_t>(lists) * k;
        sums = at;
        at += 8 * static_cast<size_t>(lists);
        list = at;
        at += 2 * kListGroups;
        total = (at + 15) / 16 * 16;
    }
};

// The merge, by CTA 0 of an item: the lists' entries as ranks, then the best of the
// lists' heads `count` times, by one warp.
__device__ __forceinline__ void merge_beams(const BeamProblem& pr, int64_t item, int k, int ranks,
                                            const unsigned long long* gathered, unsigned long long* keys,
                                            const float* sums, float scale2) {
    __shared__ BeamSum beam[kMaxBeams];
    __shared__ int win[ARGR_LOGITS_MAX_TOP];
    __shared__ int poisoned;
    const int t = threadIdx.x, nt = blockDim.x, lane = t & 31;
    const int beams = pr.beams, lists = beams * ranks, count = pr.count;
    if (t == 0) poisoned = 0;
    __syncthreads();
    for (int b = t; b < beams; b += nt) {
        const float s = pr.scores[item * beams + b];
        const float w = pr.scale ? pr.scale[item * beams + b] : 1.0f;
        BeamSum v;
        v.base = s;
        v.scale = w;
        v.m = 0.0f;
        v.state = s == neg_inf() ? kBeamGone : pr.ended && pr.ended[item * beams + b] ? kBeamEnded : kBeamLive;
        bool bad = v.state != kBeamGone && (!(fabsf(s) <= FLT_MAX) || !(w > 0.0f && w <= FLT_MAX));
        if (v.state == kBeamLive) {
            SoftSum c;
            for (int r = 0; r < ranks; ++r) {
                SoftSum d;
                d.m = sums[2 * (b * ranks + r)];
                d.s = sums[2 * (b * ranks + r) + 1];
                c.join(d, scale2);
            }
            v.m = c.m;
            if (c.s != c.s) bad = true;
            else if (c.empty()) v.state = kBeamGone;
            else v.base -= log(static_cast<double>(c.s));
        }
        if (bad) poisoned = 1;
        beam[b] = v;
    }
    __syncthreads();
    for (int i = t; i < lists * k; i += nt) {
        const int l = i / k, at = i - l * k;
        const BeamSum& v = beam[l / ranks];
        const unsigned long long g = gathered[i];
        double rank = v.base * v.scale;
        bool in;
        if (v.state == kBeamLive) {
            in = g != 0;
            if (in) rank = (v.base + (static_cast<double>(order_value(static_cast<unsigned>(g >> 32))) - v.m) * pr.inv_t) * v.scale;
        } else {
            in = v.state == kBeamEnded && at == 0 && l % ranks == 0;
        }
        keys[i] = in && !poisoned ? rank_key(rank) : 0ull;
    }
    __syncthreads();
    if (t < 32) {
        // lane l holds the lists 2 l and 2 l + 1
        int at[2] = {0, 0};
        unsigned long long head[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) head[j] = 2 * lane + j < lists ? keys[(2 * lane + j) * k] : 0ull;
        for (int r = 0; r < count; ++r) {
            const int j = head[1] > head[0];
            const unsigned long long h = j ? head[1] : head[0];
            const unsigned hi = static_cast<unsigned>(h >> 32), top = __reduce_max_sync(0xffffffffu, hi);
            const unsigned lo = hi == top ? static_cast<unsigned>(h) : 0u;
            const unsigned low = __reduce_max_sync(0xffffffffu, lo);
            const bool best = hi == top && lo == low;
            const unsigned holds = __ballot_sync(0xffffffffu, best);
            if ((top | low) == 0u) {  // nothing is left
                for (int i = r + lane; i < count; i += 32) win[i] = -1;
                break;
            }
            if (lane == __ffs(holds) - 1) {
                const int l = 2 * lane + j, p = j ? at[1] : at[0];
                win[r] = l * k + p;
                const unsigned long long next = p + 1 < k ? keys[l * k + p + 1] : 0ull;
                if (j) {
                    head[1] = next;
                    at[1] = p + 1;
                } else {
                    head[0] = next;
                    at[0] = p + 1;
                }
            }
        }
    }
    __syncthreads();
    for (int r = t; r < count; r += nt) {
        const int i = win[r];
        int64_t token = -1, parent = -1;
        float score = poisoned ? quiet_nan() : neg_inf();
        if (i >= 0) {
            parent = i / k / ranks;
            const BeamSum& v = beam[parent];
            const unsigned long long g = gathered[i];
            token = v.state == kBeamEnded ? pr.end_token : key_index(g);
            score = static_cast<float>(v.state == kBeamEnded
                                           ? v.base
                                           : v.base + (static_cast<double>(order_value(static_cast<unsigned>(g >> 32))) - v.m) * pr.inv_t);
        }
        pr.tokens[item * count + r] = token;
        pr.parents[item * count + r] = parent;
        pr.out_scores[item * count + r] = score;
    }
}

template <class Tag, int BLOCK, int PER_SM>
__global__ void __launch_bounds__(BLOCK, PER_SM) beam_select_kernel(const BeamProblem pr, float scale2, int cluster,
                                                                    int ranks, int seg_slots) {
    using R = typename Tag::raw;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ float red[96];
    __shared__ int count[3];
    const int t = threadIdx.x;
    const int cta = static_cast<int>(blockIdx.x % cluster), rank = cta % ranks, groups = cluster / ranks;
    const int64_t item = blockIdx.x / cluster;
    const int k = pr.rows.top_k, lists = pr.beams * ranks;
    const BeamLayout lay(k, lists, seg_slots, kGroupElems<Tag>);
    TopShared sh;
    sh.room = cand_room(k, kGroupElems<Tag>);
    sh.big = reinterpret_cast<unsigned*>(dyn + lay.big);
    sh.cand = reinterpret_cast<unsigned long long*>(dyn + lay.cand);
    sh.best = reinterpret_cast<unsigned long long*>(dyn + lay.best);
    sh.list = reinterpret_cast<unsigned short*>(dyn + lay.list);
    sh.count = count;
    unsigned long long* gathered = reinterpret_cast<unsigned long long*>(dyn + lay.gathered);
    float* sums = reinterpret_cast<float*>(dyn + lay.sums);
    allow_dependents();
    if (cluster > 1) cluster_ready();
    if (cta / ranks < pr.beams) prefetch_part<Tag>(pr.rows, item * pr.beams + cta / ranks, rank, ranks);
    grid_dependency_wait();
    if (cluster > 1) cluster_wait();
    const unsigned to_lists = cluster > 1 ? cluster_addr(smem_u32(gathered), 0) : 0;
    const unsigned to_sums = cluster > 1 ? cluster_addr(smem_u32(sums), 0) : 0;
    for (int b = cta / ranks; b < pr.beams; b += groups) {
        const int64_t r = item * pr.beams + b;
        if (pr.scores[r] == neg_inf() || (pr.ended && pr.ended[r])) continue;  // (alike in every thread)
        const R* row = static_cast<const R*>(pr.rows.x) + r * pr.rows.row_stride;
        const Part<Tag> part(row, pr.rows.cols, rank, ranks);
        SoftSum c;
        int have = 0;
        for (int at = 0;;) {
            const Segment<Tag> sg = part.segment(at);
            SoftSum d;
            unsigned most = 0;
            scan_segment<Tag, false, true, false>(d, row, sg, scale2, sh.big, nullptr, most, row + part.end());
            d.t = 0.0f;
            c.join(d, scale2);
            if (at + sg.body >= part.count) softsum_to(c, scale2, red);
            have = take_segment<Tag>(row, sg, k, have, most, sh);
            at += sg.body;
            if (at >= part.count) break;
        }
        if (t < 32) c = softsum_from(scale2, red);
        const int l = b * ranks + rank;
        if (cluster > 1) {
            if (t == 0) {
                st_cluster(to_sums + 8 * l, c.m);
                st_cluster(to_sums + 8 * l + 4, c.s);
            }
            for (int i = t; i < k; i += blockDim.x) st_cluster(to_lists + 8 * (l * k + i), i < have ? sh.best[i] : 0ull);
        } else {
            if (t == 0) {
                sums[2 * l] = c.m;
                sums[2 * l + 1] = c.s;
            }
            for (int i = t; i < k; i += blockDim.x) gathered[l * k + i] = i < have ? sh.best[i] : 0ull;
        }
        __syncthreads();  // `red` and the best have been read
    }
    if (cluster > 1) {
        cluster_arrive();
        cluster_wait();
        if (cta != 0) return;
    }
    merge_beams(pr, item, k, ranks, gathered, reinterpret_cast<unsigned long long*>(dyn + lay.ranks), sums, scale2);
}

template <class Tag, int BLOCK, int PER_SM>
cudaError_t launch_beam_cluster(const BeamProblem& pr, int block, int cluster, int ranks) {
    auto kern = beam_select_kernel<Tag, BLOCK, PER_SM>;
    static KernelLaunchCache cache;
    const int64_t parts = (pr.rows.cols / kGroupElems<Tag> + ranks - 1) / ranks;
    const int seg_slots = static_cast<int>((parts < kSegGroups ? parts : kSegGroups) + 2 + 3) / 4 * 4;
    const size_t smem = BeamLayout(pr.rows.top_k, pr.beams * ranks, seg_slots, kGroupElems<Tag>).total;
    cudaError_t e = ensure_smem_limit(kern, smem + 8192, cache);  // with the static part
    if (e != cudaSuccess) return e;
    if (cluster > 1) {
        bool ok = false;
        if (cluster > 8 && (e = allow_big_cluster(kern, cache)) != cudaSuccess) return e;
        if ((e = cluster_fits(kern, dim3(static_cast<unsigned>(cluster)), block, cluster, smem, cache, &ok)) != cudaSuccess)
            return e;
        if (!ok) return cudaErrorInvalidClusterSize;
    }
    argr_plan p = {};
    p.flags = ARGR_PLAN_PDL;
    return launch_ex_smem(kern, dim3(static_cast<unsigned>(pr.items * cluster)), dim3(block), cluster, smem, p,
                          pr.rows.stream, pr, kLog2E / pr.rows.temperature, cluster, ranks, seg_slots);
}

// A CTA per beam (up to 16 in a cluster, the beams in turns past that), and several to a beam while
// every CTA has an SM of its own and two groups per thread.
template <class Tag>
cudaError_t launch_beam_select_t(const BeamProblem& pr, const argr_caps& caps) {
    const int most = caps.max_cluster < 16 ? caps.max_cluster : 16;
    const int64_t row_groups = pr.rows.cols / kGroupElems<Tag>;
    const int groups = pr.beams < most ? pr.beams : most;
    int ranks = 1;
    while (2 * ranks * groups <= most && groups == pr.beams && 2 * pr.items * groups * ranks <= caps.sm_count &&
           row_groups / (2 * ranks) >= 128)
        ranks *= 2;
    const int cluster = groups * ranks;
    const int64_t per_cta = row_groups / ranks, n = pr.items * cluster;
    const int k = pr.rows.top_k;
    int block = 512;
    if (n > caps.sm_count) {
        block = 256;
        while (block > 32 && per_cta <= 8 * block && n > (block == 256 ? 3 : 640 / block) * static_cast<int64_t>(caps.sm_count))
            block /= 2;
        while (block < 256 && block < 2 * k) block *= 2;
    } else {
        while (block > 32 && block / 2 >= per_cta && block > 2 * k) block /= 2;
    }
    if (block > 256 || n * block <= static_cast<int64_t>(caps.sm_count) * 512)
        return launch_beam_cluster<Tag, 512, 1>(pr, block, cluster, ranks);
    return block > 128 ? launch_beam_cluster<Tag, 256, 3>(pr, block, cluster, ranks)
                       : launch_beam_cluster<Tag, 128, 5>(pr, block, cluster, ranks);
}

}  // namespace argr
