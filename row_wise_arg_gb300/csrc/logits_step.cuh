// A distillation step, loss and gradient, with one read of the row.
//
// A cluster of C CTAs holds a row in shared memory, a chunk each (asynchronous
// 16-byte copies; a thread later uses just the units that it copied, so it
// waits for its own copies alone). First pass: softmax sums of the chunk, exchanged
// across the cluster. Second pass: the gradient, from shared memory. So x is
// read once and the gradient written once, where a forward and a backward kernel
// read x twice; the exponential is taken twice. Several small CTAs per SM, at
// different points of this, keep both directions of the memory busy.
#pragma once

#include "logits_grad.cuh"

namespace argr {

constexpr int kStepMaxBlock = 256;
constexpr int kStepStages = 4;

__device__ __forceinline__ void copy_async16(unsigned dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// 16-byte units of a chunk that a thread takes four at a time: unit j of batch b
// is t + (4 b + j) nt.
template <class Tag>
__device__ __forceinline__ void load_batch(Group<Tag>& v, const uint4* data, int first, int units) {
    constexpr uint32_t none = std::is_same<Tag, TagF32>::value ? 0xff800000u
                              : std::is_same<Tag, TagBF16>::value ? 0xff80ff80u : 0xfc00fc00u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int u = first + j * static_cast<int>(blockDim.x);
        const uint4 q = u < units ? data[u] : make_uint4(none, none, none, none);
        v.w[4 * j] = q.x;
        v.w[4 * j + 1] = q.y;
        v.w[4 * j + 2] = q.z;
        v.w[4 * j + 3] = q.w;
    }
}

template <class Tag, bool TAIL>
__global__ void __launch_bounds__(kStepMaxBlock, 4) distill_step_kernel(const LogitsProblem pr, float scale2,
                                                                        int ranks, int max_units) {
    using R = typename Tag::raw;
    constexpr int E = kGroupElems<Tag>;
    constexpr int P = 16 / static_cast<int>(sizeof(R));  // elements of a unit
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ float red[96];
    __shared__ float parts[4 * kMaxRanks];
    __shared__ float row_stats[3];
    __shared__ unsigned ends[2];  // the named elements of the ragged ends, a bit each
    const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5;
    const int rank = static_cast<int>(blockIdx.x % ranks);
    uint4* data = reinterpret_cast<uint4*>(dyn);
    const Slots sl(dyn + 16 * static_cast<size_t>(max_units), pr.slots);
    // a byte of bits per unit for the elements that slots name
    unsigned char* named = dyn + 16 * static_cast<size_t>(max_units) + Slots::bytes(pr.slots);
    grid_dependency_wait();
    allow_dependents();
    const int64_t row_slots = gridDim.x / ranks;
    for (int64_t r = blockIdx.x / ranks; r < pr.rows; r += row_slots) {
        if (ranks > 1) cluster_arrive();
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        R* out = static_cast<R*>(pr.grad) + r * pr.grad_stride;
        const Part<Tag> part(row, pr.cols, rank, ranks);
        const int units = part.count * (kGroupBytes / 16);
        const int lo = part.begin(), hi = part.end(), body = part.align + part.first * E, tail = body + units * P;
        const int batches = (units + 4 * nt - 1) / (4 * nt);
        const unsigned base = smem_u32(data);
#pragma unroll
        for (int s = 0; s < kStepStages; ++s) {
            for (int b = batches * s / kStepStages; b < batches * (s + 1) / kStepStages; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int u = t + (4 * b + j) * nt;
                    if (u < units) copy_async16(base + 16 * u, row + body + static_cast<int64_t>(u) * P);
                }
            copy_commit();
        }
        // the ragged ends, an element per lane: the head with the first warp, the tail with the last
        const bool has_head = warp == 0 && lane < body - lo, has_tail = warp == (nt >> 5) - 1 && lane < hi - tail;
        const float x_head = has_head ? widen_elem<Tag>(row[lo + lane]) : 0.0f;
        const float x_tail = has_tail ? widen_elem<Tag>(row[tail + lane]) : 0.0f;
        load_slots<Tag>(pr, r, row, rank == 0 ? 0 : lo, rank == 0 ? pr.cols : hi, sl);
        bool drop_head = false, drop_tail = false;
        if constexpr (TAIL) {
            for (int i = t; i < (units + 3) / 4; i += nt) reinterpret_cast<unsigned*>(named)[i] = 0u;
            if (t < 2) ends[t] = 0u;
        }
        const Teacher q = teacher_of(pr, sl);
        if constexpr (TAIL) {
            for (int i = t; i < pr.slots; i += nt) {
                const int j = sl.id[i];
                if (j >= body && j < tail) {
                    const int u = (j - body) / P;
                    atomicOr(reinterpret_cast<unsigned*>(named) + (u >> 2), 1u << (8 * (u & 3) + (j - body) % P));
                } else if (j >= lo && j < hi) {
                    atomicOr(&ends[j >= tail], 1u << (j >= tail ? j - tail : j - lo));
                }
            }
            __syncthreads();
            drop_head = ends[0] >> lane & 1u;
            drop_tail = ends[1] >> lane & 1u;
        }
        SoftSum c;
        if (has_head && !drop_head) c.add(x_head, scale2);
        if (has_tail && !drop_tail) c.add(x_tail, scale2);
#pragma unroll
        for (int s = 0; s < kStepStages; ++s) {
            if (s == 0) copy_wait<kStepStages - 1>();
            else if (s == 1) copy_wait<kStepStages - 2>();
            else if (s == 2) copy_wait<kStepStages - 3>();
            else copy_wait<0>();
            for (int b = batches * s / kStepStages; b < batches * (s + 1) / kStepStages; ++b) {
                Group<Tag> v;
                const int first = t + 4 * b * nt;
                load_batch<Tag>(v, data, first, units);
                if constexpr (TAIL) {
                    unsigned bits = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (first + j * nt < units) bits |= static_cast<unsigned>(named[first + j * nt]) << (P * j);
                    if (bits) v.drop(bits);
                }
                add_group<Tag, false>(c, v, v.largest(), scale2);
            }
        }
        c.t = 0.0f;
        c = block_softsum(c, scale2, red);
        SoftSum d;  // with the tail: this chunk's elements that slots name
        if constexpr (TAIL) {
            for (int i = t; i < pr.slots; i += nt)
                if (sl.id[i] >= lo && sl.id[i] < hi) d.add(sl.x[i], scale2);
            d = block_softsum(d, scale2, red);
        }
        if (ranks > 1) {
            cluster_wait();
            if (t < ranks) {
                const unsigned at = cluster_addr(smem_u32(parts), t) + 16 * rank;
                st_cluster(at, c.m);
                st_cluster(at + 4, c.s);
                st_cluster(at + 8, d.m);
                st_cluster(at + 12, d.s);
            }
            cluster_arrive();
            cluster_wait();
            if (t < 32) {
                c = SoftSum();
                d = SoftSum();
                if (t < ranks) {
                    c.m = parts[4 * t];
                    c.s = parts[4 * t + 1];
                    d.m = parts[4 * t + 2];
                    d.s = parts[4 * t + 3];
                }
                c = warp_softsum(c, scale2);
                d = warp_softsum(d, scale2);
            }
        }
        if (t == 0) {
            SoftSum all = c;
            all.join(d, scale2);
            c.rebase(all.m, scale2);
            row_stats[0] = all.empty() ? neg_inf() : all.m;
            row_stats[1] = all.empty() ? neg_inf() : logf(all.s);
            row_stats[2] = c.empty() ? neg_inf() : logf(c.s);
        }
        __syncthreads();
        const float m = row_stats[0], ln_s = row_stats[1], ln_rest = row_stats[2];
        const GradWeights w(pr, q, pr.grad_logprob[r], m, ln_s, ln_rest);
        const auto f = [&](float x) { return narrow_elem<Tag>(w.dense * ex2((x - w.m) * scale2 - w.ls2)); };
        if (w.none) {
            const R fill = narrow_elem<Tag>(w.dense);
            for (int j = lo + t; j < hi; j += nt) out[j] = fill;
        } else if (((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0) {
            const f32x2 minus = pack2(-w.m, -w.m), scale = pack2(scale2, scale2), shift = pack2(-w.ls2, -w.ls2);
            for (int b = 0; b < batches; ++b) {
                Group<Tag> v;
                const int first = t + 4 * b * nt;
                load_batch<Tag>(v, data, first, units);
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    float a, e;
                    v.pair(i, a, e);
                    unpack2(fma2(add2(pack2(a, e), minus), scale, shift), a, e);
                    v.set_pair(i, w.dense * ex2(a), w.dense * ex2(e));
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int u = first + j * nt;
                    if (u < units)
                        *reinterpret_cast<uint4*>(out + body + static_cast<int64_t>(u) * P) =
                            make_uint4(v.w[4 * j], v.w[4 * j + 1], v.w[4 * j + 2], v.w[4 * j + 3]);
                }
            }
            if (has_head) out[lo + lane] = f(x_head);
            if (has_tail) out[tail + lane] = f(x_tail);
        } else {
            // the gradient lies otherwise than x: element by element, from everybody's units
            __syncthreads();
            const R* mine = reinterpret_cast<const R*>(data);
            for (int j = t; j < units * P; j += nt) out[body + j] = f(widen_elem<Tag>(mine[j]));
            if (has_head) out[lo + lane] = f(x_head);
            if (has_tail) out[tail + lane] = f(x_tail);
        }
        __syncthreads();
        if (!w.none)
            for (int i = t; i < pr.slots; i += nt) {
                const int j = sl.id[i];
                if (j >= lo && j < hi) out[j] = narrow_elem<Tag>(w.named(sl.x[i], sl.v[i] - q.shift, scale2));
            }
        if (rank == 0) {
            const float loss = row_loss(pr, q, sl, m, ln_s, ln_rest, red);
            if (t == 0) {
                if (pr.loss) pr.loss[r] = loss;
                pr.stats[r] = make_float4(m, ln_s, ln_rest, 0.0f);
            }
        }
        __syncthreads();
    }
}

}  // namespace argr
