// A distillation step, loss and gradient, with one read of the row.
//
// A cluster of C CTAs holds a row in shared memory, a part each, fetched by bulk
// copies (kStepStages of them, an mbarrier each) while the teacher's side is read.
// First pass: softmax sums of the part, a stage as it lands, exchanged across the cluster.
// Second pass: the gradient, from shared memory. So x is read once and the
// gradient written once, where a forward and a backward kernel read x twice; the
// exponential is taken twice. Parts of about 40 KB, so that five CTAs or more per SM, at
// different points of this, keep both directions of the memory busy.
//
//   p_j = exp2((x_j - m) scale2 - log2 s), (m, s) joined over the cluster;
//   dx_j = w p_j, and at the elements that slots name (Q + tail) p_j - q_j. With a
//   tail bucket the named elements are left out of the sums (-inf in their place in shared
//   memory) and summed by themselves, and w p_j is w' times the element's share of the tail.
//
// A CTA's time is a chain: copies, sums, exchange, gradient; what is not memory
// in it (about half) bounds the kernel. Hence: every warp sends its own sums to every
// CTA and joins all of them itself (one cluster barrier, no CTA-wide reduction before
// or after it), and nothing is loaded where it is used.
//
// [1024, 202048] bf16, 64 slots and a tail: 152 us, 5.4 TB/s read and written (a forward and a
// backward kernel: 80 + 122 us). [333, 50021] f32, 100 slots, rows 50064 apart and the gradient's
// 50021: 35.4 us, 3.8 TB/s. Where a row's gradient lies otherwise than the row modulo 16 bytes, as
// of three rows of four there, it is stored element by element: [1024, 50257] bf16, 64 slots and a
// tail, 49 us, with rows 50304 apart 62 us.
// Tried and slower: reading the part a second time from L2 instead of keeping it; a
// persistent CTA that sums one row while it writes the gradient of the one before
// (273 against 198 us then); loads per thread instead of bulk copies; a bit map of the
// named elements instead of -inf in their place.
//
// The waits for copies are bounded. One that runs out is recorded
// (argreduce_read_error); its CTA goes on with what is in shared memory, so that the cluster's
// barriers are kept, waits again for the copies and sums in flight, and the row's outputs
// are undefined.
#pragma once

#include "logits_forward.cuh"
#include "logits_grad.cuh"

namespace argr {

constexpr int kStepMaxBlock = 256;
constexpr int kStepStages = 4;

// 16-byte units of a part that a thread takes four at a time: unit j of batch b
// is t + (4 b + j) nt. Past the last unit (FULL: there is none) every element is -inf.
template <class Tag, bool FULL>
__device__ __forceinline__ void load_batch(Group<Tag>& v, const uint4* data, int first, int units) {
    constexpr uint32_t none = std::is_same<Tag, TagF32>::value ? 0xff800000u
                              : std::is_same<Tag, TagBF16>::value ? 0xff80ff80u : 0xfc00fc00u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int u = first + j * static_cast<int>(blockDim.x);
        const uint4 q = FULL || u < units ? data[u] : make_uint4(none, none, none, none);
        v.w[4 * j] = q.x;
        v.w[4 * j + 1] = q.y;
        v.w[4 * j + 2] = q.z;
        v.w[4 * j + 3] = q.w;
    }
}

template <class Tag, bool TAIL>
__global__ void __launch_bounds__(kStepMaxBlock, 4) distill_step_kernel(const LogitsProblem pr, float scale2,
                                                                        int ranks, int max_units, int flags) {
    using R = typename Tag::raw;
    constexpr int E = kGroupElems<Tag>;
    constexpr int P = 16 / static_cast<int>(sizeof(R));  // elements of a unit
    extern __shared__ __align__(16) unsigned char dyn[];
    // of every warp of the cluster: (m, s), and the same of the elements that slots name
    __shared__ __align__(16) uint4 parts[kMaxRanks * kStepMaxBlock / 32];
    __shared__ __align__(8) unsigned long long bars[kStepStages + 1];  // the stages', and the exchange's
    __shared__ GradWeights weights;
    __shared__ unsigned ends[2];  // the named elements of the ragged ends, a bit each
    const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5, warps = nt >> 5;
    const int rank = static_cast<int>(blockIdx.x % ranks);
    uint4* data = reinterpret_cast<uint4*>(dyn);
    const Slots sl(dyn + 16 * static_cast<size_t>(max_units), pr.slots);
    const unsigned bar = smem_u32(bars);
    if (t == 0) {
        for (int s = 0; s <= kStepStages; ++s) mbar_init(bar + 8 * s, 1);
        mbar_init_fence();
    }
    allow_dependents();
    grid_dependency_wait();
    __syncthreads();
    const int64_t row_slots = gridDim.x / ranks;
    unsigned parity = 0;
    bool dead = false;  // a wait ran out
    for (int64_t r = blockIdx.x / ranks; r < pr.rows; r += row_slots, parity ^= 1) {
        if (ranks > 1) cluster_ready();  // (the first time: the barriers are initialised)
        const R* row = static_cast<const R*>(pr.x) + r * pr.row_stride;
        R* out = static_cast<R*>(pr.grad) + r * pr.grad_stride;
        const Part<Tag> part(row, pr.cols, rank, ranks);
        const int units = part.count * (kGroupBytes / 16);
        const int lo = part.begin(), hi = part.end(), body = part.align + part.first * E, tail = body + units * P;
        const int batches = (units + 4 * nt - 1) / (4 * nt), full = units / (4 * nt);
        if (t == 0 && !dead) {
            fence_proxy_async_smem();  // the row before has been read (a barrier ago)
            for (int s = 0; s < kStepStages; ++s) {
                const int u0 = batches * s / kStepStages * 4 * nt;
                const int u1 = min(units, batches * (s + 1) / kStepStages * 4 * nt);
                const unsigned bytes = u1 > u0 ? 16u * static_cast<unsigned>(u1 - u0) : 0u;
                mbar_arrive_expect_tx(bar + 8 * s,
                                      bytes + ((flags & ARGR_PLAN_TEST_EXPIRE) && s == kStepStages - 1 ? 16u : 0u));
                if (bytes)
                    bulk_copy_g2s(smem_u32(data) + 16 * u0, row + body + static_cast<int64_t>(u0) * P, bytes, bar + 8 * s);
            }
        }
        // the ragged ends, an element per lane: the head with the first warp, the tail with the last
        const bool has_head = warp == 0 && lane < body - lo, has_tail = warp == warps - 1 && lane < hi - tail;
        const float x_head = has_head ? widen_elem<Tag>(row[lo + lane]) : 0.0f;
        const float x_tail = has_tail ? widen_elem<Tag>(row[tail + lane]) : 0.0f;
        float grad_loss;  // asked for now: the compiler would load it where it is used, a DRAM latency late
        asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(grad_loss) : "l"(pr.grad_logprob + r));
        load_slots<Tag>(pr, r, row, rank == 0 ? 0 : lo, rank == 0 ? pr.cols : hi, sl);
        if constexpr (TAIL) {
            if (t < 2) ends[t] = 0u;
        }
        __syncthreads();
        // the teacher's sums in the first warp; with the tail, the sums of this part's named elements in the second
        if (warp == 0) {
            const Teacher q = warp_teacher(pr, sl);
            if (lane == 0) *sl.sums = q;
        }
        SoftSum d;
        const int d_warp = warps > 1 ? 1 : 0;
        if constexpr (TAIL) {
            if (warp == d_warp) {
                for (int i = lane; i < pr.slots; i += 32)
                    if (sl.id[i] >= lo && sl.id[i] < hi) d.add(sl.x[i], scale2);
                d = warp_softsum(d, scale2);
            }
        }
        bool landed = true;
        const unsigned long long limit = (flags & ARGR_PLAN_TEST_EXPIRE) ? 2ull * 1000 * 1000 : kWaitLimitNs;
        if constexpr (TAIL) {
            // -inf in the place of the elements that slots name: nothing to the sums, 0 to the dense gradient
            for (int s = 0; s < kStepStages; ++s)
                if (!dead) landed = mbar_wait_bounded(bar + 8 * s, parity, limit) && landed;
            R* mine = reinterpret_cast<R*>(data);
            for (int i = t; i < pr.slots; i += nt) {
                const int j = sl.id[i];
                if (j >= body && j < tail) mine[j - body] = narrow_elem<Tag>(neg_inf());
                else if (j >= lo && j < hi) atomicOr(&ends[j >= tail], 1u << (j >= tail ? j - tail : j - lo));
            }
        }
        __syncthreads();
        const bool drop_head = TAIL && (ends[0] >> lane & 1u), drop_tail = TAIL && (ends[1] >> lane & 1u);
        SoftSum c;
        if (has_head && !drop_head) c.add(x_head, scale2);
        if (has_tail && !drop_tail) c.add(x_tail, scale2);
        for (int s = 0; s < kStepStages; ++s) {
            if (!TAIL && !dead) landed = mbar_wait_bounded(bar + 8 * s, parity, limit) && landed;
            for (int b = batches * s / kStepStages; b < batches * (s + 1) / kStepStages; ++b) {
                Group<Tag> v;
                const int first = t + 4 * b * nt;
                if (b < full) load_batch<Tag, true>(v, data, first, units);
                else load_batch<Tag, false>(v, data, first, units);
                add_group<Tag, false>(c, v, v.largest(), scale2);
            }
        }
        // every warp's sums to every CTA, which joins them in each of its warps
        c.t = 0.0f;
        c = warp_softsum(c, scale2);
        const uint4 mine = make_uint4(__float_as_uint(c.m), __float_as_uint(c.s), __float_as_uint(d.m), __float_as_uint(d.s));
        if (ranks > 1) {
            cluster_wait();
            if (t == 0) mbar_arrive_expect_tx(bar + 8 * kStepStages, 16u * static_cast<unsigned>(ranks * warps));
            if (lane < ranks)
                st_async_v4(cluster_addr(smem_u32(&parts[rank * warps + warp]), lane), mine,
                            cluster_addr(bar + 8 * kStepStages, lane));
            const unsigned long long t0 = global_timer_ns();
            bool here = mbar_try_wait_cluster(bar + 8 * kStepStages, parity);
            while (!here && global_timer_ns() - t0 <= kWaitLimitNs) here = mbar_try_wait_cluster(bar + 8 * kStepStages, parity);
            landed = landed && here;
        } else {
            if (lane == 0) parts[warp] = mine;
            __syncthreads();
        }
        c = SoftSum();
        d = SoftSum();
        for (int i = lane; i < ranks * warps; i += 32) {
            const uint4 v = parts[i];
            SoftSum o;
            o.m = __uint_as_float(v.x);
            o.s = __uint_as_float(v.y);
            c.join(o, scale2);
            if constexpr (TAIL) {
                o.m = __uint_as_float(v.z);
                o.s = __uint_as_float(v.w);
                o.t = 0.0f;
                d.join(o, scale2);
            }
        }
        c = warp_softsum(c, scale2);
        SoftSum all = c;
        if constexpr (TAIL) all.join(warp_softsum(d, scale2), scale2);
        const float m = all.empty() ? neg_inf() : all.m;
        const float ln_s = all.empty() ? neg_inf() : logf(all.s);
        const float ln_rest = TAIL ? tail_log(pr, c, all.m, ln_s) : ln_s;
        const GradWeights w(pr, *sl.sums, grad_loss, m, ln_s, ln_rest, TAIL ? c.m : m, TAIL ? logf(c.s) : ln_rest);
        if (t == 0) weights = w;  // for the named elements: they come last
        const auto f = [&](float x) { return narrow_elem<Tag>(w.dense * ex2((x - w.dense_m) * scale2 - w.dense_ls2)); };
        // every element that slots name has been read, by all CTAs, before the first is written
        if (w.none) {
            const R fill = narrow_elem<Tag>(w.dense);
            for (int j = lo + t; j < hi; j += nt) out[j] = fill;
        } else {
            if (((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0) {
                const f32x2 minus = pack2(-w.dense_m, -w.dense_m), scale = pack2(scale2, scale2);
                const f32x2 shift = pack2(-w.dense_ls2, -w.dense_ls2), dense = pack2(w.dense, w.dense);
                uint4* to = reinterpret_cast<uint4*>(out + body);
                const auto grads = [&](Group<Tag>& v) {
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) {
                        float a, e;
                        v.pair(i, a, e);
                        unpack2(fma2(add2(pack2(a, e), minus), scale, shift), a, e);
                        unpack2(mul2(pack2(ex2(a), ex2(e)), dense), a, e);
                        v.set_pair(i, a, e);
                    }
                };
                for (int b = 0; b < full; ++b) {
                    Group<Tag> v;
                    const int first = t + 4 * b * nt;
                    load_batch<Tag, true>(v, data, first, units);
                    grads(v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        to[first + j * nt] = make_uint4(v.w[4 * j], v.w[4 * j + 1], v.w[4 * j + 2], v.w[4 * j + 3]);
                }
                if (full < batches) {
                    Group<Tag> v;
                    const int first = t + 4 * full * nt;
                    load_batch<Tag, false>(v, data, first, units);
                    grads(v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (first + j * nt < units)
                            to[first + j * nt] = make_uint4(v.w[4 * j], v.w[4 * j + 1], v.w[4 * j + 2], v.w[4 * j + 3]);
                }
            } else {
                // the gradient lies otherwise than x: element by element
                const R* mine = reinterpret_cast<const R*>(data);
                for (int j = t; j < units * P; j += nt) out[body + j] = f(widen_elem<Tag>(mine[j]));
            }
            if (has_head) out[lo + lane] = f(x_head);
            if (has_tail) out[tail + lane] = f(x_tail);
            __syncthreads();
            const Teacher q = *sl.sums;
            const GradWeights named = weights;
            for (int i = t; i < pr.slots; i += nt) {
                const int j = sl.id[i];
                if (j >= lo && j < hi) out[j] = narrow_elem<Tag>(named.named(sl.x[i], teacher_log(pr, q, sl.v[i]), scale2));
            }
        }
        if (rank == 0 && warp == 0) {
            const Teacher q = *sl.sums;
            float loss = 0.0f;
            for (int i = lane; i < pr.slots; i += 32) loss += slot_loss(pr, q, sl, i, m, ln_s);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
            if (lane == 0) {
                if (pr.loss) pr.loss[r] = whole_loss(q, loss, ln_s, ln_rest);
                pr.stats[r] = make_float4(m, ln_s, ln_rest, 0.0f);
            }
        }
        if (!__syncthreads_and(landed) && !dead) {
            // leave nothing in flight behind, and copy no more: a CTA whose wait for the exchange ran out stays
            // until those that still wait for copies, a limit per stage, have sent it their sums
            dead = true;
            if (t == 0) {
                record_device_error(kErrWaitExpired);
                for (int s = 0; s < kStepStages; ++s) mbar_wait_bounded(bar + 8 * s, parity, limit);
                if (ranks > 1) mbar_wait_bounded(bar + 8 * kStepStages, parity, (kStepStages + 1) * kWaitLimitNs);
            }
        }
    }
}

}  // namespace argr
