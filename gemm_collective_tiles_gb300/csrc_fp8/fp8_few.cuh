// matmul_fp8 for at most 32 rows (decoding): the weights' columns take the MMA's
// 128 rows and the tokens its N.
//
// Such a product reads every weight once for a handful of multiplications, so
// it should run at the speed of memory, and what stands in the way is the work
// per stage of 128 x 128 weights: with tokens as the MMA's rows a promotion
// warp would load and scale 64 accumulator columns for a few useful lanes.
// Turned round, a lane is a column of the output and loads NT values, the
// tokens, per stage.
//
//   out[t][n] = sum_b sa[t][b] * sb[b][n / 128] * P_b[n][t] + bias[n]
//
// CTA layout (384 threads, one CTA per SM): warp 0 loads, warps 1 and 3 issue
// the MMAs of alternate stages, warps 4-11 promote: quadrant warp % 4 of the
// columns, and of the stages the even ones (warps 4-7) or the odd ones.
// A cluster of up to 8 CTAs shares a tile's contraction.  At the end the sums
// of both groups and of all parts lie in shared memory; each CTA adds a share
// of the tile's outputs over them, in order of part and group, and stores them
// along the columns.
#pragma once
#include "fp8_gemm.cuh"

namespace gct {
namespace fp8 {

template <int NT>
struct FewGeo {
    static constexpr int STAGES = NT == 16 ? 10 : 8;
    static constexpr int ACCS = 8;
    // a slot belongs to one of the two issuers: a wait by parity is only valid
    // for one who sees every phase of the barrier
    static_assert(STAGES % 2 == 0 && ACCS % 2 == 0, "issuers by parity of the slot");
    static constexpr int TMEM_COLS = ACCS * NT;
    static constexpr uint32_t W_BYTES = 128 * 128, X_BYTES = NT * 128, STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr uint32_t SUMS = NT * 128;  // fp32 sums of one group
    static constexpr uint32_t TILES_BYTES = STAGES * STAGE_BYTES;
    static constexpr int NUM_BARS = 2 * STAGES + 2 * ACCS + 4;
    static constexpr uint32_t SCALE_BYTES = 8 * 2 * NT * 4;  // per promotion warp: the tokens' scales of two stages
    static constexpr uint32_t BYTES = 1024 + TILES_BYTES + 2 * SUMS * 4 + SCALE_BYTES + NUM_BARS * 8 + 32;
    static constexpr int THREADS = 384;
};

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

template <int NT>
__global__ void __launch_bounds__(FewGeo<NT>::THREADS, 1) few_rows_kernel(const __grid_constant__ GemmParams p) {
    using G = FewGeo<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t tiles = smem_u32(base);
    float* const sums = reinterpret_cast<float*>(base + G::TILES_BYTES);
    float* const scales = sums + 2 * G::SUMS;
    const uint32_t full = tiles + G::TILES_BYTES + 2 * G::SUMS * 4 + G::SCALE_BYTES, done = full + 8 * G::STAGES;
    const uint32_t acc_full = done + 8 * G::STAGES, acc_empty = acc_full + 8 * G::ACCS;
    const uint32_t parts_in = acc_empty + 8 * G::ACCS, parts_out = parts_in + 8, final_bar = parts_out + 8;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(base + (final_bar + 16 - tiles));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int S = p.split;
    const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            bar_init(full + 8 * s, 1);
            bar_init(done + 8 * s, 1);
        }
        for (int b = 0; b < G::ACCS; ++b) {
            bar_init(acc_full + 8 * b, 1);
            bar_init(acc_empty + 8 * b, 4);
        }
        bar_init(parts_in, 8 * S);
        bar_init(parts_out, 8 * S);
        bar_init(final_bar, 1);
        bar_init(final_bar + 8, 1);
        fence_mbar_init();
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
        // for the whole CTA, which waits for this thread below
        grid_wait();
        grid_release();
        const uint32_t e = *reinterpret_cast<volatile uint32_t*>(&p.ws->epoch) + 1u;
        tmem_slot[1] = e == 0u ? 1u : e;
    }
    if (warp == 1) tmem_alloc<G::TMEM_COLS, 1>(tmem_slot);
    tc_fence_before();
    __syncthreads();
    if (S > 1) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot[0];
    const Ctl ctl{p.ws, tmem_slot[1], p.wait_ns, rank};
    const int first = blockIdx.x / S, step = gridDim.x / S;
    const int lo = rank * p.part_stages, hi = min(p.stages_total, lo + p.part_stages);

    if (warp == 0) {
        if (lane == 0) {
            Ring<G::STAGES> st;
            Fills fills;
            bool ok = true;
            for (int u = first; u < p.n_units && ok; u += step)
                for (int s = lo; s < hi; ++s) {
                    if (!wait_bar(ctl, done + 8 * st.slot, st.phase ^ 1, WAIT_EMPTY)) {
                        ok = false;
                        break;
                    }
                    const uint32_t w = tiles + st.slot * G::STAGE_BYTES, bar = full + 8 * st.slot;
                    const int d = s * 128, col = u * 128;
                    bar_expect_tx(bar, G::STAGE_BYTES);
                    tma_load_2d(w, &p.tmB, p.b_mn ? col : d, p.b_mn ? d : col, bar);
                    tma_load_2d(w + G::W_BYTES, &p.tmA, d, 0, bar);
                    fills.add(st.slot, st.phase);
                    st.next();
                }
            fills.drain(ctl, full, G::STAGES);
        }
        __syncwarp();
    } else if (warp == 1 || warp == 3) {
        // two issuers take the stages in turn: each stage has its own
        // accumulator, and a stage's issue takes longer than its MMAs
        const int issuer = warp >> 1;
        const uint32_t w_adv = p.b_mn ? 256 : 2;  // a K step of 32 codes: 32 rows of 128 bytes, or 32 bytes
        const uint64_t w_desc = smem_desc(tiles, 16, 1024), x_desc = smem_desc(tiles + G::W_BYTES, 16, 1024);
        Ring<G::STAGES> st;
        Ring<G::ACCS> acc;
        bool ok = true;
        for (int u = first; u < p.n_units && ok; u += step) {
            const bool report = p.debug_skip != static_cast<uint32_t>(u) + 1;
            for (int s = lo; s < hi; ++s, st.next(), acc.next()) {
                if ((acc.slot & 1) != issuer) continue;
                if (!wait_bar(ctl, acc_empty + 8 * acc.slot, acc.phase ^ 1, WAIT_ACC_EMPTY) ||
                    !wait_bar(ctl, full + 8 * st.slot, st.phase, WAIT_FULL)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t at = st.slot * (G::STAGE_BYTES / 16);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_f8<1>(tmem + acc.slot * NT, w_desc + at + k * w_adv, x_desc + at + k * 2, p.idesc, k > 0 ? 1u : 0u);
                    umma_commit_all<1>(done + 8 * st.slot);
                    if (report) umma_commit_all<1>(acc_full + 8 * acc.slot);
                }
                __syncwarp();
            }
        }
        if (elect_one()) umma_commit_one<1>(final_bar + 8 * issuer);
        __syncwarp();
        wait_bar(ctl, final_bar + 8 * issuer, 0, WAIT_DRAIN_MMA);
    } else if (warp >= 4) {
        const int w = warp - 4, q = w & 3, group = w >> 2;
        Ring<G::ACCS> acc;
        uint32_t tiles_done = 0;
        constexpr int AHEAD = NT == 16 ? 4 : 2;
        float* const my_scales = scales + w * 2 * NT;
        bool ok = true;
        for (int u = first; u < p.n_units && ok; u += step) {
            const int col0 = u * 128;
            const bool live = col0 + q * 32 < p.N;
            unsigned long long sum[NT / 2];
#pragma unroll
            for (int i = 0; i < NT / 2; ++i) sum[i] = 0ull;
            // this group's stages; lane l fetches the scales of token l, AHEAD
            // of its stages ahead, into registers of their own, and hands them
            // round through shared memory (a read of four tokens'
            // scales costs what a shuffle of one does)
            const int mine = lo + ((lo & 1) != group);
            const float* pa = p.sa + min(lane, p.M - 1) * p.sa_rs + mine * p.sa_cs;
            const float* pb = p.sb + u * p.sb_cs + mine * p.sb_rs;
            int left = (hi - mine + 1) / 2;
            float a[AHEAD], b[AHEAD];
            auto fetch = [&](float& fa, float& fb) {
                fa = *pa;
                fb = *pb;
                if (--left > 0) {
                    pa += 2 * p.sa_cs;
                    pb += 2 * p.sb_rs;
                }
            };
            if (left > 0) {
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) fetch(a[j], b[j]);
            }
            if (mine != lo && hi > lo) acc.next();  // the other group's first stage
            for (int s = mine; s < hi && ok; s += 2 * AHEAD) {
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    if (s + 2 * j >= hi) break;
                    float* const f = my_scales + (j & 1) * NT;
                    if (lane < NT) f[lane] = a[j] * b[j];
                    fetch(a[j], b[j]);
                    if (!wait_bar(ctl, acc_full + 8 * acc.slot, acc.phase, WAIT_ACC_FULL)) {
                        ok = false;
                        break;
                    }
                    __syncwarp();  // tensor-memory loads are for the converged warp
                    tc_fence_after();
                    const uint32_t from = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc.slot * NT;
                    uint32_t r[NT];
                    if (live) {
                        tmem_ld_cols(from, r);
                        tmem_wait_regs(r);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(acc_empty + 8 * acc.slot);
                    acc.next();
                    if (s + 2 * j + 1 < hi) acc.next();
                    if (live) {
#pragma unroll
                        for (int i = 0; i < NT / 4; ++i) {
                            const ulonglong2 f4 = *reinterpret_cast<const ulonglong2*>(f + 4 * i);
                            sum[2 * i] = fma_f32x2(pack_f32x2(r[4 * i], r[4 * i + 1]), f4.x, sum[2 * i]);
                            sum[2 * i + 1] = fma_f32x2(pack_f32x2(r[4 * i + 2], r[4 * i + 3]), f4.y, sum[2 * i + 1]);
                        }
                    }
                }
            }
            if (!ok) break;

            // the sums meet: [group][token][column] of every part
            if (tiles_done > 0 && !wait_bar_cluster(ctl, parts_out, (tiles_done - 1) & 1, WAIT_PARTS)) break;
            float* to = sums + group * G::SUMS + q * 32 + lane;
#pragma unroll
            for (int i = 0; i < NT / 2; ++i) {
                float v0, v1;
                unpack_f32x2(sum[i], v0, v1);
                if (2 * i < p.M) to[(2 * i) * 128] = v0;
                if (2 * i + 1 < p.M) to[(2 * i + 1) * 128] = v1;
            }
            __syncwarp();
            if (S == 1) {
                if (lane == 0) bar_arrive(parts_in);
            } else if (lane < S) {
                mbar_arrive_cluster(map_to(parts_in, lane));
            }
            if (S == 1 ? !wait_bar(ctl, parts_in, tiles_done & 1, WAIT_PARTS)
                       : !wait_bar_cluster(ctl, parts_in, tiles_done & 1, WAIT_PARTS))
                break;
            __syncwarp();
            ++tiles_done;
            // this part's share of the tile's M x 128 outputs
            const int all = p.M * 128, share = ((all + S - 1) / S + 31) / 32 * 32;
            const int end = min(all, (rank + 1) * share);
            const uint32_t mine_at = smem_u32(sums);
            for (int i = rank * share + w * 32 + lane; i < end; i += 256) {
                float t[2 * MAX_SPLIT];
#pragma unroll
                for (int k = 0; k < MAX_SPLIT; ++k)
                    if (k < S) {
                        const uint32_t at = S == 1 ? mine_at : map_to(mine_at, k);
                        t[2 * k] = ld_shared_cluster_f32(at + i * 4);
                        t[2 * k + 1] = ld_shared_cluster_f32(at + (G::SUMS + i) * 4);
                    }
                float v = t[0] + t[1];
#pragma unroll
                for (int k = 1; k < MAX_SPLIT; ++k)
                    if (k < S) {
                        v += t[2 * k];
                        v += t[2 * k + 1];
                    }
                const int row = i >> 7, col = col0 + (i & 127);
                if (col < p.N) store_out(p, row, col, v + load_bias(p, col));
            }
            // tell the parts that their sums have been read, unless none will
            // write again: a CTA on its way out gets no more arrivals
            __syncwarp();
            if (u + step < p.n_units) {
                if (S == 1) {
                    if (lane == 0) bar_arrive(parts_out);
                } else if (lane < S) {
                    mbar_arrive_cluster(map_to(parts_out, lane));
                }
            }
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // no CTA of a cluster leaves while another may still signal its barriers
    // or read its sums
    if (S > 1) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<G::TMEM_COLS, 1>(tmem);
    }
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&p.ws->done_ctr, 1u) == gridDim.x - 1)
            *reinterpret_cast<uint4*>(p.ws) = make_uint4(ctl.epoch, 0u, 0u, 0u);
    }
}

}  // namespace fp8
}  // namespace gct
