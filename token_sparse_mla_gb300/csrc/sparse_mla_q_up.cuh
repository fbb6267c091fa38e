// The query's way into the latent space on tcgen05 tensor cores (sm_103a): the counterpart of the
// v_up projection on the input side of the attention.
//
//   out[t, h, n]       = sum_{d < DN} q[t, h, d] * W[h, d, n]            n < 512
//   out[t, h, 512 + .] = the 32 pairs of q[t, h, DN : DN + 64] turned by position t's angles
//
// q [T, h, DN + 64] bf16 (DN = 128, 192 or 256 nope dims: the geometries of the masked dense route,
// with the 64 rope dims behind them), W [h, DN, 512] bf16 (the key half of the up-projection as it
// is stored, so no transposed copy of it is needed), out [T, h, 576] bf16: what the forward reads.
//
// Writing the result is what it cannot avoid: 1152 bytes out and 2 (DN + 64) in per (token, head)
// against 1024 DN flops, so at the measured rates the products take about a third of the stores'
// time.  A GEMM per head: M = 128 tokens, N = 128 latent dims, K = DN.  Each CTA owns one (head,
// 128-dim slice) and a contiguous run of 128-token tiles; its slice of W stays in shared memory as
// the MN-major operand, token panels stream through a TMA ring, the fp32 accumulator is double
// buffered in TMEM, and the rounded tile leaves through shared memory and a TMA store (rows are
// 1152 * h bytes apart: direct stores touch a line per lane).  The rotated dims ride along: the four
// slices of a head take 32 tokens of each tile each, on warps of their own.
//
// Roles (320 threads):
//   warp 0      TMA producer (one thread): the W slice, then the token panels into the ring.
//   warp 1      MMA issuer (one thread) and TMEM owner.
//   warps 2-5   epilogue: TMEM lane quadrant -> bf16 -> shared memory -> TMA store.
//   warps 6-9   the rotated dims of this slice's quarter of the tile, eight tokens a warp.
// Every wait is bounded; a CTA that gives up drains its copies and MMAs before it leaves.
#pragma once

#include "sparse_mla_append.cuh"

namespace smla {

constexpr int kQupRows = 128;                    // tokens per tile (MMA M)
constexpr int kQupN = 128;                       // latent dims per CTA (MMA N)
constexpr int kQupSlices = kDV / kQupN;          // CTA slices per head
constexpr int kQupStages = 5;                    // 80 KB of q in flight
constexpr int kQupPanelBytes = kQupRows * 128;   // 128 tokens x 64 bf16, SW128
constexpr int kQupThreads = 320;
constexpr int kQupTmemCols = 2 * kQupN;

template <int DN>
struct QupLayout {
    static_assert(DN == 128 || DN == 192 || DN == 256, "nope dims");
    static constexpr int kPanelsK = DN / 64;
    static constexpr int kWPanel = DN * 128;                                   // [DN k][64 n], SW128
    static constexpr int kOffW = 0;                                            // two panels
    static constexpr int kOffA = kOffW + 2 * kWPanel;
    static constexpr int kOffOut = kOffA + kQupStages * kQupPanelBytes;        // [2 buffers][2 panels][128 t][64 n]
    static constexpr int kOffBar = kOffOut + 4 * kQupPanelBytes;
    static constexpr int kNumBars = 1 + 2 * kQupStages + 4 + 1;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;                    // tmem base, abort flag
    static constexpr int kBytes = kOffMisc + 16;
    static_assert(kOffA % 1024 == 0 && kOffOut % 1024 == 0, "swizzled operands need 1 KB alignment");
    static_assert(kBytes <= 232448, "shared memory budget (227 KB)");
};

enum : int {
    kQbW = 0,
    kQbFull = 1,                            // +stage
    kQbEmpty = 1 + kQupStages,              // +stage
    kQbAccFull = 1 + 2 * kQupStages,        // +buffer
    kQbAccEmpty = 3 + 2 * kQupStages,       // +buffer
    kQbDrain = 5 + 2 * kQupStages
};

struct QupParams {
    const __nv_bfloat16* q;      // [T, h, DN + 64]
    __nv_bfloat16* out;          // [T, h, 576]
    const int32_t* positions;    // [T]
    const float* cos_sin;        // [max_pos][64]
    int32_t T, h;
    int32_t max_pos, interleaved;
    int32_t cpg;                 // CTAs per (head, slice)
    int32_t mtiles;              // ceil(T / 128)
};

template <int DN>
__global__ void __launch_bounds__(kQupThreads, 1)
    sparse_mla_q_up_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_w,
                           const __grid_constant__ CUtensorMap tm_o, const QupParams p) {
    using L = QupLayout<DN>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    if (sbase & 1023u) {  // uniform across the grid: every CTA leaves before any barrier
        if (threadIdx.x == 0) atomicOr(&g_smla_error, kErrLayout);
        return;
    }
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    volatile int* sAbort = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
    auto bar = [&](int i) -> uint32_t { return sbase + L::kOffBar + 8u * i; };
    auto wait = [&](int i, uint32_t parity) -> bool {
        return ptx::mbar_wait(bar(i), parity, sAbort, &g_smla_error, kErrTimeout, kWaitLimitNs);
    };

    // this CTA: group g = (head hh, slice nh) and token tiles [j0, j1)
    const int g = static_cast<int>(blockIdx.x) / p.cpg;
    const int kc = static_cast<int>(blockIdx.x) % p.cpg;
    const int hh = g / kQupSlices, nh = g % kQupSlices;
    const int j0 = static_cast<int>(static_cast<int64_t>(kc) * p.mtiles / p.cpg);
    const int j1 = static_cast<int>(static_cast<int64_t>(kc + 1) * p.mtiles / p.cpg);
    const int nt = j1 - j0;

    if (threadIdx.x == 0) {
        *sAbort = 0;
        ptx::mbar_init(bar(kQbW), 1);
        for (int s = 0; s < kQupStages; ++s) {
            ptx::mbar_init(bar(kQbFull + s), 1);
            ptx::mbar_init(bar(kQbEmpty + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar(kQbAccFull + b), 1);
            ptx::mbar_init(bar(kQbAccEmpty + b), 4);
        }
        ptx::mbar_init(bar(kQbDrain), 1);
        ptx::fence_mbarrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(sbase + L::kOffMisc, kQupTmemCols);
        ptx::tmem_relinquish();
    }
    // launched as a programmatic dependent: q may be the previous launch's output
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc);

    if (warp == 0) {
        // ================================================================ TMA producer
        if (lane == 0 && nt > 0) {
            ptx::prefetch_tmap(&tm_q);
            ptx::prefetch_tmap(&tm_w);
            ptx::mbar_arrive_expect_tx(bar(kQbW), static_cast<uint32_t>(2 * L::kWPanel));
            for (int i = 0; i < 2; ++i)
                ptx::tma_load_3d(sbase + L::kOffW + i * L::kWPanel, &tm_w, kQupN * nh + 64 * i, 0, hh, bar(kQbW));
            int it = 0;
            bool ok = true;
            for (int j = j0; j < j1 && ok; ++j) {
                for (int pn = 0; pn < L::kPanelsK; ++pn) {
                    const int s = it % kQupStages;
                    if (it >= kQupStages && !(ok = wait(kQbEmpty + s, ((it / kQupStages) - 1) & 1))) break;
                    ptx::mbar_arrive_expect_tx(bar(kQbFull + s), static_cast<uint32_t>(kQupPanelBytes));
                    ptx::tma_load_3d(sbase + L::kOffA + s * kQupPanelBytes, &tm_q, 64 * pn, hh, kQupRows * j,
                                     bar(kQbFull + s));
                    ++it;
                }
            }
            // no copy may still be landing when the CTA leaves: W and the ring's last loads
            ptx::mbar_wait(bar(kQbW), 0, nullptr, &g_smla_error, 0u, kDrainLimitNs);
            for (int i = it - (it < kQupStages ? it : kQupStages); i < it; ++i)
                ptx::mbar_wait(bar(kQbFull + i % kQupStages), (i / kQupStages) & 1, nullptr, &g_smla_error, 0u,
                               kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================================================================ MMA issuer
        // A: 16 tokens' worth of k is 32 bytes of a K-major panel; B: 16 k rows are 2048 bytes of
        // the MN-major panels, whose 64-dim halves lie one panel apart (the descriptor's leading
        // offset)
        if (lane == 0 && nt > 0) {
            constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(kQupRows, kQupN, 0, 1);
            const uint64_t dw = ptx::smem_desc_sw128(sbase + L::kOffW, L::kWPanel, 1024);
            const uint64_t da = ptx::smem_desc_sw128(sbase + L::kOffA, 16, 1024);
            bool ok = wait(kQbW, 0);
            int it = 0;
            for (int jj = 0; jj < nt && ok; ++jj) {
                const int buf = jj & 1;
                if (jj >= 2 && !(ok = wait(kQbAccEmpty + buf, ((jj >> 1) - 1) & 1))) break;
                ptx::tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(buf * kQupN);
                for (int pn = 0; pn < L::kPanelsK; ++pn, ++it) {
                    const int s = it % kQupStages;
                    if (!(ok = wait(kQbFull + s, (it / kQupStages) & 1))) break;
                    ptx::tc_fence_after();
                    const uint64_t a0 = da + static_cast<uint64_t>((s * kQupPanelBytes) >> 4);
                    const uint64_t b0 = dw + static_cast<uint64_t>((pn * 64 * 128) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::mma_bf16_ss(d, a0 + ((kk * 32) >> 4), b0 + ((kk * 2048) >> 4), kIdesc, (pn | kk) != 0);
                    ptx::mma_commit(bar(kQbEmpty + s));
                }
                if (!ok) break;
                ptx::mma_commit(bar(kQbAccFull + buf));
            }
            ptx::mma_commit(bar(kQbDrain));
            ptx::mbar_wait(bar(kQbDrain), 0, nullptr, &g_smla_error, 0u, kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ================================================================ epilogue
        const int quad = warp & 3;  // the TMEM lane quadrant this warp may read
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const int r = quad * 32 + lane;  // token row of the tile
        const bool elected = warp == 2 && lane == 0;
        bool ok = true;
        for (int jj = 0; jj < nt; ++jj) {
            const int buf = jj & 1;
            if (lane == 0) ok = wait(kQbAccFull + buf, (jj >> 1) & 1);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            __syncwarp();
            // the store of tile jj - 2 has read its staging buffer; a warp that gave up takes all out
            if (elected) ptx::bulk_wait_group_read_1();
            if (ptx::named_bar_red_or(1, 128, !ok)) break;
            ptx::tc_fence_after();
            const uint32_t stage = sbase + L::kOffOut + buf * 2 * kQupPanelBytes + r * 128;
#pragma unroll
            for (int c = 0; c < kQupN / 32; ++c) {
                uint32_t v[32];
                SMLA_TMEM_LD16(tmem + lane_base + static_cast<uint32_t>(buf * kQupN + c * 32), v);
                SMLA_TMEM_LD16(tmem + lane_base + static_cast<uint32_t>(buf * kQupN + c * 32 + 16), v + 16);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t ch = static_cast<uint32_t>((c & 1) * 4 + e);
                    ptx::st_shared_v4(stage + (c >> 1) * kQupPanelBytes + ((ch ^ static_cast<uint32_t>(r & 7)) << 4),
                                      pack_bf16x8(reinterpret_cast<const float*>(v) + 8 * e));
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(kQbAccEmpty + buf));
            ptx::fence_proxy_async_smem();
            ptx::named_bar_sync(2, 128);
            if (elected) {  // tokens past the last fall outside the map and are not written
                for (int i = 0; i < 2; ++i)
                    ptx::tma_store_3d(&tm_o, sbase + L::kOffOut + (buf * 2 + i) * kQupPanelBytes, kQupN * nh + 64 * i, hh,
                                      (j0 + jj) * kQupRows);
                ptx::bulk_commit_group();
            }
        }
        if (elected) ptx::bulk_wait_group_read_0();  // shared memory may not be released before it is read
    } else {
        // ================================================================ the rotated dims
        constexpr int kPer = 8;  // tokens per warp: their loads are in flight together
        const bool inter = p.interleaved != 0;
        for (int j = j0; j < j1; ++j) {
            const int64_t t0 = static_cast<int64_t>(j) * kQupRows + nh * 32 + (warp - 6) * kPer;
            if (t0 >= p.T) break;
            uint32_t pair[kPer];
            float cs[kPer], sn[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int64_t t = t0 + i;
                pair[i] = 0u;
                cs[i] = sn[i] = 0.f;
                if (t < p.T) {
                    const int pos = __ldg(p.positions + t);
                    if (pos >= 0 && pos < p.max_pos) {
                        pair[i] = load_pair(p.q + (t * p.h + hh) * (DN + 64) + DN, lane, inter);
                        cs[i] = __ldg(p.cos_sin + static_cast<int64_t>(pos) * 64 + lane);
                        sn[i] = __ldg(p.cos_sin + static_cast<int64_t>(pos) * 64 + 32 + lane);
                    } else if (pos != -1 && lane == 0) {
                        atomicOr(&g_smla_error, kErrRowRange);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (t0 + i < p.T) store_turned(p.out + ((t0 + i) * p.h + hh) * kDQK + kDV, pair[i], cs[i], sn[i], lane, inter);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kQupTmemCols);
    }
}

}  // namespace smla
