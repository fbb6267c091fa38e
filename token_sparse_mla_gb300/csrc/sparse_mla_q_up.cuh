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
// time.  A GEMM per head: M = 128 tokens, K = DN, and a slice of NS latent dims per CTA whose part of
// W stays in shared memory as the MN-major operand, while token panels stream through a TMA ring.
// A wider slice reads q fewer times from L2 but leaves the ring less room.  Measured, 128- against
// 256-dim slices: 128 nope dims, 64 heads x 16384 tokens 282 / 295 us (512: 293); 192, 32 x 8192
// 90 / 82 us; 256, 16 x 16384 108 / 112 us.  So 256-dim slices for 192 nope dims, once their items fill
// the SMs, and 128-dim slices otherwise.
// The (head, token tile) items are dealt in equal contiguous runs, one CTA per SM; the CTAs of a
// run's slices go through it side by side, so that q leaves HBM once, and a run that crosses into
// another head reloads W.  The fp32 accumulators are four TMEM buffers of 128 dims, taken in turn.
// A warp of the epilogue stages 64 dims of its 32 tokens in its own piece
// of shared memory and stores them as whole 128-byte lines (a row per lane would touch 32 lines per
// instruction), so no barrier joins the epilogue's warps.
//
// Roles (448 threads):
//   warp 0       TMA producer (one thread): slices of W, token panels into the ring.
//   warp 1       MMA issuer (one thread) and TMEM owner.
//   warps 2-9    epilogue: two warps per TMEM lane quadrant, every other accumulator each.
//   warps 10-13  the rotated dims, a token per warp.
// Every wait is bounded; a CTA that gives up drains its copies and MMAs before it leaves.
#pragma once

#include "sparse_mla_append.cuh"

namespace smla {

constexpr int kQupRows = 128;                    // tokens per tile (MMA M)
constexpr int kQupN = 128;                       // latent dims per accumulator (MMA N)
constexpr int kQupAcc = 4;                       // accumulators in TMEM
constexpr int kQupPanelBytes = kQupRows * 128;   // 128 tokens x 64 bf16, SW128
constexpr int kQupEpiWarps = 8;
constexpr int kQupRopeWarps = 4;
constexpr int kQupThreads = 64 + 32 * (kQupEpiWarps + kQupRopeWarps);
constexpr int kQupMaxStages = 6;

template <int DN, int NS>
struct QupLayout {
    static_assert(DN == 128 || DN == 192 || DN == 256, "nope dims");
    static_assert(NS == 128 || NS == 256, "slice width");
    static constexpr int kPanelsK = DN / 64;
    static constexpr int kSlices = kDV / NS;
    static constexpr int kChunks = NS / kQupN;
    static constexpr int kWPanel = DN * 128;                                   // [DN k][64 n], SW128
    static constexpr int kWBytes = (NS / 64) * kWPanel;
    static constexpr int kOutBytes = kQupEpiWarps * 32 * 128;                  // 32 tokens x 64 dims per warp
    static constexpr int kFit = (232448 - 256 - kWBytes - kOutBytes) / kQupPanelBytes;
    static constexpr int kStages = kFit < kQupMaxStages ? kFit : kQupMaxStages;
    static constexpr int kOffW = 0;
    static constexpr int kOffA = kOffW + kWBytes;
    static constexpr int kOffOut = kOffA + kStages * kQupPanelBytes;
    static constexpr int kOffBar = kOffOut + kOutBytes;
    static constexpr int kNumBars = 2 + 2 * kQupMaxStages + 2 * kQupAcc + 1;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;                    // tmem base, abort flag
    static constexpr int kBytes = kOffMisc + 16;
    static_assert(kStages >= kPanelsK, "a tile's panels are all in the ring while its accumulators are formed");
    static_assert(kOffA % 1024 == 0 && kOffOut % 1024 == 0, "swizzled operands need 1 KB alignment");
    static_assert(kBytes <= 232448, "shared memory budget (227 KB)");
};

enum : int {
    kQbWFull = 0,
    kQbWEmpty = 1,                             // the MMAs of a slice are done with its W
    kQbFull = 2,                               // +stage
    kQbEmpty = 2 + kQupMaxStages,              // +stage
    kQbAccFull = 2 + 2 * kQupMaxStages,        // +buffer
    kQbAccEmpty = kQbAccFull + kQupAcc,        // +buffer
    kQbDrain = kQbAccEmpty + kQupAcc
};

struct QupParams {
    const __nv_bfloat16* q;      // [T, h, DN + 64]
    __nv_bfloat16* out;          // [T, h, 576]
    const int32_t* positions;    // [T]
    const float* cos_sin;        // [max_pos][64]
    int64_t items;               // h * mtiles
    int32_t T, h;
    int32_t max_pos, interleaved;
    int32_t mtiles;              // ceil(T / 128)
};

// Eight of a token's 64 rotated values (lane l of eight: values 8l .. 8l + 7) turned.  cs and sn are
// words 4l .. 4l + 3 of the table's cosines and sines.  Interleaved, those are the angles of the
// lane's four pairs.  Otherwise the partner values sit four lanes away and the lane's eight angles
// are its own four and that lane's, the lower ones with the lower of the two.  The whole warp calls.
template <bool INTER>
__device__ __forceinline__ uint4 turn_eight(const uint4 x, const float4 cs, const float4 sn, int lane) {
    float a[8];
    unpack_bf16x8(x, a);
    float y[8];
    const float c[4] = {cs.x, cs.y, cs.z, cs.w}, s[4] = {sn.x, sn.y, sn.z, sn.w};
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = a[2 * i] * c[i] - a[2 * i + 1] * s[i];
            y[2 * i + 1] = a[2 * i + 1] * c[i] + a[2 * i] * s[i];
        }
    } else {
        const uint4 xo = make_uint4(__shfl_xor_sync(0xffffffffu, x.x, 4), __shfl_xor_sync(0xffffffffu, x.y, 4),
                                    __shfl_xor_sync(0xffffffffu, x.z, 4), __shfl_xor_sync(0xffffffffu, x.w, 4));
        float o[8];
        unpack_bf16x8(xo, o);
        // angles 8 (l % 4) .. + 7 lie in words 4 l' .. of lanes l' = 2 (l % 4) and l' + 1
        const int src = (lane & 24) + 2 * (lane & 3);
        const float sign = (lane & 4) ? 1.f : -1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float ci = __shfl_sync(0xffffffffu, c[i & 3], src + (i >> 2));
            const float si = __shfl_sync(0xffffffffu, s[i & 3], src + (i >> 2));
            y[i] = a[i] * ci + sign * (o[i] * si);
        }
    }
    return pack_bf16x8(y);
}

// The rotated dims: they need no product, so they are dealt over the warps of the whole grid by tokens,
// all heads of a token to one warp, which then reads the token's angles once (dealt like the items, a
// head at a time, the angles alone were 256 bytes per (token, head), as much as is read and written
// here).  Eight lanes per head, 16 bytes each, and up to 32 heads' loads in flight; the next token's
// angles are loaded meanwhile.  Loads have no branch -- an unused token reads row 0 of the table, a lane
// past the last head the last head's -- because a conditional load made each wait for its own.
template <int DN, bool INTER>
__device__ __forceinline__ void turn_tokens(const QupParams& p, int first, int step, int lane) {
    constexpr int kFlight = 8;
    const int hd = lane >> 3, l8 = lane & 7;
    auto position = [&](int64_t t) -> int {
        const int pos = t < p.T ? ptx::ld(p.positions + t) : -1;
        const bool bad = pos != -1 && (pos < 0 || pos >= p.max_pos);
        if (bad && lane == 0) atomicOr(&g_smla_error, kErrRowRange);
        return bad ? -1 : pos;
    };
    auto angles = [&](int pos, int off) -> float4 {
        const uint4 v = ptx::ld_v4(p.cos_sin + static_cast<int64_t>(max(pos, 0)) * 64 + off + 4 * l8);
        return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
    };
    int64_t t = first;
    if (t >= p.T) return;
    int pos = position(t);
    float4 cs = angles(pos, 0), sn = angles(pos, 32);
    int pos1 = position(t + step);
    for (; t < p.T; t += step) {
        const int pos2 = position(t + 2 * static_cast<int64_t>(step));
        const float4 cs1 = angles(pos1, 0), sn1 = angles(pos1, 32);
#pragma unroll 1
        for (int h0 = 0; h0 < p.h; h0 += 4 * kFlight) {
            uint4 x[kFlight];
#pragma unroll
            for (int e = 0; e < kFlight; ++e) {
                const int hh = min(h0 + 4 * e + hd, p.h - 1);
                x[e] = ptx::ld_v4(p.q + (t * p.h + hh) * (DN + 64) + DN + 8 * l8);
            }
#pragma unroll
            for (int e = 0; e < kFlight; ++e) {
                const int hh = h0 + 4 * e + hd;
                uint4 r = turn_eight<INTER>(x[e], cs, sn, lane);
                if (pos < 0) r = make_uint4(0u, 0u, 0u, 0u);
                if (hh < p.h) __stcs(reinterpret_cast<uint4*>(p.out + (t * p.h + hh) * kDQK + kDV) + l8, r);
            }
        }
        pos = pos1;
        cs = cs1;
        sn = sn1;
        pos1 = pos2;
    }
}

template <int DN, int NS>
__global__ void __launch_bounds__(kQupThreads, 1)
    sparse_mla_q_up_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_w,
                           const QupParams p) {
    using L = QupLayout<DN, NS>;
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

    // this CTA's slice nh and its run of items (head, tile) = head * mtiles + tile; the CTAs of the
    // other slices have the same run
    const int nh = static_cast<int>(blockIdx.x) % L::kSlices;
    const int64_t run = blockIdx.x / L::kSlices, runs = gridDim.x / L::kSlices;
    const int64_t i0 = p.items * run / runs;
    const int nt = static_cast<int>(p.items * (run + 1) / runs - i0);
    const int h0 = static_cast<int>(i0 / p.mtiles);
    const int j0 = static_cast<int>(i0 % p.mtiles);

    if (threadIdx.x == 0) {
        *sAbort = 0;
        ptx::mbar_init(bar(kQbWFull), 1);
        ptx::mbar_init(bar(kQbWEmpty), 1);
        for (int s = 0; s < L::kStages; ++s) {
            ptx::mbar_init(bar(kQbFull + s), 1);
            ptx::mbar_init(bar(kQbEmpty + s), 1);
        }
        for (int b = 0; b < kQupAcc; ++b) {
            ptx::mbar_init(bar(kQbAccFull + b), 1);
            ptx::mbar_init(bar(kQbAccEmpty + b), 4);
        }
        ptx::mbar_init(bar(kQbDrain), 1);
        ptx::fence_mbarrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(sbase + L::kOffMisc, kQupAcc * kQupN);
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
            int it = 0, nw = 0;
            bool ok = true;
            int hh = h0, j = j0;
            for (int i = 0; i < nt && ok; ++i) {
                if (i == 0 || j == 0) {  // a head begins: its W, once the last one's MMAs are done
                    if (nw > 0 && !(ok = wait(kQbWEmpty, (nw - 1) & 1))) break;
                    ptx::mbar_arrive_expect_tx(bar(kQbWFull), static_cast<uint32_t>(L::kWBytes));
                    for (int n = 0; n < NS / 64; ++n)
                        ptx::tma_load_3d(sbase + L::kOffW + n * L::kWPanel, &tm_w, NS * nh + 64 * n, 0, hh, bar(kQbWFull));
                    ++nw;
                }
                for (int pn = 0; pn < L::kPanelsK; ++pn) {
                    const int s = it % L::kStages;
                    if (it >= L::kStages && !(ok = wait(kQbEmpty + s, ((it / L::kStages) - 1) & 1))) break;
                    ptx::mbar_arrive_expect_tx(bar(kQbFull + s), static_cast<uint32_t>(kQupPanelBytes));
                    ptx::tma_load_3d(sbase + L::kOffA + s * kQupPanelBytes, &tm_q, 64 * pn, hh, kQupRows * j,
                                     bar(kQbFull + s));
                    ++it;
                }
                if (++j == p.mtiles) {
                    j = 0;
                    ++hh;
                }
            }
            // no copy may still be landing when the CTA leaves: the last W and the ring's last loads
            ptx::mbar_wait(bar(kQbWFull), (nw - 1) & 1, nullptr, &g_smla_error, 0u, kDrainLimitNs);
            for (int i = it - (it < L::kStages ? it : L::kStages); i < it; ++i)
                ptx::mbar_wait(bar(kQbFull + i % L::kStages), (i / L::kStages) & 1, nullptr, &g_smla_error, 0u,
                               kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================================================================ MMA issuer
        // A: 16 k are 32 bytes of a K-major panel; B: 16 k rows are 2048 bytes of the MN-major
        // panels, whose 64-dim halves lie one panel apart (the descriptor's leading offset).  A
        // tile's panels serve all of the slice's accumulators; the last one releases them.
        if (lane == 0 && nt > 0) {
            constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(kQupRows, kQupN, 0, 1);
            const uint64_t dw = ptx::smem_desc_sw128(sbase + L::kOffW, L::kWPanel, 1024);
            const uint64_t da = ptx::smem_desc_sw128(sbase + L::kOffA, 16, 1024);
            bool ok = true;
            int it = 0, nw = 0, ac = 0;
            int j = j0;
            for (int i = 0; i < nt && ok; ++i) {
                if (i == 0 || j == 0) {
                    if (nw > 0) ptx::mma_commit(bar(kQbWEmpty));
                    if (!(ok = wait(kQbWFull, nw & 1))) break;
                    ++nw;
                }
                for (int c = 0; c < L::kChunks && ok; ++c, ++ac) {
                    const int buf = ac % kQupAcc;
                    if (ac >= kQupAcc && !(ok = wait(kQbAccEmpty + buf, ((ac / kQupAcc) - 1) & 1))) break;
                    ptx::tc_fence_after();
                    const uint32_t d = tmem + static_cast<uint32_t>(buf * kQupN);
                    for (int pn = 0; pn < L::kPanelsK; ++pn) {
                        const int s = (it + pn) % L::kStages;
                        if (c == 0) {
                            if (!(ok = wait(kQbFull + s, ((it + pn) / L::kStages) & 1))) break;
                            ptx::tc_fence_after();
                        }
                        const uint64_t a0 = da + static_cast<uint64_t>((s * kQupPanelBytes) >> 4);
                        const uint64_t b0 = dw + static_cast<uint64_t>((2 * c * L::kWPanel + pn * 64 * 128) >> 4);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::mma_bf16_ss(d, a0 + ((kk * 32) >> 4), b0 + ((kk * 2048) >> 4), kIdesc, (pn | kk) != 0);
                        if (c == L::kChunks - 1) ptx::mma_commit(bar(kQbEmpty + s));
                    }
                    if (ok) ptx::mma_commit(bar(kQbAccFull + buf));
                }
                it += L::kPanelsK;
                if (++j == p.mtiles) j = 0;
            }
            ptx::mma_commit(bar(kQbDrain));
            ptx::mbar_wait(bar(kQbDrain), 0, nullptr, &g_smla_error, 0u, kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp < 2 + kQupEpiWarps) {
        // ================================================================ epilogue
        // Accumulator ac (counted over the CTA) belongs to the warps of part ac % 2.
        const int quad = warp & 3;  // the TMEM lane quadrant this warp may read
        const int part = (warp - 2) >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t stage = sbase + L::kOffOut + (warp - 2) * 32 * 128;
        int hh = h0, j = j0;
        int ac = 0;
        bool ok = true;
        for (int i = 0; i < nt && ok; ++i) {
            const int64_t t0 = static_cast<int64_t>(j) * kQupRows + quad * 32;
#pragma unroll 1
            for (int c = 0; c < L::kChunks; ++c, ++ac) {
                if ((ac & 1) != part) continue;
                const int buf = ac % kQupAcc;
                if (lane == 0) ok = wait(kQbAccFull + buf, (ac / kQupAcc) & 1);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                __syncwarp();
                if (!ok) break;
                ptx::tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t v[32];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            SMLA_TMEM_LD16(tmem + lane_base + static_cast<uint32_t>(buf * kQupN + half * 64 + q * 32 + e * 16),
                                           v + 16 * e);
                        ptx::tmem_wait_ld(v);
                        if (half == 1 && q == 1) {
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(bar(kQbAccEmpty + buf));
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            ptx::st_shared_v4(stage + lane * 128 + ((static_cast<uint32_t>(4 * q + e) ^ static_cast<uint32_t>(lane & 7)) << 4),
                                              pack_bf16x8(reinterpret_cast<const float*>(v) + 8 * e));
                    }
                    __syncwarp();
                    // eight lanes store one token's 128 bytes, four tokens per instruction
                    __nv_bfloat16* dst = p.out + (t0 * p.h + hh) * kDQK + NS * nh + c * kQupN + half * 64 + (lane & 7) * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = 4 * e + (lane >> 3);
                        const uint4 w = ptx::ld_shared_v4(stage + r * 128 + ((static_cast<uint32_t>(lane & 7) ^ static_cast<uint32_t>(r & 7)) << 4));
                        if (t0 + r < p.T) __stcs(reinterpret_cast<uint4*>(dst + static_cast<int64_t>(r) * p.h * kDQK), w);
                    }
                    __syncwarp();
                }
            }
            if (++j == p.mtiles) {
                j = 0;
                ++hh;
            }
        }
    } else {
        // ================================================================ the rotated dims
        const int first = static_cast<int>(blockIdx.x) * kQupRopeWarps + warp - 2 - kQupEpiWarps;
        const int step = static_cast<int>(gridDim.x) * kQupRopeWarps;
        if (p.interleaved != 0)
            turn_tokens<DN, true>(p, first, step, lane);
        else
            turn_tokens<DN, false>(p, first, step, lane);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kQupAcc * kQupN);
    }
}

}  // namespace smla
