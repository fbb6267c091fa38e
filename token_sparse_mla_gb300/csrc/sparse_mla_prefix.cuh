// Attention over a prefix that the whole batch shares, on tcgen05 tensor cores (sm_103a).
//
// Every query row (token, head) attends to the same P cache rows, those of one sequence's block
// table, so the rows of all tokens and heads are one matrix and the cache is read once for many of
// them, where the list forward gathers it per token:
//
//   s = scale q.k      over the P rows, 576 dims          O = softmax(s) . k[0:512]
//   LSE = ln sum exp(s)                                   (to be merged with each token's own part)
//
// 2 * 1088 flops per (row, key): a dense contraction, bound by the tensor cores from about 256 rows
// on.  The accumulator sets the shape: 512 fp32 columns of O fill the TMEM of one SM at 128 rows and
// leave no room for S, so two CTAs share 128 rows as one cta_group::2 MMA with M = 128.  Each CTA
// keeps 64 query rows; its D holds those rows with the first half of the N columns in TMEM lanes
// 0-63 and the second half in lanes 64-127, so O is 256 columns and S 32.  Per 64-key block (a page):
//   S[128, 64]   = Q . K^T     A: each CTA's 64 rows of Q; B: each CTA's 32 keys, all 576 dims
//   O[128, 512] += P . V       A: each CTA's 64 rows of P; B: all 64 keys, each CTA's 256 dims
// so a CTA loads 36 KB of K and 32 KB of V per block (the half of V that lies in its own K tile is
// loaded again: the MMA wants the same keys at the same offset in both CTAs, and K wants different
// ones).  Shared memory: Q 72 KB, K and V rings of two stages each, P 8 KB.
//
// Work: the (row tile, block) sequence, tile-major, is cut into equal contiguous runs, one per CTA
// pair.  A tile that lies inside one run is written out directly; a cut tile leaves an fp32 partial
// (O, running max, sum) per piece in the workspace, at most two per run, which a second kernel
// joins by log-sum-exp weights in run order (so results do not depend on timing).
//
// Rows past the prefix's end in its last page are masked in S, and zeroed in the V tile before they
// are multiplied: 0 times whatever the page holds there must stay 0.  A page number outside the
// cache masks its page; rows of a page past the cache's end are masked.
//
// Roles (bf16 rows: 192 threads; fp8 rows: 448):
//   warp 0      bf16: TMA producer (one thread).
//   warp 1      MMA issuer (one thread of the even CTA) and TMEM owner.
//   warps 2-5   softmax, rescaling and output: thread = TMEM lane, i.e. row r = lane % 64 and keys
//               32 (lane / 64) .. + 31 of a block, dims 256 (lane / 64) .. + 255 of O.  The running
//               max is moved only when it grows by more than 2^8; the two warps of a row vote per
//               block and swap maxima only then.
//   warps 6-13  fp8: producers, loading a block ahead into registers, dequantising (e4m3 -> fp32 x
//               scale -> bf16 as in the forward) into the same tiles.
// Every wait is bounded; a CTA that gives up meets the other at the final cluster barrier.
#pragma once

#include "sparse_mla_common.cuh"

namespace smla {

constexpr int kPfRows = 128;                      // query rows per CTA pair (MMA M)
constexpr int kPfHalf = 64;                       // query rows per CTA
constexpr int kPfKeys = 64;                       // keys per block: one page
constexpr int kPfStages = 2;
constexpr int kPfQBytes = kPanels * kPfHalf * 128;        // 73728
constexpr int kPfKPanel = 32 * 128;
constexpr int kPfKBytes = kPanels * kPfKPanel;            // 36864
constexpr int kPfVPanel = kPfKeys * 128;
constexpr int kPfVBytes = 4 * kPfVPanel;                  // 32768
constexpr int kPfDeqWarps = 8;
constexpr int kPfMergeThreads = 128;

template <int KVF>
struct PfRoles {
    static constexpr int kThreads = KVF == 0 ? 192 : 192 + 32 * kPfDeqWarps;
};

struct PfLayout {
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kPfQBytes;
    static constexpr int kOffV = kOffK + kPfStages * kPfKBytes;
    static constexpr int kOffP = kOffV + kPfStages * kPfVBytes;
    static constexpr int kOffX = kOffP + kPfHalf * 128;       // [2][64] values swapped by a row's two threads
    static constexpr int kOffBar = kOffX + 2 * kPfHalf * 4;
    static constexpr int kNumBars = 17;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;   // tmem base, abort flag
    static constexpr int kBytes = kOffMisc + 16;
    // TMEM columns: O [0, 256) | S x2 [256, 320)
    static constexpr int kColO = 0;
    static constexpr int kColS = 256;
    static constexpr int kTmemCols = 512;
    static_assert(kOffK % 1024 == 0 && kOffV % 1024 == 0 && kOffP % 1024 == 0, "SW128 alignment");
    static_assert(kPfKBytes % 1024 == 0 && kBytes <= 232448, "shared memory budget (227 KB)");
};

enum : int {
    kPbQFull = 0,    // even CTA: both CTAs' Q landed
    kPbQEmpty = 1,   // both: the S MMAs of the piece are done
    kPbKFull = 2,    // +stage, even CTA
    kPbKEmpty = 4,   // +stage, both
    kPbVFull = 6,    // +stage, even CTA
    kPbVEmpty = 8,   // +stage, both
    kPbSFull = 10,   // +buffer, both
    kPbSEmpty = 12,  // +buffer, even CTA
    kPbPFull = 14,   // even CTA
    kPbPvDone = 15,  // both
    kPbTail = 16     // own CTA: V of a page that the prefix ends in
};

struct PfParams {
    const void* kv;
    const int32_t* pages;        // [nblk]
    __nv_bfloat16* out;          // [rows, 512]
    float* lse;                  // [rows]
    float* part_o;               // [2 * runs][slot_rows][512]
    float* part_ml;              // [2 * runs][slot_rows][2]: running max (log2 units), sum
    int64_t rows;                // T * h
    int64_t prefix;              // P
    int64_t num_slots;
    int64_t work;                // tiles * nblk
    int32_t nblk, runs;
    int32_t slot_rows;           // min(128, rows)
    float sm_scale_log2;
};

// Rows of block b that take part, given its page number (0 .. 64), and whether the page is in the cache.
__device__ __forceinline__ int pf_valid(const PfParams& p, int b, int page) {
    if (page < 0 || static_cast<int64_t>(page) * kPfKeys >= p.num_slots) return 0;
    const int64_t left = p.prefix - static_cast<int64_t>(b) * kPfKeys;
    const int64_t room = p.num_slots - static_cast<int64_t>(page) * kPfKeys;
    const int64_t n = left < room ? left : room;
    return n < kPfKeys ? static_cast<int>(n) : kPfKeys;
}

// The pieces of a run, the same for every role: blocks [b0, b1) of tile t.
struct PfWalk {
    int64_t at, end;
    int32_t nblk;
    int64_t tile;
    int b0, b1;
    __device__ __forceinline__ PfWalk(const PfParams& p, int run)
        : at(p.work * run / p.runs), end(p.work * (run + 1) / p.runs), nblk(p.nblk), tile(0), b0(0), b1(0) {}
    __device__ __forceinline__ bool next() {
        if (at >= end) return false;
        tile = at / nblk;
        b0 = static_cast<int>(at - tile * nblk);
        const int64_t n = end - at < nblk - b0 ? end - at : nblk - b0;
        b1 = b0 + static_cast<int>(n);
        at += n;
        return true;
    }
};

template <int KVF>
__global__ void __launch_bounds__(PfRoles<KVF>::kThreads, 1)
    sparse_mla_prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                             const __grid_constant__ CUtensorMap tm_v, const PfParams p) {
    using L = PfLayout;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    if (sbase & 1023u) {  // uniform across the grid: every CTA leaves before any barrier
        if (threadIdx.x == 0) atomicOr(&g_smla_error, kErrLayout);
        return;
    }
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    const int run = static_cast<int>(blockIdx.x >> 1);
    volatile int* sAbort = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
    auto bar = [&](int i) -> uint32_t { return sbase + L::kOffBar + 8u * static_cast<uint32_t>(i); };
    auto even_bar = [&](int i) -> uint32_t { return ptx::map_shared_rank(bar(i), 0); };
    auto wait = [&](int i, uint32_t parity) -> bool {
        return ptx::mbar_wait_cluster(bar(i), parity, sAbort, &g_smla_error, kErrTimeout, kWaitLimitNs);
    };

    if (threadIdx.x == 0) {
        *sAbort = 0;
        ptx::mbar_init(bar(kPbQFull), 1);
        ptx::mbar_init(bar(kPbQEmpty), 1);
        for (int s = 0; s < kPfStages; ++s) {
            ptx::mbar_init(bar(kPbKFull + s), KVF == 0 ? 1 : 2 * kPfDeqWarps);
            ptx::mbar_init(bar(kPbVFull + s), KVF == 0 ? 1 : 2 * kPfDeqWarps);
            ptx::mbar_init(bar(kPbKEmpty + s), 1);
            ptx::mbar_init(bar(kPbVEmpty + s), 1);
            ptx::mbar_init(bar(kPbSFull + s), 1);
            ptx::mbar_init(bar(kPbSEmpty + s), 8);
        }
        ptx::mbar_init(bar(kPbPFull), 8);
        ptx::mbar_init(bar(kPbPvDone), 1);
        ptx::mbar_init(bar(kPbTail), 1);
        ptx::fence_mbarrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(sbase + L::kOffMisc, L::kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    // launched as a programmatic dependent: nothing above touched global memory
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    ptx::tc_fence_before();
    ptx::cluster_sync();  // both CTAs' barriers are initialised before anyone signals them
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc);

    if (warp == 0) {
        // ================================================================ TMA producer
        // Q of each piece, and for bf16 rows K and V of each block: the even CTA's thread expects
        // both CTAs' bytes on its barrier, each CTA's thread issues its own copies.
        if (lane == 0) {
            ptx::prefetch_tmap(&tm_q);
            if (KVF == 0) {
                ptx::prefetch_tmap(&tm_k);
                ptx::prefetch_tmap(&tm_v);
            }
            // K runs a block ahead of V, the order in which the tensor cores finish their stages:
            // K(x) waits for S(x - 2), V(x - 1) for PV(x - 3)
            auto page_row = [&](int b) -> int {  // a page outside the cache loads as zeros, from rows below 0
                const int page = __ldg(p.pages + b);
                return page >= 0 && static_cast<int64_t>(page) * kPfKeys < p.num_slots ? page * kPfKeys : -kPfKeys;
            };
            auto load_v = [&](int x, int b, int row) -> bool {
                const int s = x & 1;
                if (x >= kPfStages && !wait(kPbVEmpty + s, ((x >> 1) - 1) & 1)) return false;
                const uint32_t dst = sbase + L::kOffV + s * kPfVBytes;
                if (p.prefix - static_cast<int64_t>(b) * kPfKeys < kPfKeys) {
                    // the softmax warps wait for this one themselves and zero its end
                    ptx::mbar_arrive_expect_tx(bar(kPbTail), static_cast<uint32_t>(kPfVBytes));
                    ptx::tma_load_3d(dst, &tm_v, 0, row, 4 * rank, bar(kPbTail));
                } else {
                    if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kPbVFull + s), 2u * kPfVBytes);
                    ptx::tma_load_3d_pair(dst, &tm_v, 0, row, 4 * rank, even_bar(kPbVFull + s));
                }
                return true;
            };
            bool ok = true;
            int x = 0, piece = 0, row = 0, row_v = 0, b_v = 0;
            for (PfWalk w(p, run); ok && w.next(); ++piece) {
                if (piece > 0 && !(ok = wait(kPbQEmpty, (piece - 1) & 1))) break;
                if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kPbQFull), 2u * kPfQBytes);
                ptx::tma_load_3d_pair(sbase + L::kOffQ, &tm_q, 0, static_cast<int>(w.tile * kPfRows + rank * kPfHalf), 0,
                                      even_bar(kPbQFull));
                if (KVF == 0) {
                    for (int b = w.b0; ok && b < w.b1; ++b, ++x) {
                        const int s = x & 1;
                        row = page_row(b);
                        if (x >= kPfStages && !(ok = wait(kPbKEmpty + s, ((x >> 1) - 1) & 1))) break;
                        if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kPbKFull + s), 2u * kPfKBytes);
                        ptx::tma_load_3d_pair(sbase + L::kOffK + s * kPfKBytes, &tm_k, 0, row + 32 * rank, 0, even_bar(kPbKFull + s));
                        if (x > 0) ok = load_v(x - 1, b_v, row_v);
                        row_v = row;
                        b_v = b;
                    }
                }
            }
            if (KVF == 0 && ok && x > 0) load_v(x - 1, b_v, row_v);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================================================================ MMA issuer
        // Order: S(0), S(1), PV(0), S(2), PV(1), ...: the softmax of block x runs under S(x + 1).
        if (rank == 0 && lane == 0) {
            constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(kPfRows, kPfKeys, 0, 0);
            constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kPfRows, 256, 0, 1);
            const uint64_t dq = ptx::smem_desc_sw128(sbase + L::kOffQ, 16, 1024);
            const uint64_t dk = ptx::smem_desc_sw128(sbase + L::kOffK, 16, 1024);
            const uint64_t dv = ptx::smem_desc_sw128(sbase + L::kOffV, kPfVPanel, 1024);
            const uint64_t dp = ptx::smem_desc_sw128(sbase + L::kOffP, 16, 1024);
            auto issue_s = [&](int x, bool first, bool last, int piece) -> bool {
                const int s = x & 1;
                if (first && !wait(kPbQFull, piece & 1)) return false;
                if (!wait(kPbKFull + s, (x >> 1) & 1)) return false;
                if (x >= 2 && !wait(kPbSEmpty + s, ((x >> 1) - 1) & 1)) return false;
                ptx::tc_fence_after();
                const uint64_t k0 = dk + static_cast<uint64_t>((s * kPfKBytes) >> 4);
                const uint32_t d = tmem + L::kColS + s * 32;
#pragma unroll
                for (int pn = 0; pn < kPanels; ++pn)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        ptx::mma_bf16_ss_pair(d, dq + ((pn * kPfHalf * 128 + k * 32) >> 4), k0 + ((pn * kPfKPanel + k * 32) >> 4),
                                              kIdescS, (pn | k) != 0);
                ptx::mma_commit_pair(bar(kPbSFull + s));
                ptx::mma_commit_pair(bar(kPbKEmpty + s));
                if (last) ptx::mma_commit_pair(bar(kPbQEmpty));
                return true;
            };
            uint32_t v_parity = 0u;  // bit s: parity of the loads that came to V stage s (tails have their own barrier)
            auto issue_pv = [&](int x, int b, bool first) -> bool {
                const int s = x & 1;
                if (!wait(kPbPFull, x & 1)) return false;
                const bool tail = KVF == 0 && p.prefix - static_cast<int64_t>(b) * kPfKeys < kPfKeys;
                if (!tail) {
                    if (!wait(kPbVFull + s, (v_parity >> s) & 1u)) return false;
                    v_parity ^= 1u << s;
                }
                ptx::tc_fence_after();
                const uint64_t v0 = dv + static_cast<uint64_t>((s * kPfVBytes) >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        ptx::mma_bf16_ss_pair(tmem + L::kColO + 128 * i, dp + ((k * 32) >> 4),
                                              v0 + ((2 * i * kPfVPanel + k * 2048) >> 4), kIdescPV, (!first || k > 0) ? 1u : 0u);
                ptx::mma_commit_pair(bar(kPbVEmpty + s));
                ptx::mma_commit_pair(bar(kPbPvDone));
                return true;
            };
            bool ok = true;
            int x = 0, piece = 0;
            int pend_b = 0;
            bool pend_first = false, pend = false;
            for (PfWalk w(p, run); ok && w.next(); ++piece) {
                for (int b = w.b0; ok && b < w.b1; ++b, ++x) {
                    ok = issue_s(x, b == w.b0, b + 1 == w.b1, piece);
                    if (ok && pend) ok = issue_pv(x - 1, pend_b, pend_first);
                    pend = true;
                    pend_b = b;
                    pend_first = b == w.b0;
                }
            }
            if (ok && pend) issue_pv(x - 1, pend_b, pend_first);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ================================================================ softmax / output
        const int quad = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const int half = quad >> 1;                 // keys 32 half .. + 31, dims 256 half .. + 255
        const int r = (quad & 1) * 32 + lane;       // row of this CTA's 64
        const uint32_t grp = 1u + static_cast<uint32_t>(quad & 1);
        const float c = p.sm_scale_log2;
        volatile float* sX = reinterpret_cast<volatile float*>(smem + L::kOffX);
        auto warp_wait = [&](int i, uint32_t parity) -> bool {
            bool okw = true;
            if (lane == 0) okw = wait(i, parity);
            okw = __shfl_sync(0xffffffffu, okw, 0);
            __syncwarp();
            return okw;
        };
        const uint32_t s_empty0 = even_bar(kPbSEmpty), s_empty1 = even_bar(kPbSEmpty + 1), p_full = even_bar(kPbPFull);
        const uint32_t p_row = sbase + L::kOffP + r * 128;
        bool failed = false;
        int x = 0, tails = 0;
        for (PfWalk w(p, run); !failed && w.next();) {
            float m = -CUDART_INF_F, l = 0.f;
            int page = __ldg(p.pages + w.b0);
            for (int b = w.b0; b < w.b1; ++b, ++x) {
                const int valid = pf_valid(p, b, page);
                if (b + 1 < w.b1) page = __ldg(p.pages + b + 1);
                const int s = x & 1;
                uint32_t sv[32];
                float mx = -CUDART_INF_F;
                if (!failed && !warp_wait(kPbSFull + s, (x >> 1) & 1)) failed = true;
                if (!failed) {
                    ptx::tc_fence_after();
                    SMLA_TMEM_LD16(tmem + lane_base + L::kColS + s * 32, sv);
                    SMLA_TMEM_LD16(tmem + lane_base + L::kColS + s * 32 + 16, sv + 16);
                    ptx::tmem_wait_ld();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster(s ? s_empty1 : s_empty0);
                    const int n = valid - 32 * half;  // keys of this thread's 32 that take part
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 y = ptx::mul2(make_float2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])),
                                                   make_float2(c, c));
                        sv[2 * i] = __float_as_uint(y.x);
                        sv[2 * i + 1] = __float_as_uint(y.y);
                    }
                    if (n < 32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i >= n) sv[i] = __float_as_uint(-CUDART_INF_F);
                    }
                    float mxa[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int i = 0; i < 32; ++i) mxa[i & 3] = fmaxf(mxa[i & 3], __uint_as_float(sv[i]));
                    mx = fmaxf(fmaxf(mxa[0], mxa[1]), fmaxf(mxa[2], mxa[3]));
                    // P's buffer and O are free of PV(x - 1) from here on
                    if (x > 0 && !warp_wait(kPbPvDone, (x - 1) & 1)) failed = true;
                }
                if (ptx::named_bar_red_or(grp, 64u, failed || mx > m + kRescaleLog2)) {
                    // the row's max over both threads' keys (NaN: one of them gave up)
                    sX[half * kPfHalf + r] = failed ? CUDART_NAN_F : mx;
                    ptx::named_bar_sync(grp, 64u);
                    const float o = sX[(half ^ 1) * kPfHalf + r];
                    ptx::named_bar_sync(grp, 64u);
                    if (__any_sync(0xffffffffu, failed || o != o)) {
                        failed = true;
                        break;
                    }
                    const float mn = fmaxf(mx, o);
                    const bool grow = mn > m + kRescaleLog2;
                    float alpha = 1.f;
                    if (grow) {
                        alpha = m == -CUDART_INF_F ? 0.f : ptx::ex2_approx(m - mn);
                        m = mn;
                        l *= alpha;
                    }
                    if (b > w.b0 && __any_sync(0xffffffffu, grow)) {
                        ptx::tc_fence_after();
#pragma unroll 1
                        for (int cc = 0; cc < 16; ++cc) {
                            uint32_t ov[16];
                            SMLA_TMEM_LD16(tmem + lane_base + L::kColO + cc * 16, ov);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                            SMLA_TMEM_ST16(tmem + lane_base + L::kColO + cc * 16, ov);
                        }
                        ptx::tmem_wait_st();
                        ptx::tc_fence_before();
                    }
                }
                // P = 2^(x - m) as bf16, the operand of PV (its rounding averages out over the keys;
                // the sum takes the unrounded values)
                const float nm = m == -CUDART_INF_F ? 0.f : -m;
                uint32_t pk[16];
                float2 la[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) la[i] = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 d = ptx::add2(make_float2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])),
                                               make_float2(nm, nm));
                    const float2 pp = make_float2(ptx::ex2_approx(d.x), ptx::ex2_approx(d.y));
                    la[i & 3] = ptx::add2(la[i & 3], pp);
                    pk[i] = pack_bf16x2(pp.x, pp.y);
                }
                l += ((la[0].x + la[0].y) + (la[1].x + la[1].y)) + ((la[2].x + la[2].y) + (la[3].x + la[3].y));
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    ptx::st_shared_v4(p_row + ((static_cast<uint32_t>(4 * half + q) ^ static_cast<uint32_t>(r & 7)) << 4),
                                      make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]));
                const int64_t left = p.prefix - static_cast<int64_t>(b) * kPfKeys;
                if (KVF == 0 && left < kPfKeys) {
                    // the page's rows past the prefix's end, zeroed in this CTA's V tile
                    if (!warp_wait(kPbTail, tails & 1)) {
                        failed = true;
                        continue;  // the next reduction (or the one after the loop) takes the group out
                    }
                    ++tails;
                    const int first = static_cast<int>(left);
                    const int tid = (warp - 2) * 32 + lane;
                    const uint32_t vt = sbase + L::kOffV + s * kPfVBytes;
                    for (int i = tid; i < (kPfKeys - first) * 32; i += 128)
                        ptx::st_shared_v4(vt + (i & 3) * kPfVPanel + (first + (i >> 5)) * 128 + ((i >> 2) & 7) * 16,
                                          make_uint4(0u, 0u, 0u, 0u));
                }
                ptx::fence_proxy_async_all();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(p_full);
            }
            // ---- the piece's rows: O / l as bf16 and the natural-log LSE if the tile is whole, else
            // the unnormalised partial
            if (!failed && !warp_wait(kPbPvDone, (x - 1) & 1)) failed = true;
            ptx::tc_fence_after();
            sX[half * kPfHalf + r] = failed ? CUDART_NAN_F : l;
            if (ptx::named_bar_red_or(grp, 64u, failed)) {
                failed = true;
                break;
            }
            const float lt = l + sX[(half ^ 1) * kPfHalf + r];
            ptx::named_bar_sync(grp, 64u);
            const int64_t row = w.tile * kPfRows + rank * kPfHalf + r;
            const bool live = row < p.rows;
            const bool whole = w.b0 == 0 && w.b1 == p.nblk;
            const int64_t slot = 2 * static_cast<int64_t>(run) + (p.work * run / p.runs / p.nblk == w.tile ? 0 : 1);
            const int64_t prow = slot * p.slot_rows + rank * kPfHalf + r;
            const float inv = lt > 0.f || lt != lt ? 1.0f / lt : 0.f;
            if (live && half == 0) {
                if (whole) {
                    p.lse[row] = lt == 0.f ? -CUDART_INF_F : (m + log2f(lt)) * 0.69314718055994531f;
                } else {
                    p.part_ml[2 * prow] = m;
                    p.part_ml[2 * prow + 1] = lt;
                }
            }
#pragma unroll 1
            for (int cc = 0; cc < 16; ++cc) {
                uint32_t ov[16];
                SMLA_TMEM_LD16(tmem + lane_base + L::kColO + cc * 16, ov);
                ptx::tmem_wait_ld();
                if (live && whole) {
                    uint4* dst = reinterpret_cast<uint4*>(p.out + row * kDV + 256 * half + 16 * cc);
                    uint32_t u[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        u[e] = pack_bf16x2(__uint_as_float(ov[2 * e]) * inv, __uint_as_float(ov[2 * e + 1]) * inv);
                    dst[0] = make_uint4(u[0], u[1], u[2], u[3]);
                    dst[1] = make_uint4(u[4], u[5], u[6], u[7]);
                } else if (live) {
                    uint4* dst = reinterpret_cast<uint4*>(p.part_o + prow * kDV + 256 * half + 16 * cc);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dst[e] = make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
                }
            }
            ptx::tc_fence_before();  // before the next piece's first PV overwrites O
        }
    } else if constexpr (KVF == 1) {
        // ================================================================ producers of fp8 rows
        // Per block: this CTA's 32 keys in full (four rows of 512 codes per warp, 16 codes a lane) and
        // the other 32 keys' 256 dims (16 lanes per key), loaded a block ahead into registers.  The
        // two 16-byte stores of a lane go to neighbouring chunks; every other group of four lanes
        // takes the odd one first, so that eight lanes cover eight chunks (no bank conflict).
        const int pw = warp - 6;
        const int tid = pw * 32 + lane;
        const int swap = (lane >> 2) & 1;
        const uint8_t* kv8 = static_cast<const uint8_t*>(p.kv);
        const int64_t at0 = p.work * run / p.runs;
        const int n = static_cast<int>(p.work * (run + 1) / p.runs - at0);
        uint4 lat[6], rope;
        float scl[6];
        auto load = [&](int b) {
            const int page = __ldg(p.pages + b);
            const int valid = pf_valid(p, b, page);
            const uint8_t* base = kv8 + static_cast<int64_t>(page) * kPfKeys * kFp8RowBytes;
#pragma unroll
            for (int u = 0; u < 6; ++u) {
                const int i = tid + 256 * (u - 4);
                const int key = u < 4 ? 32 * rank + pw + 8 * u : 32 * (rank ^ 1) + (i >> 4);
                const int c16 = u < 4 ? lane : 16 * rank + (i & 15);
                lat[u] = make_uint4(0u, 0u, 0u, 0u);
                scl[u] = 0.f;
                if (key < valid) {
                    const uint8_t* src = base + key * kFp8RowBytes;
                    lat[u] = ptx::ld_nc_v4(src + 16 * c16);
                    scl[u] = ptx::ld_nc_f32(src + 512 + 4 * (c16 >> 3));
                }
            }
            const int key = 32 * rank + (tid >> 3);
            rope = make_uint4(0u, 0u, 0u, 0u);
            if (key < valid) rope = ptx::ld_nc_v4(base + key * kFp8RowBytes + 528 + 16 * (tid & 7));
        };
        auto convert = [&](const uint4 v, float sc, uint4 (&o)[2]) {
            o[0] = make_uint4(ptx::e4m3x2_scaled_bf16x2(v.x & 0xFFFFu, sc), ptx::e4m3x2_scaled_bf16x2(v.x >> 16, sc),
                              ptx::e4m3x2_scaled_bf16x2(v.y & 0xFFFFu, sc), ptx::e4m3x2_scaled_bf16x2(v.y >> 16, sc));
            o[1] = make_uint4(ptx::e4m3x2_scaled_bf16x2(v.z & 0xFFFFu, sc), ptx::e4m3x2_scaled_bf16x2(v.z >> 16, sc),
                              ptx::e4m3x2_scaled_bf16x2(v.w & 0xFFFFu, sc), ptx::e4m3x2_scaled_bf16x2(v.w >> 16, sc));
        };
        auto put = [&](uint32_t row_addr, uint32_t ch, int row, const uint4 (&o)[2]) {
            const uint32_t sw = static_cast<uint32_t>(row & 7);
            const uint32_t c0 = ch + swap, c1 = ch + (swap ^ 1);
            ptx::st_shared_v4(row_addr + ((c0 ^ sw) << 4), swap ? o[1] : o[0]);
            ptx::st_shared_v4(row_addr + ((c1 ^ sw) << 4), swap ? o[0] : o[1]);
        };
        int b = static_cast<int>(at0 % p.nblk);
        if (n > 0) load(b);
        for (int x = 0; x < n; ++x) {
            const int s = x & 1;
            bool ok = true;
            if (x >= kPfStages) {
                if (lane == 0) ok = wait(kPbKEmpty + s, ((x >> 1) - 1) & 1) && wait(kPbVEmpty + s, ((x >> 1) - 1) & 1);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                __syncwarp();
                if (!ok) break;
            }
            const uint32_t sK = sbase + L::kOffK + s * kPfKBytes, sV = sbase + L::kOffV + s * kPfVBytes;
            const uint32_t ch = static_cast<uint32_t>((lane & 3) * 2);
#pragma unroll
            for (int u = 0; u < 6; ++u) {
                uint4 o[2];
                convert(lat[u], scl[u], o);
                if (u < 4) {
                    const int row = pw + 8 * u;
                    put(sK + (lane >> 2) * kPfKPanel + row * 128, ch, row, o);
                    if ((lane >> 4) == rank) put(sV + ((lane >> 2) & 3) * kPfVPanel + (32 * rank + row) * 128, ch, row, o);
                } else {
                    const int i = tid + 256 * (u - 4);
                    const int key = 32 * (rank ^ 1) + (i >> 4);
                    put(sV + ((i & 15) >> 2) * kPfVPanel + key * 128, ch, key, o);
                }
            }
            const int row = tid >> 3;
            ptx::st_shared_v4(sK + 8 * kPfKPanel + row * 128 + ((static_cast<uint32_t>(tid & 7) ^ static_cast<uint32_t>(row & 7)) << 4),
                              rope);
            ptx::fence_proxy_async_all();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive_cluster(even_bar(kPbKFull + s));
                ptx::mbar_arrive_cluster(even_bar(kPbVFull + s));
            }
            if (++b == p.nblk) b = 0;
            if (x + 1 < n) load(b);
        }
    }
    // ---- both CTAs are done with each other's shared memory, barriers and TMEM
    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, L::kTmemCols);
    }
}

// Joins the pieces of cut tiles, one CTA per query row: weights 2^(m_i - M) of the running maxima,
// pieces in run order.  Reads what the pieces wrote once (from L2 as a rule).
__global__ void __launch_bounds__(kPfMergeThreads) sparse_mla_prefix_merge_kernel(const PfParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t row = blockIdx.x;
    const int64_t tile = row / kPfRows;
    const int rt = static_cast<int>(row % kPfRows);
    auto run_of = [&](int64_t b) -> int { return static_cast<int>(((b + 1) * p.runs - 1) / p.work); };
    const int k0 = run_of(tile * p.nblk), k1 = run_of((tile + 1) * p.nblk - 1);
    if (k0 == k1) return;  // the tile lies inside one run, which wrote it
    auto slot_row = [&](int k) -> int64_t {
        const int64_t slot = 2 * static_cast<int64_t>(k) + (p.work * k / p.runs / p.nblk == tile ? 0 : 1);
        return slot * p.slot_rows + rt;
    };
    float m = -CUDART_INF_F;
    for (int k = k0; k <= k1; ++k) m = fmaxf(m, p.part_ml[2 * slot_row(k)]);
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int kk = k0; kk <= k1; kk += 4) {
        float4 v[4];
        float wt[4], lk[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            wt[u] = lk[u] = 0.f;
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (kk + u <= k1) {
                const int64_t sr = slot_row(kk + u);
                const float mk = p.part_ml[2 * sr];
                lk[u] = p.part_ml[2 * sr + 1];
                wt[u] = mk == -CUDART_INF_F ? 0.f : ptx::ex2_approx(mk - m);
                // a piece without a key has no O of its own (its sum is 0), whatever its slot holds
                if (lk[u] != 0.f) v[u] = reinterpret_cast<const float4*>(p.part_o + sr * kDV)[threadIdx.x];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            l += wt[u] * lk[u];
            acc.x += wt[u] * v[u].x;
            acc.y += wt[u] * v[u].y;
            acc.z += wt[u] * v[u].z;
            acc.w += wt[u] * v[u].w;
        }
    }
    const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
    reinterpret_cast<uint2*>(p.out + row * kDV)[threadIdx.x] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (threadIdx.x == 0) p.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
}

// The result over no keys: O = 0, LSE = -inf.
__global__ void __launch_bounds__(256) sparse_mla_prefix_empty_kernel(const PfParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = i0; i < p.rows * (kDV / 8); i += step) reinterpret_cast<uint4*>(p.out)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t i = i0; i < p.rows; i += step) p.lse[i] = -CUDART_INF_F;
}

}  // namespace smla
