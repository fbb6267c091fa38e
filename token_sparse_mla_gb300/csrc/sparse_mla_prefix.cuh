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
// 0-63 and the second half in lanes 64-127, so O is 256 columns and S 64.  Per block of 128 keys
// (two pages):
//   S[128, 128]  = Q . K^T     A: each CTA's 64 rows of Q; B: each CTA's page of 64 keys, all 576 dims
//   O[128, 512] += P . V       A: each CTA's 64 rows of P; B: both pages, each CTA's 256 dims
// Back to back, an MMA of this form takes 32 cycles at N = 128 and 64 at N = 256 (4060 multiply-adds a
// cycle and SM, the dense rate) but 25 at N = 64, so blocks of one page would lose a third of S; a block
// of two is 36 * 32 + 16 * 64 = 2190 cycles.  The nearer bound is shared memory: operands of S 144 KB
// and of PV 96 KB, 136 KB written by TMA and P's 16 KB are 3140 cycles at 128 bytes a cycle; measured
// (76 tiles, 16384 keys against 8192) 1.73 us a block, 3260 cycles at the 1.89 GHz of a run of seconds, and
// 1.6 us, 1700 TFLOP/s, in a short one.  What the shape costs is room: Q 72 KB, K 72 KB, V 64 KB and P 16 KB leave one stage of each, so K is refilled in two groups of
// panels and V and P page by page, each as soon as its last MMA is done.  (The half of V that lies in a
// CTA's own K tile is loaded again: the MMA wants the same keys at the same offset in both CTAs, and K
// wants different ones.)
//
// fp8 rows are first expanded to bf16 rows in the workspace (sparse_mla_prefix_expand_kernel), in
// prefix order: dequantising in the main kernel would be repeated for every 128 query rows, and with
// eight warps at it a block of 64 keys took 3.7 us.  The product code x scale is rounded to bf16, the
// MMA's operand type, as in the forward.
//
// Work: the (row tile, block) sequence, tile-major, is cut into equal contiguous runs, one per CTA
// pair: as many as there are pairs, or the same number for each tile where that is shorter (the host's
// plan weighs them: 256 rows x 16384 keys took 26 us in 76 runs, 20 in 64).  A tile that lies inside one run is written out directly; a cut tile leaves an fp32 partial (O,
// running max, sum) per piece in the workspace, at most two per run, which a second kernel joins by
// log-sum-exp weights in run order (so results do not depend on timing).
//
// Rows past the prefix's end in its last page are masked in S, and zeroed in the V tile before they
// are multiplied: 0 times whatever the page holds there must stay 0.  A page number outside the
// cache masks its page; rows of a page past the cache's end are masked.
//
// Roles (384 threads):
//   warp 0      TMA producer (one thread).
//   warp 1      S issuer (one thread of the even CTA) for dims 0 .. 319, and TMEM owner.
//   warps 2-9   softmax, rescaling and output, two warps per TMEM lane quadrant: row r = lane % 64,
//               page lane / 64 of a block and 32 of its keys, dims 256 (lane / 64) .. + 255 of O and
//               128 of those.  The running max is moved only when it grows by more than 2^8; the four
//               warps of a row vote per block and swap maxima only then.  (One warp per quadrant took
//               2.4 us a block, longer than the block's MMAs.)
//   warp 10     PV issuer, warp 11 S issuer for dims 320 .. 575 (one thread of the even CTA each).
// Every wait is bounded; a CTA that gives up meets the other at the final cluster barrier.
#pragma once

#include "sparse_mla_common.cuh"

namespace smla {

constexpr int kPfRows = 128;                      // query rows per CTA pair (MMA M)
constexpr int kPfHalf = 64;                       // query rows per CTA
constexpr int kPfPage = 64;                       // rows per page
constexpr int kPfKeys = 2 * kPfPage;              // keys per block
constexpr int kPfSoftmaxWarps = 8;
constexpr int kPfPvWarp = 2 + kPfSoftmaxWarps;
constexpr int kPfS2Warp = kPfPvWarp + 1;
constexpr int kPfThreads = 32 * (kPfS2Warp + 1);
constexpr int kPfPanel = 64 * 128;                // 64 rows x 64 bf16, SW128
constexpr int kPfQBytes = kPanels * kPfPanel;
constexpr int kPfGroupA = 5;                      // K in two groups of panels, 0 .. 4 and 5 .. 8, each with an
constexpr int kPfGroupB = kPanels - kPfGroupA;    // issuing thread, a refill and an accumulator of its own
static_assert(kPfGroupB == 4, "the second group is loaded by V's map (four panels)");
constexpr int kPfVPage = 4 * kPfPanel;            // one page, this CTA's 256 dims
constexpr int kPfMergeThreads = 512;
constexpr int kPfExpandThreads = 128;
constexpr int kPfExpandRows = 4;                  // rows per warp

struct PfLayout {
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kPfQBytes;
    static constexpr int kOffV = kOffK + kPfQBytes;
    static constexpr int kOffP = kOffV + 2 * kPfVPage;        // two panels; output staging between pieces
    static constexpr int kOffX = kOffP + 2 * kPfPanel;        // [4][64] values swapped by a row's four threads
    static constexpr int kOffBar = kOffX + 4 * kPfHalf * 4;
    static constexpr int kNumBars = 18;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;   // tmem base, abort flag
    static constexpr int kBytes = kOffMisc + 16;
    // TMEM columns: O [0, 256) | two buffers of (S of the first group, S of the second), 64 each
    static constexpr int kColO = 0;
    static constexpr int kColS = 256;
    static constexpr int kSBuf = 2 * kPfPage;
    static_assert(kColS + 2 * kSBuf <= 512, "TMEM columns");
    static constexpr int kTmemCols = 512;
    static_assert(kBytes <= 232448, "shared memory budget (227 KB)");
};

enum : int {
    kPbQFull = 0,    // even CTA: both CTAs' Q landed
    kPbQEmpty = 1,   // both: the S MMAs of the piece are done
    kPbKFull = 2,    // +group, even CTA
    kPbKEmpty = 4,   // +group, both
    kPbVFull = 6,    // +page of the block, even CTA
    kPbVEmpty = 8,   // +page, both: the page's PV MMAs and all before them are done
    kPbSFull = 10,   // +buffer, both
    kPbSEmpty = 12,  // +buffer, even CTA
    kPbPFull = 14,   // +page, even CTA
    kPbTail = 16,    // own CTA: V of a page that the prefix ends in
    kPbDrain = 17    // even CTA: everything the issuers issued is done
};

struct PfParams {
    const void* kv;              // the cache
    __nv_bfloat16* expanded;     // bf16 rows in prefix order (fp8 caches), or nullptr
    const int32_t* pages;        // [npages]
    __nv_bfloat16* out;          // [rows, 512]
    float* lse;                  // [rows]
    // partials of cut tiles, rows in groups of 32 with neighbouring rows next to each other, so that a
    // warp (a lane per row) stores and loads whole lines
    float* part_o;               // [2 * runs][slot_groups][128][32][4]: dims 4 j .. 4 j + 3 of 32 rows
    float* part_ml;              // [2 * runs][slot_groups][2][32]: running max (log2 units), sum
    int64_t rows;                // T * h
    int64_t prefix;              // P
    int64_t num_slots;
    int64_t tiles;               // ceil(rows / 128)
    int64_t work;                // tiles * nblk
    int32_t npages, nblk, runs;
    int32_t slot_groups;         // groups of 32 rows in a tile: ceil(min(128, rows) / 32)
    float sm_scale_log2;
};

// Page number of page i of the prefix (-1 past its end).
__device__ __forceinline__ int pf_page(const PfParams& p, int i) { return i < p.npages ? ptx::ld(p.pages + i) : -1; }

__device__ __forceinline__ bool pf_in_cache(const PfParams& p, int page) {
    return page >= 0 && static_cast<int64_t>(page) * kPfPage < p.num_slots;
}

// Rows of page i of the prefix that take part (0 .. 64), given its page number.
__device__ __forceinline__ int pf_valid(const PfParams& p, int i, int page) {
    if (!pf_in_cache(p, page)) return 0;
    const int64_t left = p.prefix - static_cast<int64_t>(i) * kPfPage;
    const int64_t room = p.num_slots - static_cast<int64_t>(page) * kPfPage;
    const int64_t n = left < room ? left : room;
    return n < kPfPage ? static_cast<int>(n) : kPfPage;
}

// Whether page i is one whose end has to be zeroed in V.  (Expanded rows past the end are zeros.)
__device__ __forceinline__ bool pf_tail(const PfParams& p, int i) {
    return p.expanded == nullptr && i == p.npages - 1 && p.prefix % kPfPage != 0;
}

// The pieces of a run, the same for every role: blocks [b0, b1) of tile t.
struct PfWalk {
    int64_t left;    // blocks of the run still to come
    int64_t tile;
    int32_t nblk;
    int b0, b1;
    bool first;      // the run's first piece
    __device__ __forceinline__ PfWalk(const PfParams& p, int run) : nblk(p.nblk), b1(0), first(true) {
        const int64_t at = p.work * run / p.runs;
        left = p.work * (run + 1) / p.runs - at;
        tile = at / nblk;
        b0 = static_cast<int>(at - tile * nblk);
    }
    // first call: the first piece; later calls: the next tile's
    __device__ __forceinline__ bool next() {
        if (b1 != 0) {
            b0 = 0;
            ++tile;
            first = false;
        }
        if (left <= 0) return false;
        const int64_t n = left < nblk - b0 ? left : nblk - b0;
        b1 = b0 + static_cast<int>(n);
        left -= n;
        return true;
    }
};

__global__ void __launch_bounds__(kPfThreads, 1)
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
        return ptx::mbar_wait(bar(i), parity, sAbort, &g_smla_error, kErrTimeout, kWaitLimitNs);
    };

    if (threadIdx.x == 0) {
        *sAbort = 0;
        for (int i = 0; i < L::kNumBars; ++i) {
            const bool by_warps = i == kPbSEmpty || i == kPbSEmpty + 1;                // both CTAs' softmax warps
            const bool by_half = i == kPbPFull || i == kPbPFull + 1;                   // those of the page
            const bool by_two = i == kPbQEmpty || i == kPbSFull || i == kPbSFull + 1;  // both S issuers
            ptx::mbar_init(bar(i), by_warps ? 2 * kPfSoftmaxWarps : by_half ? kPfSoftmaxWarps : i == kPbDrain ? 3 : by_two ? 2 : 1);
        }
        ptx::fence_mbarrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(sbase + L::kOffMisc, L::kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tmap(&tm_q);
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
    }
    PfWalk w(p, run);
    const bool any = w.next();
    // launched as a programmatic dependent: nothing above touched global memory
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    // the producer's page numbers are loaded ahead and looked at only where their rows are asked for
    // (the first two under the cluster barrier)
    int pg0 = -1, pg1 = -1;
    if (warp == 0 && lane == 0) {
        pg0 = pf_page(p, 2 * w.b0);
        pg1 = pf_page(p, 2 * w.b0 + 1);
    }
    ptx::tc_fence_before();
    __syncwarp();         // the cluster barrier wants its warps whole
    ptx::cluster_sync();  // both CTAs' barriers are initialised before anyone signals them
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc);

    if (warp == 0) {
        // ================================================================ TMA producer
        // The even CTA's thread expects both CTAs' bytes on its barrier, each CTA's thread issues its
        // own copies.  K runs a block ahead of V, the order in which the tensor cores release them:
        // K(x) waits for S(x - 1), V(x - 1) for PV(x - 2).
        if (lane == 0) {
            auto load_v = [&](int x, int b, int row0, int row1) -> bool {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (x > 0 && !wait(kPbVEmpty + i, (x - 1) & 1)) return false;
                    const uint32_t dst = sbase + L::kOffV + i * kPfVPage;
                    if (pf_tail(p, 2 * b + i)) {  // the softmax warps wait for this one themselves and zero its end
                        ptx::mbar_arrive_expect_tx(bar(kPbTail), static_cast<uint32_t>(kPfVPage));
                        ptx::tma_load_3d(dst, &tm_v, 0, i ? row1 : row0, 4 * rank, bar(kPbTail));
                    } else {
                        if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kPbVFull + i), 2u * kPfVPage);
                        ptx::tma_load_3d_pair(dst, &tm_v, 0, i ? row1 : row0, 4 * rank, even_bar(kPbVFull + i));
                    }
                }
                return true;
            };
            // this CTA's page of the next block, into L2 while the current one is waited for: loaded from HBM
            // only when K's buffer is free it would be too late (1024 rows x 65536 keys: 129 us without, 105
            // with; two blocks ahead 106, three 107, 1 row x 131072 50 / 42 / 44 / 48: the first blocks wait
            // behind them)
            auto prefetch = [&](int b) {
                const int i = 2 * b + rank;
                if (i >= p.npages) return;
                const __nv_bfloat16* src = p.expanded + static_cast<int64_t>(i) * kPfPage * kDQK;
                int n = kPfPage;
                if (p.expanded == nullptr) {
                    const int page = pf_page(p, i);
                    n = pf_valid(p, i, page);
                    src = static_cast<const __nv_bfloat16*>(p.kv) + static_cast<int64_t>(page) * kPfPage * kDQK;
                }
                if (n > 0) ptx::bulk_prefetch_l2(src, static_cast<uint32_t>(n * kDQK * 2));
            };
            auto first_row = [&](int i, int page) -> int {  // of page i; one that is not there loads as zeros, from rows below 0
                if (p.expanded != nullptr) return i < p.npages ? i * kPfPage : -kPfPage;
                return pf_in_cache(p, page) ? page * kPfPage : -kPfPage;
            };
            bool ok = true;
            int x = 0, piece = 0, b_v = 0;
            int row_v0 = 0, row_v1 = 0;
            for (bool more = any; ok && more; more = w.next(), ++piece) {
                if (piece > 0 && !(ok = wait(kPbQEmpty, (piece - 1) & 1))) break;
                if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kPbQFull), 2u * kPfQBytes);
                ptx::tma_load_3d_pair(sbase + L::kOffQ, &tm_q, 0, static_cast<int>(w.tile * kPfRows + rank * kPfHalf), 0,
                                      even_bar(kPbQFull));
                if (piece > 0) {
                    pg0 = pf_page(p, 2 * w.b0);
                    pg1 = pf_page(p, 2 * w.b0 + 1);
                }
                for (int b = w.b0; ok && b < w.b1; ++b, ++x) {
                    const int row0 = first_row(2 * b, pg0), row1 = first_row(2 * b + 1, pg1);
                    const int mine = rank == 0 ? row0 : row1;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (x > 0 && !(ok = wait(kPbKEmpty + g, (x - 1) & 1))) break;
                        const uint32_t bytes = static_cast<uint32_t>((g ? kPfGroupB : kPfGroupA) * kPfPanel);
                        if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kPbKFull + g), 2u * bytes);
                        ptx::tma_load_3d_pair(sbase + L::kOffK + g * kPfGroupA * kPfPanel, g ? &tm_v : &tm_k, 0, mine,
                                              g * kPfGroupA, even_bar(kPbKFull + g));
                    }
                    prefetch(b + 1);
                    pg0 = pf_page(p, 2 * b + 2);  // in flight under the waits
                    pg1 = pf_page(p, 2 * b + 3);
                    if (ok && x > 0) ok = load_v(x - 1, b_v, row_v0, row_v1);
                    row_v0 = row0;
                    row_v1 = row1;
                    b_v = b;
                }
            }
            if (ok && x > 0) ok = load_v(x - 1, b_v, row_v0, row_v1);
            // every copy has landed and been used, and no release of a stage is still on its way to
            // this CTA's barriers, before it leaves
            for (int g = 0; ok && g < 2; ++g) ok = wait(kPbKEmpty + g, (x - 1) & 1);
            for (int i = 0; ok && i < 2; ++i) ok = wait(kPbVEmpty + i, (x - 1) & 1);
            if (ok) ok = wait(kPbQEmpty, (piece - 1) & 1);
            if (!ok) {  // gave up: copies in flight complete on the other CTA's barriers; leave them time to land
                const uint64_t t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 2000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1 || warp == kPfS2Warp) {
        // ================================================================ S issuers
        // Issuing an MMA costs its thread more time (45 cycles and more, its operands being moved to
        // uniform registers each time, and as much again for waits and commits) than the tensor cores
        // take for one of S (32), so S is two sums over the dims, each issued by a thread of its own
        // into an accumulator of its own; the softmax adds them.
        if (rank == 0 && lane == 0) {
            constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(kPfRows, kPfKeys, 0, 0);
            const bool ga = warp == 1;
            const uint32_t off = ga ? 0u : static_cast<uint32_t>(kPfGroupA * kPfPanel);
            const uint64_t dq = ptx::smem_desc_sw128(sbase + L::kOffQ + off, 16, 1024);
            const uint64_t dk = ptx::smem_desc_sw128(sbase + L::kOffK + off, 16, 1024);
            const uint32_t d0 = tmem + L::kColS + (ga ? 0 : kPfPage);
            const int g = ga ? 0 : 1;
            bool ok = true;
            int x = 0, piece = 0;
            for (bool more = any; ok && more; more = w.next(), ++piece) {
                if (!(ok = wait(kPbQFull, piece & 1))) break;
                for (int b = w.b0; ok && b < w.b1; ++b, ++x) {
                    const int s = x & 1;
                    if (x >= 2 && !(ok = wait(kPbSEmpty + s, ((x >> 1) - 1) & 1))) break;
                    if (!(ok = wait(kPbKFull + g, x & 1))) break;
                    ptx::tc_fence_after();
                    const uint32_t d = d0 + s * L::kSBuf;
#pragma unroll
                    for (int pn = 0; pn < kPfGroupB; ++pn)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ptx::mma_bf16_ss_pair(d, dq + ((pn * kPfPanel + k * 32) >> 4), dk + ((pn * kPfPanel + k * 32) >> 4),
                                                  kIdescS, (pn | k) != 0);
                    if (ga) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ptx::mma_bf16_ss_pair(d, dq + ((kPfGroupB * kPfPanel + k * 32) >> 4),
                                                  dk + ((kPfGroupB * kPfPanel + k * 32) >> 4), kIdescS, 1u);
                    }
                    ptx::mma_commit_pair(bar(kPbSFull + s));
                    ptx::mma_commit_pair(bar(kPbKEmpty + g));
                    if (b + 1 == w.b1) ptx::mma_commit_pair(bar(kPbQEmpty));
                }
            }
            // nothing is in flight when TMEM is freed, also after giving up
            ptx::mma_commit_pair_local(bar(kPbDrain));
            ptx::mbar_wait(bar(kPbDrain), 0, nullptr, &g_smla_error, 0u, kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp == kPfPvWarp) {
        // ================================================================ PV issuer
        // A thread of its own, for the same reason.
        if (rank == 0 && lane == 0) {
            constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kPfRows, 256, 0, 1);
            const uint64_t dv = ptx::smem_desc_sw128(sbase + L::kOffV, kPfPanel, 1024);
            const uint64_t dp = ptx::smem_desc_sw128(sbase + L::kOffP, 16, 1024);
            uint32_t v_parity = 0u;  // bit i: parity of the loads that came to V page i (tails have their own barrier)
            bool ok = true;
            int x = 0;
            for (bool more = any; ok && more; more = w.next()) {
                for (int b = w.b0; ok && b < w.b1; ++b, ++x) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (!(ok = wait(kPbPFull + i, x & 1))) break;
                        if (!pf_tail(p, 2 * b + i)) {
                            if (!(ok = wait(kPbVFull + i, (v_parity >> i) & 1u))) break;
                            v_parity ^= 1u << i;
                        }
                        ptx::tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int n = 0; n < 2; ++n)
                                ptx::mma_bf16_ss_pair(tmem + L::kColO + 128 * n, dp + ((i * kPfPanel + k * 32) >> 4),
                                                      dv + ((i * kPfVPage + 2 * n * kPfPanel + k * 2048) >> 4), kIdescPV,
                                                      (b != w.b0 || i > 0 || k > 0) ? 1u : 0u);
                        ptx::mma_commit_pair(bar(kPbVEmpty + i));
                    }
                }
            }
            // nothing is in flight when TMEM is freed, also after giving up
            ptx::mma_commit_pair_local(bar(kPbDrain));
            ptx::mbar_wait(bar(kPbDrain), 0, nullptr, &g_smla_error, 0u, kDrainLimitNs);
        }
        __syncwarp();
    } else {
        // ================================================================ softmax / output
        const int quad = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const int half = quad >> 1;                 // page of the block, dims 256 half .. + 255
        const int sub = (warp - 2) >> 2;            // keys 32 sub .. + 31 of the page, 128 of the dims
        const int part = 2 * half + sub;            // which of the row's four threads
        const int r = (quad & 1) * 32 + lane;       // row of this CTA's 64
        const uint32_t grp = 1u + static_cast<uint32_t>(quad & 1);
        // logits as |c| times +-s, so that their max is that of +-s and one fma gives log2 of P
        const float c = fabsf(p.sm_scale_log2);
        const bool flip = p.sm_scale_log2 < 0.f;
        volatile float* sX = reinterpret_cast<volatile float*>(smem + L::kOffX);
        auto warp_wait = [&](int i, uint32_t parity) -> bool {
            bool okw = true;
            if (lane == 0) okw = wait(i, parity);
            okw = __shfl_sync(0xffffffffu, okw, 0);
            __syncwarp();
            return okw;
        };
        const uint32_t s_empty0 = even_bar(kPbSEmpty), s_empty1 = even_bar(kPbSEmpty + 1), p_full = even_bar(kPbPFull + half);
        const uint32_t p_row = sbase + L::kOffP + half * kPfPanel + r * 128;
        const int ocol0 = L::kColO + 128 * sub;
        bool failed = false;
        int x = 0, tails = 0;
        for (bool more = any; !failed && more; more = w.next()) {
            float m = -CUDART_INF_F, l = 0.f;
            int page = pf_page(p, 2 * w.b0 + half);
            for (int b = w.b0; b < w.b1; ++b, ++x) {
                const int n = pf_valid(p, 2 * b + half, page) - 32 * sub;  // keys of this thread's 32 that take part
                page = pf_page(p, 2 * b + 2 + half);
                const int s = x & 1;
                uint32_t sv[32];
                float mx = -CUDART_INF_F;
                if (!failed && !warp_wait(kPbSFull + s, (x >> 1) & 1)) failed = true;
                if (!failed) {
                    ptx::tc_fence_after();
                    uint32_t sw[32];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        SMLA_TMEM_LD16(tmem + lane_base + L::kColS + s * L::kSBuf + 32 * sub + 16 * q, sv + 16 * q);
                        SMLA_TMEM_LD16(tmem + lane_base + L::kColS + s * L::kSBuf + kPfPage + 32 * sub + 16 * q, sw + 16 * q);
                    }
                    ptx::tmem_wait_ld(sv, sw);
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster(s ? s_empty1 : s_empty0);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 y = ptx::add2(make_float2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])),
                                                   make_float2(__uint_as_float(sw[2 * i]), __uint_as_float(sw[2 * i + 1])));
                        sv[2 * i] = __float_as_uint(y.x);
                        sv[2 * i + 1] = __float_as_uint(y.y);
                    }
                    if (flip) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) sv[i] ^= 0x80000000u;
                    }
                    if (n < 32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i >= n) sv[i] = __float_as_uint(-CUDART_INF_F);
                    }
                    float mxa[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) mxa[i] = fmaxf(__uint_as_float(sv[i]), __uint_as_float(sv[i + 4]));
#pragma unroll
                    for (int i = 8; i < 32; i += 8)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mxa[j] = ptx::max3(mxa[j], __uint_as_float(sv[i + j]), __uint_as_float(sv[i + j + 4]));
                    mx = fmaxf(fmaxf(mxa[0], mxa[1]), fmaxf(mxa[2], mxa[3]));
                    // (scale 0: every logit is 0.  A row of NaN only: P and the sum carry it.)
                    mx *= c;
                    if (n <= 0 || mx != mx) mx = -CUDART_INF_F;
                }
                if (ptx::named_bar_red_or(grp, 128u, failed || mx > m + kRescaleLog2)) {
                    // the row's max over its four threads' keys (NaN: one of them gave up)
                    sX[part * kPfHalf + r] = failed ? CUDART_NAN_F : mx;
                    ptx::named_bar_sync(grp, 128u);
                    const float o0 = sX[r], o1 = sX[kPfHalf + r], o2 = sX[2 * kPfHalf + r], o3 = sX[3 * kPfHalf + r];
                    ptx::named_bar_sync(grp, 128u);
                    const float mn = ptx::max_nan(ptx::max_nan(o0, o1), ptx::max_nan(o2, o3));
                    if (__any_sync(0xffffffffu, mn != mn)) {
                        failed = true;
                        break;
                    }
                    const bool grow = mn > m + kRescaleLog2;
                    float alpha = 1.f;
                    if (grow) {
                        alpha = m == -CUDART_INF_F ? 0.f : ptx::ex2_approx(m - mn);
                        m = mn;
                        l *= alpha;
                    }
                    if (b > w.b0 && __any_sync(0xffffffffu, grow)) {
                        // O is complete up to the last block: page 1 of PV(x - 1) is done.  The wait cannot pass
                        // on the phase of PV(x - 2): the page 1 warps saw that one complete in block x - 1 and
                        // have since met this warp in the vote above.  (A page 0 warp has waited for page 0
                        // only, so on a barrier that no warp follows block by block it could be two phases
                        // behind, which a parity cannot tell.)
                        if (!warp_wait(kPbVEmpty + 1, (x - 1) & 1)) failed = true;
                        if (!failed) {
                            ptx::tc_fence_after();
#pragma unroll 1
                            for (int cc = 0; cc < 8; ++cc) {
                                uint32_t ov[16];
                                SMLA_TMEM_LD16(tmem + lane_base + ocol0 + cc * 16, ov);
                                ptx::tmem_wait_ld(ov);
#pragma unroll
                                for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                                SMLA_TMEM_ST16(tmem + lane_base + ocol0 + cc * 16, ov);
                            }
                            ptx::tmem_wait_st();
                            ptx::tc_fence_before();
                        }
                        // Page 0's MMAs add to all 512 dims, also to the lanes of the page 1 warps, but its
                        // barrier counts the page 0 warps only.  So the rows' four warps meet here: a store of
                        // any of them comes before this barrier, this before the page 0 warps' arrival on
                        // kPbPFull, that (both row groups', both CTAs') before the issuer's MMAs.  The branch
                        // is the same in the four: a row's max, and with it `grow`, is the same in its threads.
                        failed = ptx::named_bar_red_or(grp, 128u, failed);
                        if (failed) break;
                    }
                }
                // P = 2^(c s - m) as bf16, the operand of PV (its rounding averages out over the keys;
                // the sum takes the unrounded values).  A masked key holds -inf, which only a scale of 0
                // would not keep out.
                const float nm = m == -CUDART_INF_F ? 0.f : -m;
                float2 la[4];
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 4; ++i) la[i] = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 d = ptx::fma2(make_float2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])),
                                               make_float2(c, c), make_float2(nm, nm));
                    float2 pp = make_float2(ptx::ex2_approx(d.x), ptx::ex2_approx(d.y));
                    if (n < 32) {
                        if (2 * i >= n) pp.x = 0.f;
                        if (2 * i + 1 >= n) pp.y = 0.f;
                    }
                    la[i & 3] = ptx::add2(la[i & 3], pp);
                    pk[i] = ptx::cvt_bf16x2(pp.x, pp.y);
                }
                l += ((la[0].x + la[0].y) + (la[1].x + la[1].y)) + ((la[2].x + la[2].y) + (la[3].x + la[3].y));
                // P's panel of this page is one buffer: the page's MMAs of PV(x - 1) have read it
                if (x > 0 && !warp_wait(kPbVEmpty + half, (x - 1) & 1)) {
                    failed = true;
                    continue;  // the next reduction (or the one after the loop) takes the group out
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    ptx::st_shared_v4(p_row + ((static_cast<uint32_t>(4 * sub + q) ^ static_cast<uint32_t>(r & 7)) << 4),
                                      make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]));
                if (pf_tail(p, 2 * b + half)) {
                    // the page's rows past the prefix's end, zeroed in this CTA's V tile by the page's warps
                    if (!warp_wait(kPbTail, tails & 1)) {
                        failed = true;
                        continue;
                    }
                    ++tails;
                    const int first = static_cast<int>(p.prefix % kPfPage);
                    const int tid = (2 * sub + (quad & 1)) * 32 + lane;
                    const uint32_t vt = sbase + L::kOffV + half * kPfVPage;
                    for (int j = tid; j < (kPfPage - first) * 32; j += 128)
                        ptx::st_shared_v4(vt + (j & 3) * kPfPanel + (first + (j >> 5)) * 128 + ((j >> 2) & 7) * 16,
                                          make_uint4(0u, 0u, 0u, 0u));
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(p_full);
            }
            // ---- the piece's rows: O / l as bf16 and the natural-log LSE if the tile is whole, else
            // the unnormalised partial
            sX[part * kPfHalf + r] = l;
            failed = ptx::named_bar_red_or(grp, 128u, failed);
            // O is complete: page 1 of the last PV is done (after the barrier, for the reason given at the rescale)
            if (!failed && !warp_wait(kPbVEmpty + 1, (x - 1) & 1)) failed = true;
            ptx::tc_fence_after();
            const float lt = (sX[r] + sX[kPfHalf + r]) + (sX[2 * kPfHalf + r] + sX[3 * kPfHalf + r]);
            const int64_t row0 = w.tile * kPfRows + rank * kPfHalf + (quad & 1) * 32;  // the warp's first row
            const int live = p.rows - row0 < 32 ? static_cast<int>(p.rows - row0) : 32;  // rows of the warp, if any
            const bool whole = w.b0 == 0 && w.b1 == p.nblk;
            const int64_t pgroup = (2 * static_cast<int64_t>(run) + (w.first ? 0 : 1)) * p.slot_groups + 2 * rank + (quad & 1);
            const float inv = lt > 0.f || lt != lt ? 1.0f / lt : 0.f;
            if (!failed && lane < live && part == 0) {
                if (whole) {
                    p.lse[row0 + lane] = lt == 0.f ? -CUDART_INF_F : (m + log2f(lt)) * 0.69314718055994531f;
                } else {
                    p.part_ml[64 * pgroup + lane] = m;
                    p.part_ml[64 * pgroup + 32 + lane] = lt;
                }
            }
            // Out: 32 rows x 64 bytes at a time through this warp's eighth of P's buffer (free until the
            // next block's P): whole sectors, where a row per lane would touch 32 lines at once.  Partials
            // go as they are, each instruction 512 contiguous bytes.
            if (!failed && live > 0) {
                const uint32_t stage = sbase + L::kOffP + (warp - 2) * 32 * 64;
                float4* part = reinterpret_cast<float4*>(p.part_o) + (pgroup * 128 + 64 * half + 32 * sub) * 32 + lane;
#pragma unroll 1
                for (int cc = 0; cc < 2; ++cc) {  // 64 columns of O are read at a time
                    uint32_t ov[64];
#pragma unroll
                    for (int q = 0; q < 4; ++q) SMLA_TMEM_LD16(tmem + lane_base + ocol0 + cc * 64 + 16 * q, ov + 16 * q);
                    ptx::tmem_wait_ld(ov);
                    if (whole) {
                        __nv_bfloat16* dst = p.out + row0 * kDV + 256 * half + 128 * sub + 64 * cc + (lane & 3) * 8;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t v[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    v[j] = ptx::cvt_bf16x2(__uint_as_float(ov[32 * u + 8 * e + 2 * j]) * inv,
                                                           __uint_as_float(ov[32 * u + 8 * e + 2 * j + 1]) * inv);
                                ptx::st_shared_v4(stage + lane * 64 + ((static_cast<uint32_t>(e) ^ static_cast<uint32_t>((lane >> 1) & 3)) << 4),
                                                  make_uint4(v[0], v[1], v[2], v[3]));
                            }
                            __syncwarp();
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int rr = 8 * e + (lane >> 2);
                                const uint4 v = ptx::ld_shared_v4(stage + rr * 64 + ((static_cast<uint32_t>(lane & 3) ^ static_cast<uint32_t>((rr >> 1) & 3)) << 4));
                                if (rr < live) *reinterpret_cast<uint4*>(dst + rr * kDV + 32 * u) = v;
                            }
                            __syncwarp();
                        }
                    } else if (lane < live) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            part[(16 * cc + e) * 32] = make_float4(__uint_as_float(ov[4 * e]), __uint_as_float(ov[4 * e + 1]),
                                                                   __uint_as_float(ov[4 * e + 2]), __uint_as_float(ov[4 * e + 3]));
                    }
                }
            }
            ptx::tc_fence_before();  // before the next piece's first PV overwrites O
            // every warp's staging is read before the next P is written over it; and all leave together
            failed = ptx::named_bar_red_or(3u, 32u * kPfSoftmaxWarps, failed);
        }
    }
    // ---- both CTAs are done with each other's shared memory, barriers and TMEM
    ptx::tc_fence_before();
    __syncwarp();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, L::kTmemCols);
    }
}

// The prefix's fp8 rows as bf16 rows in prefix order (e4m3 -> fp32 x scale -> bf16, as in the forward),
// zeros for rows that take no part: 656 bytes in and 1152 out.  A warp takes four rows of a page, their
// loads in flight together.
__global__ void __launch_bounds__(kPfExpandThreads) sparse_mla_prefix_expand_kernel(const PfParams p) {
    constexpr int kRows = kPfExpandRows;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t i = ((static_cast<int64_t>(blockIdx.x) * kPfExpandThreads + threadIdx.x) >> 5) * kRows;
    if (i >= static_cast<int64_t>(p.npages) * kPfPage) return;
    const int pg = static_cast<int>(i / kPfPage), in_page = static_cast<int>(i % kPfPage);
    const int page = ptx::ld(p.pages + pg);
    const int valid = pf_valid(p, pg, page);
    const uint8_t* row0 = static_cast<const uint8_t*>(p.kv) + (static_cast<int64_t>(page) * kPfPage + in_page) * kFp8RowBytes;
    // lane l: codes [8l, 8l + 8) and [256 + 8l, 256 + 8l + 8), so that both stores are 512 contiguous bytes
    uint2 a[kRows], b[kRows];
    float sa[kRows], sb[kRows];
    uint32_t rope[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        a[u] = b[u] = make_uint2(0u, 0u);
        sa[u] = sb[u] = 0.f;
        rope[u] = 0u;
        if (in_page + u < valid) {
            const uint8_t* row = row0 + u * kFp8RowBytes;
            a[u] = ptx::ld(reinterpret_cast<const uint2*>(row) + lane);
            b[u] = ptx::ld(reinterpret_cast<const uint2*>(row) + 32 + lane);
            sa[u] = ptx::ld(reinterpret_cast<const float*>(row + 512) + (lane >> 4));
            sb[u] = ptx::ld(reinterpret_cast<const float*>(row + 520) + (lane >> 4));
            rope[u] = ptx::ld(reinterpret_cast<const uint32_t*>(row + 528) + lane);
        }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        uint4* dst = reinterpret_cast<uint4*>(p.expanded + (i + u) * kDQK);
        dst[lane] = make_uint4(ptx::e4m3x2_scaled_bf16x2(a[u].x & 0xFFFFu, sa[u]), ptx::e4m3x2_scaled_bf16x2(a[u].x >> 16, sa[u]),
                               ptx::e4m3x2_scaled_bf16x2(a[u].y & 0xFFFFu, sa[u]), ptx::e4m3x2_scaled_bf16x2(a[u].y >> 16, sa[u]));
        dst[32 + lane] = make_uint4(ptx::e4m3x2_scaled_bf16x2(b[u].x & 0xFFFFu, sb[u]), ptx::e4m3x2_scaled_bf16x2(b[u].x >> 16, sb[u]),
                                    ptx::e4m3x2_scaled_bf16x2(b[u].y & 0xFFFFu, sb[u]), ptx::e4m3x2_scaled_bf16x2(b[u].y >> 16, sb[u]));
        reinterpret_cast<uint32_t*>(dst + 64)[lane] = rope[u];
    }
}

// Joins the pieces of cut tiles by log-sum-exp weights.  A CTA takes 32 query rows (a lane each) and
// 64 / PARTS dims, four per warp; PARTS warps share the pieces of four dims, each every PARTS-th piece in
// order with the loads of a batch in flight together, and meet in shared memory in a fixed order.  Every
// load is a whole line, and what the pieces wrote is read once, from L2 as a rule.  PARTS is the largest
// of 4, 2 and 1 with which the grid is at most three CTAs per SM (two run at a time; held to 40 registers
// for three, 256 rows x 16384 keys took 23.7 us in all instead of 20.2): few tiles are cut into many
// pieces (one warp over all 38 pieces of 256 rows took 20 us, a round of latency per eight pieces, twice;
// four take 5), many tiles into few.
template <int PARTS>
struct PfJoin {
    static constexpr int kChunks = kPfMergeThreads / 32 / PARTS;  // of four dims
    static constexpr int kDims = 4 * kChunks;                     // per CTA
};

// One CTA's share of a cut tile: rows 32 group .. (`live` of them, from out / lse on), dims kDims dg .. .  Piece
// k0 lies in slot first_slot, piece k of k0 + 1 .. k1 in slot 2 k.
template <int PARTS>
__device__ __forceinline__ void pf_join(const float* slots_o, const float* slots_ml, int slot_groups, int group, int dg, int k0, int k1,
                                        int first_slot, int live, __nv_bfloat16* out, float* lse) {
    constexpr int kChunks = PfJoin<PARTS>::kChunks;
    constexpr int kDims = PfJoin<PARTS>::kDims;
    constexpr int kFlight = 4;
    __shared__ float4 s_acc[PARTS][kChunks][32];
    __shared__ float s_m[PARTS][32], s_l[PARTS][32];
    __shared__ uint2 s_out[32][kChunks + 1];
    const int lane = threadIdx.x & 31;
    const int chunk = (threadIdx.x >> 5) % kChunks, part = (threadIdx.x >> 5) / kChunks;
    auto group_of = [&](int k) -> int64_t {
        return static_cast<int64_t>(k == k0 ? first_slot : 2 * k) * slot_groups + group;
    };
    const int at = lane < live ? lane : live - 1;  // a lane past the last row repeats it and stores nothing
    const float4* part_o = reinterpret_cast<const float4*>(slots_o) + (dg * kChunks + chunk) * 32 + at;
    float m = -CUDART_INF_F, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int kk = k0 + part; kk <= k1; kk += PARTS * kFlight) {
        float4 v[kFlight];
        float mk[kFlight], lk[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int64_t g = group_of(min(kk + PARTS * u, k1));
            mk[u] = ptx::ld(slots_ml + 64 * g + at);
            lk[u] = ptx::ld(slots_ml + 64 * g + 32 + at);
            v[u] = ptx::ld(part_o + g * (128 * 32));
        }
        float mn = m;
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (kk + PARTS * u > k1) {
                mk[u] = -CUDART_INF_F;
                lk[u] = 0.f;
                v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            mn = fmaxf(mn, mk[u]);
        }
        // a piece without a key has the sum 0 and zero rows: P was 0 and V had no NaN (one whose logits are all NaN has no max
        // either, and its NaN stays: 0 times it)
        const float keep = m == -CUDART_INF_F ? 0.f : ptx::ex2_approx(m - mn);
        m = mn;
        l *= keep;
        acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const float wt = mk[u] == -CUDART_INF_F ? 0.f : ptx::ex2_approx(mk[u] - m);
            l += wt * lk[u];
            acc.x += wt * v[u].x;
            acc.y += wt * v[u].y;
            acc.z += wt * v[u].z;
            acc.w += wt * v[u].w;
        }
    }
    if constexpr (PARTS > 1) {
        s_acc[part][chunk][lane] = acc;
        if (chunk == 0) {
            s_m[part][lane] = m;
            s_l[part][lane] = l;
        }
        __syncthreads();
        m = -CUDART_INF_F;
#pragma unroll
        for (int q = 0; q < PARTS; ++q) m = fmaxf(m, s_m[q][lane]);
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (part == 0) {
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                const float wt = s_m[q][lane] == -CUDART_INF_F ? 0.f : ptx::ex2_approx(s_m[q][lane] - m);
                const float4 o = s_acc[q][chunk][lane];
                l += wt * s_l[q][lane];
                acc.x += wt * o.x;
                acc.y += wt * o.y;
                acc.z += wt * o.z;
                acc.w += wt * o.w;
            }
        }
    }
    if (part == 0) {
        const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
        s_out[lane][chunk] = make_uint2(ptx::cvt_bf16x2(acc.x * inv, acc.y * inv), ptx::cvt_bf16x2(acc.z * inv, acc.w * inv));
        if (dg == 0 && chunk == 0 && lane < live)
            lse[lane] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
    }
    __syncthreads();
    const int r = threadIdx.x / kChunks, c = threadIdx.x % kChunks;  // neighbouring threads store a row's bytes
    if (r < live) reinterpret_cast<uint2*>(out + static_cast<int64_t>(r) * kDV + dg * kDims)[c] = s_out[r][c];
}

template <int PARTS>
__global__ void __launch_bounds__(kPfMergeThreads) sparse_mla_prefix_merge_kernel(const PfParams p) {
    constexpr int kDims = PfJoin<PARTS>::kDims;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int dg = static_cast<int>(blockIdx.x % (kDV / kDims));
    const int group = static_cast<int>(blockIdx.x / (kDV / kDims)) % p.slot_groups;
    // the tile: with more tiles than runs most are whole, and the candidates are those that the runs'
    // boundaries fall into (the first boundary of a tile stands for it)
    int64_t tile = blockIdx.x / (kDV / kDims) / p.slot_groups;
    if (p.tiles > p.runs) {
        const int64_t k = tile + 1;
        const int64_t at = p.work * k / p.runs;
        tile = at / p.nblk;
        if (at % p.nblk == 0 || p.work * (k - 1) / p.runs > tile * p.nblk) return;
    }
    const int64_t row0 = tile * kPfRows + group * 32;
    if (row0 >= p.rows) return;
    auto run_of = [&](int64_t b) -> int { return static_cast<int>(((b + 1) * p.runs - 1) / p.work); };
    const int k0 = run_of(tile * p.nblk), k1 = run_of((tile + 1) * p.nblk - 1);
    if (k0 == k1) return;  // the tile lies inside one run, which wrote it
    // this tile is the first piece of every run that starts inside it; the run that it begins in
    // keeps it in its second slot, unless that run starts with it
    const int first_slot = 2 * k0 + (p.work * k0 / p.runs == tile * p.nblk ? 0 : 1);
    const int live = p.rows - row0 < 32 ? static_cast<int>(p.rows - row0) : 32;
    pf_join<PARTS>(p.part_o, p.part_ml, p.slot_groups, group, dg, k0, k1, first_slot, live, p.out + row0 * kDV, p.lse + row0);
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
