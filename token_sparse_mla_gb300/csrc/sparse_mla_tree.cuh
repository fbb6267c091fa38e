// Attention of every sequence's drafted tokens over that sequence's cached rows and the drafted tokens they
// descend from, on tcgen05 tensor cores (sm_103a).
//
//   s = scale q.k   over the keys p < len (all of them) and len + j (where bit j of the token's mask is set)
//   O = softmax(s) . k[0:512],   LSE = ln sum exp(s)
//
// The tile is the prefix kernel's (sparse_mla_prefix.cuh): a CTA pair holds 128 rows (token, head) of one
// sequence as one cta_group::2 MMA, 512 fp32 columns of O over the pair's TMEM, blocks of 128 keys through
// one stage of K and V, S in two accumulators from two issuing threads, PV by a third, eight softmax warps.
// What differs:
//
// Bound.  A decode batch has few rows per sequence and every sequence its own rows in the cache: at up to
// 128 rows a block is 147 KB from HBM for one tile.  76 pairs at the tile's pace of 1.65 us a block
// take 6.8 TB/s, HBM's rate: rows short of 128 cost no traffic that a smaller tile would save.  (What one could save is
// shared memory, for a second stage of K and V, which fp8 rows lack most; not built.)
//
// Work.  How many rows and keys there are is known on the device only.  Every CTA sums the cost of all
// sequences' tiles (blocks, and kTrTileCost for a tile's queries, first block and epilogue) and takes its
// pair's equal share of the sequence of blocks.  A tile that lies inside one run is written out; a cut one
// leaves an fp32 partial per piece, and the run that begins it leaves a note of where they are for the
// join, so that the join needs to know nothing of the plan.
//
// Masks.  A block that reaches past the cached rows takes each row's 32 bits of the tree.  A drafted row
// that a token does not see has probability 0 there, but 0 times infinity or NaN would still spoil O: in
// pages that reach past the cached rows the V tile is cleaned in shared memory before it is multiplied (rows
// past the end zeroed, values that are not finite in the drafted rows zeroed: a token that does see such a
// row has its NaN from S, but for a logit of -infinity, which counts for nothing).
//
// fp8.  Shared memory has no room for a block's codes, so eight more warps take them through registers, eight rows of
// each page a warp, the next block's in flight as soon as this one's are written: its own page into K, as the MMA
// wants it, and its dims of both pages into V, once the last block's V has been multiplied (those of its own
// page are copied from K).  So half of the codes are converted in both CTAs.  (Expanded into a ring in global
// memory and loaded from there, a block took 5.0 us: 11 TB/s of traffic through L2.  The other CTA's half of V
// from its K: by bulk copies 3000 to 4700 cycles for 32 KB, by stores into its shared memory 2000, and 3000
// more until a fence and a release had waited for them.  Four warps for K and four for V: 4.1 us; so 3.4, and 3.6
// from HBM: what bounds it is how fast the expansion warps issue, 1900 cycles for K, 1600 for V and 1100 for the copy of 6600
// a block, in part beside S, which has shared memory to itself.  V's own part kept in registers instead of copied
// from K was no faster.)
//
// Roles (384 threads, 640 with fp8):
//   warps 0-7    softmax, rescaling and output: TMEM quadrant warp % 4, keys 32 (warp / 4) .. of a page
//   warp 8       TMA producer (one thread)
//   warp 9       S issuer for dims 0 .. 319, and TMEM owner
//   warp 10      PV issuer, warp 11 S issuer for dims 320 .. 575 (one thread of the even CTA each)
//   warps 12-19  expansion of fp8 rows
// Every wait is bounded; a CTA that gives up meets the other at the final cluster barrier.
#pragma once

#include "sparse_mla_batch.cuh"
#include "sparse_mla_prefix.cuh"

namespace smla {

constexpr int kTrSoftmaxWarps = 8;
constexpr int kTrTmaWarp = 8, kTrS1Warp = 9, kTrPvWarp = 10, kTrS2Warp = 11, kTrExpandWarp = 12;
constexpr int kTrExpandWarps = 8;
constexpr int kTrExpandRows = kPage / kTrExpandWarps;
constexpr int kTrTileCost = 3;   // what a piece costs beside its blocks, in blocks

template <int KVF>
__host__ __device__ constexpr int tree_threads() {
    return 32 * (kTrExpandWarp + (KVF ? kTrExpandWarps : 0));
}

// Registers per thread with fp8: 640 threads are launched with 96 each, and the warpgroups that issue and expand give some
// of theirs to the two of the softmax.  (More than the launch's total in all would wait forever.)
constexpr int kTrRegsLaunch = 96, kTrRegsSoftmax = 112, kTrRegsIssue = 80, kTrRegsExpand = 88;
static_assert(tree_threads<1>() * kTrRegsLaunch <= 65536, "registers of a block");
static_assert(32 * (kTrSoftmaxWarps * kTrRegsSoftmax + 4 * kTrRegsIssue + kTrExpandWarps * kTrRegsExpand) <= tree_threads<1>() * kTrRegsLaunch,
              "shares of the block's registers");

// Barriers of the prefix kernel, then:
enum : int {
    kTbTail = kPbTail,           // +page of the block, own CTA: V of a page that has to be cleaned; fp8: of every page
    kTbDrain = kTbTail + 2,      // even CTA
    kTbMade = kTbDrain + 1,      // fp8, even CTA: both CTAs' K is expanded, and its rotated dims landed
    kTbCount = kTbMade + 1
};

struct TrLayout {
    static constexpr int kOffQ = PfLayout::kOffQ, kOffK = PfLayout::kOffK, kOffV = PfLayout::kOffV, kOffP = PfLayout::kOffP;
    static constexpr int kOffX = PfLayout::kOffX;  // values swapped by a row's four threads; sums of the plan at the start
    static constexpr int kOffBar = PfLayout::kOffBar;
    static constexpr int kOffMisc = kOffBar + kTbCount * 8;  // tmem base, abort flag, the run's start
    static constexpr int kBytes = kOffMisc + 64;
    static_assert(kBytes <= 232448, "shared memory budget (227 KB)");
};

// Where a run begins: sequence, tile and its index over all sequences, the tile's first cost unit, the
// units of the run.
struct TrStart {
    int64_t at, end, tile_at;  // [at, end) of the run; where the tile begins
    int64_t total;
    int32_t b, tile, tile_index, tiles;  // tiles: of all sequences
};

struct TrParams {
    BatchParams bp;
    __nv_bfloat16* out;          // [T, h, 512]
    float* lse;                  // [T, h]
    float* part_o;               // partials as in the prefix kernel, two slots per pair
    float* part_ml;
    int4* job_list;              // [jobs]: first row, rows, first slot, last run of a cut tile; rows 0: none
    int32_t pairs, jobs, by_tile, slot_groups;  // by_tile: job i is tile i's, else the one that run i begins
    float sm_scale_log2;
};

__device__ __forceinline__ int tree_tiles(const TrParams& p, const Seq& s) {
    return static_cast<int>((static_cast<int64_t>(s.n) * p.bp.h + kPfRows - 1) / kPfRows);
}
__device__ __forceinline__ int tree_blocks(const Seq& s) { return (s.keys + kPfKeys - 1) / kPfKeys; }

// All threads of the CTA: the start of pair `run`'s share, into *start (shared memory).
__device__ __forceinline__ void tree_plan(const TrParams& p, int run, int threads, int64_t* scratch, TrStart* start) {
    const int per = (p.bp.B + threads - 1) / threads;
    const int b0 = min(ptx::behind(static_cast<int>(threadIdx.x)) * per, p.bp.B), b1 = min(b0 + per, p.bp.B);
    int64_t cost = 0, tiles = 0;
    for (int b = b0; b < b1; ++b) {
        const Seq s = load_seq(p.bp, b);
        const int t = tree_tiles(p, s);
        tiles += t;
        cost += static_cast<int64_t>(t) * (tree_blocks(s) + kTrTileCost);
    }
    int64_t at, total, first_tile, all_tiles;
    block_prefix2(cost, tiles, scratch, threads / 32, at, total, first_tile, all_tiles);
    const int runs = static_cast<int>(min(total, static_cast<int64_t>(p.pairs)));
    const int64_t from = run < runs ? share_of(total, run, runs) : total, to = run < runs ? share_of(total, run + 1, runs) : total;
    if (from >= total) {
        if (threadIdx.x == 0) *start = TrStart{total, total, total, total, p.bp.B, 0, 0, static_cast<int32_t>(all_tiles)};
    } else if (at <= from && from < at + cost) {
        int b = b0;
        for (;; ++b) {
            const Seq s = load_seq(p.bp, b);
            const int t = tree_tiles(p, s);
            const int64_t c = tree_blocks(s) + kTrTileCost;
            if (from < at + t * c) {
                const int64_t i = from - at < (1 << 30) ? static_cast<int32_t>(from - at) / static_cast<int32_t>(c) : (from - at) / c;
                *start = TrStart{from, to, at + i * c, total, b, static_cast<int32_t>(i), static_cast<int32_t>(first_tile + i),
                                 static_cast<int32_t>(all_tiles)};
                break;
            }
            at += t * c;
            first_tile += t;
        }
    }
    __syncthreads();
}

// The pieces of a run, the same for every role: blocks [b0, b1) of a tile of sequence b.
struct TrWalk {
    int64_t at, end;  // of the tile's cost units, relative to the tile's first
    Seq s;
    int b, tile, tiles, tile_index, nblk;
    int b0, b1;
    bool first;
    __device__ __forceinline__ TrWalk(const TrParams& p, const TrStart& st) : b(st.b), tile(st.tile), tile_index(st.tile_index), first(true) {
        at = st.at - st.tile_at;
        end = st.end - st.tile_at;
        b0 = b1 = -1;
        if (b < p.bp.B) {
            s = load_seq(p.bp, b);
            tiles = tree_tiles(p, s);
            nblk = tree_blocks(s);
        }
    }
    __device__ __forceinline__ bool next(const TrParams& p) {
        if (b1 >= 0) {
            end -= nblk + kTrTileCost;
            at = 0;
            ++tile;
            ++tile_index;
            first = false;
        }
        if (at >= end) return false;
        if (b1 >= 0 && tile == tiles) {
            tile = 0;
            do {
                if (++b >= p.bp.B) return false;
                s = load_seq(p.bp, b);
                tiles = tree_tiles(p, s);
            } while (tiles == 0);
            nblk = tree_blocks(s);
        }
        b0 = static_cast<int>(max(at - kTrTileCost, static_cast<int64_t>(0)));
        b1 = static_cast<int>(min(end - kTrTileCost, static_cast<int64_t>(nblk)));
        return b1 > b0;  // a run that ends before the tile's first block leaves it to the next one
    }
    __device__ __forceinline__ bool whole() const { return b0 == 0 && b1 == nblk; }
    __device__ __forceinline__ int64_t row0() const { return static_cast<int64_t>(tile) * kPfRows; }  // within the sequence
};

// Whether page i holds positions that V has to be cleaned of: drafted rows, or the end.
__device__ __forceinline__ bool tree_tail(const Seq& s, int i) { return (i + 1) * kPage > s.len && i * kPage < s.keys; }

// An expansion warp's eight rows of an fp8 page, kParts * 256 codes of each, on their way to shared memory: lane l has codes
// [8l, 8l + 8) of every part, and of row l % 8 the scales of codes [128 (l / 16), ..) of every part.  (The rotated
// dims come by TMA.)
template <int kParts>
struct TrCodes {
    uint2 a[kParts][kTrExpandRows];
    float sc[kParts];
    // rows from `row` on of page i, codes from `first` (of the row's 512) on
    __device__ __forceinline__ void load(const BatchParams& p, const Seq& s, int i, int page, int row, int first) {
        const int lane = threadIdx.x & 31;
        const int n = page_rows(p, s, i, page) - row;
        const uint8_t* src = static_cast<const uint8_t*>(p.kv) + (static_cast<int64_t>(page) * kPage + row) * kFp8RowBytes;
        const float* scales = reinterpret_cast<const float*>(src + lane % kTrExpandRows * kFp8RowBytes + 512) + first / 128 + (lane >> 4);
        src += first + 8 * lane;
        if (n >= kTrExpandRows) {
#pragma unroll
            for (int e = 0; e < kParts; ++e) {
#pragma unroll
                for (int u = 0; u < kTrExpandRows; ++u) a[e][u] = ptx::ld_l1_v2(src + u * kFp8RowBytes + 256 * e);
                sc[e] = ptx::ld_f32(scales + 2 * e);
            }
        } else {  // rows that take no part become zeros
#pragma unroll
            for (int e = 0; e < kParts; ++e) {
#pragma unroll
                for (int u = 0; u < kTrExpandRows; ++u) {
                    a[e][u] = make_uint2(0u, 0u);
                    if (u < n) a[e][u] = ptx::ld_l1_v2(src + u * kFp8RowBytes + 256 * e);
                }
                sc[e] = lane % kTrExpandRows < n ? ptx::ld_f32(scales + 2 * e) : 0.f;
            }
        }
    }
    // All rows, to those of a tile from `to` on, four panels a part: codes x scale in fp32 rounded to bf16 as in the
    // forward; chunk c of a panel's row r lies at 16 (c ^ r % 8), so each store is conflict-free.  A loop over groups of
    // four that moves the registers along: straight-line code for all rows is fetched more slowly than it runs.
    __device__ __forceinline__ void store(uint32_t to) {
        const int lane = threadIdx.x & 31;
        const uint32_t at0 = to + (lane >> 3) * kPfPanel;
#pragma unroll 1
        for (int u0 = 0; u0 < kTrExpandRows; u0 += 4) {
#pragma unroll
            for (int e = 0; e < kParts; ++e) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float s = __shfl_sync(0xffffffffu, sc[e], (lane & 16) + u0 + u);
                    const uint2 x = a[e][u];
                    const uint2 lo = ptx::e4m3x4_scaled_bf16x4(x.x, make_float2(s, s)), hi = ptx::e4m3x4_scaled_bf16x4(x.y, make_float2(s, s));
                    ptx::st_shared_v4(at0 + 4 * e * kPfPanel + (u0 + u) * 128 + (((lane & 7) ^ ((u0 & 4) + u)) << 4),
                                      make_uint4(lo.x, lo.y, hi.x, hi.y));
                }
#pragma unroll
                for (int u = 0; u < kTrExpandRows - 4; ++u) a[e][u] = a[e][u + 4];
            }
        }
    }
};

template <int KVF>
__global__ void __launch_bounds__(tree_threads<KVF>(), 1)
    sparse_mla_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const TrParams p) {
    using L = TrLayout;
    constexpr int kThreads = tree_threads<KVF>();
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
    TrStart* start = reinterpret_cast<TrStart*>(smem + L::kOffMisc + 8);
    auto bar = [&](int i) -> uint32_t { return sbase + L::kOffBar + 8u * static_cast<uint32_t>(i); };
    auto even_bar = [&](int i) -> uint32_t { return ptx::map_shared_rank(bar(i), 0); };
    auto wait = [&](int i, uint32_t parity) -> bool {
        return ptx::mbar_wait(bar(i), parity, sAbort, &g_smla_error, kErrTimeout, kWaitLimitNs);
    };

    if (threadIdx.x == 0) {
        *sAbort = 0;
        for (int i = 0; i < kTbCount; ++i) {
            const bool by_warps = i == kPbSEmpty || i == kPbSEmpty + 1;                // both CTAs' softmax warps
            const bool by_half = i == kPbPFull || i == kPbPFull + 1;                   // those of the page
            const bool by_two = i == kPbQEmpty || i == kPbSFull || i == kPbSFull + 1;  // both S issuers
            const bool by_page = KVF == 1 && (i == kTbTail || i == kTbTail + 1);       // the expansion warps of the page's CTA
            ptx::mbar_init(bar(i), by_warps ? 2 * kTrSoftmaxWarps : by_half ? kTrSoftmaxWarps : i == kTbMade ? 2 * kTrExpandWarps + 1
                                   : by_page ? kTrExpandWarps : i == kTbDrain ? 3 : by_two ? 2 : 1);
        }
        ptx::fence_mbarrier_init();
    }
    if (warp == kTrS1Warp) {
        ptx::tmem_alloc_pair(sbase + L::kOffMisc, PfLayout::kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    if (warp == kTrTmaWarp && lane == 0) {
        ptx::prefetch_tmap(&tm_q);
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
    }
    ptx::tc_fence_before();
    __syncwarp();           // the cluster barrier wants its warps whole
    ptx::cluster_arrive();  // both CTAs' barriers are initialised before anyone signals them
    // launched as a programmatic dependent: nothing above touched global memory
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    tree_plan(p, run, kThreads, reinterpret_cast<int64_t*>(smem + L::kOffX), start);
    __syncwarp();
    ptx::cluster_wait();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc);

    if (warp >= kTrSoftmaxWarps && warp < kTrExpandWarp) {
        if constexpr (KVF == 1) ptx::regs_down<kTrRegsIssue>();
        if (warp == kTrTmaWarp) {
            // ================================================================ TMA producer
            TrWalk w(p, *start);
            const bool any = w.next(p);
            // As in the prefix kernel: the even CTA's thread expects both CTAs' bytes on its barrier, K runs a
            // block ahead of V, pages are brought into L2 a block ahead.
            if (p.by_tile && run == 0 && rank == 0)
                for (int i = start->tiles + lane; i < p.jobs; i += 32) p.job_list[i] = make_int4(0, 0, 0, 0);
            if (lane == 0) {
                int4 job = make_int4(0, 0, 0, 0);
                auto load_v = [&](int x, bool tail0, bool tail1, int row0, int row1) -> bool {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (x > 0 && !wait(kPbVEmpty + i, (x - 1) & 1)) return false;
                        const uint32_t dst = sbase + L::kOffV + i * kPfVPage;
                        if (i ? tail1 : tail0) {  // the softmax warps wait for this one themselves and clean it
                            ptx::mbar_arrive_expect_tx(bar(kTbTail + i), static_cast<uint32_t>(kPfVPage));
                            ptx::tma_load_3d(dst, &tm_v, 0, i ? row1 : row0, 4 * rank, bar(kTbTail + i));
                        } else {
                            if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kPbVFull + i), 2u * kPfVPage);
                            ptx::tma_load_3d_pair(dst, &tm_v, 0, i ? row1 : row0, 4 * rank, even_bar(kPbVFull + i));
                        }
                    }
                    return true;
                };
                // a page that is not there loads as zeros, from rows below 0
                auto first_row = [&](int page) -> int { return page_in_cache(p.bp, page) ? page * kPage : -kPage; };
                auto prefetch = [&](int i) {
                    if (i >= 2 * w.b1) return;
                    const int pg = page_of(p.bp, w.b, w.s, i);
                    const int n = page_rows(p.bp, w.s, i, pg);
                    if (n > 0)
                        ptx::bulk_prefetch_l2(static_cast<const char*>(p.bp.kv) + static_cast<int64_t>(pg) * kPage * (KVF ? kFp8RowBytes : kDQK * 2),
                                              static_cast<uint32_t>(n * (KVF ? kFp8RowBytes : kDQK * 2)));
                };
                bool ok = true;
                int x = 0, piece = 0;
                bool tail_v0 = false, tail_v1 = false;
                int row_v0 = 0, row_v1 = 0;
                for (bool more = any; ok && more; more = w.next(p), ++piece) {
                    if (rank == 0 && w.b0 == 0) {
                        const int64_t runs = min(start->total, static_cast<int64_t>(p.pairs));
                        const int64_t tile_end = start->end - w.end + w.nblk + kTrTileCost;
                        if (!w.whole()) {
                            const int64_t rows = static_cast<int64_t>(w.s.n) * p.bp.h - w.row0();
                            job = make_int4(static_cast<int>(static_cast<int64_t>(w.s.first) * p.bp.h + w.row0()),
                                            static_cast<int>(min(rows, static_cast<int64_t>(kPfRows))), 2 * run + (w.first ? 0 : 1),
                                            static_cast<int>((tile_end * runs - 1) / start->total));
                        }
                        if (p.by_tile && w.tile_index < p.jobs) p.job_list[w.tile_index] = w.whole() ? make_int4(0, 0, 0, 0) : job;
                    }
                    if (piece > 0 && !(ok = wait(kPbQEmpty, (piece - 1) & 1))) break;
                    if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kPbQFull), 2u * kPfQBytes);
                    ptx::tma_load_3d_pair(sbase + L::kOffQ, &tm_q, 0,
                                          static_cast<int>(static_cast<int64_t>(w.s.first) * p.bp.h + w.row0() + rank * kPfHalf), 0,
                                          even_bar(kPbQFull));
                    if constexpr (KVF == 1) {
                        for (int b = w.b0; ok && b < w.b1; ++b, ++x) {
                            if (b == w.b0) prefetch(2 * b + 2 + rank);
                            prefetch(2 * b + 4 + rank);
                            if (x > 0 && !(ok = wait(kPbKEmpty + 1, (x - 1) & 1))) break;
                            if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kTbMade), 2u * kPfPanel);
                            ptx::tma_load_2d_pair(sbase + L::kOffK + 8 * kPfPanel, &tm_k, 528, first_row(page_of(p.bp, w.b, w.s, 2 * b + rank)),
                                                  even_bar(kTbMade));
                        }
                        continue;
                    }
                    int pg0 = page_of(p.bp, w.b, w.s, 2 * w.b0), pg1 = page_of(p.bp, w.b, w.s, 2 * w.b0 + 1);
                    for (int b = w.b0; ok && b < w.b1; ++b, ++x) {
                        const int row0 = first_row(pg0), row1 = first_row(pg1);
                        const int mine = rank == 0 ? row0 : row1;
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            if (x > 0 && !(ok = wait(kPbKEmpty + g, (x - 1) & 1))) break;
                            const uint32_t bytes = static_cast<uint32_t>((g ? kPfGroupB : kPfGroupA) * kPfPanel);
                            if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kPbKFull + g), 2u * bytes);
                            ptx::tma_load_3d_pair(sbase + L::kOffK + g * kPfGroupA * kPfPanel, g ? &tm_v : &tm_k, 0, mine,
                                                  g * kPfGroupA, even_bar(kPbKFull + g));
                        }
                        prefetch(2 * b + 2 + rank);
                        pg0 = page_of(p.bp, w.b, w.s, 2 * b + 2);
                        pg1 = page_of(p.bp, w.b, w.s, 2 * b + 3);
                        if (ok && x > 0) ok = load_v(x - 1, tail_v0, tail_v1, row_v0, row_v1);
                        row_v0 = row0;
                        row_v1 = row1;
                        tail_v0 = tree_tail(w.s, 2 * b);
                        tail_v1 = tree_tail(w.s, 2 * b + 1);
                    }
                }
                if (KVF == 0 && ok && x > 0) ok = load_v(x - 1, tail_v0, tail_v1, row_v0, row_v1);
                if (rank == 0 && !p.by_tile) p.job_list[run] = job;
                // every copy has landed and been used, and no release of a stage is still on its way to
                // this CTA's barriers, before it leaves
                if (x > 0) {
                    for (int g = 0; ok && g < 2; ++g) ok = wait(kPbKEmpty + g, (x - 1) & 1);
                    // (with fp8 the softmax warps see the last of these; this thread has not followed them)
                    for (int i = 0; KVF == 0 && ok && i < 2; ++i) ok = wait(kPbVEmpty + i, (x - 1) & 1);
                    if (ok) ok = wait(kPbQEmpty, (piece - 1) & 1);
                }
                if (!ok) {  // gave up: copies in flight complete on the other CTA's barriers; leave them time to land
                    const uint64_t t0 = ptx::globaltimer_ns();
                    while (ptx::globaltimer_ns() - t0 < 2000000ull) {
                    }
                }
            }
            __syncwarp();
        } else if (warp == kTrS1Warp || warp == kTrS2Warp) {
            // ================================================================ S issuers, as in the prefix kernel
            TrWalk w(p, *start);
            const bool any = w.next(p);
            if (rank == 0 && lane == 0) {
                constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(kPfRows, kPfKeys, 0, 0);
                const bool ga = warp == kTrS1Warp;
                const uint32_t off = ga ? 0u : static_cast<uint32_t>(kPfGroupA * kPfPanel);
                const uint64_t dq = ptx::smem_desc_sw128(sbase + L::kOffQ + off, 16, 1024);
                const uint64_t dk = ptx::smem_desc_sw128(sbase + L::kOffK + off, 16, 1024);
                const uint32_t d0 = tmem + PfLayout::kColS + (ga ? 0 : kPfPage);
                const int g = ga ? 0 : 1;
                bool ok = true;
                int x = 0, piece = 0;
                for (bool more = any; ok && more; more = w.next(p), ++piece) {
                    if (!(ok = wait(kPbQFull, piece & 1))) break;
                    for (int b = w.b0; ok && b < w.b1; ++b, ++x) {
                        const int s = x & 1;
                        if (x >= 2 && !(ok = wait(kPbSEmpty + s, ((x >> 1) - 1) & 1))) break;
                        if (!(ok = wait(KVF == 1 ? kTbMade : kPbKFull + g, x & 1))) break;
                        ptx::tc_fence_after();
                        const uint32_t d = d0 + s * PfLayout::kSBuf;
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
                ptx::mma_commit_pair_local(bar(kTbDrain));
                ptx::mbar_wait(bar(kTbDrain), 0, nullptr, &g_smla_error, 0u, kDrainLimitNs);
            }
            __syncwarp();
        } else {
            // ================================================================ PV issuer
            TrWalk w(p, *start);
            const bool any = w.next(p);
            if (rank == 0 && lane == 0) {
                constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kPfRows, 256, 0, 1);
                const uint64_t dv = ptx::smem_desc_sw128(sbase + L::kOffV, kPfPanel, 1024);
                const uint64_t dp = ptx::smem_desc_sw128(sbase + L::kOffP, 16, 1024);
                uint32_t v_parity = 0u;  // bit i: parity of the loads that came to V page i (tails have their own barriers)
                bool ok = true;
                int x = 0;
                for (bool more = any; ok && more; more = w.next(p)) {
                    for (int b = w.b0; ok && b < w.b1; ++b, ++x) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (!(ok = wait(kPbPFull + i, x & 1))) break;
                            if (KVF == 0 && !tree_tail(w.s, 2 * b + i)) {
                                if (!(ok = wait(kPbVFull + i, (v_parity >> i) & 1u))) break;
                                v_parity ^= 1u << i;
                            }
                            ptx::tc_fence_after();
#pragma unroll
                            for (int k = 0; k < 4; ++k)
#pragma unroll
                                for (int n = 0; n < 2; ++n)
                                    ptx::mma_bf16_ss_pair(tmem + PfLayout::kColO + 128 * n, dp + ((i * kPfPanel + k * 32) >> 4),
                                                          dv + ((i * kPfVPage + 2 * n * kPfPanel + k * 2048) >> 4), kIdescPV,
                                                          (b != w.b0 || i > 0 || k > 0) ? 1u : 0u);
                            ptx::mma_commit_pair(bar(kPbVEmpty + i));
                        }
                    }
                }
                // nothing is in flight when TMEM is freed, also after giving up
                ptx::mma_commit_pair_local(bar(kTbDrain));
                ptx::mbar_wait(bar(kTbDrain), 0, nullptr, &g_smla_error, 0u, kDrainLimitNs);
            }
            __syncwarp();
        }
    } else if (warp >= kTrExpandWarp) {
        // ================================================================ expansion of fp8 rows
        if constexpr (KVF == 1) {
            ptx::regs_down<kTrRegsExpand>();
            TrWalk w(p, *start);
            const bool any = w.next(p);
            const int row = kTrExpandRows * (warp - kTrExpandWarp);
            auto warp_wait = [&](int i, uint32_t parity) -> bool {
                return ptx::mbar_wait_warp(bar(i), parity, sAbort, &g_smla_error, kErrTimeout, kWaitLimitNs);
            };
            bool ok = true;
            int x = 0;
            for (bool more = any; ok && more; more = w.next(p)) {
                auto page = [&](int b, int i) -> int { return b < w.b1 ? page_of(p.bp, w.b, w.s, 2 * b + i) : -1; };
                TrCodes<2> own;    // this CTA's page, all codes: K
                TrCodes<1> other;  // the other CTA's, those of this CTA's dims: V
                auto load_own = [&](int b, int pg) { own.load(p.bp, w.s, 2 * b + rank, pg, row, 0); };
                auto load_other = [&](int b, int pg) { other.load(p.bp, w.s, 2 * b + (rank ^ 1), pg, row, 256 * rank); };
                load_own(w.b0, page(w.b0, rank));
                load_other(w.b0, page(w.b0, rank ^ 1));
                int pg_own = page(w.b0 + 1, rank), pg_other = page(w.b0 + 1, rank ^ 1);
                for (int b = w.b0; b < w.b1; ++b, ++x) {
                    // the last block's S has read the K tile
                    if (x > 0 && !(ok = warp_wait(kPbKEmpty, (x - 1) & 1) && warp_wait(kPbKEmpty + 1, (x - 1) & 1))) break;
                    own.store(sbase + L::kOffK + row * 128);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster(even_bar(kTbMade));
                    // A fence waits for the loads before it, too: the next block's come right behind one (4.05 us a block from HBM
                    // with all of them behind the last fence, 3.85 so, 5.3 with all of them before it)
                    load_own(b + 1, pg_own);
                    pg_own = page(b + 2, rank);
                    // the last block's V has been multiplied: this CTA's dims of its own page are in the K tile, panels
                    // 4 rank .. 4 rank + 3
                    if (x > 0 && !(ok = warp_wait(kPbVEmpty + rank, (x - 1) & 1))) break;
                    {
                        const uint32_t from = sbase + L::kOffK + 4 * rank * kPfPanel + row * 128 + lane * 16;
                        const uint32_t into = sbase + L::kOffV + rank * kPfVPage + row * 128 + lane * 16;
#pragma unroll 1
                        for (int j = 0; j < 4; j += 2) {
                            uint4 v[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) v[u] = ptx::ld_shared_v4(from + (j + (u >> 1)) * kPfPanel + (u & 1) * 512);
#pragma unroll
                            for (int u = 0; u < 4; ++u) ptx::st_shared_v4(into + (j + (u >> 1)) * kPfPanel + (u & 1) * 512, v[u]);
                        }
                    }
                    if (x > 0 && !(ok = warp_wait(kPbVEmpty + (rank ^ 1), (x - 1) & 1))) break;
                    other.store(sbase + L::kOffV + (rank ^ 1) * kPfVPage + row * 128);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane < 2) ptx::mbar_arrive(bar(kTbTail + lane));
                    load_other(b + 1, pg_other);
                    pg_other = page(b + 2, rank ^ 1);
                }
            }
        }
    } else {
        // ================================================================ softmax / output
        if constexpr (KVF == 1) ptx::regs_up<kTrRegsSoftmax>();
        TrWalk w(p, *start);
        const bool any = w.next(p);
        const int quad = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const int half = quad >> 1;            // page of the block, dims 256 half .. + 255
        const int sub = warp >> 2;             // keys 32 sub .. + 31 of the page, 128 of the dims
        const int part = 2 * half + sub;       // which of the row's four threads
        const int r = (quad & 1) * 32 + lane;  // row of this CTA's 64
        const uint32_t grp = 1u + static_cast<uint32_t>(quad & 1);
        // logits as |c| times +-s, so that their max is that of +-s and one fma gives log2 of P
        const float c = fabsf(p.sm_scale_log2);
        const bool flip = p.sm_scale_log2 < 0.f;
        volatile float* sX = reinterpret_cast<volatile float*>(smem + L::kOffX);
        auto warp_wait = [&](int i, uint32_t parity) -> bool {
            return ptx::mbar_wait_warp(bar(i), parity, sAbort, &g_smla_error, kErrTimeout, kWaitLimitNs);
        };
        const uint32_t s_empty0 = even_bar(kPbSEmpty), s_empty1 = even_bar(kPbSEmpty + 1), p_full = even_bar(kPbPFull + half);
        const uint32_t p_row = sbase + L::kOffP + half * kPfPanel + r * 128;
        const int ocol0 = PfLayout::kColO + 128 * sub;
        bool failed = false;
        int x = 0, tails = 0;
        for (bool more = any; !failed && more; more = w.next(p)) {
            float m = -CUDART_INF_F, l = 0.f;
            // (rows past the sequence's last are another's, or garbage: never stored)
            const int token = min(static_cast<int>(w.row0() + rank * kPfHalf + r) / p.bp.h, w.s.n - 1);
            int page = page_of(p.bp, w.b, w.s, 2 * w.b0 + half);
            for (int b = w.b0; b < w.b1; ++b, ++x) {
                const int i_page = 2 * b + half, key = i_page * kPage + 32 * sub;
                // which of this thread's 32 keys take part
                uint32_t bits = low_bits(page_rows(p.bp, w.s, i_page, page) - 32 * sub);
                if (key + 32 > w.s.len) bits &= seen_bits(p.bp, w.s, token, key);
                const bool masked = __any_sync(0xffffffffu, bits != 0xffffffffu);
                page = page_of(p.bp, w.b, w.s, i_page + 2);
                const int s = x & 1;
                uint32_t sv[32];
                float mx = -CUDART_INF_F;
                if (!failed && !warp_wait(kPbSFull + s, (x >> 1) & 1)) failed = true;
                if (!failed) {
                    ptx::tc_fence_after();
                    uint32_t sw[32];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        SMLA_TMEM_LD16(tmem + lane_base + PfLayout::kColS + s * PfLayout::kSBuf + 32 * sub + 16 * q, sv + 16 * q);
                        SMLA_TMEM_LD16(tmem + lane_base + PfLayout::kColS + s * PfLayout::kSBuf + kPfPage + 32 * sub + 16 * q, sw + 16 * q);
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
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((bits >> i) & 1u)) sv[i] = __float_as_uint(-CUDART_INF_F);
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
                    if (bits == 0u || mx != mx) mx = -CUDART_INF_F;
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
                        // O is complete up to the last block: page 1 of PV(x - 1) is done (the prefix kernel says
                        // why page 1's barrier, and why it cannot be two phases old)
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
                        // the row's four warps meet: page 0's MMAs add to the dims of the page 1 warps too
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
                    if (masked) {
                        if (!((bits >> (2 * i)) & 1u)) pp.x = 0.f;
                        if (!((bits >> (2 * i + 1)) & 1u)) pp.y = 0.f;
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
                const bool tail = tree_tail(w.s, i_page);
                if (KVF == 1 || tail) {
                    if (!warp_wait(kTbTail + half, tails & 1)) {
                        failed = true;
                        continue;
                    }
                    ++tails;
                }
                if (tail) {
                    // this CTA's V tile of the page, cleaned by the page's warps: rows past the end, and what
                    // is not finite in the drafted rows
                    const int drafted = max(w.s.len - i_page * kPage, 0), end = min(w.s.keys - i_page * kPage, kPage);
                    const int tid = (2 * sub + (quad & 1)) * 32 + lane;
                    const uint32_t vt = sbase + L::kOffV + half * kPfVPage;
#pragma unroll 1
                    for (int j = tid; j < (kPage - drafted) * 32; j += 128) {
                        const int row = drafted + (j >> 5);
                        const uint32_t at = vt + (j & 3) * kPfPanel + row * 128 + ((j >> 2) & 7) * 16;
                        uint32_t v[4] = {0u, 0u, 0u, 0u};
                        if (row < end) {
                            const uint4 q = ptx::ld_shared_v4(at);
                            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((v[e] & 0x7f80u) == 0x7f80u) v[e] &= 0xffff0000u;
                                if ((v[e] & 0x7f800000u) == 0x7f800000u) v[e] &= 0xffffu;
                            }
                        }
                        ptx::st_shared_v4(at, make_uint4(v[0], v[1], v[2], v[3]));
                    }
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
            const int64_t seq_row = w.row0() + rank * kPfHalf + (quad & 1) * 32;  // the warp's first row
            const int live = static_cast<int>(min(static_cast<int64_t>(w.s.n) * p.bp.h - seq_row, static_cast<int64_t>(32)));
            const int64_t row0 = static_cast<int64_t>(w.s.first) * p.bp.h + seq_row;
            const bool whole = w.whole();
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
                constexpr int kCols = KVF == 1 ? 32 : 64;
                const uint32_t stage = sbase + L::kOffP + warp * 32 * 64;
                float4* part = reinterpret_cast<float4*>(p.part_o) + (pgroup * 128 + 64 * half + 32 * sub) * 32 + lane;
#pragma unroll 1
                for (int cc = 0; cc < 128 / kCols; ++cc) {  // 64 columns of O are read at a time (with fp8 32, for registers)
                    uint32_t ov[kCols];
#pragma unroll
                    for (int q = 0; q < kCols / 16; ++q) SMLA_TMEM_LD16(tmem + lane_base + ocol0 + cc * kCols + 16 * q, ov + 16 * q);
                    ptx::tmem_wait_ld(ov);
                    if (whole) {
                        __nv_bfloat16* dst = p.out + row0 * kDV + 256 * half + 128 * sub + kCols * cc + (lane & 3) * 8;
#pragma unroll
                        for (int u = 0; u < kCols / 32; ++u) {
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
                        for (int e = 0; e < kCols / 4; ++e)
                            part[(kCols / 4 * cc + e) * 32] = make_float4(__uint_as_float(ov[4 * e]), __uint_as_float(ov[4 * e + 1]),
                                                                   __uint_as_float(ov[4 * e + 2]), __uint_as_float(ov[4 * e + 3]));
                    }
                }
            }
            ptx::tc_fence_before();  // before the next piece's first PV overwrites O
            // every warp's staging is read before the next P is written over it; and all leave together
            failed = ptx::named_bar_red_or(3u, 32u * kTrSoftmaxWarps, failed);
        }
    }
    // ---- both CTAs are done with each other's shared memory, barriers and TMEM
    ptx::tc_fence_before();
    __syncwarp();
    ptx::cluster_sync();
    if (warp == kTrS1Warp) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, PfLayout::kTmemCols);
    }
}

// Joins the pieces of a cut tile, as the prefix kernel's join does, from the note that its first run left.
template <int PARTS>
__global__ void __launch_bounds__(kPfMergeThreads) sparse_mla_tree_merge_kernel(const TrParams p) {
    constexpr int kSlices = kDV / PfJoin<PARTS>::kDims;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int dg = static_cast<int>(blockIdx.x % kSlices);
    const int group = static_cast<int>(blockIdx.x / kSlices) % p.slot_groups;
    const int4 job = ptx::ld(p.job_list + blockIdx.x / kSlices / p.slot_groups);
    const int live = min(job.y - 32 * group, 32);
    if (live <= 0) return;
    const int64_t row0 = static_cast<int64_t>(job.x) + 32 * group;
    pf_join<PARTS>(p.part_o, p.part_ml, p.slot_groups, group, dg, job.z >> 1, job.w, job.z, live, p.out + row0 * kDV, p.lse + row0);
}

// The same where there are many cut tiles of few pieces each: a warp takes 32 rows (a lane each) and 32 dims,
// two pieces' loads in flight, and stores its row's 64 bytes itself.  (As small CTAs that do 64 dims and meet
// in shared memory, 2432 of them took 17 us for 8 sequences of 4096 rows, most of it the latency of four
// waves.)
constexpr int kTrJoinThreads = 256;

__global__ void __launch_bounds__(kTrJoinThreads) sparse_mla_tree_join_kernel(const TrParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = static_cast<int>(blockIdx.x & 1);  // of the dims
    const int group = static_cast<int>(blockIdx.x >> 1) % p.slot_groups;
    const int4 job = ptx::ld(p.job_list + static_cast<int>(blockIdx.x >> 1) / p.slot_groups);
    const int live = min(job.y - 32 * group, 32);
    if (live <= 0) return;
    const int at = min(lane, live - 1);  // a lane past the last row repeats it and stores nothing
    const int first = job.z >> 1, last = job.w, chunk = 64 * part + 8 * warp;
    float m = -CUDART_INF_F, l = 0.f;
    float4 acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = first; k <= last; k += 2) {
        float mk[2], lk[2];
        float4 v[2][8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int kk = min(k + u, last);
            const int64_t g = static_cast<int64_t>(kk == first ? job.z : 2 * kk) * p.slot_groups + group;
            mk[u] = ptx::ld(p.part_ml + 64 * g + at);
            lk[u] = ptx::ld(p.part_ml + 64 * g + 32 + at);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = ptx::ld(reinterpret_cast<const float4*>(p.part_o) + (g * 128 + chunk + e) * 32 + at);
        }
        if (k + 1 > last) {  // no second piece
            mk[1] = -CUDART_INF_F;
            lk[1] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[1][e] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float mn = fmaxf(m, fmaxf(mk[0], mk[1]));
        // A piece without a max weighs 0 and is added all the same: without a key its sum and rows are 0 (P was 0 and V had
        // nothing that is not finite), but where all that a row sees of it is NaN, they are NaN, and 0 times that stays.
        const float keep = m == -CUDART_INF_F ? 0.f : ptx::ex2_approx(m - mn);
        m = mn;
        l *= keep;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = make_float4(acc[e].x * keep, acc[e].y * keep, acc[e].z * keep, acc[e].w * keep);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float wt = mk[u] == -CUDART_INF_F ? 0.f : ptx::ex2_approx(mk[u] - m);
            l += wt * lk[u];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc[e].x += wt * v[u][e].x;
                acc[e].y += wt * v[u][e].y;
                acc[e].z += wt * v[u][e].z;
                acc[e].w += wt * v[u][e].w;
            }
        }
    }
    if (lane >= live) return;
    const int64_t row = static_cast<int64_t>(job.x) + 32 * group + lane;
    const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
    if (chunk == 0) p.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
    uint4* out = reinterpret_cast<uint4*>(p.out + row * kDV + 4 * chunk);
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        out[e / 2] = make_uint4(ptx::cvt_bf16x2(acc[e].x * inv, acc[e].y * inv), ptx::cvt_bf16x2(acc[e].z * inv, acc[e].w * inv),
                                ptx::cvt_bf16x2(acc[e + 1].x * inv, acc[e + 1].y * inv), ptx::cvt_bf16x2(acc[e + 1].z * inv, acc[e + 1].w * inv));
}

}  // namespace smla
