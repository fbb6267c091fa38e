// The attention weight that every cached row of a batch has gathered, on tcgen05 tensor cores (sm_103a):
//
//   out[b][p] = decay * prev[b][p] (cached rows) + sum over sequence b's tokens t and heads of exp(s - lse[t])
//   s = scale q.k over 576 dims, for the rows p that token t sees (sparse_mla_tree.cuh), lse from that attention
//
// The second look at the keys that the sums need: an LSE is known only when its row's attention is done.
//
// The product is turned round: keys are the MMA's rows, so that a key's probabilities lie in one TMEM lane
// and its sum is a thread's own, without atomics and in a fixed order.  A CTA pair takes 256 keys of a
// sequence (cta_group::2, M = 256: 128 keys per CTA) against up to 256 rows (token, head), half of which each
// CTA holds; the 576 dims go through in nine panels of 64.
//
// One operand of a pair stays in shared memory, the other streams through a ring of panels:
//   up to 256 rows in the sequence: its queries stay, keys stream.  Bound by HBM, 1152 bytes a key: 256 keys
//     are 3.3 us for 76 pairs at 6.8 TB/s, the MMAs at most 36 * 128 cycles = 2.4 us.
//   more: a tile of keys stays and the queries stream from L2, tile after tile, so that a key's sum still is
//     one thread's.  Bound by that stream, 295 KB a row tile and pair: 3.9 us, where the MMAs take 2.4.
// Both operands have the same layout (rows x 9 panels, SW128), so the two forms differ in who loads what and in
// which descriptor is A.  The ring's depth sets the pace where the operand streams (64 KB in flight per CTA gave
// 42 GB/s per SM, from HBM and from L2 alike), so it takes what the other operand leaves: eight stages if no
// sequence of the batch has more than 128 rows, else five (with fp8 five and three, beside the codes).
//
// Issuing: a panel costs its thread 500 cycles and more (four MMAs at 70 to 100, a wait and a commit): nine of them
// are 2.5 us a tile, 4 beside the expansion of fp8 rows.  Where no sequence has more than 128 rows, TMEM holds two
// accumulators in each of two buffers, so two threads issue every other panel, each into its own, and the sums add
// them (37 sequences of 8191 fp8 rows: 66 -> 60 us).  A stage of the ring is always the same thread's, which so follows
// every phase of its barriers.  With more rows the MMAs themselves take 512 cycles a panel and one thread issues.
//
// Work: tiles of 256 keys, each whole in one pair, in equal shares of their cost (kWt... below).
//
// fp8 codes come by TMA, 128 of every row at a time, into a ring of their own, and eight more warps expand them, each
// 16 of the CTA's 128 keys, two panels at a time into the ring of panels (or the operand that stays); the rotated
// dims come by TMA as they are.  (Codes loaded into registers: 7 us a tile, because the fence after a panel's
// stores waits for the loads that are meant to run ahead.  Expanded into global memory and loaded from there:
// 6.4 us, L2 took the writes no faster.  One panel at a time: 4.4; two, with one thread issuing: 4.1.  With two 3.7,
// and 3.5 with the products in pairs.)  Where no sequence has more than 128 rows, each half of the warps has every other
// pair of panels and a slot of the ring for it, which the issuer of the slot waits for and frees as one, 32 rows a
// warp: half as many waits and fences a tile, and one half's waits beside the other's work (57.6 -> 55 us, L2: 3.1 to
// 3.6 us a tile).  The codes' ring is far enough ahead without a prefetch into L2 (one tile ahead 56.3, two 60).
//
// Roles (384 threads, 640 with fp8):
//   warps 0-7    elements of sequences without tokens; then sums: TMEM quadrant warp % 4 (32 keys), half warp / 4 of
//                the tile's columns
//   warp 8       TMA producer (one thread)
//   warps 9-10   MMA issuers (one thread of the even CTA each); warp 9 owns the TMEM
//   warp 11      elements past a sequence's last key
//   warps 12-19  expansion of fp8 rows
// Every wait is bounded; a CTA that gives up meets the other at the final cluster barrier.
#pragma once

#include "sparse_mla_batch.cuh"

namespace smla {

constexpr int kWtKeys = 256;      // keys per tile (pair)
constexpr int kWtHalf = 128;      // per CTA
constexpr int kWtRows = 256;      // rows (token, head) per tile
// stages of the ring, and of the ring of fp8 codes; Few: no sequence has more than kWtRowsFew rows
constexpr int kWtStages = 5, kWtStagesFew = 8;
constexpr int kWtStagesFp8 = 3, kWtStagesFewFp8 = 5;  // the latter: two pairs of panels, and one for the rotated dims
static_assert(kWtStagesFew % 2 == 0, "a stage is always the same issuer's");
constexpr int kWtRopeAt = kWtStagesFewFp8 - 1;
constexpr int kWtRaw = 2, kWtRawFew = 4;  // 128 rows x 128 codes each: two panels
constexpr int kWtRowsFew = 128;      // rows of a sequence up to which the deeper ring has room
constexpr int kWtPanel = 128 * 128;  // 128 rows x 64 bf16, SW128
constexpr int kWtSumWarps = 8;
constexpr int kWtTmaWarp = 8, kWtMmaWarp = 9, kWtFillWarp = 11, kWtExpandWarp = 12;
constexpr int kWtExpandWarps = 8;
constexpr int kWtExpandRows = kWtHalf / kWtExpandWarps;  // 16
// costs in tenths of a microsecond: a sequence's queries and first keys; a tile whose keys stream; one whose
// keys stay, and each of its row tiles
constexpr int kWtCostSeq = 30, kWtCostStream = 34, kWtCostStay = 20, kWtCostRows = 24;

template <int KVF>
__host__ __device__ constexpr int weights_threads() {
    return 32 * (kWtExpandWarp + (KVF ? kWtExpandWarps : 0));
}

enum : int {
    kWbStayFull = 0,                        // even CTA: both CTAs' part of the operand that stays, by TMA
    kWbStayMade = 1,                        // even CTA: the same, expanded, with the rotated dims by TMA
    kWbStayEmpty = 2,                       // both
    kWbFull = 3,                            // +stage, even CTA: by TMA
    kWbMade = kWbFull + kWtStagesFew,       // +stage, even CTA: expanded
    kWbEmpty = kWbMade + kWtStagesFew,      // +stage, both
    kWbSFull = kWbEmpty + kWtStagesFew,     // +buffer, both
    kWbSEmpty = kWbSFull + 2,               // +buffer, even CTA
    kWbDrain = kWbSEmpty + 2,               // even CTA
    kWbRawFull = kWbDrain + 1,              // +stage, own CTA: codes
    kWbRawEmpty = kWbRawFull + kWtRawFew,   // +stage, own CTA
    kWbCount = kWbRawEmpty + kWtRawFew
};

struct WtLayout {
    static constexpr int kOffStay = 0;                               // 9 panels of 128 rows, or of 64
    static constexpr int kOffRing = kPanels * kWtPanel, kOffRingFew = kOffRing / 2;
    static constexpr int kOffLse = kOffRing + kWtStages * kWtPanel;  // [2][256]: minus the rows' LSE
    static constexpr int kOffRaw = kOffRing + kWtStagesFp8 * kWtPanel, kOffRawFew = kOffRingFew + kWtStagesFewFp8 * kWtPanel;
    static_assert(kOffRingFew + kWtStagesFew * kWtPanel <= kOffLse, "ring");
    static_assert(kOffRaw + kWtRaw * kWtPanel <= kOffLse && kOffRawFew + kWtRawFew * kWtPanel <= kOffLse, "codes");
    static constexpr int kOffX = kOffLse + 2 * kWtRows * 4;          // [128]: sums of the columns' second half; the plan's sums
    static constexpr int kOffBar = kOffX + kWtHalf * 4;
    static constexpr int kOffMisc = kOffBar + kWbCount * 8;          // tmem base, abort flag, the run's start
    static constexpr int kBytes = kOffMisc + 8 + 40;
    static_assert(kBytes <= 232448, "shared memory budget (227 KB)");
};

struct WtStart {
    int64_t at, end, seq_at;  // the run [at, end) in cost units; where its first sequence begins
    int32_t b;
    int32_t few;              // no sequence has more than kWtRowsFew rows
};

struct WtParams {
    BatchParams bp;
    const float* lse;      // [T, h]
    const float* prev;     // [B, nb * 64] or nullptr
    float* out;            // [B, nb * 64]
    int32_t pairs;
    float scale, decay;
};

__device__ __forceinline__ int weights_row_tiles(const WtParams& p, const Seq& s) {
    return static_cast<int>((static_cast<int64_t>(s.n) * p.bp.h + kWtRows - 1) / kWtRows);
}
__device__ __forceinline__ int weights_tile_cost(int row_tiles) {
    return row_tiles <= 1 ? kWtCostStream : kWtCostStay + kWtCostRows * row_tiles;
}
__device__ __forceinline__ int weights_key_tiles(const Seq& s) { return s.n == 0 ? 0 : (s.keys + kWtKeys - 1) / kWtKeys; }

// All threads of the CTA: the start of pair `run`'s share, into *start (shared memory).
__device__ __forceinline__ void weights_plan(const WtParams& p, int run, int threads, int64_t* scratch, WtStart* start) {
    const int per = (p.bp.B + threads - 1) / threads;
    const int b0 = min(ptx::behind(static_cast<int>(threadIdx.x)) * per, p.bp.B), b1 = min(b0 + per, p.bp.B);
    auto cost_of = [&](const Seq& s) -> int64_t {
        return s.n == 0 ? 0 : kWtCostSeq + static_cast<int64_t>(weights_key_tiles(s)) * weights_tile_cost(weights_row_tiles(p, s));
    };
    int64_t cost = 0, many = 0;
    for (int b = b0; b < b1; ++b) {
        const Seq s = load_seq(p.bp, b);
        cost += cost_of(s);
        many += static_cast<int64_t>(s.n) * p.bp.h > kWtRowsFew;
    }
    int64_t at, total, wide_before, wide;  // wide: sequences of more than kWtRowsFew rows
    block_prefix2(cost, many, scratch, threads / 32, at, total, wide_before, wide);
    const int few = wide == 0;
    const int64_t from = share_of(total, run, p.pairs), to = share_of(total, run + 1, p.pairs);
    if (from >= to) {
        if (threadIdx.x == 0) *start = WtStart{0, 0, 0, p.bp.B, few};
    } else if (at <= from && from < at + cost) {
        int b = b0;
        for (;; ++b) {
            const int64_t c = cost_of(load_seq(p.bp, b));
            if (from < at + c) break;
            at += c;
        }
        *start = WtStart{from, to, at, b, few};
    }
    __syncthreads();
}

// The pieces of a run, the same for every role: key tiles [k0, k1) of sequence b.  A tile belongs to the
// run that its first cost unit lies in.
struct WtWalk {
    int64_t at, end;  // relative to the sequence's first unit
    Seq s;
    int b, row_tiles, cost, key_tiles;
    int k0, k1;
    bool begun;
    __device__ __forceinline__ WtWalk(const WtParams& p, const WtStart& st) : b(st.b), begun(false) {
        at = st.at - st.seq_at;
        end = st.end - st.seq_at;
        if (b < p.bp.B) load(p);
    }
    __device__ __forceinline__ void load(const WtParams& p) {
        s = load_seq(p.bp, b);
        row_tiles = weights_row_tiles(p, s);
        cost = weights_tile_cost(row_tiles);
        key_tiles = weights_key_tiles(s);
    }
    __device__ __forceinline__ bool next(const WtParams& p) {
        for (;;) {
            if (begun) {
                if (s.n) {
                    end -= kWtCostSeq + static_cast<int64_t>(key_tiles) * cost;
                    at = 0;
                }
                if (end <= 0 || ++b >= p.bp.B) return false;
                load(p);
            } else if (at >= end) {
                return false;
            }
            begun = true;
            k0 = first_from(at);
            k1 = first_from(end);
            if (k1 > k0) return true;
        }
    }
    // the first tile whose first unit lies at x or later
    __device__ __forceinline__ int first_from(int64_t x) const {
        const int64_t y = x - kWtCostSeq;
        return y <= 0 ? 0 : static_cast<int>(min((y + cost - 1) / cost, static_cast<int64_t>(key_tiles)));
    }
    // rows of row tile i, and the MMA's columns for them
    __device__ __forceinline__ int rows(const WtParams& p, int i) const {
        return static_cast<int>(min(static_cast<int64_t>(s.n) * p.bp.h - static_cast<int64_t>(i) * kWtRows, static_cast<int64_t>(kWtRows)));
    }
    __device__ __forceinline__ int columns(const WtParams& p, int i) const { return (rows(p, i) + 31) & ~31; }
};

// A place in the ring of stages, the same for everybody who goes along it.
struct WtStage {
    int at, stages, round;
    __device__ __forceinline__ explicit WtStage(int n) : at(0), stages(n), round(0) {}
    __device__ __forceinline__ void next() {
        if (++at == stages) {
            at = 0;
            ++round;
        }
    }
    __device__ __forceinline__ bool used() const { return round > 0; }                 // this stage has been filled before
    __device__ __forceinline__ uint32_t last() const { return (round - 1) & 1; }       // parity of its last release
};

// The elements that no tile covers, by warp `first` of `stride`: of sequences without tokens all (kIdle), of the others
// those past the last key.  Chunks of 4096 positions; a lane looks at one, so that the many without work cost little.
template <bool kIdle>
__device__ __forceinline__ void weights_fill(const WtParams& p, int first, int stride) {
    constexpr int kChunk = 4096, kLoads = kIdle ? 8 : 4;  // idle: loads in flight a lane, eight warps of them
    const int lane = threadIdx.x & 31;
    const int width = p.bp.nb * kPage, chunks = (width + kChunk - 1) / kChunk;
    const int64_t total = static_cast<int64_t>(p.bp.B) * chunks;
    for (int64_t c0 = ptx::behind(first); c0 < total; c0 += 32 * static_cast<int64_t>(stride)) {
        const int64_t c = c0 + static_cast<int64_t>(lane) * stride;
        int b = 0, from = 0, to = 0, len = 0;
        if (c < total) {
            b = static_cast<int>(c / chunks);
            from = static_cast<int>(c % chunks) * kChunk;
            to = min(from + kChunk, width);
            const Seq s = load_seq(p.bp, b);
            len = s.len;
            if (!kIdle) from = max(from, s.keys);
            if ((s.n == 0) != kIdle) to = 0;
        }
        for (uint32_t left = __ballot_sync(0xffffffffu, from < to); left; left &= left - 1u) {
            const int l = __ffs(left) - 1;
            const int64_t row = static_cast<int64_t>(__shfl_sync(0xffffffffu, b, l)) * width;
            const int i0 = __shfl_sync(0xffffffffu, from, l) + lane, i1 = __shfl_sync(0xffffffffu, to, l);
            const int n = kIdle && p.prev ? __shfl_sync(0xffffffffu, len, l) : 0;
            for (int i = i0; i < i1; i += 32 * kLoads) {
                float x[kLoads];
#pragma unroll
                for (int u = 0; u < kLoads; ++u) x[u] = i + 32 * u < n ? p.prev[row + i + 32 * u] : 0.f;
#pragma unroll
                for (int u = 0; u < kLoads; ++u)
                    if (i + 32 * u < i1) p.out[row + i + 32 * u] = i + 32 * u < n ? p.decay * x[u] : 0.f;
            }
        }
    }
}

template <int KVF>
__global__ void __launch_bounds__(weights_threads<KVF>(), 1)
    sparse_mla_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                              const __grid_constant__ CUtensorMap tm_codes, const WtParams p) {
    using L = WtLayout;
    constexpr int kThreads = weights_threads<KVF>();
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
    WtStart* start = reinterpret_cast<WtStart*>(smem + L::kOffMisc + 8);
    auto bar = [&](int i) -> uint32_t { return sbase + L::kOffBar + 8u * static_cast<uint32_t>(i); };
    auto even_bar = [&](int i) -> uint32_t { return ptx::map_shared_rank(bar(i), 0); };
    auto wait = [&](int i, uint32_t parity) -> bool {
        return ptx::mbar_wait(bar(i), parity, sAbort, &g_smla_error, kErrTimeout, kWaitLimitNs);
    };

    if (threadIdx.x == 0) {
        *sAbort = 0;
        for (int i = 0; i < kWbCount; ++i) {
            const bool by_warps = i == kWbSEmpty || i == kWbSEmpty + 1;                // both CTAs' sum warps
            const bool by_expand = i == kWbStayMade || (i >= kWbMade && i < kWbMade + kWtStagesFew);  // both CTAs' expansion warps
            const bool by_own = i >= kWbRawEmpty;                                                       // this CTA's
            const bool by_two = i == kWbStayEmpty || i == kWbSFull || i == kWbSFull + 1 || i == kWbDrain;  // both issuers
            ptx::mbar_init(bar(i), by_warps ? 2 * kWtSumWarps : by_two ? 2 : by_own ? kWtExpandWarps : by_expand ? 2 * kWtExpandWarps + (i == kWbStayMade ? 1 : 0) : 1);
        }
        ptx::fence_mbarrier_init();
    }
    if (warp == kWtMmaWarp) {
        ptx::tmem_alloc_pair(sbase + L::kOffMisc, 512);
        ptx::tmem_relinquish_pair();
    }
    if (warp == kWtTmaWarp && lane == 0) {
        ptx::prefetch_tmap(&tm_q);
        ptx::prefetch_tmap(&tm_k);
        if (KVF == 1) ptx::prefetch_tmap(&tm_codes);
    }
    ptx::tc_fence_before();
    __syncwarp();           // the cluster barrier wants its warps whole
    ptx::cluster_arrive();  // both CTAs' barriers are initialised before anyone signals them
    // launched as a programmatic dependent: nothing above touched global memory
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    weights_plan(p, run, kThreads, reinterpret_cast<int64_t*>(smem + L::kOffX), start);
    WtWalk w(p, *start);
    const bool any = w.next(p);
    __syncwarp();
    ptx::cluster_wait();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc);
    const bool few = start->few != 0;
    const int stages = KVF ? (few ? kWtStagesFewFp8 : kWtStagesFp8) : few ? kWtStagesFew : kWtStages;
    const int raw_stages = few ? kWtRawFew : kWtRaw;
    const uint32_t raw = sbase + (few ? L::kOffRawFew : L::kOffRaw);
    const uint32_t ring = sbase + (few ? L::kOffRingFew : L::kOffRing);
    const int stay_panel = few ? kWtPanel / 2 : kWtPanel;

    if (warp == kWtTmaWarp) {
        // ================================================================ TMA producer
        // The even CTA's thread expects both CTAs' bytes on its barrier, each CTA's thread issues its own copies.
        if (lane == 0) {
            bool ok = true;
            int stays = 0;          // operands that stayed so far
            WtStage st(stages);
            int row0 = 0, row1 = 0;  // rows of the tile's two pages
            auto begin_stay = [&]() -> bool {
                if (stays > 0 && !wait(kWbStayEmpty, (stays - 1) & 1)) return false;
                ++stays;
                return true;
            };
            // the stage is this thread's to fill
            auto begin_stage = [&]() -> bool {
                if (st.used() && !wait(kWbEmpty + st.at, st.last())) return false;
                if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kWbFull + st.at), 2u * kWtPanel);
                return true;
            };
            auto load_keys = [&](uint32_t dst, int pn, uint32_t b) {
                ptx::tma_load_3d_pair(dst, &tm_k, 0, row0, pn, b);
                ptx::tma_load_3d_pair(dst + kWtPanel / 2, &tm_k, 0, row1, pn, b);
            };
            // a page that is not there loads as zeros, from rows below 0
            auto first_row = [&](int page) -> int { return page_in_cache(p.bp, page) ? page * kPage : -kPage; };
            auto prefetch = [&](int i) {  // page i, into L2
                const int pg = page_of(p.bp, w.b, w.s, i);
                const int n = page_rows(p.bp, w.s, i, pg);
                if (n > 0)
                    ptx::bulk_prefetch_l2(static_cast<const char*>(p.bp.kv) + static_cast<int64_t>(pg) * kPage * (KVF ? kFp8RowBytes : kDQK * 2),
                                          static_cast<uint32_t>(n * (KVF ? kFp8RowBytes : kDQK * 2)));
            };
            WtStage raw_st(raw_stages);
            auto load_codes = [&](int pair) -> bool {  // those of panels 2 pair and 2 pair + 1
                if (raw_st.used() && !wait(kWbRawEmpty + raw_st.at, raw_st.last())) return false;
                const uint32_t dst = raw + raw_st.at * kWtPanel, b = bar(kWbRawFull + raw_st.at);
                ptx::mbar_arrive_expect_tx(b, static_cast<uint32_t>(kWtPanel));
                ptx::tma_load_2d(dst, &tm_codes, 128 * pair, row0, b);
                ptx::tma_load_2d(dst + kWtPanel / 2, &tm_codes, 128 * pair, row1, b);
                raw_st.next();
                return true;
            };
            bool others = false;  // the last piece's keys stayed
            int tiles = 0;
            for (bool more = any; ok && more; more = w.next(p)) {
                const bool stream_keys = w.row_tiles == 1;
                const int q0 = w.s.first * p.bp.h;
                if (stream_keys) {
                    if (!(ok = begin_stay())) break;
                    if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kWbStayFull), 2u * kPanels * static_cast<uint32_t>(stay_panel));
                    const int row = q0 + rank * (w.columns(p, 0) / 2);
                    for (int pn = 0; pn < kPanels; ++pn)
                        for (int half = 0; half < (few ? 1 : 2); ++half)
                            ptx::tma_load_3d_pair(sbase + L::kOffStay + pn * stay_panel + half * kWtPanel / 2, &tm_q, 0,
                                                  row + half * kPage, pn, even_bar(kWbStayFull));
                }
                // the stages that the expansion warps filled have been used before this thread fills them: barriers that it
                // does not follow could be more than one phase behind, which a parity cannot tell
                if (KVF == 1 && !stream_keys && !others && stays > 0 && !(ok = wait(kWbStayEmpty, (stays - 1) & 1))) break;
                others = !stream_keys;
                for (int k = w.k0; ok && k < w.k1; ++k, ++tiles) {
                    const int i_page = 4 * k + 2 * rank;
                    row0 = first_row(page_of(p.bp, w.b, w.s, i_page));
                    row1 = first_row(page_of(p.bp, w.b, w.s, i_page + 1));
                    if (KVF == 0 && k + 1 < w.k1) {
                        prefetch(i_page + 4);
                        prefetch(i_page + 5);
                    }
                    if (KVF == 1)
                        for (int pair = 0; ok && pair < 4; ++pair) ok = load_codes(pair);
                    if (!ok) break;
                    if (stream_keys) {
                        for (int pn = 0; ok && pn < kPanels; ++pn, st.next())
                            if (KVF == 0 && (ok = begin_stage())) load_keys(ring + st.at * kWtPanel, pn, even_bar(kWbFull + st.at));
                    } else {
                        if (KVF == 1) {
                            ++stays;  // the expansion warps'
                        } else {
                            if (!(ok = begin_stay())) break;
                            if (rank == 0) ptx::mbar_arrive_expect_tx(bar(kWbStayFull), 2u * kPanels * kWtPanel);
                            for (int pn = 0; pn < kPanels; ++pn) load_keys(sbase + L::kOffStay + pn * kWtPanel, pn, even_bar(kWbStayFull));
                        }
                        for (int i = 0; ok && i < w.row_tiles; ++i) {
                            const int row = q0 + i * kWtRows + rank * (w.columns(p, i) / 2);
                            for (int pn = 0; ok && pn < kPanels; ++pn, st.next())
                                if ((ok = begin_stage())) {
                                    const uint32_t dst = ring + st.at * kWtPanel, b = even_bar(kWbFull + st.at);
                                    ptx::tma_load_3d_pair(dst, &tm_q, 0, row, pn, b);
                                    ptx::tma_load_3d_pair(dst + kWtPanel / 2, &tm_q, 0, row + kPage, pn, b);
                                }
                        }
                    }
                }
            }
            // every copy has landed and been used, and no release is still on its way to this CTA's barriers,
            // before it leaves
            if (ok && stays > 0) ok = wait(kWbStayEmpty, (stays - 1) & 1);
            if (KVF == 1 && few) {
                for (int slot = 0; ok && stays > 0 && slot < 2; ++slot) ok = wait(kWbEmpty + 2 * slot, 1u);  // (two uses a tile)
                if (ok && stays > 0) ok = wait(kWbEmpty + kWtRopeAt, (tiles - 1) & 1);
            } else {
                for (int u = 0; ok && u < stages; ++u, st.next())
                    if (st.used()) ok = wait(kWbEmpty + st.at, st.last());
            }
            if (!ok) {  // gave up: copies in flight complete on the other CTA's barriers; leave them time to land
                const uint64_t t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 2000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == kWtMmaWarp || warp == kWtMmaWarp + 1) {
        // ================================================================ MMA issuers
        // (With more than kWtRowsFew rows the first does everything, the second's releases too.)
        if (rank == 0 && lane == 0) {
            const int me = warp - kWtMmaWarp;
            const uint64_t d_stay = ptx::smem_desc_sw128(sbase + L::kOffStay, 16, 1024);
            const uint64_t d_ring = ptx::smem_desc_sw128(ring, 16, 1024);
            bool ok = true;
            uint32_t full = 0u, made = 0u, stay_full = 0u, stay_made = 0u;  // parities, by stage
            int item = 0;
            WtStage st(stages);
            auto wait_stay = [&](bool expanded) -> bool {
                uint32_t& parity = expanded ? stay_made : stay_full;
                const bool r = wait(expanded ? kWbStayMade : kWbStayFull, parity);
                parity ^= 1u;
                return r;
            };
            const bool both = !few && me == 0;
            auto commit = [&](int i) {
                ptx::mma_commit_pair(bar(i));
                if (both) ptx::mma_commit_pair(bar(i));
            };
            for (bool more = any && (few || me == 0); ok && more; more = w.next(p)) {
                const bool stream_keys = w.row_tiles == 1;
                const bool expanded = KVF == 1 && stream_keys;  // what streams
                if (stream_keys && !(ok = wait_stay(false))) break;
                for (int k = w.k0; ok && k < w.k1; ++k) {
                    if (!stream_keys && !(ok = wait_stay(KVF == 1))) break;
                    for (int i = 0; ok && i < w.row_tiles; ++i, ++item) {
                        const int buf = item & 1;
                        if (item >= 2 && !(ok = wait(kWbSEmpty + buf, ((item >> 1) - 1) & 1))) break;
                        const uint32_t idesc = ptx::idesc_bf16_f32(kWtKeys, w.columns(p, i), 0, 0);
                        const uint32_t d = tmem + buf * kWtRows + me * kWtRowsFew;
                        // Two loops on purpose: the wide one has no time to spare (a panel's MMAs take 512 cycles, its issue about
                        // 500; with the choice of stages inside one loop the wide batches lost 4 per cent).
                        if (!few) {
                            for (int pn = 0; pn < kPanels; ++pn, st.next()) {
                                const bool by_warps = expanded && pn < kPanels - 1;
                                uint32_t& parity = by_warps ? made : full;
                                if (!(ok = wait((by_warps ? kWbMade : kWbFull) + st.at, (parity >> st.at) & 1u))) break;
                                parity ^= 1u << st.at;
                                ptx::tc_fence_after();
                                const uint64_t stay = d_stay + ((pn * stay_panel) >> 4), moving = d_ring + ((st.at * kWtPanel) >> 4);
                                const uint64_t a = stream_keys ? moving : stay, b = stream_keys ? stay : moving;
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    ptx::mma_bf16_ss_pair(d, a + ((kk * 32) >> 4), b + ((kk * 32) >> 4), idesc, (pn | kk) != 0);
                                ptx::mma_commit_pair(bar(kWbEmpty + st.at));
                            }
                        } else if (KVF == 1) {  // pairs of panels, each issuer those of its slot; the rotated dims are the second's
                            const uint64_t moving = d_ring + ((2 * me * kWtPanel) >> 4);
                            if (me == 1) {
                                if (!(ok = wait(kWbFull + kWtRopeAt, item & 1))) break;
                                ptx::tc_fence_after();
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    ptx::mma_bf16_ss_pair(d, d_ring + ((kWtRopeAt * kWtPanel + kk * 32) >> 4),
                                                          d_stay + (((kPanels - 1) * (kWtPanel / 2) + kk * 32) >> 4), idesc, kk > 0);
                                ptx::mma_commit_pair(bar(kWbEmpty + kWtRopeAt));
                            }
#pragma unroll 1
                            for (uint32_t h = 0; h < 2; ++h) {
                                if (!(ok = wait(kWbMade + 2 * me, h))) break;
                                ptx::tc_fence_after();
                                const uint64_t stay = d_stay + (((4 * h + 2 * me) * (kWtPanel / 2)) >> 4);
                                const bool more_of_it = me == 1 || h > 0;
#pragma unroll
                                for (int kk = 0; kk < 8; ++kk)
                                    ptx::mma_bf16_ss_pair(d, moving + (((kk >> 2) * kWtPanel + (kk & 3) * 32) >> 4),
                                                          stay + (((kk >> 2) * (kWtPanel / 2) + (kk & 3) * 32) >> 4), idesc, kk > 0 || more_of_it);
                                ptx::mma_commit_pair(bar(kWbEmpty + 2 * me));
                            }
                        } else {  // the keys stream past the queries; the stages of the issuer's own parity
                            bool first = true;  // nothing issued for this item yet
                            for (int pn = 0; pn < kPanels; ++pn, st.next()) {
                                const uint32_t now = (full >> st.at) & 1u;
                                full ^= 1u << st.at;
                                if ((st.at & 1) != me) continue;
                                if (!(ok = wait(kWbFull + st.at, now))) break;
                                ptx::tc_fence_after();
                                const uint64_t stay = d_stay + ((pn * stay_panel) >> 4), moving = d_ring + ((st.at * kWtPanel) >> 4);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    ptx::mma_bf16_ss_pair(d, moving + ((kk * 32) >> 4), stay + ((kk * 32) >> 4), idesc, kk > 0 || !first);
                                ptx::mma_commit_pair(bar(kWbEmpty + st.at));
                                first = false;
                            }
                        }
                        if (ok) commit(kWbSFull + buf);
                    }
                    if (ok && !stream_keys) commit(kWbStayEmpty);
                }
                if (ok && stream_keys) commit(kWbStayEmpty);
            }
            // nothing is in flight when TMEM is freed, also after giving up
            ptx::mma_commit_pair_local(bar(kWbDrain));
            ptx::mbar_wait(bar(kWbDrain), 0, nullptr, &g_smla_error, 0u, kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp >= kWtExpandWarp) {
        // ================================================================ expansion of fp8 rows
        if constexpr (KVF == 1) {
            // this warp's rows of the CTA's 128 keys; few: of every other pair of panels, twice as many
            const int slot = (warp - kWtExpandWarp) >> 2, rows = few ? 2 * kWtExpandRows : kWtExpandRows;
            const int row = few ? rows * ((warp - kWtExpandWarp) & 3) : rows * (warp - kWtExpandWarp);
            bool ok = true, others = false;  // the last piece's keys stayed
            int stays = 0, tile = 0;
            WtStage st(stages), raw_st(raw_stages);
            auto warp_wait = [&](int i, uint32_t parity) -> bool {
                return ptx::mbar_wait_warp(bar(i), parity, sAbort, &g_smla_error, kErrTimeout, kWaitLimitNs);
            };
            for (bool more = any; ok && more; more = w.next(p)) {
                const bool stream_keys = w.row_tiles == 1;
                // where keys that stay and keys that stream meet, the last operand that stayed has been used: then the
                // ring has, whose barriers these warps do not follow while queries stream
                if (others != !stream_keys) {
                    if (stays > 0 && !(ok = warp_wait(kWbStayEmpty, (stays - 1) & 1))) break;
                }
                others = !stream_keys;
                // Lane l has the scales of row l % rows of the warp's; of the codes, 16 from 16 (l % 8) on of a pair of panels, in rows
                // 4 i + l / 8.
                auto page = [&](int k, int i) -> int { return k < w.k1 ? page_of(p.bp, w.b, w.s, 4 * k + 2 * rank + i) : -1; };
                auto scales = [&](int k, int pg) -> float4 {
                    const int n = page_rows(p.bp, w.s, 4 * k + 2 * rank + row / kPage, pg) - row % kPage, r = lane & (rows - 1);
                    const uint8_t* src = static_cast<const uint8_t*>(p.bp.kv) + (static_cast<int64_t>(pg) * kPage + row % kPage + r) * kFp8RowBytes;
                    return r < n ? ptx::ld_from(reinterpret_cast<const float4*>(src + 512)) : make_float4(0.f, 0.f, 0.f, 0.f);
                };
                const int part = lane & 7, rr = lane >> 3;
                const bool second = part >= 4;  // of the two panels
                int pg0 = page(w.k0, 0), pg1 = page(w.k0, 1);
                float4 sc = scales(w.k0, row < kPage ? pg0 : pg1);
                int next0 = page(w.k0 + 1, 0), next1 = page(w.k0 + 1, 1);
                for (int k = w.k0; ok && k < w.k1; ++k, ++tile) {
                    // the rotated dims, by this CTA's first expansion warp
                    auto load_rope = [&](uint32_t dst, int i) {
                        if (lane == 0) {
                            if (rank == 0) ptx::mbar_arrive_expect_tx(bar(i), 2u * kWtPanel);
                            ptx::tma_load_2d_pair(dst, &tm_k, 528, page_in_cache(p.bp, pg0) ? pg0 * kPage : -kPage, even_bar(i));
                            ptx::tma_load_2d_pair(dst + kWtPanel / 2, &tm_k, 528, page_in_cache(p.bp, pg1) ? pg1 * kPage : -kPage, even_bar(i));
                        }
                        __syncwarp();
                    };
                    if (!stream_keys) {
                        if (stays > 0 && !(ok = warp_wait(kWbStayEmpty, (stays - 1) & 1))) break;
                        ++stays;
                        if (warp == kWtExpandWarp) load_rope(sbase + L::kOffStay + (kPanels - 1) * kWtPanel, kWbStayMade);
                    } else if (few && warp == kWtExpandWarp) {
                        if (tile > 0 && !(ok = warp_wait(kWbEmpty + kWtRopeAt, (tile - 1) & 1))) break;
                        load_rope(ring + kWtRopeAt * kWtPanel, kWbFull + kWtRopeAt);
                    }
                    // 16 rows from r0 of the warp's on: codes at `from`, panels at `into`, the rows' scale `s_of` of lane r0 + their index
                    auto expand = [&](uint32_t from, uint32_t into, int r0, float s_of) {
                        uint4 v[kWtExpandRows / 4];
#pragma unroll
                        for (int i = 0; i < kWtExpandRows / 4; ++i) v[i] = ptx::ld_shared_v4(from + (row + r0 + 4 * i) * 128 + lane * 16);
                        const uint32_t dst = into + second * kWtPanel + (row + r0) * 128;
#pragma unroll
                        for (int i = 0; i < kWtExpandRows / 4; ++i) {
                            // chunk c of row r lies at 16 (c ^ r % 8); the lanes of the second panel store their two chunks in the
                            // other order, so that the eight lanes of a row hit all banks
                            const int r = 4 * i + rr, c = 2 * (part & 3);
                            const float s = __shfl_sync(0xffffffffu, s_of, r0 + r);
                            const uint32_t x0 = second ? v[i].z : v[i].x, y0 = second ? v[i].w : v[i].y;
                            const uint32_t x1 = second ? v[i].x : v[i].z, y1 = second ? v[i].y : v[i].w;
                            const uint2 a0 = ptx::e4m3x4_scaled_bf16x4(x0, make_float2(s, s)), b0 = ptx::e4m3x4_scaled_bf16x4(y0, make_float2(s, s));
                            ptx::st_shared_v4(dst + r * 128 + (((c + second) ^ (r & 7)) << 4), make_uint4(a0.x, a0.y, b0.x, b0.y));
                            const uint2 a1 = ptx::e4m3x4_scaled_bf16x4(x1, make_float2(s, s)), b1 = ptx::e4m3x4_scaled_bf16x4(y1, make_float2(s, s));
                            ptx::st_shared_v4(dst + r * 128 + (((c + !second) ^ (r & 7)) << 4), make_uint4(a1.x, a1.y, b1.x, b1.y));
                        }
                    };
                    if (few) {
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            const int pair = 2 * h + slot, use = 2 * tile + h;  // of the pair's slot
                            if (!(ok = warp_wait(kWbRawFull + pair, tile & 1))) break;
                            if (use > 0 && !(ok = warp_wait(kWbEmpty + 2 * slot, (use - 1) & 1))) break;
                            const float s = h ? (slot ? sc.w : sc.z) : (slot ? sc.y : sc.x);
#pragma unroll 1
                            for (int r0 = 0; r0 < 2 * kWtExpandRows; r0 += kWtExpandRows)
                                expand(raw + pair * kWtPanel, ring + 2 * slot * kWtPanel, r0, s);
                            ptx::fence_proxy_async_smem();
                            __syncwarp();
                            // (twice each: the barriers count eight warps a CTA)
                            if (lane < 2) {
                                ptx::mbar_arrive_cluster(even_bar(kWbMade + 2 * slot));
                                ptx::mbar_arrive(bar(kWbRawEmpty + pair));
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int pair = 0; pair < 4; ++pair) {
                            if (!(ok = warp_wait(kWbRawFull + raw_st.at, raw_st.round & 1))) break;
                            WtStage st2 = st;
                            uint32_t into = sbase + L::kOffStay + 2 * pair * kWtPanel;
                            int apart = 0;  // how much further than the next the second panel lies
                            if (stream_keys) {
                                st2.next();
                                if (st.used() && !(ok = warp_wait(kWbEmpty + st.at, st.last()))) break;
                                if (st2.used() && !(ok = warp_wait(kWbEmpty + st2.at, st2.last()))) break;
                                into = ring + st.at * kWtPanel;
                                apart = second ? (st2.at - st.at - 1) * kWtPanel : 0;
                            }
                            expand(raw + raw_st.at * kWtPanel, into + apart, 0, sc.x);
                            sc = make_float4(sc.y, sc.z, sc.w, 0.f);
                            ptx::fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(bar(kWbRawEmpty + raw_st.at));
                            raw_st.next();
                            if (stream_keys) {
                                if (lane < 2) ptx::mbar_arrive_cluster(even_bar(kWbMade + (lane ? st2.at : st.at)));
                                st = st2;
                                st.next();
                            }
                        }
                    }
                    if (!ok) break;
                    if (!few && stream_keys) {
                        if (warp == kWtExpandWarp) {
                            if (st.used() && !(ok = warp_wait(kWbEmpty + st.at, st.last()))) break;
                            load_rope(ring + st.at * kWtPanel, kWbFull + st.at);
                        }
                        st.next();
                    } else if (!stream_keys) {
                        if (lane == 0) ptx::mbar_arrive_cluster(even_bar(kWbStayMade));
                        for (int i = 0; i < w.row_tiles * kPanels; ++i) st.next();
                    }
                    // (after the last fence, which would wait for these)
                    pg0 = next0;
                    pg1 = next1;
                    sc = scales(k + 1, row < kPage ? pg0 : pg1);
                    next0 = page(k + 2, 0);
                    next1 = page(k + 2, 1);
                }
                if (stream_keys) ++stays;  // the queries, the producer's
            }
        }
    } else if (warp >= kWtFillWarp) {
        // ================================================================ elements that no tile covers
        weights_fill<false>(p, blockIdx.x, gridDim.x);
    } else {
        // ================================================================ sums
        weights_fill<true>(p, static_cast<int>(blockIdx.x) * kWtSumWarps + warp, static_cast<int>(gridDim.x) * kWtSumWarps);
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const int tid = threadIdx.x;  // 0 .. 255
        volatile float* sX = reinterpret_cast<volatile float*>(smem + L::kOffX);
        const uint32_t s_lse = sbase + L::kOffLse;
        const float2 scale2 = make_float2(p.scale, p.scale);
        const float2 log2e2 = make_float2(1.4426950408889634f, 1.4426950408889634f);
        const int width = p.bp.nb * kPage;
        const uint32_t s_empty0 = even_bar(kWbSEmpty), s_empty1 = even_bar(kWbSEmpty + 1);
        auto warp_wait = [&](int i, uint32_t parity) -> bool {
            return ptx::mbar_wait_warp(bar(i), parity, sAbort, &g_smla_error, kErrTimeout, kWaitLimitNs);
        };
        // minus the LSE of row tid of row tile i: the table's entry.  +inf, of a row that adds nothing, is kept out of the sums
        // as keys that a token does not see are (a NaN logit would pass through any number).
        auto entry = [&](int i) -> float {
            if (tid >= w.rows(p, i)) return -CUDART_INF_F;
            return -ptx::ld_from(p.lse + static_cast<int64_t>(w.s.first) * p.bp.h + static_cast<int64_t>(i) * kWtRows + tid);
        };
        bool failed = false;
        int item = 0;
        uint32_t tables = 0u;  // bit 0: which of the two tables comes next, bit 1: rows of the last one add nothing
        for (bool more = any; !failed && more; more = w.next(p)) {
            float mine = entry(0);
            for (int k = w.k0; !failed && k < w.k1; ++k) {
                const int key = k * kWtKeys + rank * kWtHalf + 32 * quad + lane;
                const int i_page = (k * kWtKeys + rank * kWtHalf + 32 * quad) / kPage;
                const bool valid = (key % kPage) < page_rows(p.bp, w.s, i_page, page_of(p.bp, w.b, w.s, i_page));
                float* dst = p.out + static_cast<int64_t>(w.b) * width + key;
                float before = 0.f;
                if (half == 0 && key < w.s.len && p.prev) before = p.decay * p.prev[static_cast<int64_t>(w.b) * width + key];
                const bool tail = k * kWtKeys + rank * kWtHalf + 32 * quad + 32 > w.s.len;  // drafted rows among the warp's keys
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                for (int i = 0; i < w.row_tiles; ++i, ++item) {
                    if (w.row_tiles > 1 || k == w.k0) {  // the row tile's table, the next one's entry on its way
                        const bool nothing = mine == CUDART_INF_F;
                        reinterpret_cast<volatile float*>(smem + L::kOffLse)[(tables & 1u) * kWtRows + tid] = mine;
                        tables = (tables & 1u) ^ 1u;
                        if (w.row_tiles > 1) mine = entry(i + 1 < w.row_tiles ? i + 1 : 0);
                        if (ptx::named_bar_red_or(1u, 32u * kWtSumWarps, failed || nothing)) {
                            tables |= 2u;
                            failed = ptx::named_bar_red_or(1u, 32u * kWtSumWarps, failed);
                        }
                        if (failed) break;
                    }
                    const uint32_t table = s_lse + (~tables & 1u) * kWtRows * 4;
                    const int buf = item & 1;
                    const int columns = w.columns(p, i) / 2, c_first = half * columns;
                    const int limit = min(w.rows(p, i) - c_first, columns);  // this half's columns that are rows
                    if (!failed && !warp_wait(kWbSFull + buf, (item >> 1) & 1)) failed = true;
                    if (failed) continue;
                    ptx::tc_fence_after();
                    // 16 columns at a time, the next ones' logits on their way
                    const uint32_t s_at = tmem + lane_base + buf * kWtRows + c_first;
                    auto add = [&](const uint32_t* sv, int c0) {
                        float pr[16];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint4 nl = ptx::ld_shared_v4(table + (c_first + c0 + 4 * e) * 4);
                            const float2 y0 = ptx::mul2(ptx::fma2(make_float2(__uint_as_float(sv[4 * e]), __uint_as_float(sv[4 * e + 1])), scale2,
                                                                  make_float2(__uint_as_float(nl.x), __uint_as_float(nl.y))), log2e2);
                            const float2 y1 = ptx::mul2(ptx::fma2(make_float2(__uint_as_float(sv[4 * e + 2]), __uint_as_float(sv[4 * e + 3])), scale2,
                                                                  make_float2(__uint_as_float(nl.z), __uint_as_float(nl.w))), log2e2);
                            pr[4 * e] = ptx::ex2_approx(y0.x);
                            pr[4 * e + 1] = ptx::ex2_approx(y0.y);
                            pr[4 * e + 2] = ptx::ex2_approx(y1.x);
                            pr[4 * e + 3] = ptx::ex2_approx(y1.y);
                        }
                        if (tail || (tables & 2u) || c0 + 16 > limit) {
                            // lane l < 16: which of the warp's 32 keys column c0 + l sees
                            uint32_t seen = 0u;
                            if (lane < 16 && c0 + lane < limit && ptx::ld_shared_f32(table + (c_first + c0 + lane) * 4) != CUDART_INF_F)
                                seen = seen_bits(p.bp, w.s, (i * kWtRows + c_first + c0 + lane) / p.bp.h, key - lane);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (!((__shfl_sync(0xffffffffu, seen, e) >> lane) & 1u)) pr[e] = 0.f;
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[e & 1] = ptx::add2(acc[e & 1], make_float2(pr[2 * e], pr[2 * e + 1]));
                    };
                    uint32_t sv0[16], sv1[16];
                    if (!few) {
                        if (limit > 0) SMLA_TMEM_LD16(s_at, sv0);
#pragma unroll 1
                        for (int c0 = 0; c0 < limit; c0 += 32) {
                            ptx::tmem_wait_ld16(sv0);
                            if (c0 + 16 < limit) SMLA_TMEM_LD16(s_at + c0 + 16, sv1);
                            add(sv0, c0);
                            if (c0 + 16 < limit) {
                                ptx::tmem_wait_ld16(sv1);
                                if (c0 + 32 < limit) SMLA_TMEM_LD16(s_at + c0 + 32, sv0);
                                add(sv1, c0 + 16);
                            }
                        }
                    } else {  // the two issuers' accumulators
#pragma unroll 1
                        for (int c0 = 0; c0 < limit; c0 += 16) {
                            SMLA_TMEM_LD16(s_at + c0, sv0);
                            SMLA_TMEM_LD16(s_at + kWtRowsFew + c0, sv1);
                            ptx::tmem_wait_ld16(sv0);
                            ptx::tmem_wait_ld16(sv1);
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float2 y = ptx::add2(make_float2(__uint_as_float(sv0[e]), __uint_as_float(sv0[e + 1])),
                                                           make_float2(__uint_as_float(sv1[e]), __uint_as_float(sv1[e + 1])));
                                sv0[e] = __float_as_uint(y.x);
                                sv0[e + 1] = __float_as_uint(y.y);
                            }
                            add(sv0, c0);
                        }
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster(buf ? s_empty1 : s_empty0);
                }
                const float sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                if (half == 1) sX[32 * quad + lane] = sum;
                failed = ptx::named_bar_red_or(1u, 32u * kWtSumWarps, failed);
                const float other = sX[32 * quad + lane];
                if (w.row_tiles == 1) ptx::named_bar_sync(1u, 32u * kWtSumWarps);  // (else the next table's barrier comes before the next sum)
                if (!failed && half == 0 && key < w.s.keys) *dst = before + (valid ? sum + other : 0.f);
            }
        }
    }
    // ---- both CTAs are done with each other's shared memory, barriers and TMEM
    ptx::tc_fence_before();
    __syncwarp();
    ptx::cluster_sync();
    if (warp == kWtMmaWarp) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, 512);
    }
}

}  // namespace smla
