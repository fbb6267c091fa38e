// Eviction from the paged cache by gathered attention weight (sm_103a).
//
// A sequence of n rows keeps its first `sinks` and last `recent` ones and, of the rest, those with the
// largest weights, `budget` rows in all, ties to the lower position; the kept rows are copied, in order, into
// pages of the sequence's new table, and their weights go with them.  The pages that it leaves are read
// only (another sequence may share them), so that nothing here depends on the order of reads and writes.
//
// Selection: a cluster of one to eight CTAs per sequence, equal shares of its positions.  A radix select on an
// order-preserving key in four digits (9, 8, 8 and 7 bits): each CTA counts its keys' digits in shared
// memory, and every CTA adds up the cluster's histograms through distributed shared memory (2 KB from each; three
// digits of 2048 bins spent 15 us apiece on it at 32 sequences).  The keys stay in registers while a CTA's
// share is at most 8192.  Then the counts above and at the threshold go round, and
// ballots over 32 consecutive positions place the kept ones in order.
//
// Copy: 2 * 1152 (or 656) bytes a row and nothing else, bound by HBM; a warp takes four rows (eight of the
// shorter ones) with all its 16-byte loads in flight, and looks up the next ones' places under them.  Sinks and recent
// rows are copied while the selection runs (32 sequences x 16384 rows cut to 4096, 512 of them recent: 66.5 -> 63.7 us in
// all, 128 x 8191 fp8 to 2001: 74 -> 71.8; the copy's 47 us of the first are 5.6 TB/s).
#pragma once

#include "sparse_mla_batch.cuh"
#include "sparse_mla_topk.cuh"

namespace smla {

constexpr int kEvMaxCluster = 8;
constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvPerLane = 16;                             // positions a lane per step
constexpr int kEvStep = kEvThreads * kEvPerLane;           // positions a CTA per step
constexpr int kEvBins = 512;
constexpr int kEvCopyThreads = 256;

struct EvParams {
    const int32_t* tables;      // [B, nb]
    const int32_t* lengths;     // [B]
    const float* weights;       // [B, nb * 64]
    const int32_t* new_tables;  // [B, new_nb]
    int32_t* kept;              // [B, budget]
    int32_t* new_lengths;       // [B]
    float* new_weights;         // [B, new_nb * 64]
    void* cache;
    int64_t num_slots;
    int32_t B, nb, new_nb, budget, sinks, recent;
    int32_t cluster;            // CTAs per sequence
};

template <int KVF>
__host__ __device__ constexpr int evict_copy_rows() {  // a warp's at a time
    return KVF ? 8 : 4;
}

// Order-preserving key; NaN ranks below everything.
__device__ __forceinline__ uint32_t weight_key(float x) { return x != x ? 0u : score_key(x); }

__global__ void __launch_bounds__(kEvThreads) sparse_mla_evict_select_kernel(const EvParams p) {
    __shared__ __align__(16) uint32_t s_hist[2][kEvBins];
    __shared__ uint32_t s_warp[kEvWarps], s_warp2[kEvWarps];
    __shared__ uint32_t s_sel[3];
    __shared__ uint32_t s_count[2];  // keys above the threshold (and rows kept in any case), keys at it
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    const int cluster = p.cluster;
    const int b = static_cast<int>(blockIdx.x) / cluster;
    auto sync = [&]() {
        if (cluster > 1) ptx::cluster_sync();
        else __syncthreads();
    };
    const int width = p.nb * kPage, new_width = p.new_nb * kPage;
    const float* w = p.weights + static_cast<int64_t>(b) * width;
    int32_t* kept = p.kept + static_cast<int64_t>(b) * p.budget;
    float* new_w = p.new_weights + static_cast<int64_t>(b) * new_width;
    const int n = min(max(ptx::ld(p.lengths + b), 0), width);
    const int k = min(n, p.budget);
    if (rank == 0 && tid == 0) p.new_lengths[b] = k;
    for (int i = k + rank * kEvThreads + tid; i < p.budget; i += cluster * kEvThreads) kept[i] = -1;
    for (int i = k + rank * kEvThreads + tid; i < new_width; i += cluster * kEvThreads) new_w[i] = 0.f;
    if (n <= p.budget) {  // uniform across the cluster
        for (int i = rank * kEvThreads + tid; i < n; i += cluster * kEvThreads) {
            kept[i] = i;
            new_w[i] = ptx::ld(w + i);
        }
        return;
    }
    // budget < n, so that sinks + recent <= budget < n
    const int mid0 = p.sinks, mid1 = n - p.recent;
    uint32_t need = static_cast<uint32_t>(p.budget - p.sinks - p.recent);  // of [mid0, mid1)
    const int share = ((n + cluster - 1) / cluster + 31) & ~31;
    const int seg0 = min(rank * share, n), seg1 = min(seg0 + share, n);
    // a CTA's step: warp's positions c + 512 warp + 32 e + lane
    auto load = [&](int c, float (&x)[kEvPerLane]) {
#pragma unroll
        for (int e = 0; e < kEvPerLane; ++e) {
            const int i = c + kEvPerLane * 32 * warp + 32 * e + lane;
            x[e] = i < seg1 ? ptx::ld(w + i) : 0.f;
        }
    };
    float x[kEvPerLane];
    const bool held = seg1 - seg0 <= kEvStep;
    if (held) load(seg0, x);
    // ---- the threshold key, digit by digit
    uint32_t prefix = 0u, pmask = 0u;
    if (need > 0u) {
#pragma unroll 1
        for (int d = 0; d < 4; ++d) {
            const int shift = d == 0 ? 23 : d == 1 ? 15 : d == 2 ? 7 : 0;
            const uint32_t digit = d == 0 ? 0x1ffu : d == 3 ? 0x7fu : 0xffu;
            uint32_t* hist = s_hist[d & 1];
            hist[tid] = 0u;
            __syncthreads();
            for (int c = seg0; c < seg1; c += kEvStep) {
                if (!held) load(c, x);
#pragma unroll
                for (int e = 0; e < kEvPerLane; ++e) {
                    const int i = c + kEvPerLane * 32 * warp + 32 * e + lane;
                    const uint32_t key = weight_key(x[e]);
                    if (i >= mid0 && i < mid1 && i < seg1 && (key & pmask) == prefix) atomicAdd(&hist[(key >> shift) & digit], 1u);
                }
            }
            sync();  // (the other buffer's readers of two digits ago are done, too)
            // bins 4 j .. 4 j + 3, from the top: thread tid < 128 has j = 127 - tid
            if (warp < kEvBins / 128) {
                const uint32_t at = ptx::smem_u32(hist + kEvBins - 4 - 4 * tid);
                uint32_t c4[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int r = 0; r < kEvMaxCluster; ++r) {
                    if (r < cluster) {
                        const float4 v = ptx::ld_shared_cluster_v4(ptx::map_shared_rank(at, r));
                        c4[0] += __float_as_uint(v.x);
                        c4[1] += __float_as_uint(v.y);
                        c4[2] += __float_as_uint(v.z);
                        c4[3] += __float_as_uint(v.w);
                    }
                }
                const uint32_t mine = c4[0] + c4[1] + c4[2] + c4[3];
                uint32_t incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                if (lane == 31) s_warp[warp] = incl;
                ptx::named_bar_sync(1u, kEvBins / 4);
                uint32_t above = incl - mine;
#pragma unroll
                for (int q = 0; q < kEvBins / 128; ++q)
                    if (q < warp) above += s_warp[q];
                if (above < need && need <= above + mine) {
#pragma unroll
                    for (int j = 3; j >= 0; --j) {
                        if (above < need && need <= above + c4[j]) {
                            s_sel[0] = static_cast<uint32_t>(kEvBins - 4 - 4 * tid + j);
                            s_sel[1] = above;
                            s_sel[2] = c4[j];
                        }
                        above += c4[j];
                    }
                }
            }
            __syncthreads();
            prefix |= s_sel[0] << shift;
            pmask |= digit << shift;
            need -= s_sel[1];
            if (s_sel[2] == need) break;  // every key with this prefix is kept: the digits below do not matter
            // (s_sel and s_warp are written again after the next digit's barriers)
        }
    }
    // ---- what every position is: 2 kept in any case, 1 at the threshold
    auto kind = [&](int i, float x) -> int {
        if (i >= seg1) return 0;
        if (i < mid0 || i >= mid1) return 2;
        if (pmask == 0u) return 0;  // nothing of the middle
        const uint32_t key = weight_key(x) & pmask;
        return key > prefix ? 2 : key == prefix ? 1 : 0;
    };
    uint32_t over = 0u, equal = 0u;
    for (int c = seg0; c < seg1; c += kEvStep) {
        if (!held) load(c, x);
#pragma unroll
        for (int e = 0; e < kEvPerLane; ++e) {
            const int t = kind(c + kEvPerLane * 32 * warp + 32 * e + lane, x[e]);
            over += t == 2;
            equal += t == 1;
        }
    }
    over = __reduce_add_sync(0xffffffffu, over);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        s_warp[warp] = over;
        s_warp2[warp] = equal;
    }
    __syncthreads();
    if (tid < 2) {
        uint32_t sum = 0u;
        for (int q = 0; q < kEvWarps; ++q) sum += tid ? s_warp2[q] : s_warp[q];
        s_count[tid] = sum;
    }
    sync();
    uint32_t base_over = 0u, base_equal = 0u;
    for (int r = 0; r < rank; ++r) {
        base_over += __float_as_uint(ptx::ld_shared_cluster_f32(ptx::map_shared_rank(ptx::smem_u32(&s_count[0]), r)));
        base_equal += __float_as_uint(ptx::ld_shared_cluster_f32(ptx::map_shared_rank(ptx::smem_u32(&s_count[1]), r)));
    }
    // ---- the kept positions in order
    for (int c = seg0; c < seg1; c += kEvStep) {
        if (!held) load(c, x);
        uint32_t two = 0u, one = 0u;  // bit e: position e of the lane
        uint32_t wo = 0u, we = 0u;
#pragma unroll
        for (int e = 0; e < kEvPerLane; ++e) {
            const int t = kind(c + kEvPerLane * 32 * warp + 32 * e + lane, x[e]);
            two |= static_cast<uint32_t>(t == 2) << e;
            one |= static_cast<uint32_t>(t == 1) << e;
            wo += t == 2;
            we += t == 1;
        }
        wo = __reduce_add_sync(0xffffffffu, wo);
        we = __reduce_add_sync(0xffffffffu, we);
        __syncthreads();  // the last step's sums are read
        if (lane == 0) {
            s_warp[warp] = wo;
            s_warp2[warp] = we;
        }
        __syncthreads();
        uint32_t before_over = base_over, before_equal = base_equal;
#pragma unroll
        for (int q = 0; q < kEvWarps; ++q) {
            if (q < warp) {
                before_over += s_warp[q];
                before_equal += s_warp2[q];
            }
            base_over += s_warp[q];
            base_equal += s_warp2[q];
        }
        const uint32_t lower = (1u << lane) - 1u;
#pragma unroll
        for (int e = 0; e < kEvPerLane; ++e) {
            const uint32_t m2 = __ballot_sync(0xffffffffu, (two >> e) & 1u), m1 = __ballot_sync(0xffffffffu, (one >> e) & 1u);
            const uint32_t o = before_over + __popc(m2 & lower), q = before_equal + __popc(m1 & lower);
            if (((two >> e) & 1u) || (((one >> e) & 1u) && q < need)) {
                const uint32_t place = o + min(q, need);
                if (place < static_cast<uint32_t>(k)) {  // always; the check keeps every store in the row
                    kept[place] = c + kEvPerLane * 32 * warp + 32 * e + lane;
                    new_w[place] = x[e];
                }
            }
            before_over += __popc(m2);
            before_equal += __popc(m1);
        }
    }
    sync();  // the others' reads of this CTA's counts are done
}

// Rows kept[b][i] of the old tables into rows i of the new ones.  Starts beside the selection, which has seen everything
// before it done when it lets its dependents start.
template <int KVF>
__global__ void __launch_bounds__(kEvCopyThreads, 3) sparse_mla_evict_copy_kernel(const EvParams p) {
    constexpr int kChunks = KVF ? kFp8RowBytes / 16 : kDQK * 2 / 16;  // 16-byte chunks of a row: 41 or 72
    constexpr int kRows = evict_copy_rows<KVF>();
    constexpr int kLoads = (kChunks * kRows + 31) / 32;
    ptx::grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    char* cache = static_cast<char*>(p.cache);
    const int always = p.sinks + p.recent;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kEvCopyThreads / 32);
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kEvCopyThreads + threadIdx.x) >> 5;
#pragma unroll 1
    for (int phase = 0; phase < 2; ++phase) {
        // New positions i: first those whose rows are known without the selection, the sinks and the recent ones; then the
        // others', from the list.
        if (phase == 1) ptx::grid_dependency_wait();
        const int count = phase == 0 ? always : p.budget - always;
        const int groups = (count + kRows - 1) / kRows;
        const int64_t all = static_cast<int64_t>(groups) * p.B;
        // lane u < kRows: where row u of group g comes from and goes to
        auto places = [&](int64_t g, int64_t& from, int64_t& to) {
            from = to = -1;
            if (g >= all || lane >= kRows) return;
            const int b = static_cast<int>(g / groups), j = static_cast<int>(g % groups) * kRows + lane;
            if (j >= count) return;
            int i = p.sinks + j, pos;
            if (phase == 0) {
                const int n = min(max(ptx::ld(p.lengths + b), 0), p.nb * kPage);
                i = j < p.sinks ? j : p.budget - always + j;
                pos = n <= p.budget ? (i < n ? i : -1) : j < p.sinks ? i : n - p.budget + i;
            } else {
                // written since this kernel began, perhaps beside lengths or tables that the first phase has brought into L1
                pos = ptx::ld_gpu_s32(p.kept + static_cast<int64_t>(b) * p.budget + i);
            }
            if (pos < 0) return;
            const int old_page = ptx::ld(p.tables + static_cast<int64_t>(b) * p.nb + pos / kPage);
            const int new_page = ptx::ld(p.new_tables + static_cast<int64_t>(b) * p.new_nb + i / kPage);
            from = static_cast<int64_t>(old_page) * kPage + pos % kPage;
            to = static_cast<int64_t>(new_page) * kPage + i % kPage;
            if (from < 0 || from >= p.num_slots || to < 0 || to >= p.num_slots) {
                atomicOr(&g_smla_error, kErrRowRange);
                to = -1;
            }
        };
        int64_t from, to;
        places(first, from, to);
        for (int64_t g = first; g < all; g += step) {
            uint4 v[kLoads];
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int c = lane + 32 * j, u = c / kChunks;
                const int64_t f = __shfl_sync(0xffffffffu, from, u & 31), t = __shfl_sync(0xffffffffu, to, u & 31);
                if (u < kRows && t >= 0) v[j] = ptx::ld_v4(cache + f * (kChunks * 16) + (c - u * kChunks) * 16);
            }
            const int64_t dst = to;
            places(g + step, from, to);
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int c = lane + 32 * j, u = c / kChunks;
                const int64_t t = __shfl_sync(0xffffffffu, dst, u & 31);
                if (u < kRows && t >= 0) *reinterpret_cast<uint4*>(cache + t * (kChunks * 16) + (c - u * kChunks) * 16) = v[j];
            }
        }
    }
}

}  // namespace smla
