// A batch of sequences over the paged cache, each with its own block table, cached rows and drafted
// tokens: what the tree attention and the gathered weights read alike.  Everything that says how much work
// there is (lengths, starts) lives on the device, so that one captured call serves a growing batch; the
// kernels cut their work themselves.
#pragma once

#include "sparse_mla_common.cuh"

namespace smla {

constexpr int kPage = 64;                   // rows per page
constexpr int kMaxBlocks = (1 << 25) - 8;   // pages of a sequence: positions, and some past them, fit 31 bits

struct BatchParams {
    const void* kv;           // the cache
    const int32_t* tables;    // [B, nb]: position i of sequence b is slot tables[b][i / 64] * 64 + i % 64
    const int32_t* lengths;   // [B]: cached rows before the drafted ones
    const int32_t* starts;    // [B + 1]: sequence b's tokens are starts[b] .. starts[b + 1] - 1
    const uint32_t* mask;     // [T, words]: bit j of a token's words: it sees drafted token j; nullptr: a chain
    int64_t num_slots;
    int32_t B, nb, words, T, h;
};

// One sequence, its numbers brought into range: whatever the arrays hold, tokens stay inside [0, T) and
// positions inside the block table.
struct Seq {
    int first, n;   // tokens [first, first + n)
    int len, keys;  // cached rows, and with the drafted ones
};

__device__ __forceinline__ Seq load_seq(const BatchParams& p, int b) {
    Seq s;
    s.first = min(max(__ldg(p.starts + b), 0), p.T);
    s.n = min(max(__ldg(p.starts + b + 1), s.first), p.T) - s.first;
    const int most = p.nb * kPage;
    s.len = min(max(__ldg(p.lengths + b), 0), most);
    s.keys = static_cast<int>(min(static_cast<int64_t>(s.len) + s.n, static_cast<int64_t>(most)));
    return s;
}

__device__ __forceinline__ int page_of(const BatchParams& p, int b, const Seq& s, int i) {  // -1 past the end
    return i * kPage < s.keys ? __ldg(p.tables + static_cast<int64_t>(b) * p.nb + i) : -1;
}

__device__ __forceinline__ bool page_in_cache(const BatchParams& p, int page) {
    return page >= 0 && static_cast<int64_t>(page) * kPage < p.num_slots;
}

// Rows of page i that take part (0 .. 64), given its page number.
__device__ __forceinline__ int page_rows(const BatchParams& p, const Seq& s, int i, int page) {
    if (!page_in_cache(p, page)) return 0;
    const int64_t room = p.num_slots - static_cast<int64_t>(page) * kPage;
    const int left = s.keys - i * kPage;
    return static_cast<int>(min(static_cast<int64_t>(min(left, kPage)), room));
}

// Which of the 32 keys from position `key` on token i of the sequence sees (bit k: key + k), as far as the
// tree goes: all cached rows, of the drafted ones those of its mask, or in a chain those up to itself.
__device__ __forceinline__ uint32_t seen_bits(const BatchParams& p, const Seq& s, int i, int key) {
    const int j = key - s.len;  // drafted token at the first key
    if (j <= -32) return 0xffffffffu;
    if (p.mask == nullptr) {
        const int c = i + 1 - j;
        return c >= 32 ? 0xffffffffu : c <= 0 ? 0u : (1u << c) - 1u;
    }
    const uint32_t* m = p.mask + static_cast<int64_t>(s.first + i) * p.words;
    if (j < 0) return (__ldg(m) << -j) | ((1u << -j) - 1u);
    const int w = j >> 5;
    const uint32_t lo = w < p.words ? __ldg(m + w) : 0u, hi = w + 1 < p.words ? __ldg(m + w + 1) : 0u;
    return __funnelshift_r(lo, hi, j & 31);
}

// The first `n` of 32 bits (n may lie outside 0 .. 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// Sums over the CTA's threads (at most 32 warps): of the threads before this one, and of all.  `scratch`
// holds 32 values, written only before the barrier and read only after it.
__device__ __forceinline__ void block_prefix(int64_t x, int64_t* scratch, int warps, int64_t& before, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    before = incl - x;
    total = 0;
    for (int w = 0; w < warps; ++w) {
        const int64_t v = scratch[w];
        if (w < warp) before += v;
        total += v;
    }
}

// Four fp8 rows on their way to bf16 rows of 1152 bytes: the loads, and, later, codes x scale in fp32 rounded to
// bf16 as in the forward, and the stores.  `n` of the four take part (0 .. 4), the others become zeros.
struct Fp8Rows4 {
    // lane l: codes [8l, 8l + 8) and [256 + 8l, 256 + 8l + 8), so that both stores are 512 contiguous bytes
    uint2 a[4], b[4];
    float sa[4], sb[4];
    uint32_t rope[4];
    __device__ __forceinline__ void load(const uint8_t* src, int n) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            a[u] = b[u] = make_uint2(0u, 0u);
            sa[u] = sb[u] = 0.f;
            rope[u] = 0u;
            if (u < n) {
                const uint8_t* row = src + u * kFp8RowBytes;
                a[u] = __ldg(reinterpret_cast<const uint2*>(row) + lane);
                b[u] = __ldg(reinterpret_cast<const uint2*>(row) + 32 + lane);
                sa[u] = __ldg(reinterpret_cast<const float*>(row + 512) + (lane >> 4));
                sb[u] = __ldg(reinterpret_cast<const float*>(row + 520) + (lane >> 4));
                rope[u] = __ldg(reinterpret_cast<const uint32_t*>(row + 528) + lane);
            }
        }
    }
    __device__ __forceinline__ void store(__nv_bfloat16* dst) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint4* out = reinterpret_cast<uint4*>(dst + u * kDQK);
            out[lane] = make_uint4(ptx::e4m3x2_scaled_bf16x2(a[u].x & 0xFFFFu, sa[u]), ptx::e4m3x2_scaled_bf16x2(a[u].x >> 16, sa[u]),
                                   ptx::e4m3x2_scaled_bf16x2(a[u].y & 0xFFFFu, sa[u]), ptx::e4m3x2_scaled_bf16x2(a[u].y >> 16, sa[u]));
            out[32 + lane] = make_uint4(ptx::e4m3x2_scaled_bf16x2(b[u].x & 0xFFFFu, sb[u]), ptx::e4m3x2_scaled_bf16x2(b[u].x >> 16, sb[u]),
                                        ptx::e4m3x2_scaled_bf16x2(b[u].y & 0xFFFFu, sb[u]), ptx::e4m3x2_scaled_bf16x2(b[u].y >> 16, sb[u]));
            reinterpret_cast<uint32_t*>(out + 64)[lane] = rope[u];
        }
    }
};

// A warp's `rows` consecutive rows of page i of a sequence, from `row` on, and how many of them take part.
struct Fp8Source {
    const uint8_t* src;
    int n;
    __device__ __forceinline__ Fp8Source(const BatchParams& p, const Seq& s, int i, int page, int row)
        : src(static_cast<const uint8_t*>(p.kv) + (static_cast<int64_t>(page) * kPage + row) * kFp8RowBytes), n(page_rows(p, s, i, page) - row) {}
    __device__ __forceinline__ void prefetch(int rows) const {  // into L2
        if (n > 0 && (threadIdx.x & 31) == 0) ptx::bulk_prefetch_l2(src, static_cast<uint32_t>(min(n, rows) * kFp8RowBytes));
    }
    __device__ __forceinline__ void load(Fp8Rows4& r, int u) const { r.load(src + u * kFp8RowBytes, n - u); }
};

}  // namespace smla
