// A batch of sequences over the paged cache, each with its own block table, cached rows and drafted
// tokens: what the tree attention and the gathered weights read alike.  Everything that says how much work
// there is (lengths, starts) lives on the device, so that one captured call serves a growing batch; the
// kernels cut their work themselves.
#pragma once

#include "sparse_mla_common.cuh"

namespace smla {

constexpr int kPage = 64;                   // rows per page
constexpr int kMaxBlocks = (1 << 25) - 256;  // pages of a sequence: positions, and 16000 past them (a loop's step), fit 31 bits

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
// (The loads below may be moved by the compiler, so b is a number from behind the kernel's wait for the one before.)
struct Seq {
    int first, n;   // tokens [first, first + n)
    int len, keys;  // cached rows, and with the drafted ones
};

__device__ __forceinline__ Seq load_seq(const BatchParams& p, int b) {
    Seq s;
    s.first = min(max(ptx::ld_from(p.starts + b), 0), p.T);
    s.n = min(max(ptx::ld_from(p.starts + b + 1), s.first), p.T) - s.first;
    const int most = p.nb * kPage;
    s.len = min(max(ptx::ld_from(p.lengths + b), 0), most);
    s.keys = static_cast<int>(min(static_cast<int64_t>(s.len) + s.n, static_cast<int64_t>(most)));
    return s;
}

__device__ __forceinline__ int page_of(const BatchParams& p, int b, const Seq& s, int i) {  // -1 past the end
    return i * kPage < s.keys ? ptx::ld_from(p.tables + static_cast<int64_t>(b) * p.nb + i) : -1;
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
    if (j < 0) return (ptx::ld_from(m) << -j) | ((1u << -j) - 1u);
    const int w = j >> 5;
    const uint32_t lo = w < p.words ? ptx::ld_from(m + w) : 0u, hi = w + 1 < p.words ? ptx::ld_from(m + w + 1) : 0u;
    return __funnelshift_r(lo, hi, j & 31);
}

// The first `n` of 32 bits (n may lie outside 0 .. 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// Sums of two values over the CTA's threads: of the threads before this one, and of all.  `scratch` holds two
// values for every warp, written only before the barrier and read only after it.
__device__ __forceinline__ void block_prefix2(int64_t x, int64_t y, int64_t* scratch, int warps, int64_t& x_before, int64_t& x_all,
                                              int64_t& y_before, int64_t& y_all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t xi = x, yi = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t xo = __shfl_up_sync(0xffffffffu, xi, o), yo = __shfl_up_sync(0xffffffffu, yi, o);
        if (lane >= o) {
            xi += xo;
            yi += yo;
        }
    }
    if (lane == 31) {
        scratch[2 * warp] = xi;
        scratch[2 * warp + 1] = yi;
    }
    __syncthreads();
    x_before = xi - x;
    y_before = yi - y;
    x_all = y_all = 0;
#pragma unroll 4
    for (int w = 0; w < warps; ++w) {
        const longlong2 v = *reinterpret_cast<const longlong2*>(scratch + 2 * w);
        if (w < warp) {
            x_before += v.x;
            y_before += v.y;
        }
        x_all += v.x;
        y_all += v.y;
    }
}

// x * k / n, in 32 bits where they do (k <= n < 2^16)
__device__ __forceinline__ int64_t share_of(int64_t x, int k, int n) {
    if (x < (1 << 16)) return static_cast<uint32_t>(x) * static_cast<uint32_t>(k) / static_cast<uint32_t>(n);
    return x * k / n;
}

}  // namespace smla
