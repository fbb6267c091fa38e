// Appending rows to the paged latent cache: the latent (optionally through its RMS norm), the
// rotated part turned by its position, and both packed as the rows that the forward kernels read.
//
// For token t with input row [c (512) | k (64)], position pos and slot s:
//
//   n      = c * rsqrt(mean(c^2) + eps) * w        (or c itself without norm weights)
//   k'     = the 32 pairs of k turned by the angles of row pos of the cos/sin table:
//            (a, b) -> (a cos - b sin, b cos + a sin), pairs (2i, 2i + 1) or (i, i + 32)
//   bf16   row s = [bf16(n) | bf16(k')]
//   fp8    row s = [e4m3(n / scale) | 4 x fp32 scale | bf16(k')], per 128 latent values
//          scale = max|n| / 448 (1 for a tile of zeros), round to nearest even, saturated
//
// All arithmetic is fp32 and every value is rounded once, when it is stored.  A NaN in a tile is
// carried into its scale, so the tile reads back as NaN rather than as a finite value.
//
// A stream over HBM: 1152 bytes in and 1152 (656) out per token, nothing reused, so one warp per
// token keeps a row in registers and needs no shared memory.  Lane l holds word l of the rotated
// part (and words l and 32 + l of the table row) and 16 latent values: for
// bf16 rows dims [8l, 8l + 8) and [256 + 8l, 256 + 8l + 8), so that each 16-byte instruction covers
// 512 contiguous bytes of the row; for fp8 rows dims [16l, 16l + 16), so that a scale tile is 8
// neighbouring lanes and the codes leave as one 512-byte store.
#pragma once

#include "sparse_mla_common.cuh"

namespace smla {

constexpr int kAppendThreads = 128;  // four tokens per CTA: 32 decode tokens spread over 8 SMs

struct AppendParams {
    const __nv_bfloat16* kv;      // [T] rows of 576, `kv_stride` elements apart
    const int32_t* positions;     // [T]
    const int32_t* slots;         // [T]
    const float* cos_sin;         // [max_pos][64]: 32 cos, 32 sin
    const __nv_bfloat16* norm_w;  // [512] or nullptr
    void* cache;                  // [num_slots] rows
    int64_t kv_stride;
    int64_t num_slots;
    int32_t T;
    int32_t max_pos;
    float eps;
    int32_t interleaved;
};

// two fp32 values as an e4m3 pair (lo in the low byte), nearest even, saturated to +-448
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4 v, float* x) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// A 64-wide rotated part is held by a warp as word `lane` (two neighbouring values) of it and word
// `lane` of the cosines and of the sines.  Interleaved, a lane's two values are its pair.  Otherwise
// the partner of values 2l and 2l + 1 sits 16 lanes away and the angles of both lanes' values are
// words 2 (l % 16) and 2 (l % 16) + 1, fetched by shuffles: two-byte loads and stores of the halves
// would cost four times the memory instructions.  The whole warp calls it.  Products and sum are
// fp32, the result is rounded to bf16 once.
__device__ __forceinline__ uint32_t turn_pair(uint32_t pair, float cs, float sn, int lane, bool interleaved) {
    const float a = __uint_as_float(pair << 16), b = __uint_as_float(pair & 0xFFFF0000u);
    if (interleaved) return pack_bf16x2(a * cs - b * sn, b * cs + a * sn);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, pair, 16);
    const int l = 2 * (lane & 15);
    const float c0 = __shfl_sync(0xffffffffu, cs, l), c1 = __shfl_sync(0xffffffffu, cs, l + 1);
    float s0 = __shfl_sync(0xffffffffu, sn, l), s1 = __shfl_sync(0xffffffffu, sn, l + 1);
    if (lane < 16) {
        s0 = -s0;
        s1 = -s1;
    }
    return pack_bf16x2(a * c0 + __uint_as_float(other << 16) * s0, b * c1 + __uint_as_float(other & 0xFFFF0000u) * s1);
}

// KVF: 0 = bf16 rows, 1 = fp8 rows
template <int KVF>
__global__ void __launch_bounds__(kAppendThreads) sparse_mla_append_kernel(const AppendParams p) {
    // launched as a programmatic dependent: nothing before this touches global memory
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x) >> 5;
    if (t >= p.T) return;
    // the loads of the row and of the norm's weights need neither the slot nor the position: all are in
    // flight together (volatile, so that none sinks behind the checks: 4096 tokens to fp8 3.8 us with the
    // weights asked for there, 3.45 here; past L1, where every warp asks L2 for the same lines, 9.9)
    const __nv_bfloat16* src = p.kv + t * p.kv_stride;
    const uint4* src16 = reinterpret_cast<const uint4*>(src);
    const int c0 = KVF == 0 ? lane : 2 * lane;       // this lane's 16-byte chunks of the latent
    const int c1 = KVF == 0 ? 32 + lane : 2 * lane + 1;
    const uint4 v0 = ptx::ld_nc_v4(src16 + c0);
    const uint4 v1 = ptx::ld_nc_v4(src16 + c1);
    const uint32_t pair = __float_as_uint(ptx::ld_nc_f32(src + kDV + 2 * lane));
    uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
    if (p.norm_w != nullptr) {
        w0 = ptx::ld_nc_l1_v4(reinterpret_cast<const uint4*>(p.norm_w) + c0);
        w1 = ptx::ld_nc_l1_v4(reinterpret_cast<const uint4*>(p.norm_w) + c1);
    }
    const int slot = __ldg(p.slots + t);
    const int pos = __ldg(p.positions + t);
    if (slot == -1) return;  // an unused place of a padded batch
    if (slot < 0 || static_cast<int64_t>(slot) >= p.num_slots || pos < 0 || pos >= p.max_pos) {
        if (lane == 0) atomicOr(&g_smla_error, kErrRowRange);
        return;  // nothing is written for this token; the next status read says so
    }
    const float* cs = p.cos_sin + static_cast<int64_t>(pos) * 64;
    const float cosv = __ldg(cs + lane), sinv = __ldg(cs + 32 + lane);

    float x[16];
    unpack_bf16x8(v0, x);
    unpack_bf16x8(v1, x + 8);
    if (p.norm_w != nullptr) {
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sq = fmaf(x[i], x[i], sq);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        const float r = rsqrtf(sq * (1.0f / kDV) + p.eps);
        float w[16];
        unpack_bf16x8(w0, w);
        unpack_bf16x8(w1, w + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
    }
    const uint32_t turned = turn_pair(pair, cosv, sinv, lane, p.interleaved != 0);
    if constexpr (KVF == 0) {
        __nv_bfloat16* row = static_cast<__nv_bfloat16*>(p.cache) + static_cast<int64_t>(slot) * kDQK;
        uint4* row16 = reinterpret_cast<uint4*>(row);
        row16[c0] = pack_bf16x8(x);
        row16[c1] = pack_bf16x8(x + 8);
        reinterpret_cast<uint32_t*>(row + kDV)[lane] = turned;
    } else {
        float amax = fabsf(x[0]);
#pragma unroll
        for (int i = 1; i < 16; ++i) amax = ptx::max_nan(amax, fabsf(x[i]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) amax = ptx::max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float scale = __fdiv_rn(amax, 448.f);
        if (scale == 0.f) scale = 1.f;  // a tile of zeros (or of values too small for a scale): codes 0
        // code = e4m3(x / scale), the quotient rounded to fp32 first, by Markstein's correction: with y = 1/b
        // correctly rounded, q = a y (off by two units at most) and r = a - b q in an fma, q + r y is a / b to
        // 2^-45 before its one rounding, three operations per value where the scale is far from the ends of
        // the range (a division per value made the kernel compute-bound).  Where r would underflow, the code
        // is 0 either way.
        float q[16];
        if (scale > 0x1p-100f && scale < 0x1p100f) {
            const float y = __fdiv_rn(1.f, scale);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float q0 = x[i] * y;
                q[i] = fmaf(fmaf(-q0, scale, x[i]), y, q0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) q[i] = __fdiv_rn(x[i], scale);
        }
        uint32_t code[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            code[i] = pack_e4m3x2(q[4 * i], q[4 * i + 1]) | (pack_e4m3x2(q[4 * i + 2], q[4 * i + 3]) << 16);
        uint8_t* row = static_cast<uint8_t*>(p.cache) + static_cast<int64_t>(slot) * kFp8RowBytes;
        reinterpret_cast<uint4*>(row)[lane] = make_uint4(code[0], code[1], code[2], code[3]);
        if ((lane & 7) == 0) reinterpret_cast<float*>(row + kDV)[lane >> 3] = scale;
        reinterpret_cast<uint32_t*>(row + kDV + 16)[lane] = turned;
    }
}

}  // namespace smla
