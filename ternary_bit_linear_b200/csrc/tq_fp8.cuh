// tq_fp8.cuh -- quantisation to e4m3 with one fp32 scale per block of 128.
//
//   s = max(max_block |x|, 1e-20) / 448          (fp32, IEEE division)
//   q = e4m3(fp32(x / s))                         (half to even, saturating)
//
// 448 is e4m3's largest value, so a block's largest element uses the whole
// range.  The floor keeps s and every quotient near a rounding border a
// normal fp32 number.  Blocks are 1 x 128 along a row (activations,
// gradients), 128 x 1 down a column with the codes written transposed (the
// operands of a contraction over rows), or 128 x 128 (weights).
//
// All forms read x once and are bound by memory: 5 bytes of traffic per fp32
// element (3 per bf16 element), one more with the transposed codes.
#pragma once

#include <cuda_bf16.h>

#include "tq_act.cuh"
#include "tq_common.cuh"

namespace tq {

constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.0f;
constexpr float kFp8Floor = 1e-20f;

__device__ __forceinline__ float fp8_scale(float amax) { return __fdiv_rn(fmaxf(amax, kFp8Floor), kFp8Max); }

// Codes of x / s for four elements, lowest address first; s per element, or one.
__device__ __forceinline__ uint32_t fp8_codes4(float4 v, float4 s) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(__fdiv_rn(v.y, s.y)), "f"(__fdiv_rn(v.x, s.x)));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(__fdiv_rn(v.w, s.w)), "f"(__fdiv_rn(v.z, s.z)));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ uint32_t fp8_codes4(float4 v, float s) { return fp8_codes4(v, make_float4(s, s, s, s)); }

__device__ __forceinline__ float abs_max4(float4 v) {
    return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// Four elements at column c (c % 4 == 0) of a row of C elements; zeros past the
// row.  VEC: C % 4 == 0, so the four are one aligned 16- or 8-byte load.
template <bool BF16, bool VEC>
__device__ __forceinline__ float4 fp8_load4(const void *x, int64_t row, int64_t C, int64_t c) {
    if (BF16) {
        const __nv_bfloat16 *p = reinterpret_cast<const __nv_bfloat16 *>(x) + row * C;
        if (VEC) {
            if (c >= C) return make_float4(0.f, 0.f, 0.f, 0.f);
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p + c));
            return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                               __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
        }
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = c + i < C ? __bfloat162float(p[c + i]) : 0.0f;
        return make_float4(v[0], v[1], v[2], v[3]);
    }
    const float *p = reinterpret_cast<const float *>(x) + row * C;
    if (VEC) return c < C ? __ldg(reinterpret_cast<const float4 *>(p + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = c + i < C ? __ldg(p + c + i) : 0.0f;
    return make_float4(v[0], v[1], v[2], v[3]);
}

// ---------------------------------------------------------------------------
// 1 x 128 blocks.  One warp takes 512 columns of one row: four blocks, each of
// its lanes four consecutive elements of each, so a block's maximum is one
// warp reduction and its 128 codes one coalesced store.
// ---------------------------------------------------------------------------
constexpr int kFp8RowWarps = 8;

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(32 * kFp8RowWarps)
    tq_fp8_rows_kernel(const void *__restrict__ x, int64_t R, int64_t C, int64_t ldq, int64_t segs,
                       uint8_t *__restrict__ q, float *__restrict__ s) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * kFp8RowWarps + (threadIdx.x >> 5);
    const int64_t row = id / segs, c0 = (id - row * segs) * 512 + 4 * lane;
    if (row >= R) return;
    float4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = fp8_load4<BF16, VEC>(x, row, C, c0 + 128 * j);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float sc = fp8_scale(warp_max(abs_max4(v[j])));
        const int64_t c = c0 + 128 * j;
        if (c < ldq) *reinterpret_cast<uint32_t *>(q + row * ldq + c) = fp8_codes4(v[j], sc);
        if (lane == 0 && c < C) s[(c >> 7) * R + row] = sc;
    }
}

// The same after RMSNorm (x * rsqrt(mean x^2 + eps) * gain, the sum in fp64,
// the product rounded once to fp32 as the fused layer's prologue does): one
// CTA per row, the row read a second time from cache.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kActThreads)
    tq_fp8_rows_norm_kernel(const void *__restrict__ x, int64_t R, int64_t C, int64_t ldq,
                            const float *__restrict__ gain, float eps, uint8_t *__restrict__ q,
                            float *__restrict__ s) {
    __shared__ double redd[32];
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double ss = 0.0;
    for (int64_t c = 4 * threadIdx.x; c < C; c += 4 * kActThreads) {
        const float4 v = fp8_load4<BF16, VEC>(x, row, C, c);
        ss = __fma_rn((double)v.x, (double)v.x, ss);
        ss = __fma_rn((double)v.y, (double)v.y, ss);
        ss = __fma_rn((double)v.z, (double)v.z, ss);
        ss = __fma_rn((double)v.w, (double)v.w, ss);
    }
    ss = block_sum_d<kActThreads>(ss, redd);
    const double r = __ddiv_rn(1.0, __dsqrt_rn(__dadd_rn(__ddiv_rn(ss, (double)C), (double)eps)));
    for (int64_t b = 128 * warp; b < ldq; b += 128 * (kActThreads / 32)) {
        const int64_t c = b + 4 * lane;
        float4 v = fp8_load4<BF16, VEC>(x, row, C, c);
        float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double g = gain && c + i < C ? (double)__ldg(gain + c + i) : 1.0;
            e[i] = __double2float_rn(__dmul_rn(__dmul_rn((double)e[i], r), g));
        }
        v = make_float4(e[0], e[1], e[2], e[3]);
        const float sc = fp8_scale(warp_max(abs_max4(v)));
        if (c < ldq) *reinterpret_cast<uint32_t *>(q + row * ldq + c) = fp8_codes4(v, sc);
        if (lane == 0) s[(b >> 7) * R + row] = sc;
    }
}

// ---------------------------------------------------------------------------
// Tiles of 128 x 128: the 128 x 128 form, and both forms with the transposed
// codes.  A tile holds whole blocks of every kind, so x is read once for
// both outputs.  Warp w holds rows 16 w .. 16 w + 15 of the tile in registers,
// lane l the columns 4 l .. 4 l + 3: a row's maximum is a warp reduction, a
// column's meets in shared memory, and a thread's 16 rows of one column are
// 16 consecutive bytes of the transposed codes, which pass through shared
// memory to leave in whole 128-byte rows.
// ---------------------------------------------------------------------------
template <bool BF16, bool VEC, bool SQUARE, bool TRANS>
__global__ void __launch_bounds__(256)
    tq_fp8_tile_kernel(const void *__restrict__ x, int64_t R, int64_t C, int64_t ldq, int64_t ldt,
                       uint8_t *__restrict__ q, float *__restrict__ s, uint8_t *__restrict__ qt,
                       float *__restrict__ st) {
    __shared__ __align__(16) uint8_t tile[TRANS ? 128 * 128 : 16];
    __shared__ float red[8][128];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t cb = blockIdx.x, CB = gridDim.x;
    const int64_t c = cb * 128 + 4 * lane;
    for (int64_t rb = blockIdx.y; rb * 128 < R; rb += gridDim.y) {
        const int64_t r0 = rb * 128 + 16 * warp;
        float4 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = r0 + i < R ? fp8_load4<BF16, VEC>(x, r0 + i, C, c) : make_float4(0.f, 0.f, 0.f, 0.f);
        float sq = 0.0f;
        if (SQUARE) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) m = fmaxf(m, abs_max4(v[i]));
            m = warp_max(m);
            if (lane == 0) red[0][warp] = m;
            __syncthreads();
            sq = fp8_scale(warp_max(red[0][lane & 7]));
            if (threadIdx.x == 0) {
                s[rb * CB + cb] = sq;
                if (TRANS) st[cb * ((R + 127) >> 7) + rb] = sq;
            }
        } else if (TRANS) {
            float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                m.x = fmaxf(m.x, fabsf(v[i].x));
                m.y = fmaxf(m.y, fabsf(v[i].y));
                m.z = fmaxf(m.z, fabsf(v[i].z));
                m.w = fmaxf(m.w, fabsf(v[i].w));
            }
            *reinterpret_cast<float4 *>(&red[warp][4 * lane]) = m;
        }
        // codes in x's own order
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float sc = SQUARE ? sq : fp8_scale(warp_max(abs_max4(v[i])));
            w[i] = fp8_codes4(v[i], sc);
            if (r0 + i < R) {
                if (c < ldq) *reinterpret_cast<uint32_t *>(q + (r0 + i) * ldq + c) = w[i];
                if (!SQUARE && lane == 0) s[cb * R + r0 + i] = sc;
            }
        }
        if (TRANS) {
            if (!SQUARE) {  // the columns' own scales and codes
                __syncthreads();
                float4 m = *reinterpret_cast<const float4 *>(&red[0][4 * lane]);
#pragma unroll
                for (int k = 1; k < 8; ++k) {
                    const float4 t = *reinterpret_cast<const float4 *>(&red[k][4 * lane]);
                    m = make_float4(fmaxf(m.x, t.x), fmaxf(m.y, t.y), fmaxf(m.z, t.z), fmaxf(m.w, t.w));
                }
                const float4 sc = make_float4(fp8_scale(m.x), fp8_scale(m.y), fp8_scale(m.z), fp8_scale(m.w));
                if (warp == 0) {
                    const float e[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (c + k < C) st[rb * C + c + k] = e[k];
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[i] = fp8_codes4(v[i], sc);
            }
            // byte e of words 4k .. 4k + 3 -> word k of column e's 16 rows.  Chunk
            // (16 rows) w of column col sits at chunk w ^ (col / 4 % 8): a quarter
            // warp's stores and reads hit eight different chunks.
            uint4 t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                t[k] = transpose_bytes4x4(make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
            uint4 *d = reinterpret_cast<uint4 *>(tile) + 32 * lane + (warp ^ (lane & 7));
            d[0] = make_uint4(t[0].x, t[1].x, t[2].x, t[3].x);
            d[8] = make_uint4(t[0].y, t[1].y, t[2].y, t[3].y);
            d[16] = make_uint4(t[0].z, t[1].z, t[2].z, t[3].z);
            d[24] = make_uint4(t[0].w, t[1].w, t[2].w, t[3].w);
            __syncthreads();
            const int64_t tr = rb * 128 + 16 * (lane & 7);  // 16 bytes of a transposed row per lane
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int col = 32 * k + 4 * warp + (lane >> 3);
                if (cb * 128 + col < C && tr < ldt)
                    *reinterpret_cast<uint4 *>(qt + (cb * 128 + col) * ldt + tr) =
                        reinterpret_cast<const uint4 *>(tile)[8 * col + ((lane & 7) ^ ((col >> 2) & 7))];
            }
        }
        __syncthreads();  // red and tile are written again
    }
}

}  // namespace tq
