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
// All forms read x once (after RMSNorm twice, the second time from cache).  The least
// traffic is 5 bytes per fp32 element (3 per bf16 element), one more with the transposed
// codes; fp32 rows and 128 x 128 blocks come near the time of it, the others are held
// up by their instructions, which a bf16 element does not halve.
#pragma once

#include <cuda_bf16.h>

#include "tq_act.cuh"
#include "tq_common.cuh"

namespace tq {

constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.0f;
constexpr float kFp8Floor = 1e-20f;

__device__ __forceinline__ float fp8_scale(float amax) { return __fdiv_rn(fmaxf(amax, kFp8Floor), kFp8Max); }

// A block's scale and its correctly rounded reciprocal.
struct Fp8Scale {
    float s, inv;
};
__device__ __forceinline__ Fp8Scale fp8_block_scale(float amax) {
    const float s = fp8_scale(amax);
    return Fp8Scale{s, __frcp_rn(s)};
}

// fp32(v / s) from the reciprocal: Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor" (1990): a quotient within one unit, here v inv
// corrected once, becomes the correctly rounded one by its exact remainder times
// the correctly rounded reciprocal.  The remainders of quotients near a rounding
// border of e4m3 are normal numbers (the floor of s).  The remainders are taken with
// the opposite sign, q s - v, so that a quotient of -0 stays one: v = -0 leaves +0, and
// -0 + (-0) inv is -0, where -0 + (+0) inv would be +0.  An infinite s has inv = 0,
// and v * 0 is what v / s would be.
__device__ __forceinline__ float fp8_quotient(float v, Fp8Scale k) {
    const float q0 = __fmul_rn(v, k.inv);
    const float q1 = __fmaf_rn(-__fmaf_rn(q0, k.s, -v), k.inv, q0);
    const float q2 = __fmaf_rn(-__fmaf_rn(q1, k.s, -v), k.inv, q1);
    return k.inv == 0.0f ? q0 : q2;
}

// Codes of four quotients, lowest address first.
__device__ __forceinline__ uint32_t fp8_pack4(float x, float y, float z, float w) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y), "f"(x));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(w), "f"(z));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ uint32_t fp8_codes4(float4 v, Fp8Scale k) {
    return fp8_pack4(fp8_quotient(v.x, k), fp8_quotient(v.y, k), fp8_quotient(v.z, k), fp8_quotient(v.w, k));
}

__device__ __forceinline__ float abs_max4(float4 v) {
    return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// One step of a reduction of several maxima at once: a lane keeps the second of
// two (`up`) or the first, joined with its partner's of the same.
__device__ __forceinline__ void fp8_halve(float &first, float second, bool up, int off) {
    const float give = up ? first : second, keep = up ? second : first;
    first = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, off));
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
// warp reduction and its 128 codes one coalesced store.  11008 x 4096 fp32: 36 us,
// 6.2 TB/s; bf16: 34 us, 4.0 TB/s.
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
    // the four maxima by halving exchanges: block lane / 8's ends up in every lane
    float m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = abs_max4(v[j]);
    fp8_halve(m[0], m[2], lane & 16, 16);
    fp8_halve(m[1], m[3], lane & 16, 16);
    fp8_halve(m[0], m[1], lane & 8, 8);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], off));
    const Fp8Scale mine = fp8_block_scale(m[0]);
    const int64_t b = (c0 - 4 * lane) / 128 + (lane >> 3);
    if (!(lane & 7) && b * 128 < C) s[b * R + row] = mine.s;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const Fp8Scale sc{__shfl_sync(0xffffffffu, mine.s, 8 * j), __shfl_sync(0xffffffffu, mine.inv, 8 * j)};
        const int64_t c = c0 + 128 * j;
        if (c < ldq) *reinterpret_cast<uint32_t *>(q + row * ldq + c) = fp8_codes4(v[j], sc);
    }
}

// The same after RMSNorm (x * rsqrt(mean x^2 + eps) * gain, the sum in fp64,
// the product rounded once to fp32 as the fused layer's prologue does): one
// CTA per row, the row read a second time from cache.  2048 x 4096 bf16: 16.7 us;
// 11008 x 4096 fp32: 77 us, 2.9 TB/s: two chains of fp64 operations with a reduction over
// the CTA between them.
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
    if (!isfinite(r)) {
        // A NaN in the row, or an empty row without an eps: every element is a NaN, which no
        // maximum takes in.  Apart from the loop, where 0 r would make NaNs of the zeros
        // past the row too, and a test for them cost 3 %.
        for (int64_t c = threadIdx.x; c < ldq; c += kActThreads) q[row * ldq + c] = c < C ? 0x7f : 0;
        for (int64_t b = threadIdx.x; b < (C + 127) / 128; b += kActThreads) s[b * R + row] = fp8_scale(0.0f);
        return;
    }
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
        const Fp8Scale sc = fp8_block_scale(warp_max(abs_max4(v)));
        if (c < ldq) *reinterpret_cast<uint32_t *>(q + row * ldq + c) = fp8_codes4(v, sc);
        if (lane == 0) s[(b >> 7) * R + row] = sc.s;
    }
}

// ---------------------------------------------------------------------------
// Tiles of 128 x 128: the 128 x 128 form, and both forms with the transposed
// codes.  A tile holds whole blocks of every kind, so x is read once for
// both outputs.  Warp w holds rows 16 w .. 16 w + 15 of the tile in registers,
// lane l the columns 4 l .. 4 l + 3: a row's maximum is a warp reduction, a
// column's meets in shared memory, and a thread's 16 rows of one column are
// 16 consecutive bytes of the transposed codes, which pass through shared
// memory to leave in whole 128-byte rows.  Three tiles per SM, so that one's loads
// run while another's maxima meet; of the 80 registers that leaves a thread, most forms
// spill some (up to 104 bytes, 260 where cols % 4 != 0).  11008 x 4096 to 128 x 128
// blocks: fp32 43.1 us, bf16 48.9 us; with the transpose 44.1 us (6.1 TB/s) and
// 58.9 us; rows and columns, whose scales differ, 60.4 us and 65.4 us, each code twice
// from its own quotient (issue slots 64 % busy).  11008 x 4094: 49 to 107 us.
// ---------------------------------------------------------------------------
template <bool BF16, bool VEC, bool SQUARE, bool TRANS>
__global__ void __launch_bounds__(256, 3)
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
        Fp8Scale sq{0.0f, 0.0f};
        if (SQUARE) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) m = fmaxf(m, abs_max4(v[i]));
            m = warp_max(m);
            if (lane == 0) red[0][warp] = m;
            __syncthreads();
            sq = fp8_block_scale(warp_max(red[0][lane & 7]));
            if (threadIdx.x == 0) {
                s[rb * CB + cb] = sq.s;
                if (TRANS) st[cb * ((R + 127) >> 7) + rb] = sq.s;
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
        // A row's maximum over the 32 lanes: halving exchanges leave row lane / 2's in
        // every lane (16 shuffles, not 80), which makes that row's scale for all.
        Fp8Scale mine{0.0f, 0.0f};
        if (!SQUARE) {
            float m[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) m[i] = abs_max4(v[i]);
#pragma unroll
            for (int n = 8; n >= 1; n >>= 1) {
                const bool up = lane & (2 * n);
#pragma unroll
                for (int i = 0; i < n; ++i) fp8_halve(m[i], m[i + n], up, 2 * n);
            }
            mine = fp8_block_scale(fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1)));
            if (!(lane & 1) && r0 + (lane >> 1) < R) s[cb * R + r0 + (lane >> 1)] = mine.s;
        }
        // codes in x's own order
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const Fp8Scale sc = SQUARE ? sq
                                       : Fp8Scale{__shfl_sync(0xffffffffu, mine.s, 2 * i),
                                                  __shfl_sync(0xffffffffu, mine.inv, 2 * i)};
            w[i] = fp8_codes4(v[i], sc);
            if (r0 + i < R && c < ldq) *reinterpret_cast<uint32_t *>(q + (r0 + i) * ldq + c) = w[i];
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
                const Fp8Scale k[4] = {fp8_block_scale(m.x), fp8_block_scale(m.y), fp8_block_scale(m.z), fp8_block_scale(m.w)};
                if (warp == 0) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < C) st[rb * C + c + e] = k[e].s;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[i] = fp8_pack4(fp8_quotient(v[i].x, k[0]), fp8_quotient(v[i].y, k[1]), fp8_quotient(v[i].z, k[2]),
                                     fp8_quotient(v[i].w, k[3]));
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
