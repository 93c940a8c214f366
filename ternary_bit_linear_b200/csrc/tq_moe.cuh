// tq_moe.cuh -- a whole mixture-of-experts feed-forward layer for the few tokens
// of a decode step, in two kernels.
//
//   l[m][e] = sum_d x[m][d] router[e][d]             (fp64 sums, rounded to fp32)
//   ids[m]  = the top_k largest l[m][.], ties to the lower index
//   w[m][j] = exp(l[m][ids_j] - max) / sum exp(l - max)   (over all experts, or the chosen ones)
//   y[m]    = sum_j w[m][j] expert_{ids_j}(x[m])
//
// and each expert the clamped SwiGLU block of three ternary layers (Hetman-2b,
// src/quantization.py, section 6 SwiGLUClamped.forward): x_q, s_x the int8
// quantisation of FWHT-512 of [RMSNorm of] x (the same for every expert), g =
// fp32(x_q . gate) * (gamma s_x), u likewise, a = clamp(SiLU(g) u), its own
// rotation and quantisation, and the down projection.  SiLU(g) u is evaluated
// in fp64 and rounded once to fp32, so that the int8 codes that follow do not
// hang on the last bits of an exponential.
//
// What bounds it: the packed weights of the chosen experts, read once (3 D F / 4
// bytes each); for one or two tokens, the chain of dependent steps.
//
//   tq_moe_route_kernel: a CTA per token quantises it; the other CTAs compute the
//     logits, a warp per expert and four tokens.
//   tq_moe_experts_kernel: one CTA per SM, launched cooperatively (all CTAs
//     resident), with three grid-wide barriers between its phases:
//       choice     every CTA picks every token's experts (cheaper than another
//                  barrier) and sorts the (token, slot) pairs by expert; an expert
//                  and up to 16 of its pairs are one "problem".
//       gate, up   a strip is 16 rows of both matrices, so that the activation
//                  follows in registers.  The strips of all problems are split
//                  into contiguous runs, one per CTA; the quantised tokens of a
//                  run's problem sit in shared memory.
//       rotation   a team of F / 512 warps per pair: FWHT, int8 codes.
//       down       strips of 32 rows, runs as before.
//       sum        y from the pairs' outputs, slots in order: no atomics, and
//                  the result does not depend on how pairs were grouped.
//   A warp streams its strips' weights from HBM into registers, several 64-byte
//   column steps ahead, and contracts them with mma.sync (u8 codes x s8): with at
//   most 16 tokens the tensor rate is no bound, and no shared memory is spent on
//   bytes that are used once.
#pragma once

#include "tq_act.cuh"
#include "tq_common.cuh"
#include "tq_gemv.cuh"

namespace tq {

constexpr int kMoeWarps = 16;
constexpr int kMoeThreads = 32 * kMoeWarps;
constexpr int kMoeMaxTokens = 64, kMoeMaxTopk = 16, kMoeMaxExperts = 256;
constexpr int kMoeMaxPairs = kMoeMaxTokens * kMoeMaxTopk;
constexpr int kMoeChunk = 16;  // pairs of one expert per problem
constexpr int kMoeMaxProblems = kMoeMaxExperts + kMoeMaxPairs / kMoeChunk;
constexpr int kMoeMaxK = 8192;  // d_model, d_ffn: 16 blocks of 512, one per warp
constexpr int kMoeRouteTokens = 4;
// partial sums of a split strip: [2][warps][2 matrices x 2 token blocks x 4][lanes]
constexpr int kMoeRedBytes = 2 * kMoeWarps * 16 * 32 * 4;

struct MoeArgs {
    const float *x, *router;  // [M][D], [E][D] or nullptr (ids, weights given)
    const uint8_t *gate, *up, *down;
    const float *gate_gamma, *up_gamma, *down_gamma;
    float *y;
    int32_t *ids;  // [M][k]
    float *weights;
    int M, D, F, E, k;
    int per_row, norm_topk, enc;
    float clamp_val;
    ActParams act;
    // workspace
    int8_t *xq;  // [M][D], chunks transposed and swizzled as the small-M GEMV reads them
    float *sx;
    int32_t *rs;
    float *logits;       // [M][E]
    unsigned *barrier;   // one counter, zeroed by the route kernel
    float *h;            // [M k][F] activations
    int8_t *hq;          // [M k][F]
    float *sh;
    int32_t *rh;
    float *out;          // [M k][D] the pairs' outputs
};

__device__ __forceinline__ void bar_sync_n(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

struct MoeRed {
    float f[kMoeWarps];
    int i[kMoeWarps];
    double d[kMoeWarps];
};

// FWHT-512 and int8 codes of a row held by a team of nw warps (warp wt has block
// wt, 16 values per lane as in tq_act.cuh; red: the team's slots).  The steps and
// roundings of tq_prologue_fwht_kernel; the codes are written in the small-M
// GEMV's layout.
__device__ __forceinline__ void moe_rot_quant(float (&f)[16], int wt, int nw, int bar, const ActParams &p, int K,
                                              int8_t *__restrict__ dst, float *__restrict__ s, int32_t *__restrict__ rowsum,
                                              float *redf, int *redi, double *redd) {
    const int lane = threadIdx.x & 31;
    if (p.sanitize) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = quench(f[i], p.eta_max);
    }
    if (p.rmsnorm) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = __fma_rn((double)f[i], (double)f[i], ss);
        ss = warp_sum_d(ss);
        if (lane == 0) redd[wt] = ss;
        bar_sync_n(bar, 32 * nw);
        ss = warp_sum_d(lane < nw ? redd[lane] : 0.0);
        const double r = __ddiv_rn(1.0, __dsqrt_rn(__dadd_rn(__ddiv_rn(ss, (double)K), (double)p.rms_eps)));
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = __double2float_rn(__dmul_rn((double)f[i], r));
    }
    fwht512_regs(f, true);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
    amax = warp_max(amax);
    if (lane == 0) redf[wt] = amax;
    bar_sync_n(bar, 32 * nw);
    amax = warp_max(lane < nw ? redf[lane] : 0.0f);
    const float eta = eta_of(amax, p);
    const float scale = __fdiv_rn(127.0f, eta);
    uint32_t *out = reinterpret_cast<uint32_t *>(dst);
    int sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int a = quant_code(f[4 * j], scale), b = quant_code(f[4 * j + 1], scale), c = quant_code(f[4 * j + 2], scale),
                  d = quant_code(f[4 * j + 3], scale);
        sum += a + b + c + d;
        const uint32_t word = pack_codes4(a, b, c, d);
        const int q0 = lane & ~3;
        uint4 q;
        q.x = __shfl_sync(0xffffffffu, word, q0);
        q.y = __shfl_sync(0xffffffffu, word, q0 + 1);
        q.z = __shfl_sync(0xffffffffu, word, q0 + 2);
        q.w = __shfl_sync(0xffffffffu, word, q0 + 3);
        const uint4 t = transpose_bytes4x4(q);
        const int idx = wt * 128 + j * 32 + lane, e = lane & 3;
        out[4 * gemv_chunk_pos(idx >> 2) + e] = e == 0 ? t.x : e == 1 ? t.y : e == 2 ? t.z : t.w;
    }
    sum = warp_sum_i(sum);
    if (lane == 0) redi[wt] = sum;
    bar_sync_n(bar, 32 * nw);
    if (wt == 0) {
        sum = warp_sum_i(lane < nw ? redi[lane] : 0);
        if (lane == 0) {
            *s = __fdiv_rn(eta, 127.0f);
            *rowsum = sum;
        }
    }
}

__device__ __forceinline__ void load_block16(float (&f)[16], const float *row, int wt) {
    const float4 *src = reinterpret_cast<const float4 *>(row + wt * 512);
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 v = __ldcg(src + j * 32 + lane);
        f[4 * j] = v.x;
        f[4 * j + 1] = v.y;
        f[4 * j + 2] = v.z;
        f[4 * j + 3] = v.w;
    }
}

// CTAs 0 .. M - 1: token blockIdx.x's codes.  The others: logits of 16 experts
// (a warp each) and 4 tokens.
__global__ void __launch_bounds__(kMoeThreads) tq_moe_route_kernel(const __grid_constant__ MoeArgs a) {
    __shared__ MoeRed red;
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.barrier = 0;
    if ((int)blockIdx.x < a.M) {
        const int nw = a.D / 512, m = blockIdx.x;
        if (warp >= nw) return;
        float f[16];
        load_block16(f, a.x + (int64_t)m * a.D, warp);
        moe_rot_quant(f, warp, nw, 1, a.act, a.D, a.xq + (int64_t)m * a.D, a.sx + m, a.rs + m, red.f, red.i, red.d);
        return;
    }
    const int u = blockIdx.x - a.M, tgroups = (a.M + kMoeRouteTokens - 1) / kMoeRouteTokens;
    const int e = u / tgroups * kMoeWarps + warp, m0 = u % tgroups * kMoeRouteTokens;
    if (e >= a.E) return;
    const int nt = a.M - m0 < kMoeRouteTokens ? a.M - m0 : kMoeRouteTokens;
    const float4 *wr = reinterpret_cast<const float4 *>(a.router + (int64_t)e * a.D);
    const float4 *xr = reinterpret_cast<const float4 *>(a.x + (int64_t)m0 * a.D);
    const int nv = a.D / 4;  // a multiple of 128
    double s[kMoeRouteTokens] = {0.0, 0.0, 0.0, 0.0};
    for (int i = lane; i < nv; i += 128) {
        float4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __ldg(wr + i + 32 * j);
#pragma unroll
        for (int t = 0; t < kMoeRouteTokens; ++t) {
            if (t >= nt) break;
            float4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = __ldg(xr + (int64_t)t * nv + i + 32 * j);
                if (a.act.sanitize) v[j] = quench4(v[j], a.act);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[t] = __fma_rn((double)v[j].x, (double)w[j].x, s[t]);
                s[t] = __fma_rn((double)v[j].y, (double)w[j].y, s[t]);
                s[t] = __fma_rn((double)v[j].z, (double)w[j].z, s[t]);
                s[t] = __fma_rn((double)v[j].w, (double)w[j].w, s[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kMoeRouteTokens; ++t) {
        const double v = warp_sum_d(s[t]);
        if (lane == 0 && t < nt) a.logits[(int64_t)(m0 + t) * a.E + e] = __double2float_rn(v);
    }
}

// Orders fp32 values as unsigned numbers; NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t moe_key(float v) {
    if (v != v) return 0u;
    const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Grid-wide barrier number `n` (1, 2, ...) on a counter that starts at 0.  All
// CTAs are resident (cooperative launch).  Bounded: false, with the timeout
// recorded, if the others do not arrive within about a second.
__device__ __forceinline__ bool moe_grid_sync(unsigned *counter, unsigned n, int *flag) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(counter, 1u);
        const unsigned want = n * gridDim.x;
        int ok = 0;
        for (int i = 0; i < (1 << 20); ++i) {
            unsigned v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
            if (v >= want) {
                ok = 1;
                break;
            }
        }
        if (!ok) flag_timeout();
        *flag = ok;
        __threadfence();
    }
    __syncthreads();
    return *flag != 0;
}

// Sums of two sets of 16 weight rows (packed rows pa + r KB and pb + r KB) over
// the column steps j0, j0 + ks, ... of 256 codes, for up to 8 NB tokens in
// shared memory.  PD steps of weights are in flight.  A word's 16 codes enter
// the MMA as two masked fields and, shifted by 4, two more; the fields masked in
// place at bit 2 have an accumulator of their own (multiples of 4).
template <int NB, int PD, bool CONV>
__device__ __forceinline__ void moe_pair_mma(int (&acc)[2][NB][4], const uint8_t *pa, const uint8_t *pb, int KB, uint32_t x_s,
                                             int XS, int ntok, int j0, int ks, int lane, int enc) {
    const int g = lane >> 2, t = lane & 3, nsteps = KB >> 6;
    const uint8_t *row[4] = {pa + (int64_t)g * KB + 16 * t, pa + (int64_t)(g + 8) * KB + 16 * t, pb + (int64_t)g * KB + 16 * t,
                             pb + (int64_t)(g + 8) * KB + 16 * t};
    uint32_t xr[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int m = g + 8 * nb < ntok ? g + 8 * nb : ntok - 1;  // rows past ntok: sums that are not used
        xr[nb] = x_s + (uint32_t)(m * XS + 64 * t);
    }
    const uint32_t xsw = (uint32_t)(t & 2) << 4;
    int d[2][2][NB][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) d[i][j][nb][0] = d[i][j][nb][1] = d[i][j][nb][2] = d[i][j][nb][3] = 0;
    uint4 w[PD][4];
#pragma unroll
    for (int p = 0; p < PD; ++p) {
        const int step = j0 + p * ks;
        if (step < nsteps) {
#pragma unroll
            for (int r = 0; r < 4; ++r) w[p][r] = ldg_stream16(row[r] + 64 * step);
        }
    }
    for (int base = j0; base < nsteps; base += PD * ks) {
#pragma unroll
        for (int p = 0; p < PD; ++p) {
            const int step = base + p * ks;
            if (step >= nsteps) break;
            uint32_t c[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                c[r][0] = w[p][r].x;
                c[r][1] = w[p][r].y;
                c[r][2] = w[p][r].z;
                c[r][3] = w[p][r].w;
                if (CONV)
#pragma unroll
                    for (int i = 0; i < 4; ++i) c[r][i] = codes_to_foundry(c[r][i], enc);
            }
            if (step + PD * ks < nsteps) {
#pragma unroll
                for (int r = 0; r < 4; ++r) w[p][r] = ldg_stream16(row[r] + 64 * (step + PD * ks));
            }
            const uint32_t xo = (uint32_t)step * 256u;
#pragma unroll
            for (int pr = 0; pr < 2; ++pr) {
                uint4 xt[NB][2];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    xt[nb][0] = lds128(xr[nb] + xo + ((uint32_t)(32 * pr) ^ xsw));
                    xt[nb][1] = lds128(xr[nb] + xo + ((uint32_t)(32 * pr + 16) ^ xsw));
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t msk = (j & 1) ? 0x0c0c0c0cu : 0x03030303u;
                    const int sh = (j & 2) * 2;
#pragma unroll
                    for (int mat = 0; mat < 2; ++mat) {
                        const uint32_t a0 = (c[2 * mat][2 * pr] >> sh) & msk, a1 = (c[2 * mat + 1][2 * pr] >> sh) & msk;
                        const uint32_t a2 = (c[2 * mat][2 * pr + 1] >> sh) & msk, a3 = (c[2 * mat + 1][2 * pr + 1] >> sh) & msk;
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            const uint4 &u = xt[nb][0], &v = xt[nb][1];
                            const uint32_t x0 = j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w;
                            const uint32_t x1 = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
                            mma_16x8x32_u8s8_pure(d[j & 1][mat][nb], a0, a1, a2, a3, x0, x1);
                        }
                    }
                }
            }
        }
    }
#pragma unroll
    for (int mat = 0; mat < 2; ++mat)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[mat][nb][i] = d[0][mat][nb][i] + (d[1][mat][nb][i] >> 2);  // exact
}

// clamp(SiLU(g) u), in fp64, rounded once before the clamp
__device__ __forceinline__ float moe_act(float g, float u, float c) {
    const double gd = (double)g;
    const float v = __double2float_rn(__dmul_rn(__ddiv_rn(gd, __dadd_rn(1.0, exp(-gd))), (double)u));
    return fminf(fmaxf(v, -c), c);
}

// A problem: expert, its pairs sorted[start .. start + count).
struct MoeProblem {
    int16_t expert, start, count;
};

struct MoeShared {
    int ids[kMoeMaxPairs];
    float w[kMoeMaxPairs];
    int16_t sorted[kMoeMaxPairs];
    int count[kMoeMaxExperts], first[kMoeMaxExperts];
    MoeProblem prob[kMoeMaxProblems];
    int nprob, flag;
    MoeRed red;
};

// The strips of one run and problem.  GATE: rows n0 .. n0 + 15 of gate and up,
// activation to a.h; else rows n0 .. n0 + 31 of down, output to a.out.
template <int NB, bool GATE, bool CONV>
__device__ __forceinline__ void moe_strips(const MoeArgs &a, const MoeShared &sm, const MoeProblem &pb, int strip0, int strip1,
                                           uint32_t x_s, int XS, int *red, int &par, int ks) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = warp / ks, kw = warp % ks, T = kMoeWarps / ks;
    const int g = lane >> 2, t = lane & 3;
    const int N = GATE ? a.F : a.D, KB = (GATE ? a.D : a.F) / 4;
    const int64_t base = (int64_t)pb.expert * N * KB;
    const int count = pb.count;
    // this lane's tokens: 8 nb + 2 t + e
    float sv[NB][2];
    int rv[NB][2], row[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 8 * nb + 2 * t + e;
            const int p = i < count ? sm.sorted[pb.start + i] : 0;
            const int src = GATE ? p / a.k : p;
            row[nb][e] = i < count ? p : -1;
            sv[nb][e] = __ldcg((GATE ? a.sx : a.sh) + src);
            rv[nb][e] = __ldcg((GATE ? a.rs : a.rh) + src);
        }
    for (int s = strip0 + team; s < strip1; s += T) {
        const int n0 = s * (GATE ? 16 : 32);
        const uint8_t *pa = (GATE ? a.gate : a.down) + base + (int64_t)n0 * KB;
        const uint8_t *pbk = GATE ? a.up + base + (int64_t)n0 * KB : pa + 16 * (int64_t)KB;
        int acc[2][NB][4];
        moe_pair_mma<NB, NB == 1 ? 4 : 2, CONV>(acc, pa, pbk, KB, x_s, XS, count, kw, ks, lane, a.enc);
        if (ks > 1) {
            int *rb = red + par * (kMoeRedBytes / 8);
            if (kw != 0) {
#pragma unroll
                for (int i = 0; i < 8 * NB; ++i) rb[(warp * 16 + i) * 32 + lane] = acc[i / (4 * NB)][i / 4 % NB][i % 4];
            }
            bar_sync_n(1 + team, 32 * ks);
            if (kw == 0) {
                for (int w2 = warp + 1; w2 < warp + ks; ++w2)
#pragma unroll
                    for (int i = 0; i < 8 * NB; ++i) acc[i / (4 * NB)][i / 4 % NB][i % 4] += rb[(w2 * 16 + i) * 32 + lane];
            }
            par ^= 1;
        }
        if (kw != 0) continue;
        // sum c of a fragment: row g (+ 8 for c >= 2), token 8 nb + 2 t + (c & 1)
        const float *g1 = GATE ? a.gate_gamma : a.down_gamma, *g2 = GATE ? a.up_gamma : a.down_gamma;
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
            const int n = n0 + g + 8 * hi;
            const float ga = __ldg(g1 + (a.per_row ? (int64_t)pb.expert * N + n : pb.expert));
            const float gb = __ldg(g2 + (a.per_row ? (int64_t)pb.expert * N + n + (GATE ? 0 : 16) : pb.expert));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int p = row[nb][e], c = 2 * hi + e;
                    if (p < 0) continue;
                    const float va = __fmul_rn(__int2float_rn(acc[0][nb][c] - rv[nb][e]), __fmul_rn(ga, sv[nb][e]));
                    const float vb = __fmul_rn(__int2float_rn(acc[1][nb][c] - rv[nb][e]), __fmul_rn(gb, sv[nb][e]));
                    if (GATE) {
                        a.h[(int64_t)p * N + n] = moe_act(va, vb, a.clamp_val);
                    } else {
                        a.out[(int64_t)p * N + n] = va;
                        a.out[(int64_t)p * N + n + 16] = vb;
                    }
                }
        }
    }
}

// One contraction phase over all problems: this CTA's run of strips.
template <bool GATE, bool CONV>
__device__ __forceinline__ void moe_contract(const MoeArgs &a, MoeShared &sm, uint8_t *dyn) {
    const int K = GATE ? a.D : a.F, N = GATE ? a.F : a.D;
    const int spp = N / (GATE ? 16 : 32);
    const int64_t total = (int64_t)sm.nprob * spp;
    const int64_t s0 = total * blockIdx.x / gridDim.x, s1 = total * (blockIdx.x + 1) / gridDim.x;
    const int run = (int)((total + gridDim.x - 1) / gridDim.x);
    // warps per strip: as many as keep every warp busy when runs are short
    int ks = kMoeWarps;
    while (ks > 1 && (kMoeWarps / ks < run || ks > K / 256)) ks >>= 1;
    const int XS = gemv_x_stride(K);
    int *red = reinterpret_cast<int *>(dyn);
    uint8_t *xb = dyn + kMoeRedBytes;
    const uint32_t x_s = smem_u32(xb);
    int par = 0;
    for (int64_t s = s0; s < s1;) {
        const int q = (int)(s / spp);
        const MoeProblem pb = sm.prob[q];
        const int64_t end = s1 < (int64_t)(q + 1) * spp ? s1 : (int64_t)(q + 1) * spp;
        __syncthreads();  // the previous problem's tokens have been read
        const int cpr = K >> 4;
        for (int i = threadIdx.x; i < pb.count * cpr; i += kMoeThreads) {
            const int r = i / cpr, c = i - r * cpr;
            const int p = sm.sorted[pb.start + r];
            cp_async16(x_s + (uint32_t)(r * XS + 16 * c), (GATE ? a.xq + (int64_t)(p / a.k) * K : a.hq + (int64_t)p * K) + 16 * c);
        }
        cp_async_wait_all();
        __syncthreads();
        const int a0 = (int)(s - (int64_t)q * spp), a1 = (int)(end - (int64_t)q * spp);
        if (pb.count <= 8)
            moe_strips<1, GATE, CONV>(a, sm, pb, a0, a1, x_s, XS, red, par, ks);
        else
            moe_strips<2, GATE, CONV>(a, sm, pb, a0, a1, x_s, XS, red, par, ks);
        s = end;
    }
}

template <bool CONV>
__global__ void __launch_bounds__(kMoeThreads, 1) tq_moe_experts_kernel(const __grid_constant__ MoeArgs a) {
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ MoeShared sm;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = a.M * a.k;

    // ---------------- choice ----------------
    for (int m = warp; m < a.M; m += kMoeWarps) {
        if (!a.router) {
            for (int j = lane; j < a.k; j += 32) {
                const int id = __ldg(a.ids + m * a.k + j);
                sm.ids[m * a.k + j] = id >= 0 && id < a.E ? id : -1;
                sm.w[m * a.k + j] = __ldg(a.weights + m * a.k + j);
            }
            continue;
        }
        constexpr int V = kMoeMaxExperts / 32;
        float l[V];
        uint32_t key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            l[i] = e < a.E ? __ldcg(a.logits + (int64_t)m * a.E + e) : 0.0f;
            key[i] = e < a.E ? moe_key(l[i]) : 0u;
        }
        uint32_t used = 0;  // bit i: expert lane + 32 i is chosen (or does not exist)
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i >= a.E) used |= 1u << i;
        float top = 0.0f, mine = 0.0f;  // the largest logit; the logit of slot `lane`
        int my_id = 0;
        for (int j = 0; j < a.k; ++j) {
            // the largest key (+ 1, so that an unused NaN beats nothing), then the lowest index
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (!(used >> i & 1u)) best = best > key[i] ? best : key[i];
            best = __reduce_max_sync(0xffffffffu, best);
            uint32_t at = 0xffffu;
            float val = 0.0f;
#pragma unroll
            for (int i = V - 1; i >= 0; --i)
                if (!(used >> i & 1u) && key[i] == best) {
                    at = (uint32_t)(lane + 32 * i);
                    val = l[i];
                }
            const uint32_t id = __reduce_min_sync(0xffffffffu, at);
            val = __shfl_sync(0xffffffffu, val, id & 31);
            if ((int)(id & 31) == lane) used |= 1u << (id >> 5);
            if (j == 0) top = val;
            if (lane == j) {
                my_id = (int)id;
                mine = val;
            }
        }
        double den;
        const double ex = lane < a.k ? exp((double)mine - (double)top) : 0.0;
        if (a.norm_topk) {
            den = warp_sum_d(ex);
        } else {
            den = 0.0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane + 32 * i < a.E) den = __dadd_rn(den, exp((double)l[i] - (double)top));
            den = warp_sum_d(den);
        }
        if (lane < a.k) {
            const float w = __double2float_rn(__ddiv_rn(ex, den));
            sm.ids[m * a.k + lane] = my_id;
            sm.w[m * a.k + lane] = w;
            if (blockIdx.x == 0) {
                a.ids[m * a.k + lane] = my_id;
                a.weights[m * a.k + lane] = w;
            }
        }
    }
    for (int e = threadIdx.x; e < a.E; e += kMoeThreads) sm.count[e] = 0;
    __syncthreads();
    // Pairs by expert, in order (every CTA must come to the same grouping): warp 0
    // ranks 32 pairs at a time among those of the same expert.
    if (warp == 0) {
        for (int pass = 0; pass < 2; ++pass) {
            for (int p0 = 0; p0 < P; p0 += 32) {
                const int p = p0 + lane;
                const int id = p < P ? sm.ids[p] : -1;
                const uint32_t same = __match_any_sync(0xffffffffu, id);
                const int rank = __popc(same & ((1u << lane) - 1u));
                const int before = id >= 0 ? sm.count[id] : 0;
                __syncwarp();
                if (id >= 0) {
                    if (pass == 1) sm.sorted[sm.first[id] + before + rank] = (int16_t)p;
                    if (rank == 0) sm.count[id] = before + __popc(same);
                }
                __syncwarp();
            }
            if (pass == 0) {
                int at = 0, np = 0;  // running sums over experts
                for (int e0 = 0; e0 < a.E; e0 += 32) {
                    const int e = e0 + lane;
                    const int c = e < a.E ? sm.count[e] : 0, n = (c + kMoeChunk - 1) / kMoeChunk;
                    int cs = c, ns = n;
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) {
                        const int v = __shfl_up_sync(0xffffffffu, cs, off), u = __shfl_up_sync(0xffffffffu, ns, off);
                        if (lane >= off) {
                            cs += v;
                            ns += u;
                        }
                    }
                    if (e < a.E) {
                        sm.first[e] = at + cs - c;
                        for (int i = 0; i < n; ++i) {
                            MoeProblem pb;
                            pb.expert = (int16_t)e;
                            pb.start = (int16_t)(at + cs - c + i * kMoeChunk);
                            pb.count = (int16_t)(c - i * kMoeChunk < kMoeChunk ? c - i * kMoeChunk : kMoeChunk);
                            sm.prob[np + ns - n + i] = pb;
                        }
                        sm.count[e] = 0;
                    }
                    at += __shfl_sync(0xffffffffu, cs, 31);
                    np += __shfl_sync(0xffffffffu, ns, 31);
                }
                if (lane == 0) sm.nprob = np;
                __syncwarp();
            }
        }
    }
    __syncthreads();

    // ---------------- gate, up, activation ----------------
    moe_contract<true, CONV>(a, sm, dyn);
    if (!moe_grid_sync(a.barrier, 1, &sm.flag)) return;
    // ---------------- rotation and codes of every pair ----------------
    {
        const int nw = a.F / 512, fit = kMoeWarps / nw, teams = fit < 15 ? fit : 15;  // named barriers 1 .. 15
        const int team = warp / nw, wt = warp % nw;
        if (team < teams) {
            for (int p = (int)blockIdx.x + team * (int)gridDim.x; p < P; p += teams * (int)gridDim.x) {
                if (sm.ids[p] < 0) continue;
                float f[16];
                load_block16(f, a.h + (int64_t)p * a.F, wt);
                moe_rot_quant(f, wt, nw, 1 + team, a.act, a.F, a.hq + (int64_t)p * a.F, a.sh + p, a.rh + p,
                              sm.red.f + team * nw, sm.red.i + team * nw, sm.red.d + team * nw);
                bar_sync_n(1 + team, 32 * nw);  // the slots of red are written again
            }
        }
    }
    if (!moe_grid_sync(a.barrier, 2, &sm.flag)) return;
    // ---------------- down ----------------
    moe_contract<false, CONV>(a, sm, dyn);
    if (!moe_grid_sync(a.barrier, 3, &sm.flag)) return;
    // ---------------- sum over the slots ----------------
    const int nv = a.D / 4;
    for (int i = (int)blockIdx.x * kMoeThreads + (int)threadIdx.x; i < a.M * nv; i += (int)gridDim.x * kMoeThreads) {
        const int m = i / nv, c = i - m * nv;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < a.k; ++j) {
            const int p = m * a.k + j;
            if (sm.ids[p] < 0) continue;
            const float w = sm.w[p];
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.out + (int64_t)p * a.D) + c);
            s = make_float4(__fmaf_rn(w, v.x, s.x), __fmaf_rn(w, v.y, s.y), __fmaf_rn(w, v.z, s.z), __fmaf_rn(w, v.w, s.w));
        }
        reinterpret_cast<float4 *>(a.y)[i] = s;
    }
}

}  // namespace tq
