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
// The least it could take is the time of the chosen experts' packed weights, read once
// (3 D F / 4 bytes each).  What bounds it is the chain of dependent phases and the waits
// between them: no pipe is full (64 tokens of 2048 x 1536, 8 of 128 experts: DRAM 41 %,
// issue slots 40 %, ALU 36 %; of 1536 x 6144, 2 of 8: 12, 34, 30 %), and the first stall
// is a barrier.  One token of 512 x 1024, 2 of 8 experts: 14.6 us.  64 tokens of 2048 x
// 1536, 8 of 128 experts: 94.9 us (302 MB, 3.2 TB/s over all).  With the choice given:
// 13.4 and 84.7 us.
//
//   tq_moe_route_kernel: a CTA per token quantises it; the other CTAs compute the
//     logits of 8 experts and four tokens each.
//   tq_moe_experts_kernel: one CTA per SM, launched cooperatively (all CTAs
//     resident), with grid-wide barriers between its phases:
//       choice     every CTA picks every token's experts (for up to 16 tokens that
//                  is cheaper than another barrier) and sorts the (token, slot)
//                  pairs by expert; an expert and up to 8 of its pairs are one
//                  "problem".
//       gate, up   a strip is 16 rows of both matrices, so that the activation
//                  follows in registers.  The strips of all problems are split
//                  into contiguous runs, one per CTA; the quantised tokens of a
//                  run's problem sit in shared memory.
//       rotation   a team of F / 512 warps per pair: FWHT, int8 codes.
//       down       strips of 32 rows, runs as before.
//       sum        y from the pairs' outputs, slots in order: no atomics, and
//                  the result does not depend on how pairs were grouped.
//       For up to 16 pairs, where it costs few steps more, a CTA contracts a strip
//       of down for every pair at once and adds them itself: down and sum without
//       the barrier between them (about 2 us).
//   A warp streams its strips' weights from HBM by asynchronous copies into a ring
//   of its own, two or four column steps (of 2 KB) ahead, across strips and problems,
//   and into the down phase from before the rotation; a lane reads only what it
//   copied itself, so the ring needs no barrier.  They are
//   contracted with mma.sync (u8 codes x s8), whose rate is no bound here; the logic
//   operations that spread the codes run at half the rate of the others, which is
//   why a code stays where it is in its byte: field j is masked in place, counts
//   4^j-fold and has sums of its own.  (Spreading them to fp16 for the twice as wide
//   fp16 mma.sync took more of them: 149 us instead of 127 at 64 x 2048 x 1536 of
//   128 experts.)
#pragma once

#include "tq_act.cuh"
#include "tq_common.cuh"
#include "tq_gemv.cuh"

namespace tq {

constexpr int kMoeWarps = 16;
constexpr int kMoeThreads = 32 * kMoeWarps;
constexpr int kMoeMaxTokens = 64, kMoeMaxTopk = 16, kMoeMaxExperts = 256;
constexpr int kMoeMaxPairs = kMoeMaxTokens * kMoeMaxTopk;
constexpr int kMoeChunk = 8;  // pairs of one expert per problem: the MMA's 8 columns
constexpr int kMoeFew = 2 * kMoeChunk;  // pairs whose codes fit the two buffers at once: tq_moe_experts_kernel<.., FEW>
constexpr int kMoeMaxProblems = kMoeMaxExperts + kMoeMaxPairs / kMoeChunk;
constexpr int kMoeMaxK = 8192;  // d_model, d_ffn: 16 blocks of 512, one per warp
constexpr int kMoeRouteTokens = 4, kMoeRouteExperts = 8;  // logits per CTA
constexpr int kMoeSlot = 8 * 32;  // 32-bit words of a warp's exchange slot
constexpr int kMoeRedBytes = kMoeWarps * kMoeSlot * 4;
static_assert(kMoeRedBytes >= kMoeMaxPairs / 32 * kMoeMaxExperts * 2, "the pair counts fit the exchange slots");

struct MoeArgs {
    const float *x, *router;  // [M][D], [E][D] or nullptr (ids, weights given)
    const uint8_t *gate, *up, *down;
    const float *gate_gamma, *up_gamma, *down_gamma;
    float *y;
    int32_t *ids;  // [M][k]
    float *weights;
    int M, D, F, E, k;
    int per_row, norm_topk, enc;
    double inv_d, inv_f;  // 1 / D, 1 / F
    // Quotients by the number of CTAs n (of less than 2^36 / n) and by a problem's
    // strips (of less than 2^32 / strips): ceil(2^36 / n), ceil(2^32 / strips).
    uint64_t by_grid;
    uint32_t by_gate, by_down;
    uint32_t by_d, by_f;       // the same for the 16-byte chunks of a token row, D / 16 and F / 16
    uint32_t by_k, by_groups;  // ceil(2^16 / k), ceil(2^16 / the route kernel's groups of tokens)
    uint32_t by_warps;         // ceil(2^8 / (F / 512))
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

// Warp-wide maximum of non-negative values: their bits order as unsigned numbers
// (a NaN's above all), and one instruction replaces five exchanges.
__device__ __forceinline__ float warp_max_nonneg(float v) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// FWHT-512 and int8 codes of a row held by a team of nw warps (warp wt has block
// wt, 16 values per lane as in tq_act.cuh; red: the team's slots).  The steps and
// roundings of tq_prologue_fwht_kernel; the codes are written in the small-M
// GEMV's layout.
__device__ __forceinline__ void moe_rot_quant(float (&f)[16], int wt, int nw, int bar, const ActParams &p, double inv_k,
                                              int8_t *__restrict__ dst, float *__restrict__ s, int32_t *__restrict__ rowsum,
                                              float *redf, int *redi, double *redd) {
    const int lane = threadIdx.x & 31;
    if (p.sanitize) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = quench(f[i], p.eta_max);
    }
    if (p.rmsnorm) {
        double sq[4] = {0.0, 0.0, 0.0, 0.0};  // four chains: this is on the critical path
#pragma unroll
        for (int i = 0; i < 16; ++i) sq[i & 3] = __fma_rn((double)f[i], (double)f[i], sq[i & 3]);
        double ss = warp_sum_d(__dadd_rn(__dadd_rn(sq[0], sq[1]), __dadd_rn(sq[2], sq[3])));
        if (lane == 0) redd[wt] = ss;
        bar_sync_n(bar, 32 * nw);
        ss = lane < nw ? redd[lane] : 0.0;
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) ss = __dadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, off));
        ss = __shfl_sync(0xffffffffu, ss, 0);
        // within 2 units of fp64 of 1 / sqrt(ss / K + eps)
        const double r = rsqrt(__fma_rn(ss, inv_k, (double)p.rms_eps));
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = __double2float_rn(__dmul_rn((double)f[i], r));
    }
    fwht512_regs(f, true);
    // Maxima by the values' bits: a NaN's are above all others', makes the scale NaN, and
    // with it every output of this row.
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
    float amax = warp_max_nonneg(__uint_as_float(top));
    if (lane == 0) redf[wt] = amax;
    bar_sync_n(bar, 32 * nw);
    amax = warp_max_nonneg(lane < nw ? redf[lane] : 0.0f);
    const float eta = amax != amax ? amax : eta_of(amax, p);
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
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) redi[wt] = sum;
    bar_sync_n(bar, 32 * nw);
    if (wt == 0) {
        sum = __reduce_add_sync(0xffffffffu, lane < nw ? redi[lane] : 0);
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

// CTAs 0 .. M - 1: token blockIdx.x's codes.  The others: logits of 8 experts and
// 4 tokens, a warp for 2 experts and a quarter of d_model (so that few tokens
// still spread over many lanes); the quarters are added in order.  Two CTAs per
// SM: the largest batches of 128 experts then take little more than one wave.
// Bound by latency: L2 loads, then one chain of fp64 sums.  64 tokens of 2048, 64
// experts, cold: 11.2 us.
__global__ void __launch_bounds__(kMoeThreads, 2) tq_moe_route_kernel(const __grid_constant__ MoeArgs a) {
    __shared__ MoeRed red;
    __shared__ double part[kMoeWarps][2 * kMoeRouteTokens];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.barrier = 0;
    if ((int)blockIdx.x < a.M) {
        const int nw = a.D / 512, m = blockIdx.x;
        if (warp >= nw) return;
        float f[16];
        load_block16(f, a.x + (int64_t)m * a.D, warp);
        moe_rot_quant(f, warp, nw, 1, a.act, a.inv_d, a.xq + (int64_t)m * a.D, a.sx + m, a.rs + m, red.f, red.i, red.d);
        return;
    }
    const int u = blockIdx.x - a.M, tgroups = (a.M + kMoeRouteTokens - 1) / kMoeRouteTokens;
    const int eg = (int)((unsigned)u * a.by_groups >> 16);
    const int e0 = eg * kMoeRouteExperts + (warp >> 2) * 2, m0 = (u - eg * tgroups) * kMoeRouteTokens;
    const int nt = a.M - m0 < kMoeRouteTokens ? a.M - m0 : kMoeRouteTokens;
    const int nv = a.D / 4, q0 = (warp & 3) * (nv / 4);  // float4; a quarter is a multiple of 32
    const float4 *wr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)  // experts past the last: the last again, not stored
        wr[i] = reinterpret_cast<const float4 *>(a.router + (int64_t)(e0 + i < a.E ? e0 + i : a.E - 1) * a.D) + q0 + lane;
    const float4 *xr = reinterpret_cast<const float4 *>(a.x + (int64_t)m0 * a.D) + q0 + lane;
    double s[2][kMoeRouteTokens];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < kMoeRouteTokens; ++t) s[i][t] = 0.0;
    for (int c = 0; c < nv / 4; c += 32) {
        float4 w[2], v[kMoeRouteTokens];
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = __ldg(wr[i] + c);
#pragma unroll
        for (int t = 0; t < kMoeRouteTokens; ++t)
            if (t < nt) v[t] = __ldg(xr + (int64_t)t * nv + c);
#pragma unroll
        for (int t = 0; t < kMoeRouteTokens; ++t) {
            if (t >= nt) break;
            if (a.act.sanitize) v[t] = quench4(v[t], a.act);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s[i][t] = __fma_rn((double)v[t].x, (double)w[i].x, s[i][t]);
                s[i][t] = __fma_rn((double)v[t].y, (double)w[i].y, s[i][t]);
                s[i][t] = __fma_rn((double)v[t].z, (double)w[i].z, s[i][t]);
                s[i][t] = __fma_rn((double)v[t].w, (double)w[i].w, s[i][t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kMoeRouteTokens; ++t) {
        if (t >= nt) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const double v = warp_sum_d(s[i][t]);
            if (lane == 0) part[warp][2 * t + i] = v;
        }
    }
    __syncthreads();
    if (threadIdx.x < kMoeRouteExperts * nt) {
        const int t = threadIdx.x / kMoeRouteExperts, i = threadIdx.x % kMoeRouteExperts, e = eg * kMoeRouteExperts + i;
        double v = 0.0;
#pragma unroll
        for (int q = 0; q < 4; ++q) v = __dadd_rn(v, part[(i >> 1) * 4 + q][2 * t + (i & 1)]);
        if (e < a.E) a.logits[(int64_t)(m0 + t) * a.E + e] = __double2float_rn(v);
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
        // release: what this CTA's threads wrote before the barrier above included
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(counter) : "memory");
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
    }
    __syncthreads();
    return *flag != 0;
}

// Adds one column step (256 codes) of two sets of 16 rows to the sums.  w: this
// lane's 16 bytes of rows g and g + 8 of each set, in shared memory 512 bytes
// apart.  Field j of a word enters the MMA masked in place (code times 4^j) and
// has an accumulator d[j] of its own.  xr: this lane's token row in shared memory
// at the step's column; xsw: its chunk swizzle.
template <bool CONV>
__device__ __forceinline__ void moe_step_mma(int (&d)[4][2][4], uint32_t w, uint32_t xr, uint32_t xsw, int enc) {
    uint32_t c[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const uint4 v = lds128(w + 512 * r);
        c[r][0] = v.x;
        c[r][1] = v.y;
        c[r][2] = v.z;
        c[r][3] = v.w;
        if (CONV)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[r][i] = codes_to_foundry(c[r][i], enc);
    }
#pragma unroll
    for (int pr = 0; pr < 2; ++pr) {
        const uint4 u = lds128(xr + ((uint32_t)(32 * pr) ^ xsw)), v = lds128(xr + ((uint32_t)(32 * pr + 16) ^ xsw));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t msk = 0x03030303u << (2 * j);
            const uint32_t x0 = j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w;
            const uint32_t x1 = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
#pragma unroll
            for (int mat = 0; mat < 2; ++mat)
                mma_16x8x32_u8s8_pure(d[j][mat], c[2 * mat][2 * pr] & msk, c[2 * mat + 1][2 * pr] & msk,
                                      c[2 * mat][2 * pr + 1] & msk, c[2 * mat + 1][2 * pr + 1] & msk, x0, x1);
        }
    }
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_groups() {  // all but the last N groups have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// clamp(SiLU(g) u), in fp64, rounded once before the clamp; a NaN stays one
__device__ __forceinline__ float moe_act(float g, float u, float c) {
    const double gd = (double)g;
    const float v = __double2float_rn(__dmul_rn(__ddiv_rn(gd, __dadd_rn(1.0, exp(-gd))), (double)u));
    return v != v ? v : fminf(fmaxf(v, -c), c);
}

// A problem: expert, its pairs sorted[start .. start + count).
struct MoeProblem {
    int16_t expert, start, count;
};

struct MoeShared {
    int ids[kMoeMaxPairs];
    float w[kMoeMaxPairs];
    int16_t sorted[kMoeMaxPairs];
    int16_t count[kMoeMaxExperts], first[kMoeMaxExperts];
    MoeProblem prob[kMoeMaxProblems];
    int16_t where[kMoeFew];  // of up to so many pairs: problem << 8 | place in it
    float few_s[kMoeFew];    // the scales and sums of codes that a CTA computes itself
    int few_r[kMoeFew];
    int nprob, flag;
    MoeRed red;
};

// This CTA's share of a contraction phase: a run of consecutive strips of all
// problems' strips.  GATE: a strip is rows n0 .. n0 + 15 of gate and up, giving
// activations; else rows n0 .. n0 + 31 of down, giving outputs.  Teams of ks warps
// share a strip's column steps, where the run's strips would leave warps without
// work in its last rounds.
struct MoeRun {
    int s0, s1;
    int lg, ks, team, kw;  // ks = 2^lg warps per strip; this warp's team and place in it
    int mine;          // its column steps kw, kw + ks, ... of a strip
    int spp;           // strips per problem
    // the next step to request: problem, strip, step; strips of that problem end at `end`
    int q, strip, end, i;
};

__device__ __forceinline__ void moe_team(MoeRun &r, int lg, int steps) {
    const int warp = threadIdx.x >> 5;
    r.lg = lg;
    r.ks = 1 << lg;
    r.team = warp >> lg;
    r.kw = warp & (r.ks - 1);
    r.mine = (steps - r.kw + r.ks - 1) >> lg;
    r.i = 0;
}

template <bool GATE>
__device__ __forceinline__ MoeRun moe_run(const MoeArgs &a, const MoeShared &sm) {
    MoeRun r;
    r.spp = GATE ? a.F / 16 : a.D / 32;
    const unsigned total = sm.nprob * r.spp, b = blockIdx.x;  // at most 384 x 512 strips
    const int steps = (GATE ? a.D : a.F) / 256;
    r.s0 = (int)((total * b) * a.by_grid >> 36);
    r.s1 = (int)((total * (b + 1)) * a.by_grid >> 36);
    const unsigned by = GATE ? a.by_gate : a.by_down;
    r.q = (int)__umulhi((unsigned)r.s0, by);
    // the run's strips in its first problem, whole problems, strips in the last one
    const int first = min(r.s1 - r.s0, (r.q + 1) * r.spp - r.s0), rest = r.s1 - r.s0 - first;
    const int whole = (int)__umulhi((unsigned)rest, by), last = rest - whole * r.spp;
    // A round of all teams takes a strip's steps, shared, and with more than one warp
    // the exchange of sums, about two steps.  64 tokens of 1536 x 6144, 8 experts:
    // 60.2 us, 61.6 us with one warp per strip; 2 of 7168 x 2048, 8 of 256: 68.7 to
    // 80.5 us; without the exchange's term 64 of 2048 x 1536, 8 of 128: 159 to 97 us.
    int best = 0, least = 0x7fffffff;
#pragma unroll
    for (int lg = 0; lg <= 4; ++lg) {
        const int up = (kMoeWarps >> lg) - 1, down = 4 - lg;
        const int rounds = ((first + up) >> down) + whole * ((r.spp + up) >> down) + ((last + up) >> down);
        const int cost = rounds * (((steps + (1 << lg) - 1) >> lg) + (lg > 0 ? 2 : 0));
        if (cost < least && (1 << lg) <= steps) {
            least = cost;
            best = lg;
        }
    }
    moe_team(r, best, steps);
    r.strip = r.s0 - r.q * r.spp + r.team;
    r.end = min(r.s1 - r.q * r.spp, r.spp);
    return r;
}

// The down phase with its sum: this CTA's strips blockIdx.x, + gridDim.x, ..., a team
// of warps per problem.  False where a warp's steps are more
// than four above the other form's: 8 tokens of 1536 x 6144, 12 steps to 6, took
// 39.6 us to 37.4 us; 4 of 2048 x 1536, 3 steps to 3, 24.0 us to 26.5 us.
// `r` is the other form's run, and becomes this one's.
__device__ __forceinline__ bool moe_run_joint(const MoeArgs &a, const MoeShared &sm, MoeRun &r) {
    if (sm.nprob == 0) return false;
    const int steps = a.F / 256, n = (int)gridDim.x;
    int mine = 4;
    while (mine > 0 && ((kMoeWarps >> mine) < sm.nprob || (1 << mine) > steps)) --mine;
    // the other form's, for the longest run (every CTA must come to the same form)
    const auto over_grid = [&](int v) { return (int)((unsigned)(v + n - 1) * a.by_grid >> 36); };
    const int run = over_grid(sm.nprob * r.spp);
    int apart = 0x7fffffff;
#pragma unroll
    for (int lg = 0; lg <= 4; ++lg)
        if ((1 << lg) <= steps)
            apart = min(apart, ((run + (kMoeWarps >> lg) - 1) >> (4 - lg)) * ((steps + (1 << lg) - 1) >> lg));
    if (over_grid(r.spp) * ((steps + (1 << mine) - 1) >> mine) > apart + 4) return false;
    moe_team(r, mine, steps);
    r.q = r.team;
    r.s1 = (r.q + 1) * r.spp;
    r.strip = (int)blockIdx.x;
    r.end = r.team < sm.nprob ? r.spp : 0;
    return true;
}

// Requests the next step of this warp's run into a slot of its ring: one group, an
// empty one past the end.
template <bool GATE, bool JOINT = false>
__device__ __forceinline__ void moe_load(const MoeArgs &a, const MoeShared &sm, MoeRun &r, uint32_t slot) {
    while (r.strip >= r.end) {  // on to the next problem of the run
        if ((r.q + 1) * r.spp >= r.s1) break;
        ++r.q;
        r.strip = r.team;
        r.end = min(r.s1 - r.q * r.spp, r.spp);
    }
    if (r.strip < r.end) {
        const int lane = threadIdx.x & 31, N = GATE ? a.F : a.D, KB = (GATE ? a.D : a.F) / 4;
        const int64_t off = ((int64_t)sm.prob[r.q].expert * N + r.strip * (GATE ? 16 : 32) + (lane >> 2)) * KB + 16 * (lane & 3) +
                            64 * (r.kw + r.ks * r.i);
        const uint8_t *p = (GATE ? a.gate : a.down) + off, *q = GATE ? a.up + off : p + 16 * KB;
        cp_async16(slot, p);
        cp_async16(slot + 512, p + 8 * KB);
        cp_async16(slot + 1024, q);
        cp_async16(slot + 1536, q + 8 * KB);
        if (++r.i == r.mine) {
            r.i = 0;
            r.strip += JOINT ? (int)gridDim.x : kMoeWarps >> r.lg;
        }
    }
    cp_async_commit();
}

__device__ __forceinline__ int moe_token(const MoeArgs &a, int p) { return (int)((unsigned)p * a.by_k >> 16); }  // p / k

// A problem's token codes into shared memory (not committed).
template <bool GATE>
__device__ __forceinline__ void moe_stage(const MoeArgs &a, const MoeShared &sm, const MoeProblem &pb, uint32_t x_s) {
    const int K = GATE ? a.D : a.F, XS = gemv_x_stride(K), cpr = K >> 4;
    for (int i = threadIdx.x; i < pb.count * cpr; i += kMoeThreads) {
        const int r = (int)__umulhi((unsigned)i, GATE ? a.by_d : a.by_f), c = i - r * cpr;
        const int p = sm.sorted[pb.start + r];
        cp_async16(x_s + (uint32_t)(r * XS + 16 * c), (GATE ? a.xq + (int64_t)moe_token(a, p) * K : a.hq + (int64_t)p * K) + 16 * c);
    }
}

// This warp's sums of a strip: its steps from the ring, which goes on behind them.
template <bool GATE, bool JOINT, bool CONV, int PD>
__device__ __forceinline__ void moe_strip_sums(const MoeArgs &a, const MoeShared &sm, MoeRun &run, uint32_t ring, int &slot,
                                               uint32_t xr, uint32_t xsw, int (&acc)[2][4]) {
    int d[4][2][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j][0][i] = d[j][1][i] = 0;
#pragma unroll 1
    for (int i = 0; i < run.mine; ++i) {
        cp_async_wait_groups<PD - 1>();
        const uint32_t from = ring + (uint32_t)(slot * 2048);
        moe_step_mma<CONV>(d, from, xr + (uint32_t)(256 * run.ks * i), xsw, a.enc);
        moe_load<GATE, JOINT>(a, sm, run, from);  // the slot takes the step PD ahead
        slot = slot + 1 == PD ? 0 : slot + 1;
    }
#pragma unroll
    for (int mat = 0; mat < 2; ++mat)
#pragma unroll
        for (int i = 0; i < 4; ++i)  // exact: d[j] is a multiple of 4^j
            acc[mat][i] = d[0][mat][i] + (d[1][mat][i] >> 2) + (d[2][mat][i] >> 4) + (d[3][mat][i] >> 6);
}

// The team's sums, in its first warp.
__device__ __forceinline__ void moe_team_sums(int (&acc)[2][4], const MoeRun &run, int *red) {
    if (run.ks == 1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (run.kw != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) red[warp * kMoeSlot + i * 32 + lane] = acc[i >> 2][i & 3];
    }
    bar_sync_n(1 + run.team, 32 * run.ks);
    if (run.kw == 0) {
        for (int w2 = warp + 1; w2 < warp + run.ks; ++w2)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i >> 2][i & 3] += red[w2 * kMoeSlot + i * 32 + lane];
    }
    bar_sync_n(1 + run.team, 32 * run.ks);  // the slots are written again
}

// A strip's projections (matrix, row, token) at [matrix][token / 2][(16 (token % 2) + row + 8 (token / 2)) % 32].
__device__ __forceinline__ int moe_value_at(int tok, int row) { return 32 * (tok >> 1) + ((16 * (tok & 1) + row + 8 * (tok >> 1)) & 31); }
__device__ __forceinline__ void moe_values(float *val, const int (&acc)[2][4], const float (&ga)[2], const float (&gb)[2],
                                           const float (&sv)[2], const int (&rv)[2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int hi = 0; hi < 2; ++hi)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = 2 * hi + e, to = moe_value_at(2 * t + e, g + 8 * hi);
            val[to] = __fmul_rn(__int2float_rn(acc[0][c] - rv[e]), __fmul_rn(ga[hi], sv[e]));
            val[128 + to] = __fmul_rn(__int2float_rn(acc[1][c] - rv[e]), __fmul_rn(gb[hi], sv[e]));
        }
}

// Token m's weights, by one warp.  mine: the logit of slot `lane`; top: the largest.
__device__ __forceinline__ void moe_weights(const MoeArgs &a, MoeShared &sm, int m, float mine, float top) {
    const int lane = threadIdx.x & 31;
    const double ex = lane < a.k ? exp((double)mine - (double)top) : 0.0;
    double den = ex;
    if (!a.norm_topk) {
        den = 0.0;
        for (int e = lane; e < a.E; e += 32) den = __dadd_rn(den, exp((double)__ldcg(a.logits + (int64_t)m * a.E + e) - (double)top));
    }
    den = warp_sum_d(den);
    if (lane < a.k) {
        const float w = __double2float_rn(__ddiv_rn(ex, den));
        sm.w[m * a.k + lane] = w;
        if (a.M > kMoeWarps || blockIdx.x == 0) a.weights[m * a.k + lane] = w;
    }
}

// The run, the first PD steps of each warp requested before.  While a problem's
// strips are contracted, the next one's codes are copied to the other buffer; the
// ring goes on from strip to strip and problem to problem.
template <bool GATE, bool CONV, int PD>
__device__ __forceinline__ void moe_contract(const MoeArgs &a, const MoeShared &sm, MoeRun &run, uint32_t ring, uint32_t x_s,
                                             int *red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = run.team, kw = run.kw, T = kMoeWarps >> run.lg, spp = run.spp;
    const int g = lane >> 2, t = lane & 3;
    const int K = GATE ? a.D : a.F, N = GATE ? a.F : a.D, XS = gemv_x_stride(K);
    const uint32_t xsw = (uint32_t)(t & 2) << 4;
    float *val = reinterpret_cast<float *>(red + warp * kMoeSlot);
    if (run.s0 >= run.s1) return;
    int buf = 0;
    const int q0 = (int)__umulhi((unsigned)run.s0, GATE ? a.by_gate : a.by_down);
    moe_stage<GATE>(a, sm, sm.prob[q0], x_s);
    cp_async_commit();
    cp_async_wait_groups<0>();
    __syncthreads();
    int slot = 0;
    for (int at = run.s0, q = q0; at < run.s1; ++q) {
        const int first = q * spp, end = min(run.s1, first + spp);
        const MoeProblem pb = sm.prob[q];
        const bool more = end < run.s1;
        if (more) moe_stage<GATE>(a, sm, sm.prob[q + 1], x_s + (uint32_t)((buf ^ 1) * kMoeChunk * XS));
        cp_async_commit();
        // this lane's tokens of a fragment: 2 t and 2 t + 1
        float sv[2];
        int rv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * t + e < pb.count ? 2 * t + e : 0;
            const int p = sm.sorted[pb.start + i], src = GATE ? moe_token(a, p) : p;
            sv[e] = __ldcg((GATE ? a.sx : a.sh) + src);
            rv[e] = __ldcg((GATE ? a.rs : a.rh) + src);
        }
        // token g of the problem (past the last: sums that are not used)
        const uint32_t xr = x_s + (uint32_t)((buf * kMoeChunk + (g < pb.count ? g : pb.count - 1)) * XS + 64 * t + 256 * kw);
        int committed = 0;  // groups of steps since the next problem's codes
        for (int s = at - first + team; s < end - first; s += T) {
            const int n0 = s * (GATE ? 16 : 32);
            // the strip's gammas, wanted at its end
            float ga[2], gb[2];
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const int64_t n = a.per_row ? (int64_t)pb.expert * N + n0 + g + 8 * hi : pb.expert;
                ga[hi] = __ldg((GATE ? a.gate_gamma : a.down_gamma) + n);
                gb[hi] = __ldg(GATE ? a.up_gamma + n : a.down_gamma + n + (a.per_row ? 16 : 0));
            }
            int acc[2][4];
            moe_strip_sums<GATE, false, CONV, PD>(a, sm, run, ring, slot, xr, xsw, acc);
            committed += run.mine;
            moe_team_sums(acc, run, red);
            if (kw != 0) continue;
            // The projections' values pass through this warp's own slot, so that the
            // lanes share what follows evenly and stores cover whole rows' stretches.
            __syncwarp();  // the slot's last readers are done
            moe_values(val, acc, ga, gb, sv, rv);
            __syncwarp();
            if (GATE) {
                for (int i = lane; i < 16 * pb.count; i += 32) {
                    const int tok = i >> 4, row = i & 15, from = moe_value_at(tok, row);
                    a.h[(int64_t)sm.sorted[pb.start + tok] * N + n0 + row] = moe_act(val[from], val[128 + from], a.clamp_val);
                }
            } else {
                for (int tok = 0; tok < pb.count; ++tok) {
                    a.out[(int64_t)sm.sorted[pb.start + tok] * N + n0 + lane] = val[128 * (lane >> 4) + moe_value_at(tok, lane & 15)];
                }
            }
        }
        if (more) {
            // the next problem's codes are in: older than the last PD - 1 groups, if so many follow them
            if (committed >= PD - 1)
                cp_async_wait_groups<PD - 1>();
            else
                cp_async_wait_groups<0>();
            __syncthreads();
            buf ^= 1;
        }
        at = end;
    }
}

// The down phase with its sum (moe_run_joint), the first steps requested before.
template <bool CONV, int PD>
__device__ __forceinline__ void moe_down_joint(const MoeArgs &a, const MoeShared &sm, MoeRun &run, uint32_t ring, uint32_t x_s,
                                               int *red, bool here) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int K = a.F, XS = gemv_x_stride(K), cpr = K >> 4;
    const MoeProblem last = sm.prob[sm.nprob - 1];
    // every pair's codes, at most 16 rows (the two buffers' room), in sorted order
    if (!here) {
        for (int i = threadIdx.x; i < (last.start + last.count) * cpr; i += kMoeThreads) {
            const int r = (int)__umulhi((unsigned)i, a.by_f), c = i - r * cpr;
            cp_async16(x_s + (uint32_t)(r * XS + 16 * c), a.hq + (int64_t)sm.sorted[r] * K + 16 * c);
        }
        cp_async_commit();
    }
    const bool active = run.team < sm.nprob;
    const MoeProblem pb = sm.prob[active ? run.team : 0];
    float sv[2];
    int rv[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = pb.start + min(2 * t + e, pb.count - 1), p = sm.sorted[i];
        sv[e] = here ? sm.few_s[i] : __ldcg(a.sh + p);
        rv[e] = here ? sm.few_r[i] : __ldcg(a.rh + p);
    }
    const uint32_t xr = x_s + (uint32_t)((pb.start + min(g, pb.count - 1)) * XS + 64 * t + 256 * run.kw);
    const uint32_t xsw = (uint32_t)(t & 2) << 4;
    if (!here) {
        cp_async_wait_groups<0>();
        __syncthreads();
    }
    int slot = 0;
    for (int s = (int)blockIdx.x; s < run.spp; s += (int)gridDim.x) {
        const int n0 = 32 * s;
        if (active) {
            float ga[2], gb[2];
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const int64_t n = a.per_row ? (int64_t)pb.expert * a.D + n0 + g + 8 * hi : pb.expert;
                ga[hi] = __ldg(a.down_gamma + n);
                gb[hi] = __ldg(a.down_gamma + n + (a.per_row ? 16 : 0));
            }
            int acc[2][4];
            moe_strip_sums<false, true, CONV, PD>(a, sm, run, ring, slot, xr, xsw, acc);
            moe_team_sums(acc, run, red);
            if (run.kw == 0) moe_values(reinterpret_cast<float *>(red + warp * kMoeSlot), acc, ga, gb, sv, rv);
        }
        __syncthreads();
        if (warp < a.M) {  // a warp per token, a lane per output
            float y = 0.0f;
            for (int j = 0; j < a.k; ++j) {
                const int p = warp * a.k + j;
                if (sm.ids[p] < 0) continue;
                const int q = sm.where[p] >> 8, tok = sm.where[p] & 255;
                const float *val = reinterpret_cast<const float *>(red + q * run.ks * kMoeSlot);
                y = __fmaf_rn(sm.w[p], val[128 * (lane >> 4) + moe_value_at(tok, lane & 15)], y);
            }
            a.y[(int64_t)warp * a.D + n0 + lane] = y;
        }
        __syncthreads();  // the values are written again
    }
    cp_async_wait_groups<0>();
}

// PD: column steps in each warp's ring (4, or 2 where longer token rows need the room).
// FEW: at most kMoeFew pairs.
template <bool CONV, int PD, bool FEW>
__global__ void __launch_bounds__(kMoeThreads, 1) tq_moe_experts_kernel(const __grid_constant__ MoeArgs a) {
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ MoeShared sm;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = a.M * a.k;

    unsigned phase = 0;  // grid barriers passed

    // ---------------- choice ----------------
    // Up to 16 tokens, a warp of every CTA for each; more, a CTA for each, and the
    // others read its choice after a barrier.
    const bool spread = a.router && a.M > kMoeWarps;
    float slot_logit = 0.0f, top_logit = 0.0f;
    for (int m = spread ? (int)blockIdx.x : warp; m < a.M; m += spread ? (int)gridDim.x : kMoeWarps) {
        if (!a.router || (spread && warp != 0)) break;
        constexpr int V = kMoeMaxExperts / 32;
        float l[V];
        uint32_t key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            l[i] = e < a.E ? __ldcg(a.logits + (int64_t)m * a.E + e) : 0.0f;
            key[i] = e < a.E ? moe_key(l[i]) : 0u;
        }
        // this lane's best expert not chosen yet (key, index; the lowest index of equals)
        uint32_t used = 0, best = 0, at = 0xffffu;
        float val = 0.0f, top = 0.0f, mine = 0.0f;  // its logit; the largest logit; the logit of slot `lane`
        auto scan = [&]() {
            best = 0;
            at = 0xffffu;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (32 * i >= a.E) break;
                const bool free = lane + 32 * i < a.E && !(used >> i & 1u);
                if (free && (at == 0xffffu || key[i] > best)) {
                    best = key[i];
                    at = (uint32_t)(lane + 32 * i);
                    val = l[i];
                }
            }
        };
        scan();
        int my_id = 0;
        for (int j = 0; j < a.k; ++j) {
            const uint32_t most = __reduce_max_sync(0xffffffffu, best);
            const uint32_t id = __reduce_min_sync(0xffffffffu, best == most ? at : 0xffffu);
            const float v = __shfl_sync(0xffffffffu, val, id & 31);
            if (j == 0) top = v;
            if (lane == j) {
                my_id = (int)id;
                mine = v;
            }
            if ((int)(id & 31) == lane) {
                used |= 1u << (id >> 5);
                scan();
            }
        }
        if (lane < a.k) {
            sm.ids[m * a.k + lane] = my_id;
            if (spread || blockIdx.x == 0) a.ids[m * a.k + lane] = my_id;
        }
        if (spread) moe_weights(a, sm, m, mine, top);
        slot_logit = mine;
        top_logit = top;
    }
    if (spread && !moe_grid_sync(a.barrier, ++phase, &sm.flag)) return;
    if (!a.router || spread)
        for (int p = threadIdx.x; p < P; p += kMoeThreads) {
            const int id = __ldcg(a.ids + p);
            sm.ids[p] = id >= 0 && id < a.E ? id : -1;
            sm.w[p] = __ldcg(a.weights + p);
        }
    if constexpr (FEW) {
        // One warp groups the pairs, experts in the order of their first pairs.
        __syncthreads();
        if (warp == 0) {
            const int id = lane < P ? sm.ids[lane] : -1;
            const uint32_t same = __match_any_sync(0xffffffffu, id);
            const int rank = __popc(same & ((1u << lane) - 1u)), c = id >= 0 && rank == 0 ? __popc(same) : 0;
            const int n = (c + kMoeChunk - 1) / kMoeChunk;
            int both = c | (n << 16);  // running sums of pairs and of problems
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, both, off);
                if (lane >= off) both += v;
            }
            const int total = __shfl_sync(0xffffffffu, both, 31);
            const int mine = both - (c | (n << 16)), lead = __shfl_sync(0xffffffffu, mine, __ffs(same) - 1);
            if (id >= 0) {  // lanes below P
                sm.sorted[(lead & 0xffff) + rank] = (int16_t)lane;
                sm.where[lane] = (int16_t)(((lead >> 16) + rank / kMoeChunk) << 8 | rank % kMoeChunk);
            }
            for (int i = 0; i < n; ++i) {
                MoeProblem pb;
                pb.expert = (int16_t)id;
                pb.start = (int16_t)((mine & 0xffff) + i * kMoeChunk);
                pb.count = (int16_t)min(c - i * kMoeChunk, kMoeChunk);
                sm.prob[(mine >> 16) + i] = pb;
            }
            if (lane == 0) sm.nprob = total >> 16;
        }
        __syncthreads();
    } else {
        // Pairs by expert, in order (every CTA must come to the same grouping).  Warps
        // rank the pairs of 32 at a time among those of the same expert and count them;
        // a thread per expert turns its counts into offsets.
        const int nch = (P + 31) / 32;
        uint16_t *counts = reinterpret_cast<uint16_t *>(dyn);  // [nch][E]
        for (int i = threadIdx.x; i < nch * a.E; i += kMoeThreads) counts[i] = 0;
        __syncthreads();
        int id_of[2] = {-1, -1}, rank[2] = {0, 0};  // chunks warp and warp + 16
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int ch = warp + kMoeWarps * c, p = 32 * ch + lane;
            if (ch >= nch) break;
            const int id = p < P ? sm.ids[p] : -1;
            const uint32_t same = __match_any_sync(0xffffffffu, id);
            id_of[c] = id;
            rank[c] = __popc(same & ((1u << lane) - 1u));
            if (id >= 0 && rank[c] == 0) counts[ch * a.E + id] = (uint16_t)__popc(same);
        }
        __syncthreads();
        if ((int)threadIdx.x < a.E) {
            int n = 0;
            for (int ch = 0; ch < nch; ++ch) {
                const int c = counts[ch * a.E + threadIdx.x];
                counts[ch * a.E + threadIdx.x] = (uint16_t)n;
                n += c;
            }
            sm.count[threadIdx.x] = (int16_t)n;
        }
        __syncthreads();
        if (warp == 0) {
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
                    sm.first[e] = (int16_t)(at + cs - c);
                    for (int i = 0; i < n; ++i) {
                        MoeProblem pb;
                        pb.expert = (int16_t)e;
                        pb.start = (int16_t)(at + cs - c + i * kMoeChunk);
                        pb.count = (int16_t)(c - i * kMoeChunk < kMoeChunk ? c - i * kMoeChunk : kMoeChunk);
                        sm.prob[np + ns - n + i] = pb;
                    }
                }
                at += __shfl_sync(0xffffffffu, cs, 31);
                np += __shfl_sync(0xffffffffu, ns, 31);
            }
            if (lane == 0) sm.nprob = np;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int ch = warp + kMoeWarps * c;
            if (id_of[c] >= 0) sm.sorted[sm.first[id_of[c]] + counts[ch * a.E + id_of[c]] + rank[c]] = (int16_t)(32 * ch + lane);
        }
        __syncthreads();
    }

    // ---------------- gate, up, activation ----------------
    int *red = reinterpret_cast<int *>(dyn);
    const uint32_t rings = smem_u32(dyn + kMoeRedBytes), x_s = rings + kMoeWarps * PD * 2048;
    const uint32_t ring = rings + (uint32_t)(warp * PD * 2048 + 16 * lane);
    {
        MoeRun run = moe_run<true>(a, sm);
        for (int p = 0; p < PD; ++p) moe_load<true>(a, sm, run, ring + 2048u * p);
        // the weights are wanted at the end: while the first loads are on their way
        if (a.router && !spread && warp < a.M) moe_weights(a, sm, warp, slot_logit, top_logit);
        moe_contract<true, CONV, PD>(a, sm, run, ring, x_s, red);
    }
    MoeRun run = moe_run<false>(a, sm);
    const bool joint = FEW && moe_run_joint(a, sm, run);
    for (int p = 0; p < PD; ++p) {  // on their way during the rotation
        if (FEW && joint)
            moe_load<false, true>(a, sm, run, ring + 2048u * p);
        else
            moe_load<false>(a, sm, run, ring + 2048u * p);
    }
    if (!moe_grid_sync(a.barrier, ++phase, &sm.flag)) {
        cp_async_wait_groups<0>();
        return;
    }
    // ---------------- rotation and codes of every pair ----------------
    // Where a CTA's teams do all pairs in one round (and the down phase reads them
    // all), every CTA does, straight into its shared memory, without a barrier after
    // it: one token of 512 x 1024 14.6 us, 16.1 us with each pair in one CTA.  Two
    // rounds cost more than the barrier (one of 1536 x 6144: 21.8 us to 20.4 us).
    bool here = false;
    int rows = 0;
    {
        const int nw = a.F / 512, fit = (int)(kMoeWarps * a.by_warps >> 8), teams = fit < 15 ? fit : 15;  // named barriers 1 .. 15
        const int team = (int)((unsigned)warp * a.by_warps >> 8), wt = warp - team * nw;
        if (FEW && joint) {
            const MoeProblem pb = sm.prob[sm.nprob - 1];
            rows = pb.start + pb.count;
            here = rows <= teams;
        }
        if (team < teams) {
            const int n = FEW && here ? 1 : (int)gridDim.x, end = FEW && here ? rows : P;
            for (int j = (FEW && here ? 0 : (int)blockIdx.x) + team * n; j < end; j += teams * n) {
                const int p = FEW && here ? sm.sorted[j] : j;
                if (sm.ids[p] < 0) continue;
                float f[16];
                load_block16(f, a.h + (int64_t)p * a.F, wt);
                int8_t *dst = FEW && here ? reinterpret_cast<int8_t *>(dyn + kMoeRedBytes + kMoeWarps * PD * 2048) + j * gemv_x_stride(a.F)
                                          : a.hq + (int64_t)p * a.F;
                moe_rot_quant(f, wt, nw, 1 + team, a.act, a.inv_f, dst, FEW && here ? sm.few_s + j : a.sh + p,
                              FEW && here ? sm.few_r + j : a.rh + p, sm.red.f + team * nw, sm.red.i + team * nw, sm.red.d + team * nw);
                bar_sync_n(1 + team, 32 * nw);  // the slots of red are written again
            }
        }
    }
    if (FEW && here) {
        __syncthreads();
    } else if (!moe_grid_sync(a.barrier, ++phase, &sm.flag)) {
        cp_async_wait_groups<0>();
        return;
    }
    // ---------------- down ----------------
    if (FEW && joint) {
        moe_down_joint<CONV, PD>(a, sm, run, ring, x_s, red, here);
        return;
    }
    moe_contract<false, CONV, PD>(a, sm, run, ring, x_s, red);
    if (!moe_grid_sync(a.barrier, ++phase, &sm.flag)) return;
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
