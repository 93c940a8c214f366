// tq_fp8_gemm.cuh -- products of e4m3 operands with a scale per block of 128,
// on the 5th-generation tensor cores.
//
//   y[m][n] = sum_b s_x[b][m] * s_w(n, b) * (sum_{k in block b} x[m][k] w[n][k])
//
// with blocks b of 128 along K, s_w one scale per 128 x 128 block of w, or
// (ROWS) one per row and block.  The scales are arbitrary fp32 numbers, so
// the tensor core sums one block only: the four MMAs (kind::f8f6f4, K = 32
// each) of a block go to a tensor-memory buffer of their own, and the epilogue
// warps add that buffer, times its scales, to fp32 sums in registers.  The
// sum of a block of exact products and the sum over blocks are both fp32.
//
// Tiles of 128 rows of w (the MMA's M, TMEM lanes) x BT tokens (its N, TMEM
// columns); w takes M so that few tokens waste no MMA rows, and a warp's store
// of one token covers 32 consecutive outputs.  Warps:
//
//   warp 0      producer (lane 0): TMA of w [128][128 B] and x [BT][128 B],
//               128-byte swizzled, into the operand ring.
//   warp 1      TMEM owner; lane 0 issues the MMAs of a step into buffer
//               step % kAccBufs and commits twice: the operand slot is free,
//               the buffer is full.
//   warp 2      scales: asynchronous copies of s_x[b][m0 ..] and s_w into a ring of
//               six or eight steps (one load from L2 takes longer than a step).
//   warps 4 ..  epilogue: 4 warps per 64 tokens (one per TMEM lane quarter),
//               a thread per row with its tokens' sums in registers; adding
//               a block takes a multiplication of scales and a multiply-add each.
//
// S = 1: persistent CTAs, tiles with tokens fastest (CTAs running at the same
// time share w tiles in L2).  S > 1: a cluster of S CTAs shares a tile, each
// with a contiguous part of the blocks; the partial sums meet in the CTAs'
// shared memory, added in the order of the parts, so the result does not
// depend on timing.
//
// What bounds it: w for few tokens (16 x 32000 x 4096: 23.9 us, 5.6 TB/s; 1 x 4096 x
// 4096, a latency, 6.3 us), for many the epilogue, whose products each meet a scale from
// shared memory (scales per row of w, 5632 x 2048 x 2048: 49.7 us, issue slots 51 %
// busy, the tensor pipe 22 %); with one scale per block of w a kernel of its own does
// without (tq_fp8_gemm_wide_kernel).
//
// Every mbarrier wait is bounded (see mbar_wait); after a timeout the kernel
// skips the remaining work, lets its copies and MMAs end and frees its tensor
// memory.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "tq_common.cuh"
#include "tq_gemv.cuh"

namespace tq {

constexpr int kFp8TileN = 128;  // rows of w per tile (MMA M)
constexpr int kFp8Step = 128;   // K per step: one block of scales

// Instruction descriptor, kind::f8f6f4: D fp32, A and B e4m3, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// Wait for this thread's tensor-memory loads; `r` holds their results only after it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :
                 : "memory");
}
// One fp32 global -> shared, asynchronously; 0 where `take` is false.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src, bool take) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(take ? 4 : 0) : "memory");
}
// Arrive on `bar` (without adding to its count) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Keeps a value in its register: derived from a special register (thread index,
// shared-memory base), it would otherwise be computed again, at that register's
// latency, wherever it is used in a loop.
__device__ __forceinline__ void pin(uint32_t &v) { asm volatile("" : "+r"(v)); }
__device__ __forceinline__ void pin(int &v) { asm volatile("" : "+r"(v)); }

// The bounded wait of loops with one every few hundred cycles: at most 2^18 + 1
// tries, each asleep for up to 4 us (about a second in all).  It reads no clock,
// which takes longer than such a wait lasts, and is a few instructions: the
// issuing warp's loop is fetched anew in every step beside the epilogue's code.
constexpr int kStepTries = 1 << 18;
__device__ __forceinline__ bool step_wait(uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
    for (int i = 0; i < kStepTries; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 4000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    flag_timeout();
    return false;
}
__device__ __forceinline__ bool warp_step_wait(uint32_t bar, uint32_t parity, int lane) {
    int ok = 0;
    if (lane == 0) ok = step_wait(bar, parity) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// True in one lane of a converged warp.  Unlike a test of the lane number it
// tells the compiler that a single thread runs what follows, so descriptors of
// copies and MMAs go to uniform registers directly.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ float4 lds_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Shared-memory address `addr` of the CTA `rank` of this cluster, read as fp32.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
    uint32_t ra;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ra) : "memory");
    return v;
}

// One output of each of a thread's tokens (the first `rows` of them), y's rows N apart.
__device__ __forceinline__ void put_as(float *p, float v) { *p = v; }
__device__ __forceinline__ void put_as(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T, int P>
__device__ __forceinline__ void store_column(T *p, int N, int rows, const float (&acc)[P]) {
#pragma unroll
    for (int c = 0; c < P; ++c, p += N)
        if (c < rows) put_as(p, acc[c]);
}
template <int P>
__device__ __forceinline__ void add_column(float *p, int N, int rows, const float (&acc)[P]) {
#pragma unroll
    for (int c = 0; c < P; ++c, p += N)
        if (c < rows) *p = __fadd_rn(*p, acc[c]);
}

template <int BT>
struct Fp8Layout {
    static constexpr int kGroups = BT > 64 ? BT / 64 : 1;  // epilogue groups of four warps
    static constexpr int kCols = BT / kGroups;             // tokens per epilogue thread
    static constexpr int kThreads = 128 + 128 * kGroups;
    static constexpr int kChunk = 16;  // TMEM columns read at a time
    static constexpr int kAccBufs = 4;
    static constexpr uint32_t kTmemCols = kAccBufs * BT;
    static constexpr int kA = kFp8TileN * kFp8Step, kB = BT * kFp8Step;
    static constexpr int kStage = kA + kB;
    // up to 32 tokens: two CTAs per SM (see the launcher), else one
    static constexpr int kCtas = BT <= 32 ? 2 : 1;
    static constexpr int kStages = BT <= 16 ? 6 : BT <= 32 ? 5 : BT <= 64 ? 8 : 6;
    static constexpr int kScaleSlots = BT <= 16 ? 6 : 8;
    static constexpr int offScale = kStages * kStage;
    static constexpr int kScales = BT + kFp8TileN;  // a slot: the tokens' scales, then w's (ROWS: 128, else one)
    static constexpr int offBar = offScale + kScaleSlots * kScales * 4;
    // barriers: full, empty [kStages], d_full, d_empty [kAccBufs], s_full, s_empty [kScaleSlots], mma_done
    static constexpr int kBars = 2 * kStages + 2 * kAccBufs + 2 * kScaleSlots + 1;
    static constexpr int offTmem = offBar + kBars * 8;
    static constexpr int kBytes = offTmem + 16;
    static constexpr int kDynamic = kBytes + 1024;  // slack for 1024-byte alignment
    static_assert(kTmemCols >= 32 && kTmemCols * kCtas <= 512, "tensor memory columns");
    static_assert((kDynamic + 1024) * kCtas <= 233472, "shared memory per SM");
    static_assert(kStage % 1024 == 0, "swizzle atoms stay aligned");
    static_assert(BT * kFp8TileN * 4 <= kStages * kStage, "the partial sums of a split fit the ring");
};

struct Fp8Args {
    const float *s_x;  // [blocks][M]
    const float *s_w;  // [blocks of N][blocks], or (ROWS) [blocks][N]
    void *y;           // [M][N] fp32 or bf16
    int M, N, K;
    int splits;        // CTAs per tile (cluster size)
    int y_bf16, accumulate;
    int w_static;      // w may be read before the previous kernel has ended
};

template <int BT, bool ROWS>
__global__ void __launch_bounds__(Fp8Layout<BT>::kThreads, Fp8Layout<BT>::kCtas)
    tq_fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ Fp8Args a) {
    using L = Fp8Layout<BT>;
    constexpr int S = L::kStages, AB = L::kAccBufs, SS = L::kScaleSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint32_t sbase = smem_u32(smem), bar0 = sbase + L::offBar;
    pin(sbase);
    pin(bar0);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto d_full = [&](int b) { return bar0 + 8u * (2 * S + b); };
    auto d_empty = [&](int b) { return bar0 + 8u * (2 * S + AB + b); };
    auto s_full = [&](int i) { return bar0 + 8u * (2 * S + 2 * AB + i); };
    auto s_empty = [&](int i) { return bar0 + 8u * (2 * S + 2 * AB + SS + i); };
    const uint32_t mma_done = bar0 + 8u * (2 * S + 2 * AB + 2 * SS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::offTmem);

    int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pin(warp);
    pin(lane);
    const int M = a.M, N = a.N, NS = a.splits;
    const int num_m = (M + BT - 1) / BT, num_n = (N + kFp8TileN - 1) / kFp8TileN;
    const int ntiles = num_m * num_n;
    const int nblk = (a.K + kFp8Step - 1) / kFp8Step;
    // this CTA's tiles first_tile + i * tile_step, and its blocks kb0 .. kb0 + nkb of each
    const int part = (int)blockIdx.x % NS;
    const int first_tile = (int)blockIdx.x / NS, tile_step = (int)gridDim.x / NS;
    const int my_tiles = (ntiles - first_tile + tile_step - 1) / tile_step;
    const int kb0 = (int)((int64_t)nblk * part / NS);
    const int nkb = (int)((int64_t)nblk * (part + 1) / NS) - kb0;
    const int total = my_tiles * nkb;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < AB; ++b) {
            mbar_init(d_full(b), 1);
            mbar_init(d_empty(b), 4 * L::kGroups);
        }
        for (int i = 0; i < SS; ++i) {
            mbar_init(s_full(i), 32);
            mbar_init(s_empty(i), 4 * L::kGroups);
        }
        mbar_init(mma_done, 1);
        fence_barrier_init();
        prefetch_tmap(&tm_x);
        prefetch_tmap(&tm_w);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------- producer ----------------
        if (elect_one()) {
            auto load_w = [&](int g) {
                const int t = first_tile + (g / nkb) * tile_step;
                tma_load_2d(sbase + (uint32_t)((g % S) * L::kStage), &tm_w, (kb0 + g % nkb) * kFp8Step,
                            (t / num_m) * kFp8TileN, full(g % S));
            };
            auto load_x = [&](int g) {
                const int t = first_tile + (g / nkb) * tile_step;
                tma_load_2d(sbase + (uint32_t)((g % S) * L::kStage + L::kA), &tm_x, (kb0 + g % nkb) * kFp8Step,
                            (t % num_m) * BT, full(g % S));
            };
            const int pre = a.w_static ? (total < S ? total : S) : 0;
            for (int g = 0; g < pre; ++g) {
                mbar_arrive_expect_tx(full(g), L::kStage);
                load_w(g);
            }
            pdl_wait();
            for (int g = 0; g < pre; ++g) load_x(g);
            int g = pre;
            for (; g < total; ++g) {
                if (!step_wait(empty(g % S), ((g / S) & 1) ^ 1)) break;
                mbar_arrive_expect_tx(full(g % S), L::kStage);
                load_w(g);
                load_x(g);
            }
            // own copies land before the CTA may exit
            for (int j = g - S < 0 ? 0 : g - S; j < g; ++j) mbar_wait(full(j % S), (j / S) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_e4m3(kFp8TileN, BT);
            pdl_wait();  // so that no wait below has to last as long as the previous kernel
            for (int g = 0; g < total; ++g) {
                const int s = g % S, b = g % AB;
                if (!step_wait(d_empty(b), ((g / AB) & 1) ^ 1) || !step_wait(full(s), (g / S) & 1)) break;
                tc_fence_after();
                const uint32_t wa = sbase + (uint32_t)(s * L::kStage), xa = wa + L::kA;
#pragma unroll
                for (int k = 0; k < kFp8Step / 32; ++k)
                    mma_f8(tmem + (uint32_t)(b * BT), smem_desc_sw128(wa + 32 * k), smem_desc_sw128(xa + 32 * k),
                           idesc, k != 0 ? 1u : 0u);
                mma_commit(empty(s));
                mma_commit(d_full(b));
            }
            // no MMA may still use tensor or shared memory when they are freed
            mma_commit(mma_done);
            mbar_wait(mma_done, 0);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------- scales ----------------
        pdl_wait();
        int g = 0;
        for (int tl = 0; tl < my_tiles; ++tl) {
            const int t = first_tile + tl * tile_step;
            const int m = (t % num_m) * BT + lane, n = (t / num_m) * kFp8TileN + lane;
            int kb = 0;
            for (; kb < nkb; ++kb, ++g) {
                if (!warp_step_wait(s_empty(g % SS), ((g / SS) & 1) ^ 1, lane)) break;
                const uint32_t dst = sbase + (uint32_t)(L::offScale + ((g % SS) * L::kScales + lane) * 4);
                const float *sx = a.s_x + (int64_t)(kb0 + kb) * M + m;
#pragma unroll
                for (int i = 0; i < BT; i += 32)
                    if (i + lane < BT) cp_async4(dst + 4 * i, m + i < M ? sx + i : a.s_x, m + i < M);
                if (ROWS) {
                    const float *sw = a.s_w + (int64_t)(kb0 + kb) * N + n;
#pragma unroll
                    for (int i = 0; i < kFp8TileN; i += 32)
                        cp_async4(dst + 4 * (BT + i), n + i < N ? sw + i : a.s_w, n + i < N);
                } else if (lane == 0) {
                    cp_async4(dst + 4 * BT, a.s_w + (int64_t)(t / num_m) * nblk + kb0 + kb, true);
                }
                cp_async_arrive(s_full(g % SS));
            }
            if (kb < nkb) break;
        }
        cp_async_wait_all();  // own copies land before the CTA may exit
    } else if (warp >= 4) {
        // ---------------- epilogue ----------------
        pdl_wait();
        const int q = warp & 3, grp = (warp - 4) >> 2;
        uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(grp * L::kCols);
        pin(lane_addr);
        bool ok = true;
        for (int tl = 0, g = 0; tl < my_tiles && ok; ++tl) {
            const int t = first_tile + tl * tile_step;
            const int n = (t / num_m) * kFp8TileN + 32 * q + lane;
            float acc[L::kCols];
#pragma unroll
            for (int i = 0; i < L::kCols; ++i) acc[i] = 0.0f;
            for (int kb = 0; kb < nkb; ++kb, ++g) {
                const int b = g % AB, i = g % SS;
                if (!warp_step_wait(s_full(i), (g / SS) & 1, lane) || !warp_step_wait(d_full(b), (g / AB) & 1, lane)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t slot = sbase + (uint32_t)(L::offScale + i * L::kScales * 4), sc = slot + 4 * grp * L::kCols;
                const float sw = lds_f32(slot + 4 * (BT + (ROWS ? 32 * q + lane : 0)));
#pragma unroll
                for (int c = 0; c < L::kCols; c += L::kChunk) {
                    uint32_t v[L::kChunk];
                    tmem_ld(lane_addr + (uint32_t)(b * BT + c), v);
                    tmem_ld_wait_for(v);
#pragma unroll
                    for (int j = 0; j < L::kChunk; j += 4) {
                        const float4 f = lds_f32x4(sc + (uint32_t)(4 * (c + j)));
                        acc[c + j] = __fmaf_rn(__uint_as_float(v[j]), __fmul_rn(f.x, sw), acc[c + j]);
                        acc[c + j + 1] = __fmaf_rn(__uint_as_float(v[j + 1]), __fmul_rn(f.y, sw), acc[c + j + 1]);
                        acc[c + j + 2] = __fmaf_rn(__uint_as_float(v[j + 2]), __fmul_rn(f.z, sw), acc[c + j + 2]);
                        acc[c + j + 3] = __fmaf_rn(__uint_as_float(v[j + 3]), __fmul_rn(f.w, sw), acc[c + j + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(d_empty(b));
                    mbar_arrive(s_empty(i));
                }
            }
            if (!ok) break;
            if (NS > 1) {
                // The last block is in: every copy into this CTA's ring and every MMA
                // reading it has ended, so the ring takes the partial sums [token][row].
                float *partial = reinterpret_cast<float *>(smem) + grp * L::kCols * kFp8TileN + 32 * q + lane;
#pragma unroll
                for (int c = 0; c < L::kCols; ++c) partial[c * kFp8TileN] = acc[c];
                break;  // one tile per cluster
            }
            const int m0 = (t % num_m) * BT + grp * L::kCols;
            if (n < N) {
                if (a.y_bf16)
                    store_column(reinterpret_cast<__nv_bfloat16 *>(a.y) + (int64_t)m0 * N + n, N, M - m0, acc);
                else if (a.accumulate)
                    add_column(reinterpret_cast<float *>(a.y) + (int64_t)m0 * N + n, N, M - m0, acc);
                else
                    store_column(reinterpret_cast<float *>(a.y) + (int64_t)m0 * N + n, N, M - m0, acc);
            }
        }
    }
    if (NS > 1) {
        // Each CTA adds a share of the tile's tokens over the parts, in order.
        __syncwarp();
        cluster_sync_all();
        if (warp >= 4) {
            const int q = warp & 3, grp = (warp - 4) >> 2;
            const int row = 32 * q + lane, n = (first_tile / num_m) * kFp8TileN + row, m0 = (first_tile % num_m) * BT;
            for (int c = part * L::kGroups + grp; c < BT; c += NS * L::kGroups) {
                if (m0 + c >= M) break;
                const uint32_t at = sbase + (uint32_t)((c * kFp8TileN + row) * 4);
                float p[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) p[r] = r < NS ? ld_cluster_f32(at, (uint32_t)r) : 0.0f;
                float sum = p[0];
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < NS) sum = __fadd_rn(sum, p[r]);
                if (n < N) {
                    const int64_t o = (int64_t)(m0 + c) * N + n;
                    if (a.y_bf16)
                        reinterpret_cast<__nv_bfloat16 *>(a.y)[o] = __float2bfloat16_rn(sum);
                    else
                        reinterpret_cast<float *>(a.y)[o] = a.accumulate ? __fadd_rn(reinterpret_cast<float *>(a.y)[o], sum) : sum;
                }
            }
        }
        __syncwarp();
        cluster_sync_all();  // the others may still be reading this CTA's partial sums
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// Many tokens: tiles of 128 tokens (TMEM lanes) x BN rows of w (TMEM columns).
// In the narrow kernel every product meets a scale that is broadcast from
// shared memory, 4 bytes per lane and product: 4 cycles per TMEM column and
// block, twice the MMAs' time.  Here a thread reads fragments of 4 tokens x 2
// consecutive rows of w (tcgen05.ld.16x256b): the tokens' scales are 4 registers
// and the scale of a block of w is one for all columns of a warp.  They come
// straight from L2, two steps ahead: a lane loads one token's, and shuffles spread
// them (a shared ring filled by a warp of its own cost a third of the kernel's time
// in barrier traffic).  2048 x 11008 x 4096: 113 us, 1.63 PFLOP/s (the narrow kernel:
// 171 us); 4096 x 8192 x 8192: 300 us, 1.83 PFLOP/s.  The MMAs alone would take
// 40 % of that, and no pipe is full (2048 x 4096 x 4096: tensor 38 %, issue slots 39 %,
// DRAM 6 %): a step is a chain of its MMAs, the epilogue's rounds of tensor-memory
// loads, each waited for (the first stall), and the buffer's way back, of which two
// buffers overlap one step.  Adding to y (accumulate) takes twice as long, 222 us at
// 2048 x 11008 x 4096: its reads of y come after the sums, between the stores.
//
//   warp 0  producer   warp 1  TMEM, MMAs
//   warps 4-11  epilogue, four warps per half of the columns; TMEM lane quarter = warp % 4
// ---------------------------------------------------------------------------
template <int BN>
struct Fp8WideLayout {
    static constexpr int kCols = BN / 2;  // columns per epilogue warp; two groups of four warps
    static constexpr int kGroups = 2;
    static constexpr int kFirstEpi = 4;
    static constexpr int kThreads = 32 * (kFirstEpi + 4 * kGroups);
    static constexpr int kInFlight = 2;   // fragment loads per wait
    // 128 columns: 128 sums per thread.  The block starts with 168 registers per
    // thread; warps 0-3 give up theirs for the epilogue warps' (128 x 64 + 256 x
    // 216 <= 384 x 168).
    static constexpr bool kMoveRegs = kCols > 64;
    static constexpr int kAccBufs = BN > 128 ? 2 : 4;
    static constexpr uint32_t kTmemCols = kAccBufs * BN;
    static constexpr int kA = 128 * kFp8Step, kB = BN * kFp8Step, kStage = kA + kB;
    static constexpr int kStages = BN > 128 ? 4 : 6;
    static constexpr int offBar = kStages * kStage;
    static constexpr int kBars = 2 * kStages + 2 * kAccBufs + 1;
    static constexpr int offTmem = offBar + kBars * 8;
    static constexpr int kBytes = offTmem + 16;
    static constexpr int kDynamic = kBytes + 1024;
    static_assert(BN == 128 || BN == 256, "an epilogue warp's columns lie in one block of w's scales");
    static_assert(kTmemCols <= 512 && kDynamic <= 232448 && kStage % 1024 == 0, "tensor and shared memory");
};

// 16 lanes x 32 columns: register 4 i + 2 h + e is lane t / 4 + 8 h, column 8 i + 2 (t % 4) + e.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Two neighbouring outputs; PAIR: both exist and the address is aligned for one store.
template <bool PAIR>
__device__ __forceinline__ void put_pair(float *p, float v0, float v1, bool two, bool add) {
    if (PAIR) {
        float2 *q = reinterpret_cast<float2 *>(p);
        float2 v = make_float2(v0, v1);
        if (add) {
            const float2 o = *q;
            v = make_float2(__fadd_rn(o.x, v0), __fadd_rn(o.y, v1));
        }
        *q = v;
    } else {
        p[0] = add ? __fadd_rn(p[0], v0) : v0;
        if (two) p[1] = add ? __fadd_rn(p[1], v1) : v1;
    }
}
template <bool PAIR>
__device__ __forceinline__ void put_pair(__nv_bfloat16 *p, float v0, float v1, bool two, bool) {
    if (PAIR) {
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v0, v1);
    } else {
        p[0] = __float2bfloat16_rn(v0);
        if (two) p[1] = __float2bfloat16_rn(v1);
    }
}

// acc[i][h][e]: column 8 i + e (+ this lane's pair) of token m + 8 h.
template <bool PAIR, typename T, int P>
__device__ __forceinline__ void put_frags(T *y, const float (&acc)[P][4][2], int m, int n, int M, int N, bool add) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        if (m + 8 * h >= M) break;
        T *p = y + (int64_t)(m + 8 * h) * N + n;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (n + 8 * i < N) put_pair<PAIR>(p + 8 * i, acc[i][h][0], acc[i][h][1], n + 8 * i + 1 < N, add);
        }
    }
}

template <int BN>
__global__ void __launch_bounds__(Fp8WideLayout<BN>::kThreads, 1)
    tq_fp8_gemm_wide_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                            const __grid_constant__ Fp8Args a) {
    using L = Fp8WideLayout<BN>;
    constexpr int S = L::kStages, AB = L::kAccBufs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint32_t sbase = smem_u32(smem), bar0 = sbase + L::offBar;
    pin(sbase);
    pin(bar0);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto d_full = [&](int b) { return bar0 + 8u * (2 * S + b); };
    auto d_empty = [&](int b) { return bar0 + 8u * (2 * S + AB + b); };
    const uint32_t mma_done = bar0 + 8u * (2 * S + 2 * AB);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::offTmem);

    int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pin(warp);
    pin(lane);
    const int M = a.M, N = a.N;
    const int num_m = (M + 127) / 128, num_n = (N + BN - 1) / BN;
    const int ntiles = num_m * num_n;
    const int nkb = (a.K + kFp8Step - 1) / kFp8Step;
    const int my_tiles = (ntiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < AB; ++b) {
            mbar_init(d_full(b), 1);
            mbar_init(d_empty(b), 4 * L::kGroups);
        }
        mbar_init(mma_done, 1);
        fence_barrier_init();
        prefetch_tmap(&tm_x);
        prefetch_tmap(&tm_w);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;

    if (warp < L::kFirstEpi) {
        if (L::kMoveRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
        // ---------------- producer ----------------
        if (elect_one()) {
            pdl_wait();
            bool ok = true;
            int s = 0, g = 0;
            uint32_t par = 1;
            for (int tl = 0; tl < my_tiles && ok; ++tl) {
                const int t = (int)blockIdx.x + tl * (int)gridDim.x;
                const int m0 = (t % num_m) * 128, n0 = (t / num_m) * BN;
                for (int kb = 0; kb < nkb; ++kb, ++g) {
                    if (!step_wait(empty(s), par)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(full(s), L::kStage);
                    const uint32_t at = sbase + (uint32_t)(s * L::kStage);
                    tma_load_2d(at, &tm_x, kb * kFp8Step, m0, full(s));
                    tma_load_2d(at + L::kA, &tm_w, kb * kFp8Step, n0, full(s));
                    if (++s == S) {
                        s = 0;
                        par ^= 1;
                    }
                }
            }
            for (int j = g - S < 0 ? 0 : g - S; j < g; ++j) mbar_wait(full(j % S), (j / S) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_e4m3(128, BN);
            pdl_wait();  // so that no wait below has to last as long as the previous kernel
            const int total = my_tiles * nkb;
            int s = 0, b = 0;
            uint32_t s_par = 0, b_par = 1;
            for (int g = 0; g < total; ++g) {
                if (!step_wait(d_empty(b), b_par) || !step_wait(full(s), s_par)) break;
                tc_fence_after();
                const uint32_t xa = sbase + (uint32_t)(s * L::kStage), wa = xa + L::kA;
#pragma unroll
                for (int k = 0; k < kFp8Step / 32; ++k)
                    mma_f8(tmem + (uint32_t)(b * BN), smem_desc_sw128(xa + 32 * k),
                           smem_desc_sw128(wa + 32 * k), idesc, k != 0 ? 1u : 0u);
                mma_commit(empty(s));
                mma_commit(d_full(b));
                if (++s == S) {
                    s = 0;
                    s_par ^= 1;
                }
                if (++b == AB) {
                    b = 0;
                    b_par ^= 1;
                }
            }
            mma_commit(mma_done);
            mbar_wait(mma_done, 0);
        }
        __syncwarp();
    }
    } else {
        // ---------------- epilogue ----------------
        if (L::kMoveRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        pdl_wait();
        const int q = warp & 3, grp = (warp - L::kFirstEpi) >> 2;
        uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(grp * L::kCols);
        pin(lane_addr);
        // Scales of one step: this lane's token, and w's block.
        struct Scales {
            float x, w;
        };
        const float *px = nullptr, *pw = nullptr;  // the next step's, in the tile being fetched
        bool has_x = false, has_w = false;
        auto aim = [&](int tl) {
            const int t = (int)blockIdx.x + tl * (int)gridDim.x;
            const int m = (t % num_m) * 128 + 32 * q + lane, n = (t / num_m) * BN + grp * L::kCols;
            has_x = m < M;
            has_w = n < N;
            px = a.s_x + (has_x ? m : 0);
            pw = a.s_w + (has_w ? (int64_t)(n >> 7) * nkb : 0);
        };
        auto fetch = [&](Scales &v) {
            v.x = has_x ? __ldg(px) : 0.0f;
            v.w = has_w ? __ldg(pw) : 0.0f;
            px += M;
            ++pw;
        };
        float acc[L::kCols / 8][4][2];
        int b = 0;
        uint32_t b_par = 0;
        // One step: add buffer b times its scales; then v takes those of two steps later.
        auto step = [&](Scales &v, bool more) {
            const float f = __fmul_rn(v.x, v.w);
            if (more) fetch(v);
            float sx[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) sx[h] = __shfl_sync(0xffffffffu, f, (lane >> 2) + 8 * h);
            if (!warp_step_wait(d_full(b), b_par, lane)) return false;
            tc_fence_after();
            // fragment f: columns 32 (f / 2) .., tokens 16 (f % 2) ..; kInFlight loads per wait
#pragma unroll
            for (int f0 = 0; f0 < L::kCols / 16; f0 += L::kInFlight) {
                uint32_t r[L::kInFlight][16];
#pragma unroll
                for (int f = 0; f < L::kInFlight; ++f)
                    tmem_ld_frag(lane_addr + ((uint32_t)(16 * ((f0 + f) & 1)) << 16) +
                                     (uint32_t)(b * BN + 32 * ((f0 + f) >> 1)), r[f]);
#pragma unroll
                for (int f = 0; f < L::kInFlight; ++f) tmem_ld_wait_for(r[f]);
#pragma unroll
                for (int f = 0; f < L::kInFlight; ++f) {
                    const int c = (f0 + f) >> 1, half = (f0 + f) & 1;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float *o = acc[4 * c + i][2 * half + h];
                            o[0] = __fmaf_rn(__uint_as_float(r[f][4 * i + 2 * h]), sx[2 * half + h], o[0]);
                            o[1] = __fmaf_rn(__uint_as_float(r[f][4 * i + 2 * h + 1]), sx[2 * half + h], o[1]);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(d_empty(b));
            if (++b == AB) {
                b = 0;
                b_par ^= 1;
            }
            return true;
        };
        Scales v0, v1;
        aim(0);
        fetch(v0);
        if (nkb > 1) fetch(v1);
        for (int tl = 0; tl < my_tiles; ++tl) {
            const int t = (int)blockIdx.x + tl * (int)gridDim.x;
            const int m = (t % num_m) * 128 + 32 * q + (lane >> 2);  // first of this lane's four tokens, 8 apart
            const int n = (t / num_m) * BN + grp * L::kCols + 2 * (lane & 3);
#pragma unroll
            for (int i = 0; i < L::kCols / 8; ++i)
#pragma unroll
                for (int h = 0; h < 4; ++h) acc[i][h][0] = acc[i][h][1] = 0.0f;
            bool ok = true;
            for (int kb = 0; kb < nkb && ok; kb += 2) {
                ok = step(v0, kb + 2 < nkb);
                if (ok && kb + 1 < nkb) ok = step(v1, kb + 3 < nkb);
            }
            if (!ok) break;
            if (tl + 1 < my_tiles) {  // the next tile's first scales, ahead of the stores
                aim(tl + 1);
                fetch(v0);
                if (nkb > 1) fetch(v1);
            }
            if (a.y_bf16) {
                __nv_bfloat16 *y = reinterpret_cast<__nv_bfloat16 *>(a.y);
                if (N & 1)
                    put_frags<false>(y, acc, m, n, M, N, false);
                else
                    put_frags<true>(y, acc, m, n, M, N, false);
            } else {
                float *y = reinterpret_cast<float *>(a.y);
                if (N & 1)
                    put_frags<false>(y, acc, m, n, M, N, a.accumulate != 0);
                else
                    put_frags<true>(y, acc, m, n, M, N, a.accumulate != 0);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

}  // namespace tq
