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
//   warps 2, 3  scales, alternate steps: s_x[b][m0 ..] (times the tile's s_w
//               unless ROWS) into a shared-memory ring, loaded two of their
//               steps ahead.
//   warps 4 ..  epilogue: 4 warps per 64 tokens (one per TMEM lane quarter),
//               a thread per row with its tokens' sums in registers; adding
//               a block takes one packed fp32 multiply-add per two outputs
//               (two packed instructions with ROWS).
//
// S = 1: persistent CTAs, tiles with tokens fastest (CTAs running at the same
// time share w tiles in L2).  S > 1: a cluster of S CTAs shares a tile, each
// with a contiguous part of the blocks; the partial sums meet in the CTAs'
// shared memory, added in the order of the parts, so the result does not
// depend on timing.
//
// Every mbarrier wait is bounded (see mbar_wait); after a timeout the kernel
// skips the remaining work, lets its copies and MMAs end and frees its tensor
// memory.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "tq_common.cuh"

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
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Wait for this thread's tensor-memory loads; `r` holds their results only after it.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :
                 : "memory");
}

// Two fp32 operations in one instruction (each rounds as the scalar one does).
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
    lo = __uint_as_float(a);
    hi = __uint_as_float(b);
}
__device__ __forceinline__ void fma2(uint64_t &acc, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
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
__device__ __forceinline__ void store_column(T *p, int N, int rows, const uint64_t (&acc)[P]) {
#pragma unroll
    for (int c = 0; c < P; ++c) {
        float v0, v1;
        unpack2(acc[c], v0, v1);
        if (2 * c < rows) put_as(p, v0);
        p += N;
        if (2 * c + 1 < rows) put_as(p, v1);
        p += N;
    }
}
template <int P>
__device__ __forceinline__ void add_column(float *p, int N, int rows, const uint64_t (&acc)[P]) {
#pragma unroll
    for (int c = 0; c < P; ++c) {
        float v0, v1;
        unpack2(acc[c], v0, v1);
        if (2 * c < rows) *p = __fadd_rn(*p, v0);
        p += N;
        if (2 * c + 1 < rows) *p = __fadd_rn(*p, v1);
        p += N;
    }
}

template <int BT>
struct Fp8Layout {
    static constexpr int kGroups = BT > 64 ? BT / 64 : 1;  // epilogue groups of four warps
    static constexpr int kCols = BT / kGroups;             // tokens per epilogue thread
    static constexpr int kThreads = 128 + 128 * kGroups;
    static constexpr int kAccBufs = BT > 128 ? 2 : 4;
    static constexpr uint32_t kTmemCols = kAccBufs * BT;   // 64, 128, 256, 512, 512
    static constexpr int kA = kFp8TileN * kFp8Step, kB = BT * kFp8Step;
    static constexpr int kStage = kA + kB;
    // up to 32 tokens: two CTAs per SM (see the launcher), else one
    static constexpr int kCtas = BT <= 32 ? 2 : 1;
    static constexpr int kStages = BT <= 16 ? 6 : BT <= 32 ? 5 : BT <= 64 ? 8 : BT <= 128 ? 6 : 4;
    static constexpr int kScaleSlots = 8;
    static constexpr int offScale = kStages * kStage;
    static constexpr int offBar = offScale + kScaleSlots * BT * 4;
    // barriers: full[S], empty[S], d_full[A], d_empty[A], s_full[8], s_empty[8], mma_done
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
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::offBar;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto d_full = [&](int b) { return bar0 + 8u * (2 * S + b); };
    auto d_empty = [&](int b) { return bar0 + 8u * (2 * S + AB + b); };
    auto s_full = [&](int i) { return bar0 + 8u * (2 * S + 2 * AB + i); };
    auto s_empty = [&](int i) { return bar0 + 8u * (2 * S + 2 * AB + SS + i); };
    const uint32_t mma_done = bar0 + 8u * (2 * S + 2 * AB + 2 * SS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::offTmem);
    float *scale_ring = reinterpret_cast<float *>(smem + L::offScale);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
            mbar_init(s_full(i), 1);
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
        if (lane == 0) {
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
                if (!mbar_wait_sleep(empty(g % S), ((g / S) & 1) ^ 1)) break;
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
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3(kFp8TileN, BT);
            for (int g = 0; g < total; ++g) {
                const int s = g % S, b = g % AB;
                if (!mbar_wait(d_empty(b), ((g / AB) & 1) ^ 1)) break;
                if (!mbar_wait(full(s), (g / S) & 1)) break;
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
    } else if (warp < 4) {
        // ---------------- scales ----------------
        pdl_wait();
        constexpr int V = (BT + 31) / 32;
        auto load = [&](int g, float (&v)[V]) {
            const int t = first_tile + (g / nkb) * tile_step, kb = kb0 + g % nkb;
            const int m0 = (t % num_m) * BT;
            const float sw = ROWS ? 1.0f : __ldg(a.s_w + (int64_t)(t / num_m) * nblk + kb);
            const float *src = a.s_x + (int64_t)kb * M;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int m = m0 + 32 * i + lane;
                v[i] = m < M && 32 * i + lane < BT ? __fmul_rn(__ldg(src + m), sw) : 0.0f;
            }
        };
        auto store = [&](int g, const float (&v)[V]) {
            if (!warp_wait_sleep(s_empty(g % SS), ((g / SS) & 1) ^ 1, lane)) return false;
            float *dst = scale_ring + (g % SS) * BT;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (32 * i + lane < BT) dst[32 * i + lane] = v[i];
            __syncwarp();
            if (lane == 0) mbar_arrive(s_full(g % SS));
            return true;
        };
        // steps g0, g0 + 2, ...; two loads in flight
        float v0[V], v1[V];
        int g = warp - 2;
        if (g < total) load(g, v0);
        if (g + 2 < total) load(g + 2, v1);
        for (; g < total; g += 4) {
            if (!store(g, v0)) break;
            if (g + 4 < total) load(g + 4, v0);
            if (g + 2 >= total || !store(g + 2, v1)) break;
            if (g + 6 < total) load(g + 6, v1);
        }
    } else {
        // ---------------- epilogue ----------------
        if (ROWS || a.accumulate) pdl_wait();
        const int q = warp & 3, grp = (warp - 4) >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(grp * L::kCols);
        bool ok = true;
        for (int tl = 0, g = 0; tl < my_tiles && ok; ++tl) {
            const int t = first_tile + tl * tile_step;
            const int n = (t / num_m) * kFp8TileN + 32 * q + lane;
            uint64_t acc[L::kCols / 2];
#pragma unroll
            for (int i = 0; i < L::kCols / 2; ++i) acc[i] = 0;
            const float *wrow = a.s_w + (n < N ? n : 0);  // ROWS: this row's scales, stride N
            float w_next = ROWS ? __ldg(wrow + (int64_t)kb0 * N) : 0.0f;
            for (int kb = 0; kb < nkb; ++kb, ++g) {
                const float w_now = w_next;
                if (ROWS && kb + 1 < nkb) w_next = __ldg(wrow + (int64_t)(kb0 + kb + 1) * N);
                const uint64_t w2 = pack2(__float_as_uint(w_now), __float_as_uint(w_now));
                const int b = g % AB, i = g % SS;
                if (!warp_wait(s_full(i), (g / SS) & 1, lane) || !warp_wait(d_full(b), (g / AB) & 1, lane)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float *sc = scale_ring + i * BT + grp * L::kCols;
#pragma unroll
                for (int c = 0; c < L::kCols / 16; ++c) {
                    uint32_t v[16];
                    tmem_ld16(lane_addr + (uint32_t)(b * BT + 16 * c), v);
                    tmem_ld_wait16(v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(sc + 16 * c + 4 * j);
                        const uint64_t p0 = pack2(v[4 * j], v[4 * j + 1]), p1 = pack2(v[4 * j + 2], v[4 * j + 3]);
                        if (ROWS) {
                            fma2(acc[8 * c + 2 * j], mul2(p0, f.x), w2);
                            fma2(acc[8 * c + 2 * j + 1], mul2(p1, f.y), w2);
                        } else {
                            fma2(acc[8 * c + 2 * j], p0, f.x);
                            fma2(acc[8 * c + 2 * j + 1], p1, f.y);
                        }
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
                for (int c = 0; c < L::kCols / 2; ++c)
                    unpack2(acc[c], partial[2 * c * kFp8TileN], partial[(2 * c + 1) * kFp8TileN]);
                break;  // one tile per cluster
            }
            if (tl == 0) pdl_wait();  // y may be read by the previous kernel
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
            pdl_wait();
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

}  // namespace tq
