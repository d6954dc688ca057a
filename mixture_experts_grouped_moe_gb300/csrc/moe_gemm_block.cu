// The matrix product in 8-bit floating point with a scale for each block of 128, as an operator of
// its own: dense or grouped by expert (the group GEMM of the AITER walk-through, section 3.2, with
// its "per_1x128" quantisation), and the weight gradient over each expert's tokens.
//
//   product   D[m][n] = sum_b sa[m][b] sb[n/128][b] sum_{k in block b} A[m][k] B[n][k]
//   gradient  D[e][m][n] = sum_{b of e} sum_{p in block b} (sa[b][m] A[m][p]) (sb[b][n] B[n][p])
//
// The scales are any fp32 values, not the power-of-two 32-element scales that the tensor core
// applies itself, so every 128-wide block of K is accumulated on its own by tcgen05.mma
// kind::f8f6f4 into a TMEM buffer, and promotion warps fold it into fp32 registers with its scales
// while the tensor core fills the next buffer.  K need not be a multiple of 128: the copies zero-fill
// past the end, and a zero code adds nothing.
//
// Bounds and figures (one GB300): large products by the hand-off of every block of K between the tensor core
// and the promotion warps (a single launch has the tensor pipe active half of the time and 36 % of the issue
// slots in use) and, back to back, by the board's power as well -- 4096 tokens top-2, N 14336, K 4096 of eight
// experts take 450 us (2.14 PFLOP/s) in launches apart at 2070 MHz and 476-492 us in a row, where the power
// limit holds the SM clock at 1680-1800 MHz; few rows by HBM -- 32 tokens, N 28672, K 4096 of eight experts in
// 147 us, 6.4 TB/s; one row, N 4096, K 14336 in 17.8 us.  The weight gradient (4096 x 14336 of eight experts,
// 841 us) fills neither the tensor pipe (24 %) nor the issue slots (40 %): its promotion waits for every load
// from TMEM before the arithmetic on it.
#include <cuda_bf16.h>

#include "gemm_common.cuh"
#include "moe_internal.h"
#include "sm100_ptx.cuh"

namespace moe {

namespace blockgemm {

struct Args {
    CUtensorMap tm_a;  // token operand (wgrad: rows of D)
    CUtensorMap tm_b;  // weight operand (wgrad: columns of D)
    const float *sa;
    int64_t sa_row, sa_blk;  // strides of sa: per row, per 128-block of K
    const float *sb;         // product: [E][ceil(N/128)][KB]; wgrad: [KB][N]
    const int32_t *expert_ids;  // expert of each block_m rows, or null (dense)
    const int32_t *npp;         // rows in use (device), or null: M
    const int32_t *counts;      // wgrad: tokens of each expert, or null (one segment: all of K)
    int64_t M;
    int N, K, E, block_m;
    void *d;
    int64_t ld_d;
    int out_f32, accumulate;
    int wide;  // rows of D start and end on 16-byte (wgrad: 32-byte) boundaries
    int *status;
};

__device__ __forceinline__ int64_t rows_in_use(const Args &a)
{
    if (!a.npp)
        return a.M;
    const int64_t n = *a.npp;
    return n < 0 ? 0 : n < a.M ? n : a.M;
}

__device__ __forceinline__ int expert_of(const Args &a, int64_t row)
{
    if (!a.expert_ids)
        return 0;
    const int e = __ldg(a.expert_ids + row / a.block_m);
    return (unsigned)e < (unsigned)a.E ? e : 0;
}

// acc[0..1] += v[0..1] * f[0..1]
__device__ __forceinline__ void ffma2v(float &acc0, float &acc1, float v0, float v1, float f0, float f1)
{
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "mov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "+f"(acc0), "+f"(acc1)
        : "f"(v0), "f"(v1), "f"(f0), "f"(f1));
}

// (acc0, acc1) += ((v0, v1) * (s0, s1)) * f, in pairs of fp32.
__device__ __forceinline__ void scaled_ffma2(float &acc0, float &acc1, float v0, float v1, float2 s, float f)
{
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "mov.b64 d, {%6, %6};\n\t"
        "mov.b64 c, {%0, %1};\n\t"
        "mul.rn.f32x2 a, a, b;\n\t"
        "fma.rn.f32x2 c, a, d, c;\n\t"
        "mov.b64 {%0, %1}, c;\n\t}"
        : "+f"(acc0), "+f"(acc1)
        : "f"(v0), "f"(v1), "f"(s.x), "f"(s.y), "f"(f));
}

// 32 lanes x 16 columns of TMEM as two 16-lane halves, and the wait for them.  Lane l of the warp gets
// of half h (v: TMEM lanes 0-15 from taddr on, u: lanes 16-31), group g of 8 columns: elements 4 g, 4 g + 1
// at (row l / 4, columns 8 g + 2 (l % 4) and the next), 4 g + 2, 4 g + 3 eight rows below.
__device__ __forceinline__ void tmem_ld_halves(uint32_t taddr, float (&v)[8], float (&u)[8])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(u[0]), "=f"(u[1]), "=f"(u[2]), "=f"(u[3]), "=f"(u[4]), "=f"(u[5]), "=f"(u[6]), "=f"(u[7])
        : "r"(taddr), "r"(taddr + (16u << 16))
        : "memory");
}

// Among the four lanes that share lane / 4: x[j] of lane l becomes x[l % 4] of lane j.
__device__ __forceinline__ void transpose4(float2 (&x)[4], int lane)
{
#pragma unroll
    for (int b = 1; b <= 2; b <<= 1) {
        const bool up = lane & b;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (!(j & b)) {
                const float2 give = up ? x[j] : x[j + b];
                const float2 got = make_float2(__shfl_xor_sync(0xffffffffu, give.x, b),
                                               __shfl_xor_sync(0xffffffffu, give.y, b));
                if (up)
                    x[j] = got;
                else
                    x[j + b] = got;
            }
    }
}

// Eight floats to a 32-byte boundary in one store (or added to what is there).
__device__ __forceinline__ void store8(float *d, float2 (&x)[4], int accumulate)
{
    if (accumulate) {
        const float4 p = reinterpret_cast<const float4 *>(d)[0], q = reinterpret_cast<const float4 *>(d)[1];
        x[0].x += p.x, x[0].y += p.y, x[1].x += p.z, x[1].y += p.w;
        x[2].x += q.x, x[2].y += q.y, x[3].x += q.z, x[3].y += q.w;
    }
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "f"(x[0].x), "f"(x[0].y),
                 "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y)
                 : "memory");
}

// All threads of the cluster, whole warps or not.
__device__ __forceinline__ void cluster_meet()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// ------------------------------------------------------------ many rows
//
// A tile is 128 rows of A x TN rows of B.  Warps: 0 TMA producer, 1 TMEM allocation and MMA issue, then
// eight for promotion and epilogue (two per TMEM lane quadrant, half of the columns each).  A weight
// gradient folds with a scale per row and one per column (about 460 instructions a warp and block, twice a
// product's; 746 of its 841 us remain with the stores left out).  Not faster there: sixteen promotion warps,
// two CTAs an SM (989 us and more), sharing the operands by cluster multicast, claiming tiles dynamically.
// Its scales come through a ring of their own: it has a second warp that copies them and a spare one (so that the promotion warps start
// a group of four), and its first four warps hand registers to the other eight (setmaxnreg): 128
// threads x 72 + 256 x 216 = 64512 = 384 x 168, all that the block is launched with.

template <int TN, bool WG>
struct Cfg {
    // 64-column products share an SM between two CTAs: small problems are bound by the chain of a block,
    // and one's hides behind the other's.
    static constexpr int kCtas = TN == 64 && !WG ? 2 : 1;
    static constexpr int kStages = TN == 256 ? 4 : TN == 128 ? 6 : WG ? 8 : 3;
    static constexpr int kABytes = 128 * 128, kBBytes = TN * 128;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kBufs = TN == 256 ? 2 : 4;  // TMEM accumulators
    static constexpr int kScaleSlots = WG ? 8 : 1;
    static constexpr int kFirstPromo = WG ? 4 : 2;
    static constexpr int kThreads = 32 * (kFirstPromo + 8);
    static constexpr int kSlot = WG ? 128 + TN : 4;  // floats: the rows' scales, then the columns'
};

constexpr int kPromoWarps = 8;
constexpr int kFewRegs = 72, kPromoRegs = 216;
static_assert(128 * kFewRegs + 32 * kPromoWarps * kPromoRegs <= 384 * 168, "within the launch's registers");
constexpr int kGroupM = 16;  // row tiles that walk the column tiles together (64: no faster)
constexpr int kMaxE = 1024;

template <int TN, bool WG>
struct __align__(1024) Smem {
    using C = Cfg<TN, WG>;
    uint8_t stage[C::kStages][C::kStageBytes];
    float scale[C::kScaleSlots][C::kSlot];
    float4 ep_out[WG ? 1 : kPromoWarps][32][4];  // a warp's 32 rows x 64 bytes on their way to D
    uint64_t full[C::kStages], empty[C::kStages];
    uint64_t tfull[C::kBufs], tempty[C::kBufs];
    uint64_t sfull[C::kScaleSlots], sempty[C::kScaleSlots];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int off[WG ? kMaxE + 1 : 1];  // wgrad: first 128-block of each expert
};

struct Tile {
    int e;
    int64_t row0;
    int col0;
    int kb0, kb1;
};

template <int TN, bool WG>
__global__ void __launch_bounds__(Cfg<TN, WG>::kThreads, Cfg<TN, WG>::kCtas) gemm_block_kernel(const __grid_constant__ Args a, int S)
{
    using C = Cfg<TN, WG>;
    constexpr int kFirstPromo = C::kFirstPromo;
    extern __shared__ uint8_t smem_raw[];
    auto &sm = *reinterpret_cast<Smem<TN, WG> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort_flag = &sm.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            mbar_init(&sm.tfull[i], 1);
            mbar_init(&sm.tempty[i], kPromoWarps);
        }
        for (int i = 0; i < C::kScaleSlots; ++i) {
            mbar_init(&sm.sfull[i], 32);
            mbar_init(&sm.sempty[i], kPromoWarps);
        }
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&a.tm_a);
        tma_prefetch_desc(&a.tm_b);
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, C::kBufs * TN);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    if (WG && warp == 2) {
        // first block of each expert: a running sum of ceil(count / 128) over the experts
        int run = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int c = !a.counts ? a.K : e < a.E ? a.counts[e] : 0;
            int v = e < a.E && c > 0 ? (c + 127) / 128 : 0;
            int incl = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d)
                    incl += o;
            }
            if (e < a.E)
                sm.off[e] = run + incl - v;
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0)
            sm.off[a.E] = run;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = sm.tmem_base;
    const int KB = (a.K + 127) / 128;
    const int64_t rows = rows_in_use(a);
    const int nmt = (int)((rows + 127) / 128);
    const int nnt = (a.N + TN - 1) / TN;
    const int ntiles = nmt * nnt * (WG ? a.E : 1);  // (the host checks that the count fits)
    // S > 1: a cluster of S CTAs takes one tile, each a part of K
    constexpr bool kSplits = TN == 64 && !WG;
    const int rank = kSplits && S > 1 ? (int)cluster_ctarank() : 0;
    const int first = kSplits ? blockIdx.x / S : blockIdx.x, step = kSplits ? gridDim.x / S : gridDim.x;

    auto get_tile = [&](int t) {
        Tile tl;
        int within = t;
        const int group = within / (kGroupM * nnt);
        within -= group * kGroupM * nnt;
        const int gsize = min(kGroupM, nmt - group * kGroupM);
        tl.row0 = (int64_t)(group * kGroupM + within % gsize) * 128;
        tl.col0 = within / gsize * TN;
        tl.e = expert_of(a, tl.row0);
        tl.kb0 = kSplits ? KB * rank / S : 0;
        tl.kb1 = kSplits ? KB * (rank + 1) / S : KB;
        return tl;
    };

    // The same order for a weight gradient, whose tiles are few blocks of K: a walk keeps its place instead of
    // the tile's number, which taken apart by divisions costs every role about 1000 cycles a tile.
    struct Walk {
        int e, group, pos;
    };
    auto settle = [&](Walk &w) {  // carry pos over into the next groups and experts
        for (;;) {
            const int count = min(kGroupM, nmt - w.group * kGroupM) * nnt;
            if (w.pos < count || w.e >= a.E)
                return;
            w.pos -= count;
            if (++w.group * kGroupM >= nmt) {
                w.group = 0;
                ++w.e;
            }
        }
    };
    auto start = [&]() {
        Walk w = {0, 0, first};
        if (ntiles > 0)
            settle(w);
        return w;
    };
    auto advance = [&](Walk &w) {
        w.pos += step;
        settle(w);
    };
    auto tile_at = [&](const Walk &w) {
        Tile tl;
        const int gsize = min(kGroupM, nmt - w.group * kGroupM);
        const int col = gsize == kGroupM ? w.pos / kGroupM : w.pos / gsize;
        tl.row0 = (int64_t)(w.group * kGroupM + w.pos - col * gsize) * 128;
        tl.col0 = col * TN;
        tl.e = w.e;
        tl.kb0 = min(sm.off[tl.e], KB);
        tl.kb1 = min(sm.off[tl.e + 1], KB);
        return tl;
    };

    if (warp >= kFirstPromo) {
        if (WG)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPromoRegs));
        const int q = warp & 3;                     // TMEM lane quadrant
        const int sub = (warp - kFirstPromo) >> 2;  // half of the columns
        constexpr int kCols = TN / 2;
        constexpr int kLd = 16;  // TMEM columns per load, two loads per wait
        const int row = q * 32 + lane;
        int buf = 0;
        uint32_t bph = 0;
        bool ok = true;
        if constexpr (WG) {
            int ss = 0;
            uint32_t sph = 0;
            // Here every column has a scale of its own.  Read as one row a lane, each would be one more
            // shared-memory pass per 32 products (1024 cycles a block, more than the copies and the
            // tensor core take); in the 16 x 256-bit shape a lane holds 4 rows x 32 of the 128 columns,
            // so it reads 32 column scales, and its pairs of columns leave as whole 32-byte sectors
            // without passing through shared memory.
            const int r0 = q * 32 + (lane >> 2), c2 = 2 * (lane & 3);
            Walk w = start();
            for (int t = first; t < ntiles; t += step, advance(w)) {
                const Tile tl = tile_at(w);
                float acc[2][kCols / 2];  // [half][4 g + i]
#pragma unroll
                for (int i = 0; i < kCols / 2; ++i)
                    acc[0][i] = acc[1][i] = 0.0f;
                for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
                    const bool s_ok = mbar_wait(&sm.sfull[ss], sph, a.status, abort_flag);
                    const float *scale = sm.scale[ss];
                    float f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        f[i] = scale[r0 + 8 * i];
                    const float2 *s2 = reinterpret_cast<const float2 *>(scale + 128 + sub * kCols + c2);
                    const bool w_ok = mbar_wait(&sm.tfull[buf], bph, a.status, abort_flag);
                    if (!__all_sync(0xffffffffu, w_ok && s_ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + buf * TN + sub * kCols;
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) {
                        float v[8], u[8];
                        const float2 x[2] = {s2[c / 2], s2[c / 2 + 4]};
                        tmem_ld_halves(tb + c, v, u);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const int i = 4 * g, o = c / 2 + i;
                            scaled_ffma2(acc[0][o], acc[0][o + 1], v[i], v[i + 1], x[g], f[0]);
                            scaled_ffma2(acc[0][o + 2], acc[0][o + 3], v[i + 2], v[i + 3], x[g], f[1]);
                            scaled_ffma2(acc[1][o], acc[1][o + 1], u[i], u[i + 1], x[g], f[2]);
                            scaled_ffma2(acc[1][o + 2], acc[1][o + 3], u[i + 2], u[i + 3], x[g], f[3]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.tempty[buf]);
                        mbar_arrive(&sm.sempty[ss]);
                    }
                    if (++buf == C::kBufs) {
                        buf = 0;
                        bph ^= 1;
                    }
                    if (++ss == C::kScaleSlots) {
                        ss = 0;
                        sph ^= 1;
                    }
                }
                if (!ok)
                    break;
                const int n0 = tl.col0 + sub * kCols;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t r = tl.row0 + r0 + 8 * i;
                    float *d = static_cast<float *>(a.d) + ((int64_t)tl.e * a.M + r) * a.N;
#pragma unroll
                    for (int g = 0; g < kCols / 8; g += 4) {
                        float2 x[4];  // columns 8 (g + j) + c2 and the next of row r
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            x[j] = make_float2(acc[i / 2][4 * (g + j) + 2 * (i & 1)],
                                               acc[i / 2][4 * (g + j) + 2 * (i & 1) + 1]);
                        if (a.wide) {  // (the same for every lane)
                            transpose4(x, lane);  // now the 8 columns of group g + lane % 4
                            const int n = n0 + 8 * (g + (lane & 3));
                            if (r < a.M && n < a.N)
                                store8(d + n, x, a.accumulate);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int n = n0 + 8 * (g + j) + c2;
                                if (r < a.M && n < a.N) {  // (N % 4 == 0: a pair of columns is in or out)
                                    d[n] = a.accumulate ? d[n] + x[j].x : x[j].x;
                                    d[n + 1] = a.accumulate ? d[n + 1] + x[j].y : x[j].y;
                                }
                            }
                        }
                    }
                }
            }
        } else {
        const int nsb = (a.N + 127) / 128;
        bool met = false;
        for (int t = first; t < ntiles; t += step) {
            const float *sa, *sb;
            int left_kb;  // blocks to go
            {
                const Tile tl = get_tile(t);
                const int64_t grow = tl.row0 + row;
                // (a row past M is never stored)
                sa = a.sa + (grow < a.M ? grow : a.M - 1) * a.sa_row + tl.kb0 * a.sa_blk;
                const int nb = min((tl.col0 + sub * kCols) / 128, nsb - 1);
                sb = a.sb + ((int64_t)tl.e * nsb + nb) * KB + tl.kb0;
                left_kb = tl.kb1 - tl.kb0;
            }
            float acc[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i)
                acc[i] = 0.0f;
            float sa_n = __ldg(sa), sb_n = __ldg(sb);
            for (; left_kb > 0; --left_kb) {
                const float f = sa_n * sb_n;
                if (left_kb > 1) {  // fetched while this block is on the tensor core
                    sa_n = __ldg(sa += a.sa_blk);
                    sb_n = __ldg(++sb);
                }
                const bool w_ok = mbar_wait(&sm.tfull[buf], bph, a.status, abort_flag);
                if (!__all_sync(0xffffffffu, w_ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + buf * TN + sub * kCols;
#pragma unroll
                for (int c = 0; c < kCols; c += 2 * kLd) {
                    float v[kLd], u[kLd];
                    tmem_ld_nowait(tb + c, v);
                    tmem_ld_nowait(tb + c + kLd, u);
                    tmem_wait_ld(v, u);
#pragma unroll
                    for (int i = 0; i < kLd; i += 2) {
                        ffma2(acc[c + i], acc[c + i + 1], v[i], v[i + 1], f);
                        ffma2(acc[c + kLd + i], acc[c + kLd + i + 1], u[i], u[i + 1], f);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.tempty[buf]);
                if (++buf == C::kBufs) {
                    buf = 0;
                    bph ^= 1;
                }
            }
            if (!ok)
                break;
            asm volatile("" : "+r"(t));  // (the tile is formed again, not kept in registers over the K loop)
            const Tile tl = get_tile(t);
            if (kSplits && S > 1) {
                // The parts meet in the stages' memory, free once every CTA of the cluster has finished
                // its part of K: CTA o adds up rows [o * own, (o + 1) * own) of the tile in the order of
                // the ranks.  Element (row r, column c) of a part is at [c][r ^ c], so that neither the
                // rows written by a warp nor the columns read by one meet a bank conflict.
                cluster_meet();
                const int own = 128 / S, owner = row / own;
                float *red = reinterpret_cast<float *>(sm.stage[0]);
                const uint32_t dst0 = cluster_map(red, owner) + (uint32_t)(rank * TN * own * 4);
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const int n = sub * kCols + c;
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(
                                     dst0 + (uint32_t)((n * own + ((row % own) ^ (n & (own - 1)))) * 4)),
                                 "f"(acc[c])
                                 : "memory");
                }
                cluster_meet();
                for (int i = (warp - kFirstPromo) * 32 + lane; i < own * TN; i += 32 * kPromoWarps) {
                    const int n = i % TN, r = i / TN;
                    float v = 0.0f;
                    for (int p = 0; p < S; ++p)
                        v += red[(p * TN + n) * own + (r ^ (n & (own - 1)))];
                    const int64_t m = tl.row0 + rank * own + r;
                    if (m < rows && tl.col0 + n < a.N) {
                        const int64_t at = m * a.ld_d + tl.col0 + n;
                        if (a.out_f32)
                            static_cast<float *>(a.d)[at] = v;
                        else
                            static_cast<__nv_bfloat16 *>(a.d)[at] = __float2bfloat16_rn(v);
                    }
                }
                met = true;
                break;
            }
            // Each lane holds one row.  Pieces of 64 bytes a row go through a per-warp shared block
            // (16-byte slot j of row r at j ^ ((r >> 1) & 3): no bank conflicts either way) and
            // leave as 8 rows x 64 contiguous bytes per store: on the way out lane l holds 16 bytes
            // at slot l % 4 of rows l / 4 + 8 i, whose addresses are formed once.
            float4(*ep)[4] = sm.ep_out[warp - kFirstPromo];
            const int rr = lane >> 2, cq = lane & 3;
            const int n0 = tl.col0 + sub * kCols;
            const int64_t left = rows - tl.row0 - q * 32;  // rows of D from lane 0's
            const int es = a.out_f32 ? 4 : 2, per = 16 / es;
            uint8_t *dst[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t r = tl.row0 + q * 32 + 8 * i + rr;
                dst[i] = 8 * i + rr < left ? static_cast<uint8_t *>(a.d) + (r * a.ld_d + n0 + per * cq) * es : nullptr;
            }
            const int n1 = n0 + per * cq;  // this lane's first column of a piece
            auto flush = [&](int c) {      // the shared block holds columns n0 + c ..
                __syncwarp();
                if (a.wide) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 o = ep[8 * i + rr][cq ^ (((8 * i + rr) >> 1) & 3)];
                        if (dst[i] && n1 + c < a.N)
                            *reinterpret_cast<float4 *>(dst[i] + c * es) = o;
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const float4 o = ep[8 * i + rr][cq ^ (((8 * i + rr) >> 1) & 3)];
                        if (8 * i + rr >= left)
                            continue;
                        uint8_t *d = dst[0] + (int64_t)8 * i * a.ld_d * es + c * es;
                        const float e4[4] = {o.x, o.y, o.z, o.w};
                        if (a.out_f32) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (n1 + c + j < a.N)
                                    reinterpret_cast<float *>(d)[j] = e4[j];
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (n1 + c + j < a.N)
                                    reinterpret_cast<uint16_t *>(d)[j] =
                                        (uint16_t)(__float_as_uint(e4[j / 2]) >> (16 * (j & 1)));
                        }
                    }
                }
                __syncwarp();
            };
            if (a.out_f32) {
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        ep[lane][j ^ ((lane >> 1) & 3)] =
                            make_float4(acc[c + 4 * j], acc[c + 4 * j + 1], acc[c + 4 * j + 2], acc[c + 4 * j + 3]);
                    flush(c);
                }
            } else {
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        ep[lane][j ^ ((lane >> 1) & 3)] = pack_bf16x8(acc + c + 8 * j, 1.0f);
                    flush(c);
                }
            }
        }
        if (kSplits && S > 1 && !met) {  // no tile, or given up: the peers' barriers still need this CTA
            cluster_meet();
            cluster_meet();
        }
        }
    } else {
        if (WG)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_b = l2_policy_evict_normal();
            const uint64_t pol_a = l2_policy_evict_last();
            int s = 0;
            uint32_t ph = 0;
            uint32_t issued = 0;  // stages with a copy issued, and its phase
            uint32_t issued_ph = 0;
            bool ok = true;
            Walk w = {};
            if (WG)
                w = start();
            for (int t = first; ok && t < ntiles; t += step) {
                Tile tl;
                if (WG) {
                    tl = tile_at(w);
                    advance(w);
                } else {
                    tl = get_tile(t);
                }
                const int brow = WG ? tl.col0 : tl.e * a.N + tl.col0;
                for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
                    if (!mbar_wait(&sm.empty[s], ph ^ 1, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t *dst = sm.stage[s];
                    mbar_arrive_expect_tx(&sm.full[s], C::kStageBytes);
                    tma_load_2d(dst, &a.tm_a, kb * 128, (int)tl.row0, &sm.full[s], pol_a);
#pragma unroll
                    for (int i = 0; i < (TN + 127) / 128; ++i)
                        tma_load_2d(dst + C::kABytes + i * 128 * 128, &a.tm_b, kb * 128, brow + i * 128, &sm.full[s],
                                    pol_b);
                    issued |= 1u << s;
                    issued_ph = (issued_ph & ~(1u << s)) | (ph << s);
                    if (++s == C::kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok) {  // let the copies in flight land before the shared memory is given up
                for (int i = 0; i < C::kStages; ++i)
                    if (issued >> i & 1) {
                        const unsigned long long t0 = global_timer_ns();
                        while (!mbar_try_wait(&sm.full[i], issued_ph >> i & 1) &&
                               global_timer_ns() - t0 < 100000000ull) {
                        }
                    }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int s = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true, any = false;
            const uint32_t idesc = make_idesc(0, 0, 128, TN);
            Walk w = {};
            if (WG)
                w = start();
            for (int t = first; ok && t < ntiles; t += step) {
                Tile tl;
                if (WG) {
                    tl = tile_at(w);
                    advance(w);
                } else {
                    tl = get_tile(t);
                }
                bool loaded = false;
                for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
                    if ((!loaded && !mbar_wait(&sm.full[s], ph, a.status, abort_flag)) ||
                        !mbar_wait(&sm.tempty[buf], bph ^ 1, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint8_t *as = sm.stage[s], *bs = sm.stage[s] + C::kABytes;
                    const int cur = s;
                    if (++s == C::kStages) {
                        s = 0;
                        ph ^= 1;
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        // the next block's copies are looked at while the queue holds MMAs of this one
                        if (kk == 2)
                            loaded = kb + 1 < tl.kb1 && mbar_try_wait(&sm.full[s], ph);
                        mma_fp8(tmem_base + buf * TN, smem_desc_sw128(as + kk * 32), smem_desc_sw128(bs + kk * 32),
                                idesc, kk > 0 ? 1u : 0u);
                    }
                    any = true;
                    mma_commit(&sm.tfull[buf]);
                    mma_commit(&sm.empty[cur]);
                    if (++buf == C::kBufs) {
                        buf = 0;
                        bph ^= 1;
                    }
                }
            }
            if (!ok && any) {
                mma_commit(&sm.drain);
                const unsigned long long t0 = global_timer_ns();
                while (!mbar_try_wait(&sm.drain, 0) && global_timer_ns() - t0 < 100000000ull) {
                }
            }
        }
    } else if (WG && warp == 2) {
        // Scales of each K block, copied ahead into a ring: fetched by the promotion warps a block
        // ahead, their latency paced the K loop, where every block is a new line.
        int ss = 0;
        uint32_t sph = 0;
        bool ok = true;
        Walk w = start();
        for (int t = first; ok && t < ntiles; t += step, advance(w)) {
            const Tile tl = tile_at(w);
            const float *sa = a.sa + (tl.row0 + lane) * a.sa_row + tl.kb0 * a.sa_blk;
            const int left = (int)min((int64_t)128, a.M - tl.row0);
            const float *sb = a.sb + tl.col0 + 4 * lane + (int64_t)tl.kb0 * a.N;
            const int col = tl.col0 + 4 * lane;
            for (int left_kb = tl.kb1 - tl.kb0; left_kb > 0; --left_kb) {
                const bool e_ok = mbar_wait(&sm.sempty[ss], sph ^ 1, a.status, abort_flag);
                if (!__all_sync(0xffffffffu, e_ok)) {
                    ok = false;
                    break;
                }
                float *dst = sm.scale[ss];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (lane + 32 * i < left)  // (rows past M are never stored)
                        cp_async_4(dst + lane + 32 * i, sa + 32 * i * a.sa_row);
#pragma unroll
                for (int i = 0; i < (TN + 127) / 128; ++i)
                    if (4 * lane + 128 * i < TN && col + 128 * i < a.N)  // (N % 4 == 0)
                        cp_async_16_zfill(dst + 128 + 4 * lane + 128 * i, sb + 128 * i, true);
                sa += a.sa_blk;
                sb += a.N;
                cp_async_arrive(&sm.sfull[ss]);
                if (++ss == C::kScaleSlots) {
                    ss = 0;
                    sph ^= 1;
                }
            }
        }
        cp_async_wait_all();
    }
    }
    if (kSplits && S > 1) {
        if (warp < kFirstPromo) {
            __syncwarp();
            cluster_meet();
            cluster_meet();
        }
        cluster_meet();  // no CTA leaves while a peer may still read or write its memory
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem_base, C::kBufs * TN);
}

// ------------------------------------------------------------- few rows
//
// Up to NP rows per expert: the weights take the tensor core's 128-row side and the NP rows of A its
// columns, so a tile streams 128 weight rows once.  A ring of 16 KB weight stages keeps the HBM
// requests in flight.  A cluster of S CTAs shares one tile, each taking a part of K; the parts are
// added through distributed shared memory in the order of the CTAs' ranks.

template <int NP>
struct FewCfg {
    static constexpr int kWBytes = 128 * 128;
    static constexpr int kXBytes = NP * 128;
    static constexpr int kStageBytes = kWBytes + kXBytes;
    static constexpr int kStages = NP == 64 ? 7 : NP == 32 ? 9 : 10;
    static constexpr int kBufs = 4;
    static constexpr int kTmem = kBufs * NP < 32 ? 32 : kBufs * NP;
    // promotion warps: one per TMEM lane quadrant, or two that share its columns
    static constexpr int kWarps = NP == 64 ? 8 : 4;
    static constexpr int kThreads = 64 + 32 * kWarps;
    static constexpr int kCols = NP * 4 / kWarps;  // columns of a warp
};

template <int NP>
struct __align__(1024) FewSmem {
    using C = FewCfg<NP>;
    uint8_t stage[C::kStages][C::kStageBytes];
    float red[NP * 128];                 // the parts of this CTA's rows: [source][column][row]
    float f[C::kWarps][2][C::kCols];     // a warp's column factors, alternating between blocks
    uint64_t full[C::kStages], empty[C::kStages];
    uint64_t tfull[C::kBufs], tempty[C::kBufs];
    uint64_t red_full, red_free;
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

template <int NP>
__global__ void __launch_bounds__(FewCfg<NP>::kThreads, 1) gemm_block_few_kernel(const __grid_constant__ Args a, int S)
{
    using C = FewCfg<NP>;
    extern __shared__ uint8_t smem_raw[];
    auto &sm = *reinterpret_cast<FewSmem<NP> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    volatile int *abort_flag = &sm.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            mbar_init(&sm.tfull[i], 1);
            mbar_init(&sm.tempty[i], C::kWarps);
        }
        mbar_init(&sm.red_full, (S > 4 ? S : 4) * (C::kWarps / 4));
        mbar_init(&sm.red_free, S * C::kWarps);
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&a.tm_a);
        tma_prefetch_desc(&a.tm_b);
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, C::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    if (S > 1)  // (the wait for it comes before the first write to a peer)
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem_base = sm.tmem_base;
    pdl_wait();
    pdl_trigger();
    const int KB = (a.K + 127) / 128;
    const int kb0 = (int)((int64_t)KB * rank / S), kb1 = (int)((int64_t)KB * (rank + 1) / S);
    const int64_t rows = rows_in_use(a);
    const int nblk = (int)((rows + NP - 1) / NP);
    const int nwt = (a.N + 127) / 128;
    const int64_t ntiles = (int64_t)nblk * nwt;
    const int first = blockIdx.x / S, step = gridDim.x / S;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_w = nblk > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
            const uint64_t pol_x = l2_policy_evict_last();
            int s = 0;
            uint32_t ph = 0, issued = 0, issued_ph = 0;
            bool ok = true;
            for (int64_t t = first; ok && t < ntiles; t += step) {
                const int b = (int)(t % nblk), wt = (int)(t / nblk);
                const int wrow = expert_of(a, (int64_t)b * NP) * a.N + wt * 128;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&sm.empty[s], ph ^ 1, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&sm.full[s], C::kStageBytes);
                    tma_load_2d(sm.stage[s], &a.tm_b, kb * 128, wrow, &sm.full[s], pol_w);
                    tma_load_2d(sm.stage[s] + C::kWBytes, &a.tm_a, kb * 128, b * NP, &sm.full[s], pol_x);
                    issued |= 1u << s;
                    issued_ph = (issued_ph & ~(1u << s)) | (ph << s);
                    if (++s == C::kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok)
                for (int i = 0; i < C::kStages; ++i)
                    if (issued >> i & 1) {
                        const unsigned long long t0 = global_timer_ns();
                        while (!mbar_try_wait(&sm.full[i], issued_ph >> i & 1) &&
                               global_timer_ns() - t0 < 100000000ull) {
                        }
                    }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int s = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true, any = false;
            const uint32_t idesc = make_idesc(0, 0, 128, NP);
            for (int64_t t = first; ok && t < ntiles; t += step)
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&sm.full[s], ph, a.status, abort_flag) ||
                        !mbar_wait(&sm.tempty[buf], bph ^ 1, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint8_t *w = sm.stage[s], *x = sm.stage[s] + C::kWBytes;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_fp8(tmem_base + buf * NP, smem_desc_sw128(w + kk * 32), smem_desc_sw128(x + kk * 32),
                                idesc, kk > 0 ? 1u : 0u);
                    any = true;
                    mma_commit(&sm.empty[s]);
                    mma_commit(&sm.tfull[buf]);
                    if (++s == C::kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                    if (++buf == C::kBufs) {
                        buf = 0;
                        bph ^= 1;
                    }
                }
            if (!ok && any) {
                mma_commit(&sm.drain);
                const unsigned long long t0 = global_timer_ns();
                while (!mbar_try_wait(&sm.drain, 0) && global_timer_ns() - t0 < 100000000ull) {
                }
            }
        }
    } else {
        constexpr int kCols = C::kCols;
        const int q = warp & 3, pw = warp - 2;
        const int col0 = pw / 4 * kCols;  // this warp's columns
        bool met = S == 1;  // the cluster's CTAs have all started
        const int row = q * 32 + lane;  // weight row of the tile
        int buf = 0;
        uint32_t bph = 0, rph = 0;
        bool ok = true;
        for (int64_t t = first; ok && t < ntiles; t += step) {
            const int b = (int)(t % nblk), wt = (int)(t / nblk);
            const int64_t x0 = (int64_t)b * NP;
            const int e = expert_of(a, x0);
            const float *sb = a.sb + ((int64_t)e * nwt + wt) * KB;
            float acc[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i)
                acc[i] = 0.0f;
            // lane c holds the next block's scale of column col0 + c
            static_assert(kCols <= 32, "a lane per column");
            float sx = 0.0f, sw = 0.0f;
            const int64_t xr = x0 + col0 + lane;
            const bool has = lane < kCols && xr < a.M;
            auto fetch = [&](int kb) {
                if (has)
                    sx = a.sa[xr * a.sa_row + kb * a.sa_blk];
                sw = sb[kb];
            };
            if (kb0 < kb1)
                fetch(kb0);
            for (int kb = kb0; kb < kb1; ++kb) {
                float *f = sm.f[pw][kb & 1];
                if (lane < kCols)
                    f[lane] = sx * sw;
                if (kb + 1 < kb1)
                    fetch(kb + 1);
                const bool w_ok = mbar_wait(&sm.tfull[buf], bph, a.status, abort_flag);
                if (!__all_sync(0xffffffffu, w_ok)) {
                    ok = false;
                    break;
                }
                __syncwarp();
                tc_fence_after();
                const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + buf * NP + col0;
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                    float v[8], u[8];
                    tmem_ld_nowait(tb + c, v);
                    tmem_ld_nowait(tb + c + 8, u);
                    tmem_wait_ld(v, u);
                    const float4 *f4 = reinterpret_cast<const float4 *>(f + c);
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 x = f4[i / 4], y = f4[2 + i / 4];
                        ffma2v(acc[c + i], acc[c + i + 1], v[i], v[i + 1], x.x, x.y);
                        ffma2v(acc[c + i + 2], acc[c + i + 3], v[i + 2], v[i + 3], x.z, x.w);
                        ffma2v(acc[c + 8 + i], acc[c + 9 + i], u[i], u[i + 1], y.x, y.y);
                        ffma2v(acc[c + 10 + i], acc[c + 11 + i], u[i + 2], u[i + 3], y.z, y.w);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.tempty[buf]);
                if (++buf == C::kBufs) {
                    buf = 0;
                    bph ^= 1;
                }
            }
            if (!ok)
                break;
            auto store = [&](int c, int n, float v) {
                if (x0 + c < rows && n < a.N) {
                    const int64_t at = (x0 + c) * a.ld_d + n;
                    if (a.out_f32)
                        static_cast<float *>(a.d)[at] = v;
                    else
                        static_cast<__nv_bfloat16 *>(a.d)[at] = __float2bfloat16_rn(v);
                }
            };
            if (S == 1) {
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    store(col0 + c, wt * 128 + row, acc[c]);
                continue;
            }
            // CTA o of the cluster adds up the tile's rows [o * own, (o + 1) * own)
            const int own = 128 / S, owner = row / own;
            if (!met) {
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
                met = true;
            }
            const bool free_ok = mbar_wait_cluster(&sm.red_free, rph ^ 1, a.status, abort_flag);
            if (!__all_sync(0xffffffffu, free_ok)) {
                ok = false;
                break;
            }
            const uint32_t dst = cluster_map(sm.red, owner) + (uint32_t)(((rank * NP + col0) * own + row % own) * 4);
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + (uint32_t)(c * own * 4)), "f"(acc[c])
                             : "memory");
            __syncwarp();
            if (lane == 0 || (own < 32 && lane == own))
                mbar_arrive_cluster(cluster_map(&sm.red_full, owner));
            const bool full_ok = mbar_wait_cluster(&sm.red_full, rph, a.status, abort_flag);
            if (!__all_sync(0xffffffffu, full_ok)) {
                ok = false;
                break;
            }
            for (int i = pw * 32 + lane; i < own * NP; i += 32 * C::kWarps) {
                float v = 0.0f;
                for (int s2 = 0; s2 < S; ++s2)
                    v += sm.red[s2 * NP * own + i];
                store(i / own, wt * 128 + rank * own + i % own, v);
            }
            __syncwarp();
            if (lane < S)
                mbar_arrive_cluster(cluster_map(&sm.red_free, lane));
            rph ^= 1;
        }
        if (!met)
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    if (S > 1 && warp < 2) {
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (S > 1)
        cluster_sync();  // no CTA leaves while a peer may still write to it
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem_base, C::kTmem);
}

// ------------------------------------------------------------- launches

// What a 64-column product of `tiles` tiles costs, in 10 ns: a block of K about 0.33 us a wave at one CTA an SM
// and 0.52 at two; the meeting of a split tile's CTAs 2.5 us.  *S: the CTAs that share a tile (each a part of
// K, four blocks at least) at the lowest cost.  (128 x 4096 x 14336: 49.9 us without a split, 32.9 with two CTAs
// a tile, 23.9 with four; 256 x 4096 x 4096: 15.3 without, 17.1 with two.)
int64_t cost64(int64_t tiles, int KB, int sms, int *S)
{
    int64_t best = INT64_MAX;
    for (int s = 1; s <= 8; s *= 2) {
        if (s > 1 && (tiles * s > 2 * sms || KB / s < 4))
            break;
        const int64_t waves = (tiles * s + 2 * sms - 1) / (2 * sms);
        const int64_t cost = waves * ((KB + s - 1) / s) * (tiles * s <= sms ? 33 : 52) + (s > 1 ? 250 : 0);
        if (cost < best) {
            best = cost;
            *S = s;
        }
    }
    return best;
}

// `clusters` clusters of S CTAs.
cudaError_t launch_cluster(void (*kern)(Args, int), const Args &a, int S, int64_t clusters, int threads, size_t smem,
                           cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * S));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, S);
}

template <int TN, bool WG>
cudaError_t launch_many(const Args &a, int64_t max_tiles, int sms, cudaStream_t st)
{
    auto kern = gemm_block_kernel<TN, WG>;
    constexpr size_t smem = sizeof(Smem<TN, WG>) + 1024;
    static_assert(smem <= 227 * 1024, "a CTA has at most 227 KB of shared memory");
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess)
        return err;
    const int64_t most = (int64_t)sms * Cfg<TN, WG>::kCtas;
    if (TN == 64 && !WG) {
        int S = 1;
        cost64(max_tiles, (a.K + 127) / 128, sms, &S);
        return launch_cluster(kern, a, S, max_tiles < most / S ? max_tiles : most / S, Cfg<TN, WG>::kThreads, smem, st);
    }
    const int grid = (int)(max_tiles < most ? max_tiles : most);
    return launch_kernel(true, kern, dim3(grid), dim3(Cfg<TN, WG>::kThreads), smem, st, a, 1);
}

template <int NP>
cudaError_t launch_few(const Args &a, int64_t max_tiles, int sms, cudaStream_t st)
{
    auto kern = gemm_block_few_kernel<NP>;
    constexpr size_t smem = sizeof(FewSmem<NP>) + 1024;
    static_assert(smem <= 227 * 1024, "a CTA has at most 227 KB of shared memory");
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess)
        return err;
    const int KB = (a.K + 127) / 128;
    // CTAs that share a tile: as many as SMs are free, four blocks of K each at least (us without and with:
    // one row, N 4096, K 14336 42.3 / 17.7; 64 rows, N 4096, K 4096 17.8 / 11.6).
    int S = 1;
    while (S < 8 && max_tiles * 2 * S <= sms && KB / (2 * S) >= 4)
        S *= 2;
    return launch_cluster(kern, a, S, max_tiles < sms / S ? max_tiles : sms / S, FewCfg<NP>::kThreads, smem, st);
}

// Columns of a tile.  A block of K costs a wave of tiles about 0.58 us with 256 columns and 0.40 with 128; 64 as
// above.  The cheapest is taken.  (us at 256 / 128 / 64 columns: 1024 x 4096 x 4096 21.1 / 29.5 / 34.1,
// 512 x 14336 x 4096 38.2 / 42.4 / 50.4, 1000 x 1416 x 2000 15.0 / 10.9 / 13.7.)
int column_tile(int64_t row_tiles, int N, int KB, int sms)
{
    const auto waves = [&](int tn) { return (row_tiles * ((N + tn - 1) / tn) + sms - 1) / sms; };
    const int64_t c256 = 58 * waves(256) * KB, c128 = 40 * waves(128) * KB;
    int S;
    const int64_t c64 = cost64(row_tiles * ((N + 63) / 64), KB, sms, &S);
    return c256 <= c128 && c256 <= c64 ? 256 : c128 <= c64 ? 128 : 64;
}

int to_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

}  // namespace blockgemm

}  // namespace moe

using namespace moe;
using namespace moe::blockgemm;

extern "C" {

int moe_gemm_fp8_block(const uint8_t *A, const float *a_scale, int a_scale_by_block, const uint8_t *B,
                       const float *b_scale, int64_t M, int N, int K, int E, int block_m,
                       const int32_t *sorted_expert_ids, const int32_t *num_tokens_post_padded, int out_type, void *D,
                       int64_t ld_d, void *ws, size_t ws_bytes, void *stream)
{
    if (M < 0 || N <= 0 || K <= 0 || E <= 0 || !A || !a_scale || !B || !b_scale || !D || !ws || ld_d < N ||
        a_scale_by_block < 0 || a_scale_by_block > 1 || (out_type != MOE_ROW_BF16 && out_type != MOE_ROW_FP32))
        return MOE_ERR_INVALID_ARG;
    const bool grouped = sorted_expert_ids != nullptr;
    if (grouped != (num_tokens_post_padded != nullptr) || (!grouped && (E != 1 || block_m != 0)))
        return MOE_ERR_INVALID_ARG;
    const int es = out_type == MOE_ROW_FP32 ? 4 : 2;
    if (misaligned(A, 16) || misaligned(B, 16) || misaligned(a_scale, 4) || misaligned(b_scale, 4) ||
        misaligned(D, es) || misaligned(ws, 4))
        return MOE_ERR_INVALID_ARG;
    if (K % 16 != 0 || K > 1 << 20 || N > 1 << 24 || (int64_t)E * N > 1 << 30 || M > 1 << 30)
        return MOE_ERR_UNSUPPORTED;
    if (grouped && block_m != 16 && block_m != 32 && block_m != 64 && (block_m <= 0 || block_m % 128 != 0))
        return MOE_ERR_UNSUPPORTED;
    if (ws_bytes < MOE_GEMM_BLOCK_WS_BYTES)
        return MOE_ERR_WORKSPACE;
    if (M == 0)
        return MOE_OK;
    const int sms = num_sms_current_device();
    if (sms <= 0)
        return MOE_ERR_CUDA;
    Args a = {};
    const int KB = (K + 127) / 128;
    a.sa = a_scale;
    a.sa_row = a_scale_by_block ? 1 : KB;
    a.sa_blk = a_scale_by_block ? M : 1;
    a.sb = b_scale;
    a.expert_ids = sorted_expert_ids;
    a.npp = num_tokens_post_padded;
    a.M = M, a.N = N, a.K = K, a.E = E, a.block_m = grouped ? block_m : 128;
    a.d = D, a.ld_d = ld_d, a.out_f32 = out_type == MOE_ROW_FP32;
    a.wide = ((reinterpret_cast<uintptr_t>(D) | (uintptr_t)(ld_d * es) | (uintptr_t)((int64_t)N * es)) & 15) == 0;
    a.status = static_cast<int *>(ws);
    const auto st = static_cast<cudaStream_t>(stream);
    // (us, few-row kernel against 64-column tiles: 64 rows, N 4096, K 14336 20.5 / 32.8; 64, N 14336, K 4096
    // 19.1 / 21.2; 32, N 4096, K 4096 11.0 / 13.8.  Sorted blocks of fewer than 128 rows have no other kernel.)
    const int few = grouped ? (block_m < 128 ? block_m : 0) : M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 0;
    const int64_t nmt = (M + 127) / 128;
    const int tn = few ? 128 : column_tile(nmt, N, (K + 127) / 128, sms);
    if (!encode_tmap_2d(&a.tm_a, A, 1, K, M, 128, few ? few : 128) ||
        !encode_tmap_2d(&a.tm_b, B, 1, K, (uint64_t)E * N, 128, tn < 128 ? tn : 128))
        return MOE_ERR_CUDA;
    if (few) {
        const int64_t tiles = (M + few - 1) / few * ((N + 127) / 128);
        return to_status(few == 16   ? launch_few<16>(a, tiles, sms, st)
                         : few == 32 ? launch_few<32>(a, tiles, sms, st)
                                     : launch_few<64>(a, tiles, sms, st));
    }
    const int64_t tiles = nmt * ((N + tn - 1) / tn);
    if (tiles > 1 << 30)
        return MOE_ERR_UNSUPPORTED;
    return to_status(tn == 256   ? launch_many<256, false>(a, tiles, sms, st)
                     : tn == 128 ? launch_many<128, false>(a, tiles, sms, st)
                                 : launch_many<64, false>(a, tiles, sms, st));
}

int moe_wgrad_fp8_block(const uint8_t *A, const float *a_scale, const uint8_t *B, const float *b_scale, int64_t P,
                        int M, int N, int E, const int32_t *expert_counts, float *D, int accumulate, void *ws,
                        size_t ws_bytes, void *stream)
{
    if (P < 0 || M <= 0 || N <= 0 || E <= 0 || !A || !a_scale || !B || !b_scale || !D || !ws || accumulate < 0 ||
        accumulate > 1 || (!expert_counts && E != 1))
        return MOE_ERR_INVALID_ARG;
    if (misaligned(A, 16) || misaligned(B, 16) || misaligned(a_scale, 4) || misaligned(b_scale, 16) ||
        misaligned(D, 4) || misaligned(ws, 4))
        return MOE_ERR_INVALID_ARG;
    if (E > kMaxE || P % 128 != 0 || N % 4 != 0 || P > 1 << 30 || M > 1 << 24 || N > 1 << 24)
        return MOE_ERR_UNSUPPORTED;
    if (ws_bytes < MOE_GEMM_BLOCK_WS_BYTES)
        return MOE_ERR_WORKSPACE;
    const int sms = num_sms_current_device();
    if (sms <= 0)
        return MOE_ERR_CUDA;
    Args a = {};
    a.sa = a_scale, a.sa_row = 1, a.sa_blk = M;
    a.sb = b_scale;
    a.counts = expert_counts;
    a.M = M, a.N = N, a.K = (int)P, a.E = E;
    a.d = D, a.ld_d = N, a.out_f32 = 1, a.accumulate = accumulate;
    a.wide = !misaligned(D, 32) && N % 8 == 0;
    a.status = static_cast<int *>(ws);
    const auto st = static_cast<cudaStream_t>(stream);
    const int64_t nmt = ((int64_t)M + 127) / 128;
    // Wide tiles for many, narrower ones where those would leave SMs idle (us at 256 / 128 / 64 columns: 4096 x
    // 14336 of eight experts 841 / 912 / 1356, 1024 x 2048 of eight 24.6 / 22.5 / 28.3, 512 x 1024 of four
    // 8.2 / 6.2 / 6.8, 256 x 512 of one over 4000 tokens 28.0 / 17.7 / 16.4).
    const int tn = nmt * ((N + 255) / 256) * E >= 4 * sms ? 256 : nmt * ((N + 127) / 128) * E >= sms / 2 ? 128 : 64;
    // P = 0: no block to read (the maps need at least one row)
    const uint64_t inner = P > 0 ? P : 128;
    if (!encode_tmap_2d(&a.tm_a, A, 1, inner, M, 128, 128) ||
        !encode_tmap_2d(&a.tm_b, B, 1, inner, N, 128, tn < 128 ? tn : 128))
        return MOE_ERR_CUDA;
    const int64_t tiles = nmt * ((N + tn - 1) / tn) * E;
    if (tiles > 1 << 30)
        return MOE_ERR_UNSUPPORTED;
    return to_status(tn == 256   ? launch_many<256, true>(a, tiles, sms, st)
                     : tn == 128 ? launch_many<128, true>(a, tiles, sms, st)
                                 : launch_many<64, true>(a, tiles, sms, st));
}

}  // extern "C"
