// Dense products of 16-bit matrices on CTA pairs, the core of the gated feed-forward block and of the
// vocabulary's cross entropy: D[M][N] = A B^T summed over K in fp32, then an epilogue on the accumulator.
//
// The two-SM tensor core (.cta_group::2) computes one 256 x NT tile per pair; CTA r of the pair holds the
// tile's A rows 128 r.. and B rows NT/2 r.. in its shared memory and the accumulator of its A rows in its
// TMEM.  Either operand may be stored with K contiguous ([rows][K]) or with its rows contiguous ([K][rows],
// an MN-major operand), so that the backward's products read the matrices as they lie and nothing is
// transposed:
//   MAJ 0: A and B [rows][K]  (x W^T);   MAJ 1: B is [K][N]  (d W);   MAJ 2: both are  (d^T x).
// Rows and K may end anywhere: TMA fills zeros past the edges of both operands.
//
// Roles (192 threads a CTA, one CTA an SM): warp 0 TMA producer, warp 1 issues the pair's MMAs (in the
// leader), warps 2..5 the epilogue of the CTA's 128 rows, which overlaps the next tile's MMAs through a
// second accumulator.  Tiles are dealt round-robin (all cost the same); groups of eight row tiles walk the
// columns together, so that 76 pairs in flight share about 8 x 10 tiles' rows through L2.
//
// Few tiles (a short batch, a narrow matrix) leave pairs idle: K is then split over S pairs a tile, which
// store fp32 partial sums, and a second kernel adds them in ascending order and applies the epilogue.
// Every sum has a fixed order: results are bitwise reproducible.
#pragma once

#include <atomic>
#include <type_traits>

#include "gemm_common.cuh"
#include "moe_internal.h"
#include "rows.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace dense {

// ------------------------------------------------------------- arguments

enum Mode {
    kStore,     // d = (acc_in + v) * *scale + add
    kGated,     // v = gate | up: h = act(gate) * up (and gate | up themselves, for the backward)
    kGatedBwd,  // v = dh: d gate | d up from the kept gate | up
    kLse,       // v = logits: each row's maximum and sum of exponentials in the tile, the target's logit
    kDlogits,   // v = logits: (softmax - one at the target) times the row's factor
};

struct Args {
    CUtensorMap tm_a, tm_b;
    int64_t M;
    int N;                // columns (gated: of h)
    int K;
    int tiles_m, tiles_n;
    int S;                // pairs that share a tile's K
    float *part;          // S > 1: partial sums
    int *status;
    // kStore: d [M] rows of N at pitch ld_d, of the rows' type or fp32; add of d's type
    void *d;
    int64_t ld_d;
    const void *add;
    int64_t ld_add;
    const float *acc_in;  // [M][N]
    const float *scale;
    int d_f32;
    // gated
    int act;
    void *h;              // [M][N]
    void *gu;             // [M][2N], kept by the forward (may be null) and read by the backward
    void *dgu;            // [M][2N]
    // cross entropy
    const int32_t *targets;
    float2 *stats;        // [M][tiles_n]
    float *target_logit;  // [M]
    const float *lse, *dloss;
    const float *dscale;  // {factor of dloss, its inverse}
    int v0, V;            // the piece's first column, the vocabulary
};

constexpr int kThreads = 192;
constexpr int kGroup = 8;
constexpr int kABytes = 128 * 128;  // 128 rows x 64 elements of K
template <int NT>
constexpr int kStageBytes = kABytes + NT / 2 * 128;
template <int NT>
constexpr int kStages = NT == 256 ? 7 : 9;

template <int NT>
struct __align__(1024) Smem {
    uint8_t stage[kStages<NT>][kStageBytes<NT>];
    uint64_t full[kStages<NT>];   // leader: both CTAs' bytes of the stage
    uint64_t empty[kStages<NT>];  // both: the MMAs have read the stage
    uint64_t tfull[2];            // both: accumulator complete
    uint64_t tempty[2];           // leader: both CTAs' epilogues have read it
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
template <int NT>
constexpr size_t kSmemBytes = sizeof(Smem<NT>) + 1024;
static_assert(kSmemBytes<256> <= 227 * 1024 && kSmemBytes<128> <= 227 * 1024, "a CTA has at most 227 KB");

// ------------------------------------------------------------ activations

// act(g) = g sigmoid(q(g)) with q = g (silu) or 2 sqrt(2/pi) (g + 0.044715 g^3) (gelu, tanh form: 1 + tanh z =
// 2 sigmoid(2z)); relu apart.  One exponential and one reciprocal an element: their errors (2^-21) vanish in the
// 16-bit rounding that follows, also where sigmoid is small, which 0.5 + 0.5 tanh would not give.
__device__ __forceinline__ float sigmoid_of(float q) { return __fdividef(1.0f, 1.0f + __expf(-q)); }

constexpr float kGeluA = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluB = 0.044715f;

__device__ __forceinline__ float act_of(float g, int act)
{
    if (act == MOE_ACT_RELU)
        return g <= 0.0f ? 0.0f : g;  // (a NaN stays one)
    const float q = act == MOE_ACT_SILU ? g : kGeluA * fmaf(kGeluB * g * g, g, g);
    return g * sigmoid_of(q);
}

// act(g) and its derivative s + g s (1 - s) q'(g)
__device__ __forceinline__ void act_grad(float g, int act, float &a, float &da)
{
    if (act == MOE_ACT_RELU) {
        a = g <= 0.0f ? 0.0f : g;
        da = g <= 0.0f ? 0.0f : 1.0f;
        return;
    }
    float q = g, dq = 1.0f;
    if (act != MOE_ACT_SILU) {
        const float g2 = g * g;
        q = kGeluA * fmaf(kGeluB * g2, g, g);
        dq = kGeluA * fmaf(3.0f * kGeluB, g2, 1.0f);
    }
    const float s = sigmoid_of(q);
    a = g * s;
    const float slope = s * (1.0f - s);
    da = slope == 0.0f ? s : fmaf(a * (1.0f - s), dq, s);  // (dq may be infinite where the slope is zero)
}

// --------------------------------------------------------------- epilogue

// 8 values to 16 bits each at a 16-byte boundary.
template <class TE>
__device__ __forceinline__ void store8(TE *dst, const float *v)
{
    *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_word(v[0], v[1], TE{}), pack_word(v[2], v[3], TE{}),
                                                 pack_word(v[4], v[5], TE{}), pack_word(v[6], v[7], TE{}));
}

template <class TE>
__device__ __forceinline__ void load8(const TE *src, float *v)
{
    const uint4 w = *reinterpret_cast<const uint4 *>(src);
    unpack_word(w.x, v[0], v[1], TE{});
    unpack_word(w.y, v[2], v[3], TE{});
    unpack_word(w.z, v[4], v[5], TE{});
    unpack_word(w.w, v[6], v[7], TE{});
}

// 32 columns from `col` of row `row` (N % 8 == 0; row < M).
template <class TE>
__device__ __forceinline__ void epi_store(const Args &a, int64_t row, int col, float (&v)[32])
{
    const float sc = a.scale ? *a.scale : 1.0f;
    if (a.acc_in) {
        const float *src = a.acc_in + row * a.N + col;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            if (col + i < a.N) {
                const float4 f = *reinterpret_cast<const float4 *>(src + i);
                v[i] += f.x, v[i + 1] += f.y, v[i + 2] += f.z, v[i + 3] += f.w;
            }
    }
    if (a.scale) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] *= sc;
    }
    if (a.d_f32) {
        float *dst = static_cast<float *>(a.d) + row * a.ld_d + col;
        const float *add = static_cast<const float *>(a.add) + row * a.ld_add + col;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            if (col + i < a.N) {
                float4 f = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                if (a.add) {
                    const float4 g = *reinterpret_cast<const float4 *>(add + i);
                    f.x += g.x, f.y += g.y, f.z += g.z, f.w += g.w;
                }
                *reinterpret_cast<float4 *>(dst + i) = f;
            }
        return;
    }
    TE *dst = static_cast<TE *>(a.d) + row * a.ld_d + col;
    const TE *add = static_cast<const TE *>(a.add) + row * a.ld_add + col;
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (col + i < a.N) {
            if (a.add) {
                float f[8];
                load8(add + i, f);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i + j] += f[j];
            }
            store8(dst + i, v + i);
        }
}

// h = act(g) u, from the unrounded products; g and u are rounded only where they are kept.
template <class TE>
__device__ __forceinline__ void epi_gated(const Args &a, int64_t row, int col, float (&g)[32], float (&u)[32])
{
    TE *hd = static_cast<TE *>(a.h) + row * a.N + col;
    if (a.gu) {
        TE *kept = static_cast<TE *>(a.gu) + row * 2 * a.N + col;
#pragma unroll
        for (int i = 0; i < 32; i += 8)
            if (col + i < a.N) {
                store8(kept + i, g + i);
                store8(kept + a.N + i, u + i);
            }
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
        g[i] = act_of(g[i], a.act) * u[i];
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (col + i < a.N)
            store8(hd + i, g + i);
}

// d gate = dh u act'(g), d up = dh act(g): rounded to 16 bits as the operands of the products that follow.
template <class TE>
__device__ __forceinline__ void epi_gated_bwd(const Args &a, int64_t row, int col, const float (&dh)[32])
{
    const TE *kept = static_cast<const TE *>(a.gu) + row * 2 * a.N + col;
    TE *out = static_cast<TE *>(a.dgu) + row * 2 * a.N + col;
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (col + i < a.N) {
            float g[8], u[8];
            load8(kept + i, g);
            load8(kept + a.N + i, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float act, slope;
                act_grad(g[j], a.act, act, slope);
                g[j] = dh[i + j] * u[j] * slope;
                u[j] = dh[i + j] * act;
            }
            store8(out + i, g);
            store8(out + a.N + i, u);
        }
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// One more 32 columns of a row's running maximum m and sum s of exp(v - m).  Columns past N count as -inf.
__device__ __forceinline__ void epi_lse(const Args &a, int col, int target, float (&v)[32], float &m, float &s,
                                        float &own, bool &has)
{
    if (col + 32 > a.N) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (col + i >= a.N)
                v[i] = -INFINITY;
    }
    const int at = target - col;
    if (at >= 0 && at < 32) {
        has = true;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i == at)
                own = v[i];
    }
    float top = v[0];
#pragma unroll
    for (int i = 1; i < 32; ++i)
        top = fmaxf(top, v[i]);
    const float was = m;
    m = fmaxf(m, top);
    const float base = m == -INFINITY ? 0.0f : m * kLog2e;  // (nothing but -inf so far: every term is 0)
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 32; ++i)
        part[i & 3] += exp2_fast(fmaf(v[i], kLog2e, -base));
    s = fmaf(s, exp2_fast(fmaf(was, kLog2e, -base)), (part[0] + part[1]) + (part[2] + part[3]));
}

// factor (softmax - one at the target), 32 columns; the pitch of the rows (a.ld_d) is a multiple of 8.
template <class TE>
__device__ __forceinline__ void epi_dlogits(const Args &a, int64_t row, int col, int target, float lse, float factor,
                                            float (&v)[32])
{
    const float base = lse * kLog2e;
    const int at = target - col;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        float p = exp2_fast(fmaf(v[i], kLog2e, -base));
        if (i == at)
            p -= 1.0f;
        v[i] = factor == 0.0f ? 0.0f : factor * p;  // (a row left out adds nothing, whatever its logits)
    }
    TE *dst = static_cast<TE *>(a.d) + row * a.ld_d + col;
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (col + i < a.N)
            store8(dst + i, v + i);
}

// -------------------------------------------------------------- the tiles

struct Tile {
    int m0, nt;    // first row, column tile
    int kb0, kb1;  // blocks of 64 of K
    int s;
};

__device__ __forceinline__ Tile tile_of(const Args &a, int t)
{
    Tile p;
    const int per = a.tiles_m * a.tiles_n;
    const int nkb = (a.K + 63) / 64;
    p.s = t / per;
    t -= p.s * per;
    p.kb0 = (int)((int64_t)nkb * p.s / a.S);
    p.kb1 = (int)((int64_t)nkb * (p.s + 1) / a.S);
    const int g = t / (kGroup * a.tiles_n);
    const int size = min(kGroup, a.tiles_m - g * kGroup);
    t -= g * kGroup * a.tiles_n;
    p.nt = t / size;
    p.m0 = (g * kGroup + t % size) * 256;
    return p;
}

// Columns of D that a tile covers.
template <int MODE, int NT>
constexpr int kCols = MODE == kGated ? NT / 2 : NT;

// Partial sums of CTA `rank` of a tile: [NT / 4][128 rows] of four columns, so that neighbouring threads (rows)
// touch neighbouring 16 bytes.
template <int NT>
__device__ __forceinline__ float4 *part_of(const Args &a, const Tile &p, int rank, int s)
{
    const int64_t tile = (int64_t)(p.m0 / 256) * a.tiles_n + p.nt;
    return reinterpret_cast<float4 *>(a.part) +
           (((int64_t)s * a.tiles_m * a.tiles_n + tile) * 2 + rank) * (NT / 4 * 128);
}

template <int MODE, int MAJ, class TE, int NT>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ Args a)
{
    using SmemT = Smem<NT>;
    constexpr int kS = kStages<NT>;
    constexpr int kHalf = NT / 2;  // B rows (accumulator columns) of one CTA
    extern __shared__ uint8_t smem_raw[];
    SmemT &sm = *reinterpret_cast<SmemT *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    volatile int *abort_flag = &sm.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kS; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.tfull[i], 1);
            mbar_init(&sm.tempty[i], 2 * 4);
        }
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&a.tm_a);
        tma_prefetch_desc(&a.tm_b);
    }
    if (warp == 1) {
        tmem_alloc_pair(&sm.tmem_base, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any signal between them
    tc_fence_after();
    const uint32_t tmem_base = sm.tmem_base;
    pdl_wait();
    pdl_trigger();

    const int items = a.tiles_m * a.tiles_n * a.S;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_normal();
            int s = 0;
            uint32_t ph = 0;
            bool ok = true, any = false;
            for (int t = first; ok && t < items; t += step) {
                const Tile p = tile_of(a, t);
                const int arow = p.m0 + rank * 128;
                // gated: CTA 0 holds gate rows, CTA 1 the matching up rows
                const int brow = MODE == kGated ? rank * a.N + p.nt * kHalf : p.nt * NT + rank * kHalf;
                for (int kb = p.kb0; kb < p.kb1; ++kb) {
                    if (!mbar_wait(&sm.empty[s], ph ^ 1, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = sm.stage[s], *sb = sm.stage[s] + kABytes;
                    const uint32_t bar = cluster_map(&sm.full[s], 0);
                    if (leader)
                        mbar_arrive_expect_tx(&sm.full[s], 2 * kStageBytes<NT>);
                    if (MAJ == 2) {
                        tma_load_2d_pair(sa, &a.tm_a, arow, kb * 64, bar, keep);
                        tma_load_2d_pair(sa + kABytes / 2, &a.tm_a, arow + 64, kb * 64, bar, keep);
                    } else {
                        tma_load_2d_pair(sa, &a.tm_a, kb * 64, arow, bar, keep);
                    }
                    if (MAJ >= 1) {
#pragma unroll
                        for (int c = 0; c < kHalf; c += 64)
                            tma_load_2d_pair(sb + c * 128, &a.tm_b, brow + c, kb * 64, bar, keep);
                    } else {
                        tma_load_2d_pair(sb, &a.tm_b, kb * 64, brow, bar, keep);
                    }
                    any = true;
                    if (++s == kS) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok && any) {
                // copies in flight complete on the leader's barriers: a bounded moment for them to land
                const unsigned long long t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 20000000ull) {
                }
            }
        }
    } else if (warp == 1) {
        if (leader && lane == 0) {
            const uint32_t type = std::is_same<TE, __nv_bfloat16>::value ? 1u : 0u;  // (fp16: 0) both operands alike
            const uint32_t idesc = make_idesc(type, type, 256, NT) | (MAJ >= 1 ? 1u << 16 : 0u) |
                                   (MAJ == 2 ? 1u << 15 : 0u);
            int s = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true, any = false;
            for (int t = first; ok && t < items; t += step) {
                const Tile p = tile_of(a, t);
                if (!mbar_wait(&sm.tempty[acc], aph ^ 1, a.status, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + acc * 256;
                for (int kb = p.kb0; kb < p.kb1; ++kb) {
                    if (!mbar_wait(&sm.full[s], ph, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint8_t *sa = sm.stage[s], *sb = sm.stage[s] + kABytes;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        // 16 of K: 32 bytes further along a K-major row, 16 rows further in an MN-major box
                        const uint64_t da = MAJ == 2 ? smem_desc_sw128_mn(sa + kk * 2048, kABytes / 2)
                                                     : smem_desc_sw128(sa + kk * 32);
                        const uint64_t db = MAJ >= 1 ? smem_desc_sw128_mn(sb + kk * 2048, 8192)
                                                     : smem_desc_sw128(sb + kk * 32);
                        mma_pair<0>(d, da, db, idesc, (kb > p.kb0 || kk > 0) ? 1u : 0u);
                    }
                    any = true;
                    mma_commit_pair(&sm.empty[s], 0x3);
                    if (++s == kS) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                if (!ok)
                    break;
                mma_commit_pair(&sm.tfull[acc], 0x3);
                if (++acc == 2) {
                    acc = 0;
                    aph ^= 1;
                }
            }
            if (!ok && any) {
                mma_commit_pair(&sm.drain, 0x1);
                const unsigned long long t0 = global_timer_ns();
                while (!mbar_try_wait(&sm.drain, 0) && global_timer_ns() - t0 < 100000000ull) {
                }
            }
        }
    } else {
        const int q = warp & 3;  // TMEM lane quadrant of this warp
        const int r = q * 32 + lane;
        int acc = 0;
        uint32_t aph = 0;
        for (int t = first; t < items; t += step) {
            const Tile p = tile_of(a, t);
            const int64_t row = p.m0 + rank * 128 + r;
            const bool live = row < a.M;
            const int c0 = p.nt * kCols<MODE, NT>;
            if (MODE == kGatedBwd && a.S == 1 && live) {
                // the kept gate | up of this thread's part of the tile: into L2 while the MMAs run
                const TE *kept = static_cast<const TE *>(a.gu) + row * 2 * a.N + c0;
                for (int c = 0; c < NT && c0 + c < a.N; c += 64) {
                    prefetch_l2(kept + c);
                    prefetch_l2(kept + a.N + c);
                }
            }
            int target = -1;
            float lse = 0.0f, factor = 0.0f;
            if ((MODE == kLse || MODE == kDlogits) && live) {
                target = a.targets[row];
                const bool counts = target >= 0 && target < a.V;
                if (MODE == kDlogits) {
                    lse = a.lse[row];
                    factor = counts ? a.dloss[row] * a.dscale[0] : 0.0f;
                }
                target = counts ? target - a.v0 : -1;
            }
            bool ok = mbar_wait(&sm.tfull[acc], aph, a.status, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                break;
            tc_fence_after();
            const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + acc * 256;
            if (a.S > 1) {
                float4 *dst = part_of<NT>(a, p, rank, p.s) + r;
#pragma unroll 1
                for (int c = 0; c < NT; c += 32) {
                    float v[32];
                    tmem_ld32(tacc + c, v);
                    if (!live)
                        continue;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        dst[(c + i) / 4 * 128] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            } else if (MODE == kGated) {
#pragma unroll 1
                for (int c = 0; c < kHalf && c0 + c < a.N; c += 32) {
                    float g[32], u[32];
                    tmem_ld32(tacc + c, g);
                    tmem_ld32(tacc + kHalf + c, u);
                    if (live)
                        epi_gated<TE>(a, row, c0 + c, g, u);
                }
            } else {
                float m = -INFINITY, s = 0.0f, own = 0.0f;
                bool has = false;
#pragma unroll 1
                for (int c = 0; c < NT && c0 + c < a.N; c += 32) {
                    float v[32];
                    tmem_ld32(tacc + c, v);
                    if (!live)
                        continue;
                    if (MODE == kStore)
                        epi_store<TE>(a, row, c0 + c, v);
                    else if (MODE == kGatedBwd)
                        epi_gated_bwd<TE>(a, row, c0 + c, v);
                    else if (MODE == kLse)
                        epi_lse(a, c0 + c, target, v, m, s, own, has);
                    else
                        epi_dlogits<TE>(a, row, c0 + c, target, lse, factor, v);
                }
                if (MODE == kLse && live) {
                    a.stats[row * a.tiles_n + p.nt] = make_float2(m, s);
                    if (has)
                        a.target_logit[row] = own;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_remote(cluster_map(&sm.tempty[acc], 0));
            if (++acc == 2) {
                acc = 0;
                aph ^= 1;
            }
        }
    }

    // both CTAs stay until the pair's last MMA, copy and remote arrive are done
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc_pair(tmem_base, 512);
}

// The partial sums of a tile added up in ascending order, then the epilogue: a block of 128 threads (rows) for
// 32 columns of one CTA's part of a tile.
template <int MODE, class TE, int NT>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Args a)
{
    constexpr int kChunks = kCols<MODE, NT> / 32;
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x % kChunks * 32, rank = blockIdx.x / kChunks & 1, t = blockIdx.x / kChunks / 2;
    Tile p;
    p.m0 = t / a.tiles_n * 256;
    p.nt = t % a.tiles_n;
    const int64_t row = p.m0 + rank * 128 + threadIdx.x;
    const int col = p.nt * kCols<MODE, NT> + c;
    if (row >= a.M || col >= a.N)
        return;
    float v[32] = {}, u[32] = {};
    for (int s = 0; s < a.S; ++s) {
        const float4 *src = part_of<NT>(a, p, rank, s) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 f = src[(c + i) / 4 * 128];
            v[i] += f.x, v[i + 1] += f.y, v[i + 2] += f.z, v[i + 3] += f.w;
        }
        if (MODE == kGated) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 f = src[(NT / 2 + c + i) / 4 * 128];
                u[i] += f.x, u[i + 1] += f.y, u[i + 2] += f.z, u[i + 3] += f.w;
            }
        }
    }
    if (MODE == kStore)
        epi_store<TE>(a, row, col, v);
    else if (MODE == kGated)
        epi_gated<TE>(a, row, col, v, u);
    else
        epi_gated_bwd<TE>(a, row, col, v);
}

// ------------------------------------------------------------------- host

// Clusters of two that can be resident at once, kept per device.
template <int MODE, int MAJ, class TE, int NT>
int max_pairs()
{
    static std::atomic<int> cache[64];  // zero until first computed
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        auto kern = gemm_kernel<MODE, MAJ, TE, NT>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<NT>) !=
            cudaSuccess)
            return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemBytes<NT>;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0)
            return 0;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Workspace of the partial sums: as many tiles as there are pairs, at most.
constexpr size_t kPartBytes = (size_t)80 * 256 * 256 * 4;

// Pairs that share a tile's K: as many as would be idle otherwise, with at least four blocks of 64 each.
inline int k_split(int64_t tiles, int K, int pairs)
{
    int S = (int)(pairs / tiles);
    const int most = (K + 63) / 64 / 4;
    if (S > most)
        S = most;
    if (S > 16)
        S = 16;
    return S < 1 ? 1 : S;
}

// D = A B^T by the rule above.  a: everything but the tiles; part: kPartBytes or null (no split).
template <int MODE, int MAJ, class TE, int NT>
cudaError_t launch(Args &a, float *part, cudaStream_t st)
{
    auto kern = gemm_kernel<MODE, MAJ, TE, NT>;
    int pairs = max_pairs<MODE, MAJ, TE, NT>();
    if (pairs <= 0)
        return cudaErrorInvalidConfiguration;
    if (pairs > 80)
        pairs = 80;
    const int64_t tm = (a.M + 255) / 256, tn = (a.N + kCols<MODE, NT> - 1) / kCols<MODE, NT>;
    if (tm * tn > 1 << 30)
        return cudaErrorInvalidValue;
    a.tiles_m = (int)tm, a.tiles_n = (int)tn;
    a.S = part ? k_split(tm * tn, a.K, pairs) : 1;
    a.part = part;
    const int64_t items = tm * tn * a.S;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<NT>);
    if (err != cudaSuccess)
        return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (items < pairs ? items : pairs)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes<NT>;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, kern, a);
    if (err != cudaSuccess || a.S == 1)
        return err;
    if constexpr (MODE == kStore || MODE == kGated || MODE == kGatedBwd)
        return launch_kernel(true, join_kernel<MODE, TE, NT>, dim3((unsigned)(tm * tn * 2 * (kCols<MODE, NT> / 32))),
                             dim3(128), 0, st, a);
    return cudaErrorInvalidValue;
}

}  // namespace dense
}  // namespace moe
