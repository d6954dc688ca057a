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
// Roles (320 threads a CTA, one CTA an SM): warp 0 TMA producer, warp 1 issues the pair's MMAs (in the
// leader), warps 2..9 the epilogue of the CTA's 128 rows (two warps a row, each half of the columns), which
// overlaps the next tile's MMAs through a second accumulator.  Tiles are dealt round-robin (those of a product
// cost the same); groups of eight row tiles walk the columns together, so that 76 pairs in flight share about
// 8 x 10 tiles' rows through L2.  Products that do not depend on one another (the gradients of x and of the
// weights) go into one launch, longest K first: one start, one tail and one rounding up to whole waves.
//
// Few tiles (a short batch, a narrow matrix) leave pairs idle: tiles are then half as wide, or K is split over S
// pairs a tile, which store fp32 partial sums, and a second kernel adds them in ascending order and applies the
// epilogue.  Every sum has a fixed order: results are bitwise reproducible.
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

constexpr int kProducts = 3;  // of one launch

struct Product {
    CUtensorMap tm_a, tm_b;
    const void *A, *B;    // from which the launch makes the maps, whose boxes go by the tile
    int64_t ld_a, ld_b;
    int64_t M;
    int N;                // columns (gated: of h; B then has 2N rows)
    int K;
    int maj;              // 0, 1 or 2, as above
    int tiles_m, tiles_n;
    int S;                // pairs that share a tile's K
    int first;            // its first item; an item is a tile, or a part of K of one
    // kStore: d [M] rows of N at pitch ld_d, of the rows' type or fp32; add of d's type
    void *d;
    int64_t ld_d;
    const void *add;
    int64_t ld_add;
    const float *acc_in;  // [M][N]
    const float *scale;
    int d_f32;
};

struct Args {
    Product p[kProducts];
    int n, items;
    float *part;          // partial sums, one accumulator an item
    int *status;
    // gated
    int act;
    void *h;              // [M][N]
    void *gu;             // [M][2N], kept by the forward (may be null) and read by the backward
    void *dgu;            // [M][2N]
    // cross entropy
    const int32_t *targets;
    float2 *stats;        // [M][pairs]
    int pairs;            // (maximum, sum) pairs of a row
    float *target_logit;  // [M]
    const float *lse, *dloss;
    const float *dscale;  // {factor of dloss, its inverse}
    int v0, V;            // the piece's first column, the vocabulary
};

constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
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

// W columns from `col` of row `row` (N % 8 == 0; row < M).
template <class TE, int W>
__device__ __forceinline__ void epi_store(const Product &a, int64_t row, int col, float (&v)[W])
{
    const float sc = a.scale ? *a.scale : 1.0f;
    if (a.acc_in) {
        const float *src = a.acc_in + row * a.N + col;
#pragma unroll
        for (int i = 0; i < W; i += 4)
            if (col + i < a.N) {
                const float4 f = *reinterpret_cast<const float4 *>(src + i);
                v[i] += f.x, v[i + 1] += f.y, v[i + 2] += f.z, v[i + 3] += f.w;
            }
    }
    if (a.scale) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            v[i] *= sc;
    }
    if (a.d_f32) {
        float *dst = static_cast<float *>(a.d) + row * a.ld_d + col;
        const float *add = static_cast<const float *>(a.add) + row * a.ld_add + col;
#pragma unroll
        for (int i = 0; i < W; i += 4)
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
    for (int i = 0; i < W; i += 8)
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
template <class TE, int W>
__device__ __forceinline__ void epi_gated(const Args &a, int64_t row, int col, float (&g)[W], float (&u)[W])
{
    const int N = a.p[0].N;
    TE *hd = static_cast<TE *>(a.h) + row * N + col;
    if (a.gu) {
        TE *kept = static_cast<TE *>(a.gu) + row * 2 * N + col;
#pragma unroll
        for (int i = 0; i < W; i += 8)
            if (col + i < N) {
                store8(kept + i, g + i);
                store8(kept + N + i, u + i);
            }
    }
#pragma unroll
    for (int i = 0; i < W; ++i)
        g[i] = act_of(g[i], a.act) * u[i];
#pragma unroll
    for (int i = 0; i < W; i += 8)
        if (col + i < N)
            store8(hd + i, g + i);
}

// d gate = dh u act'(g), d up = dh act(g): rounded to 16 bits as the operands of the products that follow.
template <class TE, int W>
__device__ __forceinline__ void epi_gated_bwd(const Args &a, int64_t row, int col, const float (&dh)[W])
{
    const int N = a.p[0].N;
    const TE *kept = static_cast<const TE *>(a.gu) + row * 2 * N + col;
    TE *out = static_cast<TE *>(a.dgu) + row * 2 * N + col;
#pragma unroll
    for (int i = 0; i < W; i += 8)
        if (col + i < N) {
            float g[8], u[8];
            load8(kept + i, g);
            load8(kept + N + i, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float act, slope;
                act_grad(g[j], a.act, act, slope);
                g[j] = dh[i + j] * u[j] * slope;
                u[j] = dh[i + j] * act;
            }
            store8(out + i, g);
            store8(out + N + i, u);
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
__device__ __forceinline__ void epi_lse(int N, int col, int target, float (&v)[32], float &m, float &s, float &own,
                                        bool &has)
{
    if (col + 32 > N) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (col + i >= N)
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

// factor (softmax - one at the target), 32 columns; the pitch of the rows (ld_d) is a multiple of 8.
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
    TE *dst = static_cast<TE *>(a.p[0].d) + row * a.p[0].ld_d + col;
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (col + i < a.p[0].N)
            store8(dst + i, v + i);
}

// -------------------------------------------------------------- the tiles

struct Tile {
    int prod;      // which product
    int m0, nt;    // first row, column tile
    int kb0, kb1;  // blocks of 64 of K
};

template <int MODE>
__device__ __forceinline__ Tile tile_of(const Args &a, int t)
{
    Tile r;
    r.prod = 0;
    if (MODE == kStore)
        while (r.prod + 1 < a.n && t >= a.p[r.prod + 1].first)
            ++r.prod;
    const Product &p = a.p[r.prod];
    t -= p.first;
    const int per = p.tiles_m * p.tiles_n;
    const int nkb = (p.K + 63) / 64;
    const int s = t / per;
    t -= s * per;
    r.kb0 = (int)((int64_t)nkb * s / p.S);
    r.kb1 = (int)((int64_t)nkb * (s + 1) / p.S);
    const int g = t / (kGroup * p.tiles_n);
    const int size = min(kGroup, p.tiles_m - g * kGroup);
    t -= g * kGroup * p.tiles_n;
    r.nt = t / size;
    r.m0 = (g * kGroup + t % size) * 256;
    return r;
}

// Columns of D that a tile covers.
template <int MODE, int NT>
constexpr int kCols = MODE == kGated ? NT / 2 : NT;

// Partial sums of CTA `rank` of an item: [NT / 4][128 rows] of four columns, so that neighbouring threads (rows)
// touch neighbouring 16 bytes.
template <int NT>
__device__ __forceinline__ float4 *part_of(const Args &a, int item, int rank)
{
    return reinterpret_cast<float4 *>(a.part) + ((int64_t)item * 2 + rank) * (NT / 4 * 128);
}

template <int MODE, class TE, int NT>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ Args a)
{
    using SmemT = Smem<NT>;
    constexpr int kS = kStages<NT>;
    constexpr int kHalf = NT / 2;  // B rows of one CTA
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
            mbar_init(&sm.tempty[i], 2 * kEpiWarps);
        }
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        fence_mbarrier_init();
        for (int i = 0; i < a.n; ++i) {
            tma_prefetch_desc(&a.p[i].tm_a);
            tma_prefetch_desc(&a.p[i].tm_b);
        }
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

    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_normal();
            int s = 0;
            uint32_t ph = 0;
            bool ok = true, any = false;
            for (int t = first; ok && t < a.items; t += step) {
                const Tile tile = tile_of<MODE>(a, t);
                const Product &p = a.p[tile.prod];
                const int maj = MODE == kStore ? p.maj : MODE == kGatedBwd ? 1 : 0;
                const int arow = tile.m0 + rank * 128;
                // gated: CTA 0 holds gate rows, CTA 1 the matching up rows
                const int brow = MODE == kGated ? rank * p.N + tile.nt * kHalf : tile.nt * NT + rank * kHalf;
                for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
                    if (!mbar_wait(&sm.empty[s], ph ^ 1, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = sm.stage[s], *sb = sm.stage[s] + kABytes;
                    const uint32_t bar = cluster_map(&sm.full[s], 0);
                    if (leader)
                        mbar_arrive_expect_tx(&sm.full[s], 2 * kStageBytes<NT>);
                    if (maj == 2) {
                        tma_load_2d_pair(sa, &p.tm_a, arow, kb * 64, bar, keep);
                        tma_load_2d_pair(sa + kABytes / 2, &p.tm_a, arow + 64, kb * 64, bar, keep);
                    } else {
                        tma_load_2d_pair(sa, &p.tm_a, kb * 64, arow, bar, keep);
                    }
                    if (maj >= 1) {
#pragma unroll
                        for (int c = 0; c < kHalf; c += 64)
                            tma_load_2d_pair(sb + c * 128, &p.tm_b, brow + c, kb * 64, bar, keep);
                    } else {
                        tma_load_2d_pair(sb, &p.tm_b, kb * 64, brow, bar, keep);
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
            int s = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true, any = false;
            for (int t = first; ok && t < a.items; t += step) {
                const Tile tile = tile_of<MODE>(a, t);
                const int maj = MODE == kStore ? a.p[tile.prod].maj : MODE == kGatedBwd ? 1 : 0;
                const uint32_t idesc = make_idesc(type, type, 256, NT) | (maj >= 1 ? 1u << 16 : 0u) |
                                       (maj == 2 ? 1u << 15 : 0u);
                if (!mbar_wait(&sm.tempty[acc], aph ^ 1, a.status, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + acc * 256;
                for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
                    if (!mbar_wait(&sm.full[s], ph, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint8_t *sa = sm.stage[s], *sb = sm.stage[s] + kABytes;
                    // 16 of K: 32 bytes further along a K-major row, 16 rows (2 KB) further in an MN-major box
                    uint64_t da = maj == 2 ? smem_desc_sw128_mn(sa, kABytes / 2) : smem_desc_sw128(sa);
                    uint64_t db = maj >= 1 ? smem_desc_sw128_mn(sb, 8192) : smem_desc_sw128(sb);
                    const uint64_t ia = maj == 2 ? 2048 >> 4 : 32 >> 4, ib = maj >= 1 ? 2048 >> 4 : 32 >> 4;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        mma_pair<0>(d, da, db, idesc, (kb > tile.kb0 || kk > 0) ? 1u : 0u);
                        da += ia, db += ib;  // (the start address is the descriptor's lowest field)
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
        const int q = warp & 3;          // TMEM lane quadrant of this warp
        const int half = (warp - 2) / 4; // its half of the columns
        const int r = q * 32 + lane;
        int acc = 0;
        uint32_t aph = 0;
        for (int t = first; t < a.items; t += step) {
            const Tile tile = tile_of<MODE>(a, t);
            const Product &p = a.p[tile.prod];
            const int64_t row = tile.m0 + rank * 128 + r;
            const bool live = row < p.M;
            constexpr int kMine = kCols<MODE, NT> / 2;              // columns of D of this warp
            const int c0 = tile.nt * kCols<MODE, NT> + half * kMine;  // the first of them
            // what the epilogue will read of memory: into L2 while the MMAs run
            if (MODE == kGatedBwd && p.S == 1 && live) {
                const TE *kept = static_cast<const TE *>(a.gu) + row * 2 * p.N + c0;
                for (int c = 0; c < kMine && c0 + c < p.N; c += 64) {
                    prefetch_l2(kept + c);
                    prefetch_l2(kept + p.N + c);
                }
            }
            if (MODE == kStore && p.S == 1 && live && p.add) {
                const int es = p.d_f32 ? 4 : 2;
                const char *add = static_cast<const char *>(p.add) + (row * p.ld_add + c0) * es;
                for (int c = 0; c < kMine && c0 + c < p.N; c += 128 / es)
                    prefetch_l2(add + c * es);
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
            if (p.S > 1) {
                float4 *dst = part_of<NT>(a, t, rank) + r;
#pragma unroll 1
                for (int c = half * kHalf; c < (half + 1) * kHalf; c += 32) {
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
                for (int c = 0; c < kMine && c0 + c < p.N; c += 32) {
                    float g[32], u[32];
                    tmem_ld32(tacc + half * kMine + c, g);
                    tmem_ld32(tacc + kHalf + half * kMine + c, u);
                    if (live)
                        epi_gated<TE>(a, row, c0 + c, g, u);
                }
            } else {
                float m = -INFINITY, s = 0.0f, own = 0.0f;
                bool has = false;
#pragma unroll 1
                for (int c = 0; c < kMine && c0 + c < p.N; c += 32) {
                    float v[32];
                    tmem_ld32(tacc + half * kMine + c, v);
                    if (!live)
                        continue;
                    if (MODE == kStore)
                        epi_store<TE>(p, row, c0 + c, v);
                    else if (MODE == kGatedBwd)
                        epi_gated_bwd<TE>(a, row, c0 + c, v);
                    else if (MODE == kLse)
                        epi_lse(p.N, c0 + c, target, v, m, s, own, has);
                    else
                        epi_dlogits<TE>(a, row, c0 + c, target, lse, factor, v);
                }
                if (MODE == kLse && live) {
                    a.stats[row * a.pairs + tile.nt * 2 + half] = make_float2(m, s);
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
// 8 columns of one CTA's part of a tile (32 columns a thread, with the parts in line: 8-17 us instead of 4).
constexpr int kJoinCols = 8;

struct JoinBlocks {
    int first[kProducts + 1];  // first block of each product (none for one that is not split)
};

template <int MODE, class TE, int NT>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Args a, JoinBlocks jb)
{
    constexpr int kChunks = kCols<MODE, NT> / kJoinCols;
    pdl_wait();
    pdl_trigger();
    int prod = 0;
    while ((int)blockIdx.x >= jb.first[prod + 1])
        ++prod;
    const Product &p = a.p[prod];
    const int b = blockIdx.x - jb.first[prod];
    const int c = b % kChunks * kJoinCols, rank = b / kChunks & 1, t = b / kChunks / 2;
    const Tile tile = tile_of<MODE>(a, p.first + t);
    const int64_t row = tile.m0 + rank * 128 + threadIdx.x;
    const int col = tile.nt * kCols<MODE, NT> + c;
    if (row >= p.M || col >= p.N)
        return;
    const int tiles = p.tiles_m * p.tiles_n;
    float v[kJoinCols] = {}, u[kJoinCols] = {};
#pragma unroll 4
    for (int s = 0; s < p.S; ++s) {
        const float4 *src = part_of<NT>(a, p.first + s * tiles + t, rank) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < kJoinCols; i += 4) {
            const float4 f = __ldcs(src + (c + i) / 4 * 128);
            v[i] += f.x, v[i + 1] += f.y, v[i + 2] += f.z, v[i + 3] += f.w;
        }
        if (MODE == kGated) {
#pragma unroll
            for (int i = 0; i < kJoinCols; i += 4) {
                const float4 f = __ldcs(src + (NT / 2 + c + i) / 4 * 128);
                u[i] += f.x, u[i + 1] += f.y, u[i + 2] += f.z, u[i + 3] += f.w;
            }
        }
    }
    if (MODE == kStore)
        epi_store<TE>(p, row, col, v);
    else if (MODE == kGated)
        epi_gated<TE>(a, row, col, v, u);
    else
        epi_gated_bwd<TE>(a, row, col, v);
}

// ------------------------------------------------------------------- host

// One more product of the launch: D [M][N] = A B^T over K, the operands' rows ld_a and ld_b elements apart.
inline Product &product(Args &a, int64_t M, int N, int K, int maj, const void *A, int64_t ld_a, const void *B,
                        int64_t ld_b)
{
    Product &p = a.p[a.n++];
    p.M = M, p.N = N, p.K = K, p.maj = maj;
    p.A = A, p.ld_a = ld_a, p.B = B, p.ld_b = ld_b;
    return p;
}

// Tensor maps of a product's operands in boxes of 64 elements x 128 rows (B: half a tile's), MN-major ones 64 x 64.
template <int MODE, int NT>
bool make_maps(Product &p)
{
    const auto map = [](CUtensorMap *m, const void *at, int64_t inner, int64_t rows, int64_t pitch, int box_rows) {
        return encode_tmap_2d_pitched(m, at, 2, inner, rows, pitch, 64, box_rows);
    };
    const int64_t b_rows = MODE == kGated ? 2 * (int64_t)p.N : p.N;
    return (p.maj == 2 ? map(&p.tm_a, p.A, p.M, p.K, p.ld_a, 64) : map(&p.tm_a, p.A, p.K, p.M, p.ld_a, 128)) &&
           (p.maj >= 1 ? map(&p.tm_b, p.B, p.N, p.K, p.ld_b, 64) : map(&p.tm_b, p.B, p.K, b_rows, p.ld_b, NT / 2));
}

// Clusters of two that can be resident at once, kept per device.
template <int MODE, class TE, int NT>
int max_pairs()
{
    static std::atomic<int> cache[64];  // zero until first computed
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        auto kern = gemm_kernel<MODE, TE, NT>;
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

// Workspace of the partial sums: there are at most as many parts as pairs.
constexpr int kMostPairs = 80;
constexpr size_t kPartBytes = (size_t)kMostPairs * 256 * 256 * 4;

template <int MODE, class TE, int NT>
cudaError_t launch_nt(Args &a, int S, int pairs, cudaStream_t st)
{
    auto kern = gemm_kernel<MODE, TE, NT>;
    JoinBlocks jb = {};
    int64_t items = 0;
    bool split = false;
    for (int i = 0; i < a.n; ++i) {
        Product &p = a.p[i];
        const int64_t tm = (p.M + 255) / 256, tn = (p.N + kCols<MODE, NT> - 1) / kCols<MODE, NT>;
        const int most = (p.K + 63) / 64;
        if (!make_maps<MODE, NT>(p))
            return cudaErrorInvalidValue;
        p.tiles_m = (int)tm, p.tiles_n = (int)tn;
        p.S = S < most ? S : most;
        p.first = (int)items;
        items += tm * tn * p.S;
        if (items > 1 << 30)
            return cudaErrorInvalidValue;
        split = split || p.S > 1;
        jb.first[i + 1] = jb.first[i] + (p.S > 1 ? (int)(tm * tn * 2 * (kCols<MODE, NT> / kJoinCols)) : 0);
    }
    for (int i = a.n; i < kProducts; ++i)
        jb.first[i + 1] = jb.first[i];
    a.items = (int)items;
    a.pairs = a.p[0].tiles_n * 2;
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
    if (err != cudaSuccess || !split)
        return err;
    if constexpr (MODE == kStore || MODE == kGated || MODE == kGatedBwd)
        return launch_kernel(true, join_kernel<MODE, TE, NT>, dim3((unsigned)jb.first[kProducts]), dim3(128), 0, st, a,
                             jb);
    return cudaErrorInvalidValue;
}

// The launch's time by its parts: waves of tiles, each the blocks of K in line (KB) and an epilogue that nothing
// hides in the last wave; a split's second kernel.  In 10 ns.
inline int64_t cost_of(int64_t tiles, int64_t KB, int S, bool wide, int pairs)
{
    const int64_t waves = (tiles * S + pairs - 1) / pairs;
    return waves * ((KB + S - 1) / S) * (wide ? 28 : 19) + (wide ? 250 : 150) + (S > 1 ? 400 : 0);
}

// The products of `a` (p[0] .. p[n - 1] but for their tiles), longest K first.  part: kPartBytes, or null (no
// split).
template <int MODE, class TE>
cudaError_t launch(Args &a, float *part, cudaStream_t st)
{
    int pairs = max_pairs<MODE, TE, 256>();  // (one CTA an SM at either width)
    if (pairs <= 0)
        return cudaErrorInvalidConfiguration;
    if (pairs > kMostPairs)
        pairs = kMostPairs;
    a.part = part;
    for (int i = 1; i < a.n; ++i)
        for (int j = i; j > 0 && a.p[j].K > a.p[j - 1].K; --j) {
            const Product t = a.p[j];
            a.p[j] = a.p[j - 1], a.p[j - 1] = t;
        }
    int64_t best = INT64_MAX;
    int S = 1;
    bool wide = true;
    for (int w = MODE == kLse ? 1 : 0; w < 2; ++w) {  // (a logit tile leaves two pairs a row, whatever its width)
        const int cols = (w ? 256 : 128) / (MODE == kGated ? 2 : 1);
        int64_t tiles = 0, blocks = 0;
        for (int i = 0; i < a.n; ++i) {
            const int64_t n = (a.p[i].M + 255) / 256 * ((a.p[i].N + cols - 1) / cols);
            tiles += n, blocks += n * ((a.p[i].K + 63) / 64);
        }
        const int64_t KB = (blocks + tiles - 1) / tiles;
        for (int s = 1; s <= 16 && (s == 1 || (part && tiles * s <= pairs && KB / s >= 4)); ++s) {
            const int64_t c = cost_of(tiles, KB, s, w, pairs);
            if (c < best)
                best = c, S = s, wide = w;
        }
    }
    if constexpr (MODE != kLse)
        if (!wide)
            return launch_nt<MODE, TE, 128>(a, S, pairs, st);
    return launch_nt<MODE, TE, 256>(a, S, pairs, st);
}

}  // namespace dense
}  // namespace moe
