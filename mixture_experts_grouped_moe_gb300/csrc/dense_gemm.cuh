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
// overlaps the next tile's MMAs through a second accumulator.  Tiles are dealt to the clusters beforehand (those of a
// product cost the same); groups of 16 row tiles walk the columns together, so that 76 pairs in flight share about
// 16 x 5 tiles' rows through L2, where they are kept (evict-last).  Products that do not depend on one another (the
// gradients of x and of the weights) go into one launch, longest K first: one start, one tail and one rounding up to
// whole waves.
//
// Few tiles (a short batch, a narrow matrix) leave pairs idle: tiles are then half as wide, or K is split over the
// S = 2 or 4 pairs of a cluster.  Each then owns 1/S of the tile's columns: the others' fp32 parts of them come
// through distributed shared memory, into the stages that no MMA reads any more, and are added in ascending order
// before the epilogue.  Every sum has a fixed order: results are bitwise reproducible.
//
// Bound by the tensor pipe for many tiles: 8192 x 4096 x 28672 and 8192 x 14336 x 4096 (a gated block's two products)
// 1.53-1.61 ms, 1.79-1.89 PFLOP/s; in a row by the board's power, 1.66 PFLOP/s (a library product: 1.69).  Few tiles
// are bound by a launch's latency (release of the predecessor 2 us, first loads 1.1, epilogue 1-2, meeting 2) and by
// what an SM takes from L2: a block of 64 of K, 32 KB a CTA, 0.29 us.
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
    kStoreLong, // the same for a long K, summed in parts
    kGated,     // v = gate | up: h = act(gate) * up (and gate | up themselves, for the backward)
    kGatedBwd,  // v = dh: d gate | d up from the kept gate | up
    kLse,       // v = logits: each row's maximum and sum of exponentials in the tile, the target's logit
    kLseLong,   // the same for a long K, summed in parts
    kDlogits,   // v = logits: (softmax - one at the target) times the row's factor
    kDlogitsLong,
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
    int first;            // its first tile
    // kStore: d [M] rows of N at pitch ld_d, of the rows' type or fp32; add of d's type
    void *d;
    int64_t ld_d;
    const void *add;
    int64_t ld_add;
    const float *acc_in;  // [M][N]
    const float *scale;
    int d_f32;
};

// Which tiles a cluster goes through.  The first product's (the longest K) are dealt round-robin.  Where its last
// round leaves some clusters without one, those first get as many rounds of the others' tiles as take the same time;
// the rest is dealt round-robin to all, from those clusters on.
struct Deal {
    int P;     // clusters
    int n0;    // the first product's tiles: q whole rounds and r more
    int q, r;
    int E;     // rounds that the clusters from r on get ahead of the rest

    // Tile k of cluster c; a number past the last tile when there is none (then there is none for any larger k).
    __host__ __device__ int tile(int c, int k) const
    {
        const int mine = q + (c < r ? 1 : 0);
        if (k < mine)
            return k * P + c;
        k -= mine;
        if (c >= r) {
            if (k < E)
                return n0 + k * (P - r) + c - r;
            k -= E;
        }
        return n0 + E * (P - r) + k * P + (c >= r ? c - r : c - r + P);
    }
};

struct Args {
    Product p[kProducts];
    int n, tiles;
    Deal deal;
    int S;                // pairs that share a tile's K, one cluster
    int *status;
    // gated
    int act;
    void *h;              // [M][N]
    void *gu;             // [M][2N], kept by the forward (may be null) and read by the backward
    void *dgu;            // [M][2N], fp16: times a power of two (gradient_factor)
    const unsigned *most; // [kMost], fp16: the largest finite |dout|, in parts, as bits
    float *back;          // the inverse of that factor
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
// Row tiles of a group (ms of a prefill's two products in a row, one box: 8 1.757, 16 1.740, 32 1.820; the box's own
// spread is 0.5 %).
constexpr int kGroup = 16;
constexpr int kABytes = 128 * 128;  // 128 rows x 64 elements of K
template <int NT>
constexpr int kStageBytes = kABytes + NT / 2 * 128;
template <int NT>
constexpr int kStages = NT == 256 ? 6 : 8;
// The tensor core truncates what it adds to its running sum: of positive products a sum loses 2.7e-6 of itself over
// K = 2048, 1.0e-5 over 4096, 3.0e-5 over 8192, 3.8e-4 over 65536 and 1.6e-3 over 262144 (of products of either sign,
// relative to the result's 2-norm: 2.1e-6, 4.4e-6, 9.1e-6, 7.6e-5, 3.0e-4).  Results that stay in 32 bits are therefore
// summed a part of a long K at a time, the parts in registers with rounding, also within each pair's share of a split
// tile; the whole goes back to TMEM for the epilogue.  The sums take most of the registers, so that the kernel that
// follows no longer starts ahead, and a change of parts costs about 0.4 us of a pair's time.
//
// The loss: 2048 at a time, 2.8e-6 at most for any K (4096 x 32000, 100 rows 54 -> 58 us, 2000 rows 295 -> 298; shorter
// rows keep the plain form).  The backward's logits go the same way: p = exp(l - lse) wants l as it was when lse was
// made of it, above all where p is near 1 and the gradient is 1 - p (a logit of 30 that lost 1.0e-5 of itself makes
// 1 - p = 1e-3 a third larger).  Weight gradients in fp32, over K rows: 4096 at a time.
constexpr int kPart = 32;      // blocks of 64 of K
constexpr int kPartRows = 64;
template <int MODE>
constexpr bool kIsLse = MODE == kLse || MODE == kLseLong;
template <int MODE>
constexpr bool kIsDlogits = MODE == kDlogits || MODE == kDlogitsLong;
template <int MODE>
constexpr bool kIsStore = MODE == kStore || MODE == kStoreLong;
template <int MODE>
constexpr bool kInParts = MODE == kStoreLong || MODE == kLseLong || MODE == kDlogitsLong;
template <int MODE>
constexpr int kPartOf = kIsStore<MODE> ? kPartRows : kPart;
constexpr int kRowsBytes = 4096;    // an epilogue warp's 32 rows of 32 columns of up to 32 bits

template <int NT>
struct __align__(1024) Smem {
    uint8_t stage[kStages<NT>][kStageBytes<NT>];
    uint8_t rows[kEpiWarps][kRowsBytes];
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
// 2 sigmoid(2z)); relu apart.  One exponential and one reciprocal an element, relative to the result also where sigmoid
// is small, which 0.5 + 0.5 tanh would not be.  The fast exponential's documented error grows with its argument, 2 +
// 1.17 |q| steps of 2^-23: 2^-20 near zero, 2^-18.4 at |q| = 20 and 2^-16.4 at 80, where bf16 still holds silu.  For
// the gelu q's own rounding adds as much.  Half a step of the 16-bit rounding that follows is 2^-12 or more.
__device__ __forceinline__ float sigmoid_of(float q) { return __fdividef(1.0f, 1.0f + __expf(-q)); }

constexpr float kGeluA = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluB = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_of(float g)
{
    if (ACT == MOE_ACT_RELU)
        return g <= 0.0f ? 0.0f : g;  // (a NaN stays one)
    const float q = ACT == MOE_ACT_SILU ? g : kGeluA * fmaf(kGeluB * g * g, g, g);
    return g * sigmoid_of(q);
}

// act(g) and its derivative s + g s (1 - s) q'(g)
template <int ACT>
__device__ __forceinline__ void act_grad(float g, float &a, float &da)
{
    if (ACT == MOE_ACT_RELU) {
        a = g <= 0.0f ? 0.0f : g;
        da = g <= 0.0f ? 0.0f : 1.0f;
        return;
    }
    float q = g, dq = 1.0f;
    if (ACT != MOE_ACT_SILU) {
        const float g2 = g * g;
        q = kGeluA * fmaf(kGeluB * g2, g, g);
        dq = kGeluA * fmaf(3.0f * kGeluB, g2, 1.0f);
    }
    const float s = sigmoid_of(q);
    a = g * s;
    const float slope = s * (1.0f - s);
    da = slope == 0.0f ? s : fmaf(a * (1.0f - s), dq, s);  // (dq may be infinite where the slope is zero)
}

// fn(a constant of the activation): the choice outside the loops over elements (inside, the branches kept a warp's
// exponentials apart: 3.7 us of a 256 x 256 tile's epilogue against 1.2).
template <class F>
__device__ __forceinline__ void with_act(int act, F fn)
{
    if (act == MOE_ACT_SILU)
        fn(std::integral_constant<int, MOE_ACT_SILU>());
    else if (act == MOE_ACT_GELU_TANH)
        fn(std::integral_constant<int, MOE_ACT_GELU_TANH>());
    else
        fn(std::integral_constant<int, MOE_ACT_RELU>());
}

// g = act(g) * u
template <int W>
__device__ __forceinline__ void gate(int act, float (&g)[W], const float (&u)[W])
{
    with_act(act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            g[i] = act_of<decltype(kind)::value>(g[i]) * u[i];
    });
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
__device__ __forceinline__ void unpack8(const uint4 &w, float *v)
{
    unpack_word(w.x, v[0], v[1], TE{});
    unpack_word(w.y, v[2], v[3], TE{});
    unpack_word(w.z, v[4], v[5], TE{});
    unpack_word(w.w, v[6], v[7], TE{});
}

template <class TE>
__device__ __forceinline__ void load8(const TE *src, float *v)
{
    unpack8<TE>(*reinterpret_cast<const uint4 *>(src), v);
}

// 32 rows x 32 columns between memory and a warp's registers, through its shared memory.  The accumulator gives a
// thread a row; 16 bytes of 32 different rows at a time would touch 32 lines a request and thrash the little L1
// that is left (a 256 x 256 tile's epilogue with `add` took 13 us, the gated backward's 23 us).  Here a request
// covers whole rows (64 or 128 bytes), and the pieces of 16 bytes are swizzled so that both orders are free of
// bank conflicts.
template <class T>
struct Rows {
    static constexpr int kP = sizeof(T) == 4 ? 8 : 4;    // pieces of a row; also: requests
    static constexpr int kV = 16 / (int)sizeof(T);       // elements of a piece
    __device__ __forceinline__ static int at(int r, int c)
    {
        return r * kP + (kP == 8 ? c ^ (r & 7) : c ^ (r >> 1 & 3));
    }

    // Rows 0 .. rows - 1 and columns 0 .. cols - 1 of p; zeros elsewhere.
    __device__ __forceinline__ static void load(const T *p, int64_t ld, int rows, int cols, int lane, uint4 *w)
    {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            const int r = i * (32 / kP) + lane / kP, c = lane % kP * kV;
            w[i] = r < rows && c < cols ? *reinterpret_cast<const uint4 *>(p + r * ld + c) : make_uint4(0, 0, 0, 0);
        }
    }
    // As loaded -> the thread's own row.
    __device__ __forceinline__ static void to_row(uint4 *buf, uint4 *w, int lane)
    {
#pragma unroll
        for (int i = 0; i < kP; ++i)
            buf[at(i * (32 / kP) + lane / kP, lane % kP)] = w[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kP; ++i)
            w[i] = buf[at(lane, i)];
        __syncwarp();
    }
    // The thread's own row -> memory.
    __device__ __forceinline__ static void store(uint4 *buf, const uint4 *w, T *p, int64_t ld, int rows, int cols,
                                                 int lane)
    {
#pragma unroll
        for (int i = 0; i < kP; ++i)
            buf[at(lane, i)] = w[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            const int r = i * (32 / kP) + lane / kP, c = lane % kP * kV;
            const uint4 v = buf[at(r, lane % kP)];
            if (r < rows && c < cols)
                *reinterpret_cast<uint4 *>(p + r * ld + c) = v;
        }
        __syncwarp();
    }
};

template <class TE>
__device__ __forceinline__ uint4 pack8(const float *v)
{
    return make_uint4(pack_word(v[0], v[1], TE{}), pack_word(v[2], v[3], TE{}), pack_word(v[4], v[5], TE{}),
                      pack_word(v[6], v[7], TE{}));
}

// 32 values of the thread's row, each rounded, to memory.
template <class TE>
__device__ __forceinline__ void put_rows(uint4 *buf, const float *v, TE *p, int64_t ld, int rows, int cols, int lane)
{
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack8<TE>(v + 8 * i);
    Rows<TE>::store(buf, w, p, ld, rows, cols, lane);
}

__device__ __forceinline__ void add4(float *v, const uint4 &w)
{
    v[0] += __uint_as_float(w.x), v[1] += __uint_as_float(w.y);
    v[2] += __uint_as_float(w.z), v[3] += __uint_as_float(w.w);
}

// The forms that follow are of one thread's row in pieces of its own (the few columns of a split tile's owner).

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
        if (a.add) {
            const float *add = static_cast<const float *>(a.add) + row * a.ld_add + col;
            float4 f[W / 4];
#pragma unroll
            for (int i = 0; i < W; i += 4)
                if (col + i < a.N)
                    f[i / 4] = *reinterpret_cast<const float4 *>(add + i);
#pragma unroll
            for (int i = 0; i < W; i += 4)
                v[i] += f[i / 4].x, v[i + 1] += f[i / 4].y, v[i + 2] += f[i / 4].z, v[i + 3] += f[i / 4].w;
        }
#pragma unroll
        for (int i = 0; i < W; i += 4)
            if (col + i < a.N)
                *reinterpret_cast<float4 *>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        return;
    }
    TE *dst = static_cast<TE *>(a.d) + row * a.ld_d + col;
    if (a.add) {
        const TE *add = static_cast<const TE *>(a.add) + row * a.ld_add + col;
        uint4 w[W / 8];
#pragma unroll
        for (int i = 0; i < W; i += 8)
            if (col + i < a.N)
                w[i / 8] = *reinterpret_cast<const uint4 *>(add + i);
#pragma unroll
        for (int i = 0; i < W; i += 8) {
            float f[8];
            unpack8<TE>(w[i / 8], f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i + j] += f[j];
        }
    }
#pragma unroll
    for (int i = 0; i < W; i += 8)
        if (col + i < a.N)
            store8(dst + i, v + i);
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
    gate(a.act, g, u);
#pragma unroll
    for (int i = 0; i < W; i += 8)
        if (col + i < N)
            store8(hd + i, g + i);
}

constexpr int kMost = 128;

// In fp16, d gate | d up are kept times 2^-e, with the largest finite |dout| in [2^e, 2^(e+1)) and e < 0: steps of
// 2^-24 would otherwise be all that is left of an output gradient far below one (a step is 6 % at 1e-6).  Its products
// are scaled back in fp32.  bf16 has fp32's range.
template <class TE>
constexpr bool kScaledGrad = std::is_same<TE, __half>::value;

// The factor (a whole warp).
__device__ __forceinline__ float gradient_factor(const unsigned *most, int lane)
{
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < kMost; i += 32)
        m = max(m, most[i + lane]);
    m = __reduce_max_sync(0xffffffffu, m);
    const float v = __half2float(__ushort_as_half((unsigned short)m));
    return v > 0.0f && v < 1.0f ? ldexpf(1.0f, -ilogbf(v)) : 1.0f;
}

// d gate = dh u act'(g), d up = dh act(g) of 8 columns, in the place of g and u: rounded to 16 bits as the operands
// of the products that follow.
template <class TE, int ACT>
__device__ __forceinline__ void gated_grad8(const float *dh, float factor, uint4 &wg, uint4 &wu)
{
    float g[8], u[8];
    unpack8<TE>(wg, g);
    unpack8<TE>(wu, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float v, slope;
        act_grad<ACT>(g[j], v, slope);
        const float d = kScaledGrad<TE> ? dh[j] * factor : dh[j];
        g[j] = d * u[j] * slope;
        u[j] = d * v;
    }
    wg = pack8<TE>(g);
    wu = pack8<TE>(u);
}

template <class TE, int W>
__device__ __forceinline__ void epi_gated_bwd(const Args &a, int64_t row, int col, const float (&dh)[W], float factor)
{
    const int N = a.p[0].N;
    const TE *kept = static_cast<const TE *>(a.gu) + row * 2 * N + col;
    TE *out = static_cast<TE *>(a.dgu) + row * 2 * N + col;
    uint4 wg[W / 8], wu[W / 8];
#pragma unroll
    for (int i = 0; i < W; i += 8)
        if (col + i < N) {
            wg[i / 8] = *reinterpret_cast<const uint4 *>(kept + i);
            wu[i / 8] = *reinterpret_cast<const uint4 *>(kept + N + i);
        }
    with_act(a.act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < W; i += 8)
            if (col + i < N)
                gated_grad8<TE, decltype(kind)::value>(dh + i, factor, wg[i / 8], wu[i / 8]);
    });
#pragma unroll
    for (int i = 0; i < W; i += 8)
        if (col + i < N) {
            *reinterpret_cast<uint4 *>(out + i) = wg[i / 8];
            *reinterpret_cast<uint4 *>(out + N + i) = wu[i / 8];
        }
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// One more W columns of a row's running maximum m and sum s of exp(v - m).  Columns past N count as -inf.
template <int W>
__device__ __forceinline__ void epi_lse(int N, int col, int target, float (&v)[W], float &m, float &s, float &own,
                                        bool &has)
{
    if (col + W > N) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (col + i >= N)
                v[i] = -INFINITY;
    }
    const int at = target - col;
    if (at >= 0 && at < W) {
        has = true;
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (i == at)
                own = v[i];
    }
    float top = v[0];
#pragma unroll
    for (int i = 1; i < W; ++i)
        top = fmaxf(top, v[i]);
    const float was = m;
    m = fmaxf(m, top);
    const float base = m == -INFINITY ? 0.0f : m * kLog2e;  // (nothing but -inf so far: every term is 0)
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < W; ++i)
        part[i & 3] += exp2_fast(fmaf(v[i], kLog2e, -base));
    s = fmaf(s, exp2_fast(fmaf(was, kLog2e, -base)), (part[0] + part[1]) + (part[2] + part[3]));
}

// factor (softmax - one at the target), W columns.
template <int W>
__device__ __forceinline__ void epi_dlogits(int col, int target, float lse, float factor, float (&v)[W])
{
    const float base = lse * kLog2e;
    const int at = target - col;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        float p = exp2_fast(fmaf(v[i], kLog2e, -base));
        if (i == at)
            p -= 1.0f;
        v[i] = factor == 0.0f ? 0.0f : factor * p;  // (a row left out adds nothing, whatever its logits)
    }
}

// What the logits' epilogues know of a row: its target's column in the piece (-1: none, or left out), lse and the
// factor of its gradient.
struct RowOf {
    int target;
    float lse, factor;
};
template <int MODE>
__device__ __forceinline__ RowOf row_of(const Args &a, int64_t row)
{
    RowOf r = {-1, 0.0f, 0.0f};
    if (row < a.p[0].M) {
        const int t = a.targets[row];
        const bool counts = t >= 0 && t < a.V;
        if (kIsDlogits<MODE>) {
            r.lse = a.lse[row];
            r.factor = counts ? a.dloss[row] * a.dscale[0] : 0.0f;
        }
        r.target = counts ? t - a.v0 : -1;
    }
    return r;
}

// -------------------------------------------------------------- the tiles

struct Tile {
    int prod;      // which product
    int m0, nt;    // first row, column tile
    int kb0, kb1;  // blocks of 64 of K
};

// Tile t, and the part of K that falls to pair s of the cluster.
template <int MODE>
__device__ __forceinline__ Tile tile_of(const Args &a, int t, int s)
{
    Tile r;
    r.prod = 0;
    if (kIsStore<MODE>)
        while (r.prod + 1 < a.n && t >= a.p[r.prod + 1].first)
            ++r.prod;
    const Product &p = a.p[r.prod];
    t -= p.first;
    const int nkb = (p.K + 63) / 64;
    const int shift = a.S >> 1;  // log2 of S = 1, 2 or 4 (nkb < 2^24)
    r.kb0 = nkb * s >> shift;
    r.kb1 = nkb * (s + 1) >> shift;
    const int g = t / (kGroup * p.tiles_n);
    const int size = min(kGroup, p.tiles_m - g * kGroup);
    t -= g * kGroup * p.tiles_n;
    r.nt = t / size;
    r.m0 = (g * kGroup + t % size) * 256;
    return r;
}

// Parts of K that a tile (a pair's share of it) is summed in.
template <int MODE>
__device__ __forceinline__ int parts_of(const Tile &t)
{
    return (t.kb1 - t.kb0 + kPartOf<MODE> - 1) / kPartOf<MODE>;
}

// Columns of D that a tile covers.
template <int MODE, int NT>
constexpr int kCols = MODE == kGated ? NT / 2 : NT;

// The parts of a split tile's accumulator to the pairs that own their columns, and the owners' epilogue.  All
// threads of the cluster.  buf: [S sources][columns / 4][128 rows] of four columns, so that neighbouring threads
// (rows) touch neighbouring 16 bytes.
template <int MODE, class TE, int NT>
__device__ __forceinline__ void meet(const Args &a, uint8_t *buf, uint32_t tmem_base, const Tile &tile, int rank,
                                     int pair, int warp, int lane, float factor)
{
    const int S = a.S, q = warp & 3, half = (warp - 2) / 4, r = q * 32 + lane;
    // accumulator columns that a pair owns: gated, as many of the gate's as of the up's
    constexpr int kSides = MODE == kGated ? 2 : 1;
    constexpr int kSide = NT / kSides;
    const int own = kSide / S;  // of each side, 32 or more
    if (warp >= 2) {
        const int acc = kInParts<MODE> ? (parts_of<MODE>(tile) - 1) & 1 : 0;
        const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + acc * 256;
#pragma unroll 1
        for (int c = half * (NT / 2); c < (half + 1) * (NT / 2); c += 16) {
            float v[16];
            tmem_ld16(tacc + c, v);
            const int side = c / kSide, at = c % kSide, owner = at / own, local = side * own + at % own;
            const uint32_t dst = cluster_map(buf, (uint32_t)(owner * 2 + rank)) +
                                 (uint32_t)(((pair * kSides * own + local) / 4 * 128 + r) * 16);
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (uint32_t)(i / 4 * 2048)),
                             "f"(v[i]), "f"(v[i + 1]), "f"(v[i + 2]), "f"(v[i + 3])
                             : "memory");
        }
    }
    __syncwarp();
    cluster_sync();
    if (warp < 2)
        return;
    const Product &p = a.p[tile.prod];
    const int64_t row = tile.m0 + rank * 128 + r;
    const int mine = own / 2;  // columns of this warp
    const int col = tile.nt * kCols<MODE, NT> + pair * own + half * mine;
    if (row >= p.M)
        return;
    const auto sum16 = [&](int local, float(&v)[16]) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = 0.0f;
        for (int s = 0; s < S; ++s) {
            const float4 *src = reinterpret_cast<const float4 *>(buf) + (s * kSides * own + local) / 4 * 128 + r;
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 f = src[i / 4 * 128];
                v[i] += f.x, v[i + 1] += f.y, v[i + 2] += f.z, v[i + 3] += f.w;
            }
        }
    };
    RowOf of = {};
    if (kIsLse<MODE> || kIsDlogits<MODE>)
        of = row_of<MODE>(a, row);
    float top = -INFINITY, exps = 0.0f, target_logit = 0.0f;
    bool has = false;
#pragma unroll 1
    for (int c = 0; c < mine && col + c < p.N; c += 16) {
        float v[16];
        sum16(half * mine + c, v);
        if constexpr (MODE == kGated) {
            float u[16];
            sum16(own + half * mine + c, u);
            epi_gated<TE>(a, row, col + c, v, u);
        } else if constexpr (kIsStore<MODE>) {
            epi_store<TE>(p, row, col + c, v);
        } else if constexpr (MODE == kGatedBwd) {
            epi_gated_bwd<TE>(a, row, col + c, v, factor);
        } else if constexpr (kIsLse<MODE>) {
            epi_lse(p.N, col + c, of.target, v, top, exps, target_logit, has);
        } else {
            epi_dlogits(col + c, of.target, of.lse, of.factor, v);
            TE *dst = static_cast<TE *>(p.d) + row * p.ld_d + col + c;  // (8 columns may go past N, into the padding)
#pragma unroll
            for (int i = 0; i < 16; i += 8)
                if (col + c + i < p.N)
                    store8(dst + i, v + i);
        }
    }
    if (kIsLse<MODE>) {
        a.stats[row * a.pairs + (tile.nt * S + pair) * 2 + half] = make_float2(top, exps);
        if (has)
            a.target_logit[row] = target_logit;
    }
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
    const int S = a.S;
    const int in_cluster = (int)cluster_ctarank();
    const int rank = in_cluster & 1, pair = in_cluster >> 1;
    const uint32_t lead = (uint32_t)(pair * 2);  // the pair's leader
    const uint16_t both = (uint16_t)(3u << (pair * 2));
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
    const int cluster = blockIdx.x / (2 * S), first = a.deal.tile(cluster, 0);
    {
        // the first tile's arithmetic before the wait: it brings the parameters it reads into the constant cache
        const Tile t = tile_of<MODE>(a, first, pair);
        const Product &p = a.p[t.prod];
        asm volatile("" ::"r"(t.kb1), "r"(t.m0), "r"(p.N), "r"(p.maj), "l"(p.M), "l"(p.d), "l"(p.add), "l"(a.status)
                     : "memory");
    }
    pdl_wait();
    pdl_trigger();

    float factor = 1.0f;  // of d gate | d up
    if (warp == 0) {
        if (lane == 0) {
            // both operands are read again by the pairs around (ms as above: evict-normal 1.740, evict-last 1.699; the
            // cross entropy's four products 2.807 and 2.726)
            const uint64_t keep = l2_policy_evict_last();
            int s = 0;
            uint32_t ph = 0;
            bool ok = true, any = false;
            for (int t = first, k = 0; ok && t < a.tiles; t = a.deal.tile(cluster, ++k)) {
                const Tile tile = tile_of<MODE>(a, t, pair);
                const Product &p = a.p[tile.prod];
                const int maj = kIsStore<MODE> ? p.maj : MODE == kGatedBwd ? 1 : 0;
                const int arow = tile.m0 + rank * 128;
                // gated: CTA 0 holds gate rows, CTA 1 the matching up rows
                const int brow = MODE == kGated ? rank * p.N + tile.nt * kHalf : tile.nt * NT + rank * kHalf;
                for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
                    if (!mbar_wait(&sm.empty[s], ph ^ 1, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = sm.stage[s], *sb = sm.stage[s] + kABytes;
                    const uint32_t bar = cluster_map(&sm.full[s], lead);
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
            for (int t = first, k = 0; ok && t < a.tiles; t = a.deal.tile(cluster, ++k)) {
                const Tile tile = tile_of<MODE>(a, t, pair);
                const int maj = kIsStore<MODE> ? a.p[tile.prod].maj : MODE == kGatedBwd ? 1 : 0;
                const uint32_t idesc = make_idesc(type, type, 256, NT) | (maj >= 1 ? 1u << 16 : 0u) |
                                       (maj == 2 ? 1u << 15 : 0u);
                const int part = kInParts<MODE> ? kPartOf<MODE> : tile.kb1 - tile.kb0;
                for (int k0 = tile.kb0; k0 < tile.kb1; k0 += part) {
                    if (!mbar_wait(&sm.tempty[acc], aph ^ 1, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + acc * 256;
                    const int k1 = min(k0 + part, tile.kb1);
                    for (int kb = k0; kb < k1; ++kb) {
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
                            mma_pair<0>(d, da, db, idesc, (kb > k0 || kk > 0) ? 1u : 0u);
                            da += ia, db += ib;  // (the start address is the descriptor's lowest field)
                        }
                        any = true;
                        mma_commit_pair(&sm.empty[s], both);
                        if (++s == kS) {
                            s = 0;
                            ph ^= 1;
                        }
                    }
                    if (!ok)
                        break;
                    mma_commit_pair(&sm.tfull[acc], both);
                    if (++acc == 2) {
                        acc = 0;
                        aph ^= 1;
                    }
                }
            }
            if (!ok && any) {
                mma_commit_pair(&sm.drain, (uint16_t)(1u << lead));
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
        if constexpr (MODE == kGatedBwd && kScaledGrad<TE>) {
            factor = gradient_factor(a.most, lane);
            if (blockIdx.x == 0 && warp == 2 && lane == 0)
                *a.back = 1.0f / factor;
        }
        for (int t = first, k = 0; t < a.tiles; t = a.deal.tile(cluster, ++k)) {
            const Tile tile = tile_of<MODE>(a, t, pair);
            const Product &p = a.p[tile.prod];
            const int64_t row = tile.m0 + rank * 128 + r;
            const bool live = row < p.M;
            constexpr int kMine = kCols<MODE, NT> / 2;              // columns of D of this warp
            const int c0 = tile.nt * kCols<MODE, NT> + half * kMine;  // the first of them
            // what the epilogue will read of memory: into L2 while the MMAs run
            if (MODE == kGatedBwd && S == 1 && live) {
                const TE *kept = static_cast<const TE *>(a.gu) + row * 2 * p.N + c0;
                for (int c = 0; c < kMine && c0 + c < p.N; c += 64) {
                    prefetch_l2(kept + c);
                    prefetch_l2(kept + p.N + c);
                }
            }
            if (kIsStore<MODE> && S == 1 && live && p.add) {
                const int es = p.d_f32 ? 4 : 2;
                const char *add = static_cast<const char *>(p.add) + (row * p.ld_add + c0) * es;
                for (int c = 0; c < kMine && c0 + c < p.N; c += 128 / es)
                    prefetch_l2(add + c * es);
            }
            RowOf of = {};
            if (kIsLse<MODE> || kIsDlogits<MODE>)
                of = row_of<MODE>(a, row);
            uint4 *buf = reinterpret_cast<uint4 *>(sm.rows[warp - 2]);
            const int64_t row0 = tile.m0 + rank * 128 + q * 32;  // the warp's rows
            const int rows = (int)max((int64_t)0, min((int64_t)32, p.M - row0));
            // the first columns of what is read, before the wait for the accumulator
            uint4 pre[8];
            const auto read = [&](int c) {
                if (rows == 0 || S > 1 || c >= kMine || c0 + c >= p.N)
                    return;
                if (kIsStore<MODE> && p.add) {
                    const int64_t at = row0 * p.ld_add + c0 + c;
                    const int cols = p.N - c0 - c;
                    if (p.d_f32)
                        Rows<float>::load(static_cast<const float *>(p.add) + at, p.ld_add, rows, cols, lane, pre);
                    else
                        Rows<TE>::load(static_cast<const TE *>(p.add) + at, p.ld_add, rows, cols, lane, pre);
                }
                if (MODE == kGatedBwd) {
                    const TE *kept = static_cast<const TE *>(a.gu) + row0 * 2 * p.N + c0 + c;
                    Rows<TE>::load(kept, 2 * (int64_t)p.N, rows, p.N - c0 - c, lane, pre);
                    Rows<TE>::load(kept + p.N, 2 * (int64_t)p.N, rows, p.N - c0 - c, lane, pre + 4);
                }
            };
            if (!kInParts<MODE>)
                read(0);
            // the CTA's rows of accumulator `acc`, this warp's half of the columns
            const auto wait = [&] {
                const bool done = __all_sync(0xffffffffu, mbar_wait(&sm.tfull[acc], aph, a.status, abort_flag));
                tc_fence_after();
                return done;
            };
            const auto at = [&] { return tmem_base + ((uint32_t)(q * 32) << 16) + acc * 256 + half * kMine; };
            const auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_remote(cluster_map(&sm.tempty[acc], lead));
                if (++acc == 2) {
                    acc = 0;
                    aph ^= 1;
                }
            };
            bool ok = true;
            if constexpr (kInParts<MODE>) {
                if (parts_of<MODE>(tile) > 1) {
                    // all parts but the last are added up here, then the last one, and the whole goes back to its place
                    float sums[kMine];
#pragma unroll
                    for (int c = 0; c < kMine; ++c)
                        sums[c] = 0.0f;
                    for (int i = parts_of<MODE>(tile); i > 1 && (ok = wait()); --i) {
#pragma unroll
                        for (int c = 0; c < kMine; c += 16) {
                            float f[16];
                            tmem_ld16(at() + c, f);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                sums[c + j] += f[j];
                        }
                        release();
                    }
                    if (!ok || !(ok = wait()))
                        break;
#pragma unroll
                    for (int c = 0; c < kMine; c += 16) {
                        float f[16];
                        tmem_ld16(at() + c, f);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            f[j] += sums[c + j];
                        tmem_st16(at() + c, f);
                    }
                } else {
                    ok = wait();
                }
                read(0);
            } else {
                ok = wait();
            }
            if (!ok)
                break;
            if (S > 1)
                break;  // the parts meet below
            const uint32_t tacc = at();
            float m = -INFINITY, e = 0.0f, own = 0.0f;
            bool has = false;
#pragma unroll 1
            for (int c = 0; c < kMine && c0 + c < p.N && rows > 0; c += 32) {
                const int col = c0 + c, cols = p.N - col;
                float v[32];
                tmem_ld32(tacc + c, v);
                if constexpr (kIsStore<MODE>) {
                    if (p.acc_in) {
                        uint4 w[8];
                        Rows<float>::load(p.acc_in + row0 * p.N + col, p.N, rows, cols, lane, w);
                        Rows<float>::to_row(buf, w, lane);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            add4(v + 4 * i, w[i]);
                    }
                    if (p.scale) {
                        const float sc = *p.scale;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] *= sc;
                    }
                    if (p.d_f32) {
                        if (p.add) {
                            Rows<float>::to_row(buf, pre, lane);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                add4(v + 4 * i, pre[i]);
                            read(c + 32);
                        }
                        uint4 w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                              __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
                        Rows<float>::store(buf, w, static_cast<float *>(p.d) + row0 * p.ld_d + col, p.ld_d, rows, cols,
                                           lane);
                    } else {
                        if (p.add) {
                            Rows<TE>::to_row(buf, pre, lane);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float f[8];
                                unpack8<TE>(pre[i], f);
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    v[8 * i + j] += f[j];
                            }
                            read(c + 32);
                        }
                        put_rows(buf, v, static_cast<TE *>(p.d) + row0 * p.ld_d + col, p.ld_d, rows, cols, lane);
                    }
                } else if constexpr (MODE == kGated) {
                    float u[32];
                    tmem_ld32(tacc + kHalf + c, u);
                    if (a.gu) {
                        TE *kept = static_cast<TE *>(a.gu) + row0 * 2 * p.N + col;
                        put_rows(buf, v, kept, 2 * (int64_t)p.N, rows, cols, lane);
                        put_rows(buf, u, kept + p.N, 2 * (int64_t)p.N, rows, cols, lane);
                    }
                    gate(a.act, v, u);
                    put_rows(buf, v, static_cast<TE *>(a.h) + row0 * p.N + col, p.N, rows, cols, lane);
                } else if constexpr (MODE == kGatedBwd) {
                    uint4 wg[4], wu[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        wg[i] = pre[i], wu[i] = pre[4 + i];
                    read(c + 32);
                    Rows<TE>::to_row(buf, wg, lane);
                    Rows<TE>::to_row(buf, wu, lane);
                    with_act(a.act, [&](auto kind) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            gated_grad8<TE, decltype(kind)::value>(v + 8 * i, factor, wg[i], wu[i]);
                    });
                    TE *out = static_cast<TE *>(a.dgu) + row0 * 2 * p.N + col;
                    Rows<TE>::store(buf, wg, out, 2 * (int64_t)p.N, rows, cols, lane);
                    Rows<TE>::store(buf, wu, out + p.N, 2 * (int64_t)p.N, rows, cols, lane);
                } else if constexpr (kIsLse<MODE>) {
                    epi_lse(p.N, col, of.target, v, m, e, own, has);
                } else {
                    epi_dlogits(col, of.target, of.lse, of.factor, v);
                    // (a last piece of 8 columns may go past N, into the rows' padding)
                    put_rows(buf, v, static_cast<TE *>(p.d) + row0 * p.ld_d + col, p.ld_d, rows, cols, lane);
                }
            }
            if (kIsLse<MODE> && live) {
                a.stats[row * a.pairs + tile.nt * 2 + half] = make_float2(m, e);
                if (has)
                    a.target_logit[row] = own;
            }
            release();
        }
    }

    if (S > 1) {
        // every MMA of the cluster has read its stages (the pair's accumulator is complete: what the epilogue warps
        // waited for)
        __syncwarp();
        tc_fence_before();
        cluster_sync();
        tc_fence_after();
        meet<MODE, TE, NT>(a, sm.stage[0], tmem_base, tile_of<MODE>(a, first, pair), rank, pair, warp, lane, factor);
    }
    // both CTAs stay until the pair's last MMA, copy and remote arrive are done
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc_pair(tmem_base, 512);
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

template <int MODE, class TE, int NT>
cudaLaunchConfig_t config_of(cudaLaunchAttribute (&attr)[2], int S, int64_t clusters, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * S * clusters));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes<NT>;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

// Clusters of S = 1, 2 or 4 pairs that can be resident at once, kept per device (one CTA an SM in every mode and at
// every width, so one kernel is asked for all of them).
template <class TE>
int max_clusters(int S)
{
    static std::atomic<int> cache[64][3];  // zero until first computed
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 0;
    std::atomic<int> &kept = cache[dev][S / 2];
    int n = kept.load(std::memory_order_relaxed);
    if (n == 0) {
        auto kern = gemm_kernel<kStore, TE, 256>;
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = config_of<kStore, TE, 256>(attr, S, 1, nullptr);
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<256>) !=
                cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0)
            return 0;
        kept.store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int MODE, class TE, int NT>
cudaError_t launch_nt(Args &a, int S, int clusters, cudaStream_t st)
{
    auto kern = gemm_kernel<MODE, TE, NT>;
    int64_t tiles = 0;
    for (int i = 0; i < a.n; ++i) {
        Product &p = a.p[i];
        const int64_t tm = (p.M + 255) / 256, tn = (p.N + kCols<MODE, NT> - 1) / kCols<MODE, NT>;
        if (!make_maps<MODE, NT>(p))
            return cudaErrorInvalidValue;
        p.tiles_m = (int)tm, p.tiles_n = (int)tn;
        p.first = (int)tiles;
        tiles += tm * tn;
        if (tiles > 1 << 30)
            return cudaErrorInvalidValue;
    }
    a.tiles = (int)tiles;
    a.S = S;
    int64_t busiest;
    a.deal = deal_of(a.p, a.n, kCols<MODE, NT>, S, S > 1 ? tiles : clusters, &busiest);
    a.pairs = a.p[0].tiles_n * S * 2;
    const cudaError_t err =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<NT>);
    if (err != cudaSuccess)
        return err;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        config_of<MODE, TE, NT>(attr, S, a.deal.P, st);
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// Tiles of one product, and what one costs: its blocks of K, or its epilogue where that takes longer (one tile's
// overlaps the next one's products).
struct Load {
    int64_t tiles, blocks;
};
inline Load load_of(const Product &p, int cols, int S)
{
    const int64_t KB = ((p.K + 63) / 64 + S - 1) / S, epilogue = cols > 128 ? 8 : 6;
    return {(p.M + 255) / 256 * ((p.N + cols - 1) / cols), KB > epilogue ? KB : epilogue};
}

// The deal of n products over at most `clusters` clusters, and the blocks of K that the busiest goes through.
inline Deal deal_of(const Product *p, int n, int cols, int S, int64_t clusters, int64_t *busiest)
{
    const Load first = load_of(p[0], cols, S);
    int64_t others = 0, blocks = 0;
    for (int i = 1; i < n; ++i) {
        const Load l = load_of(p[i], cols, S);
        others += l.tiles, blocks += l.tiles * l.blocks;
    }
    const int64_t P = first.tiles + others < clusters ? first.tiles + others : clusters;
    const int64_t q = first.tiles / P, r = first.tiles % P;
    int64_t E = 0;
    if (r > 0 && others > 0) {
        const int64_t same = first.blocks / load_of(p[1], cols, S).blocks, most = others / (P - r);
        E = same < most ? same : most;
    }
    const int64_t rest = others - E * (P - r), rounds = rest / P, more = rest % P;
    const int64_t each = others ? (blocks + others - 1) / others : 0;
    const int64_t with = r > 0 ? (q + 1) * first.blocks + (rounds + (more > P - r ? 1 : 0)) * each : 0;
    const int64_t without = q * first.blocks + (E + rounds + (more > 0 ? 1 : 0)) * each;
    *busiest = with > without ? with : without;
    return {(int)P, (int)first.tiles, (int)q, (int)r, (int)E};
}

constexpr int kMostSplit = 38;  // tiles that may be split: clusters of four CTAs that 152 SMs hold

struct Plan {
    int64_t cost;  // in 10 ns
    int S;
    bool wide;
};

// How to launch n products together.  The time is that of the busiest cluster's blocks of K, of an epilogue that
// nothing hides after the last of them, of the meeting of a split tile's pairs, and of a launch.  (Measured, us of the
// whole call, whole tiles / half-wide / whole in 2 / half-wide in 2 / whole in 4 parts of K: 1001 x 1416 x 1000 as a
// block's second product 24.9 / 22.6 / 23.6 / 22.6 / 33.2, its clusters then starting in turns; 777 x 8192 x 1000
// 168 / 157 / 145 / 136 / 158.  Gradients of 515 x 520 x 1000 in one launch 43, in three 49.)
template <int MODE>
Plan plan(const Product *p, int n, const int *clusters)
{
    Plan best = {INT64_MAX, 1, true};
    int least = p[0].K;
    for (int i = 1; i < n; ++i)
        least = p[i].K < least ? p[i].K : least;
    for (int w = kIsLse<MODE> ? 1 : 0; w < 2; ++w) {  // (a logit tile leaves two pairs a row, whatever its width)
        const int cols = (w ? 256 : 128) / (MODE == kGated ? 2 : 1);
        // (a warp of an owner finishes 16 columns at least, of each side)
        const int most = MODE == kGated && !w ? 2 : 4;
        for (int s = 1; s <= most && (s == 1 || (clusters[s] > 0 && (least + 63) / 64 / s >= 2)); s *= 2) {
            // (clusters that share a tile take one each: with more tiles than clusters they would start in turns)
            int64_t tiles = 0;
            for (int i = 0; i < n; ++i)
                tiles += (p[i].M + 255) / 256 * ((p[i].N + cols - 1) / cols);
            if (s > 1 && (tiles > clusters[s] || tiles > kMostSplit))
                continue;
            int64_t busiest;
            deal_of(p, n, cols, s, clusters[s], &busiest);
            const int64_t c = busiest * (w ? 29 : 22) + (w ? 250 : 150) + (s > 1 ? 230 : 0) + 450;
            if (c < best.cost)
                best = {c, s, w != 0};
        }
    }
    return best;
}

// Whether a product to memory needs its sum in parts of K: weight gradients in fp32 of more rows than one part, and
// what is rounded to 16 bits where the truncation comes near that (1.7e-4 of positive terms at K = 32768; half a step
// of fp16 is 4.9e-4 at most).
inline bool wants_parts(const Product &p) { return p.K > (p.maj == 2 && p.d_f32 ? 64 * kPartRows : 32768); }

// The products of `a` (p[0] .. p[n - 1]), longest K first: in one launch, the first apart from the others, or each in
// its own, whichever is fastest (a product of few tiles and a long K wants it split, one of many tiles does not).
template <int MODE, class TE>
cudaError_t launch(Args &a, cudaStream_t st)
{
    int clusters[5] = {};
    for (int s = 1; s <= 4; s *= 2)
        if ((clusters[s] = max_clusters<TE>(s)) <= 0 && s == 1)
            return cudaErrorInvalidConfiguration;
    for (int i = 1; i < a.n; ++i)
        for (int j = i; j > 0 && a.p[j].K > a.p[j - 1].K; --j) {
            const Product t = a.p[j];
            a.p[j] = a.p[j - 1], a.p[j - 1] = t;
        }
    // products [from, from + n) of a in one launch
    const auto go = [&](int from, int n, const Plan &how) {
        Args part = a;
        for (int i = 0; from && i < n; ++i)
            part.p[i] = a.p[from + i];
        part.n = n;
        if constexpr (!kIsLse<MODE>) {
            if (!how.wide)
                return launch_nt<MODE, TE, 128>(part, how.S, clusters[how.S], st);
        }
        const cudaError_t err = launch_nt<MODE, TE, 256>(part, how.S, clusters[how.S], st);
        a.pairs = part.pairs;
        return err;
    };
    const Plan all = plan<MODE>(a.p, a.n, clusters);
    if (a.n == 1)
        return go(0, 1, all);
    const Plan first = plan<MODE>(a.p, 1, clusters), others = plan<MODE>(a.p + 1, a.n - 1, clusters);
    Plan each[kProducts] = {first, others, others};
    int64_t apart = first.cost;
    for (int i = 1; i < a.n; ++i) {
        if (a.n > 2)
            each[i] = plan<MODE>(a.p + i, 1, clusters);
        apart += each[i].cost;
    }
    if (all.cost <= apart && all.cost <= first.cost + others.cost)
        return go(0, a.n, all);
    cudaError_t err = go(0, 1, first);
    if (first.cost + others.cost <= apart)
        return err != cudaSuccess ? err : go(1, a.n - 1, others);
    for (int i = 1; i < a.n && err == cudaSuccess; ++i)
        err = go(i, 1, each[i]);
    return err;
}

// The products of `a` to memory.
template <class TE>
cudaError_t launch_store(Args &a, cudaStream_t st)
{
    bool parts = false;
    for (int i = 0; i < a.n; ++i)
        parts = parts || wants_parts(a.p[i]);
    return parts ? launch<kStoreLong, TE>(a, st) : launch<kStore, TE>(a, st);
}

}  // namespace dense
}  // namespace moe
