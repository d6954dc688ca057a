// The norms before and after a block, fused with the block's gate and residual scale, and their
// gradients.  For a block output h, the residual stream and RMS norms with weights w_post, w_pre:
//   r_h = 1 / sqrt(mean(h^2) + eps)      n = h r_h (w_post + offset)      (n = h without w_post)
//   y   = residual + scale * gate * n                                     the next residual stream
//   r_y = 1 / sqrt(mean(y^2) + eps)      z = y r_y (w_pre + offset)       the next block's input
// gate: none (1), one value per column, per row, or per element.  Backward, from dy (gradient of
// the residual stream, may be absent) and dz, with yh = y r_y, hh = h r_h, u = dz (w_pre + offset):
//   D    = dy + r_y (u - yh mean(u yh))                                   = d residual
//   dw_pre = sum_rows dz yh          dn = scale * gate * D
//   v = dn (w_post + offset)         dh = r_h (v - hh mean(v hh))
//   dw_post = sum_rows dn hh         dgate = scale * n * D, summed over what it was broadcast over
//
// From HBM the forward reads h and the residual and writes y and z once each, the backward reads h, the
// residual, dy and dz and writes d residual and dh once each.  A row needs its own two sums before its
// results.  The forward keeps the row in registers between its passes.  The backward reads it again, h in
// three passes, the residual and dz in two: from shared memory where rows are copied ahead (below), else
// from global memory.  A gate per element is read in every pass that uses it.  All sums are fp32.  z is
// computed from y before y's rounding, and the backward forms the same unrounded y again from h and the
// residual: reading the rounded y instead would cost the same bytes and leave the sums over the rows off
// by bf16's 2^-9.  The column sums (dw, per-column dgate) are kept in registers over the rows that a block walks and written as one partial row per block;
// a second launch adds the partial rows in order, so the gradients are bitwise reproducible.
//
// A row's two sums are a chain of barriers, so a block that loads its next row only after this one
// leaves HBM idle most of the time.  The blocks are persistent and copy the next rows ahead into
// shared memory (cp.async; each thread copies exactly the pieces that it will read itself, so no
// barrier guards the ring).  8192 rows of 4096 bf16 with a gate per column: forward 44 us (6.0 TB/s; 103 us
// without the ring), forward and backward 153 (250), 8192 rows of 2048 86 (123), of 4096 fp32 214 (384).
// 2048 rows of 16384 have the ring in the forward only (64-68 us, 73 without): two rows of the backward's four
// arrays are more than an SM's shared memory, and forward and backward take 303 us.  A third row in the
// ring was no faster (155 and 48 us again, fp32 220).  Rows that are no whole number of 16-byte pieces go by
// single elements and without the ring (8192 rows of 401, forward: 17.8 us; of 1001 46.5, with the backward
// 170); the widest of those (over 4096 elements) no longer fit a thread's registers, 8192 rows of 4097 taking
// 300 us forward and 1760 with the backward.
#include "moe_internal.h"
#include "rows.cuh"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxH = 16384;
constexpr int kSlots = 2;  // rows of a block's ring in shared memory

struct NormArgs {
    const void *h, *residual, *gate, *w_post, *w_pre;
    int gate_kind;
    int64_t T;
    int H;
    float scale, offset, eps;
    void *y, *z;
    float *r_h, *r_y;
    // backward
    const void *dy, *dz;
    void *dres, *dh, *dgate;
    float *part;  // [blocks][2][H]: the blocks' column sums
};

// The rows that a block walks (blockIdx.x, + gridDim.x, ...), each of N arrays, a thread's pieces of
// them.  RING: copied ahead into shared memory; otherwise loaded when wanted.
template <typename V, int NV, int N, bool RING>
struct RowRing {
    const V *src[N];  // null: not read
    V *ring;
    int64_t T;
    int units, slot;

    __device__ __forceinline__ void init(int64_t rows, int nunits)
    {
        extern __shared__ __align__(16) uint8_t smem[];
        ring = reinterpret_cast<V *>(smem);
        T = rows, units = nunits, slot = 0;
        if (RING)
            for (int i = 0; i < kSlots; ++i)
                fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
    }
    __device__ __forceinline__ void fetch(int64_t t, int to)
    {
        if (t < T)
#pragma unroll
            for (int a = 0; a < N; ++a)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int u = threadIdx.x + i * blockDim.x;
                    if (src[a] && u < units)
                        cp_async_16_zfill(ring + (to * N + a) * units + u, src[a] + t * units + u, true);
                }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // Wait for this thread's pieces of the block's next row.
    __device__ __forceinline__ void wait()
    {
        if (RING) {
            static_assert(kSlots == 2, "every copy but the kSlots - 1 newer ones");
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        }
    }
    // Piece i of array a of that row (row t).
    __device__ __forceinline__ V at(int64_t t, int a, int i) const
    {
        const int u = threadIdx.x + i * blockDim.x;
        return RING ? ring[(slot * N + a) * units + u] : src[a][t * units + u];
    }
    // Row t's pieces have been read: its place takes the row kSlots further on.
    __device__ __forceinline__ void next(int64_t t)
    {
        if (RING) {
            fetch(t + (int64_t)kSlots * gridDim.x, slot);
            slot ^= 1;
        }
    }
};

// Sum of v over the block's threads (every thread gets it); `buf` alternates between calls.
__device__ __forceinline__ float block_sum(float v, float (*buf)[kMaxWarps], int which)
{
    v = warp_sum(v);
    const int nw = blockDim.x >> 5;
    if (nw == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        buf[which][threadIdx.x >> 5] = v;
    __syncthreads();
    float s = (threadIdx.x & 31) < nw ? buf[which][threadIdx.x & 31] : 0.0f;
    return warp_sum(s);
}

// weight + offset of a piece's elements, 1 without a weight
template <typename T, int VEC>
__device__ __forceinline__ void weight_piece(const void *w, float offset, int u, float (&f)[VEC])
{
    if (w) {
        unpack<T, VEC>(static_cast<const Piece<T, VEC> *>(w)[u], f);
#pragma unroll
        for (int c = 0; c < VEC; ++c)
            f[c] += offset;
    } else {
#pragma unroll
        for (int c = 0; c < VEC; ++c)
            f[c] = 1.0f;
    }
}

// What multiplies h * rstd(h) (and a row's or an element's gate) in y: scale * (w_post + offset) and, with
// a gate per column, that gate.  The same for every row: a thread keeps its columns' in registers.
template <typename T, int VEC>
__device__ __forceinline__ void branch_factor(const NormArgs &a, int u, float (&k)[VEC])
{
    weight_piece<T, VEC>(a.w_post, a.offset, u, k);
    float g[VEC];
    if (a.gate_kind == MOE_GATE_CHANNEL)
        unpack<T, VEC>(static_cast<const Piece<T, VEC> *>(a.gate)[u], g);
#pragma unroll
    for (int c = 0; c < VEC; ++c)
        k[c] *= a.gate_kind == MOE_GATE_CHANNEL ? a.scale * g[c] : a.scale;
}

// FULL: a gate per element.
template <typename T, int VEC, int NV, bool RING, bool FULL>
__global__ void __launch_bounds__(kMaxThreads, RING && NV == 1 ? 2 : 1) norm_kernel(const NormArgs a)
{
    using V = Piece<T, VEC>;
    __shared__ float s_buf[2][kMaxWarps];
    const int units = a.H / VEC;
    const float inv_h = 1.0f / (float)a.H;
    RowRing<V, NV, 2, RING> in = {{static_cast<const V *>(a.h), static_cast<const V *>(a.residual)}};
    pdl_wait();
    pdl_trigger();
    in.init(a.T, units);
    float k[NV][VEC], wi[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = threadIdx.x + i * blockDim.x;
        if (u < units) {
            branch_factor<T, VEC>(a, u, k[i]);
            weight_piece<T, VEC>(a.w_pre, a.offset, u, wi[i]);
        }
    }
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        in.wait();
        float f = a.gate_kind == MOE_GATE_TOKEN ? row_to_f(static_cast<const T *>(a.gate)[t]) : 1.0f;
        V h[NV], r[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (threadIdx.x + i * blockDim.x < units) {
                h[i] = in.at(t, 0, i);
                r[i] = in.at(t, 1, i);
            }
        float r_h = 1.0f;
        if (a.w_post) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (threadIdx.x + i * blockDim.x < units) {
                    float x[VEC];
                    unpack<T, VEC>(h[i], x);
#pragma unroll
                    for (int c = 0; c < VEC; ++c)
                        sum = fmaf(x[c], x[c], sum);
                }
            r_h = rsqrtf(fmaf(block_sum(sum, s_buf, 0), inv_h, a.eps));
        }
        in.next(t);
        f *= r_h;
        float y[NV][VEC];
        float ysum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u >= units)
                continue;
            float x[VEC], res[VEC], g[VEC];
            unpack<T, VEC>(h[i], x);
            unpack<T, VEC>(r[i], res);
            if (FULL)
                unpack<T, VEC>(static_cast<const V *>(a.gate)[t * units + u], g);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                y[i][c] = fmaf(k[i][c], FULL ? x[c] * f * g[c] : x[c] * f, res[c]);
                ysum = fmaf(y[i][c], y[i][c], ysum);
            }
            static_cast<V *>(a.y)[t * units + u] = pack<T, VEC>(y[i]);
        }
        if (threadIdx.x == 0 && a.r_h)
            a.r_h[t] = r_h;
        if (a.w_pre) {
            const float r_y = rsqrtf(fmaf(block_sum(ysum, s_buf, 1), inv_h, a.eps));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int u = threadIdx.x + i * blockDim.x;
                if (u >= units)
                    continue;
#pragma unroll
                for (int c = 0; c < VEC; ++c)
                    y[i][c] *= r_y * wi[i][c];
                static_cast<V *>(a.z)[t * units + u] = pack<T, VEC>(y[i]);
            }
            if (threadIdx.x == 0 && a.r_y)
                a.r_y[t] = r_y;
        }
        // a row uses both halves of s_buf once; the half written first in the next row was last
        // read before this row's second sum, except when only one norm is on
        if (!a.w_post || !a.w_pre)
            __syncthreads();
    }
}

// With hh = h r_h and, per row or element, hg = gate * hh (a gate per column is part of k):
//   y = residual + k hg       D = dy + r_y dz wi - y r_y^2 mean(dz wi y r_y)
//   t = k D    (v = gate t)   mean of v hh, and a row's dgate, from the sum of t hh
//   column sums  c_post += D hg, c_pre += dz y r_y
// dw_post and a column's dgate are c_post times what is left of scale, gate and weight.
template <typename T, int VEC, int NV, bool RING, bool FULL>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const NormArgs a)
{
    using V = Piece<T, VEC>;
    __shared__ float s_buf[2][kMaxWarps];
    const int units = a.H / VEC;
    const float inv_h = 1.0f / (float)a.H;
    RowRing<V, NV, 4, RING> in = {{static_cast<const V *>(a.h), static_cast<const V *>(a.w_pre ? a.residual : nullptr),
                                   static_cast<const V *>(a.dy), static_cast<const V *>(a.dz)}};
    pdl_wait();
    pdl_trigger();
    in.init(a.T, units);
    float c_post[NV][VEC], c_pre[NV][VEC], k[NV][VEC], wi[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = threadIdx.x + i * blockDim.x;
        if (u < units) {
            branch_factor<T, VEC>(a, u, k[i]);
            weight_piece<T, VEC>(a.w_pre, a.offset, u, wi[i]);
        }
#pragma unroll
        for (int c = 0; c < VEC; ++c)
            c_post[i][c] = c_pre[i][c] = 0.0f;
    }
    // the next row's statistics and gate, fetched a row ahead
    float next_rh = 1.0f, next_ry = 0.0f, next_gate = 1.0f;
    auto fetch_row = [&](int64_t t) {
        if (t >= a.T)
            return;
        if (a.w_post)
            next_rh = a.r_h[t];
        if (a.w_pre)
            next_ry = a.r_y[t];
        if (a.gate_kind == MOE_GATE_TOKEN)
            next_gate = row_to_f(static_cast<const T *>(a.gate)[t]);
    };
    fetch_row(blockIdx.x);
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * units;
        in.wait();
        const float r_h = next_rh, r_y = next_ry, gate = next_gate;
        fetch_row(t + gridDim.x);
        // (y is formed in both passes: kept in registers next to the column sums it would spill)
        float m1 = 0.0f;
        if (a.w_pre) {
            const float f = r_h * gate;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int u = threadIdx.x + i * blockDim.x;
                if (u >= units)
                    continue;
                float h[VEC], r[VEC], dz[VEC], g[VEC];
                unpack<T, VEC>(in.at(t, 0, i), h);
                unpack<T, VEC>(in.at(t, 1, i), r);
                unpack<T, VEC>(in.at(t, 3, i), dz);
                if (FULL)
                    unpack<T, VEC>(static_cast<const V *>(a.gate)[row + u], g);
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    const float p = dz[c] * fmaf(k[i][c], FULL ? h[c] * f * g[c] : h[c] * f, r[c]);
                    c_pre[i][c] = fmaf(p, r_y, c_pre[i][c]);
                    sum = fmaf(p, wi[i][c], sum);
                }
            }
            m1 = block_sum(sum, s_buf, 0) * inv_h * r_y * r_y * r_y;
        }
        float v[NV][VEC];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u >= units)
                continue;
            float hh[VEC], hg[VEC], D[VEC], g[VEC];
            unpack<T, VEC>(in.at(t, 0, i), hh);
            if (FULL)
                unpack<T, VEC>(static_cast<const V *>(a.gate)[row + u], g);
            unpack<T, VEC>(a.dy ? in.at(t, 2, i) : piece_zero<T, VEC>(), D);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                hh[c] *= r_h;
                hg[c] = hh[c] * (FULL ? g[c] : gate);
            }
            if (a.w_pre) {
                float r[VEC], dz[VEC];
                unpack<T, VEC>(in.at(t, 1, i), r);
                unpack<T, VEC>(in.at(t, 3, i), dz);
#pragma unroll
                for (int c = 0; c < VEC; ++c)
                    D[c] = fmaf(r_y * dz[c], wi[i][c], fmaf(-fmaf(k[i][c], hg[c], r[c]), m1, D[c]));
            }
            static_cast<V *>(a.dres)[row + u] = pack<T, VEC>(D);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                c_post[i][c] = fmaf(D[c], hg[c], c_post[i][c]);
                v[i][c] = k[i][c] * D[c];
                D[c] = v[i][c] * hh[c];
                if (FULL) {
                    sum = fmaf(D[c], g[c], sum);
                    v[i][c] *= g[c];
                } else {
                    sum += D[c];
                }
            }
            if (FULL)
                static_cast<V *>(a.dgate)[row + u] = pack<T, VEC>(D);
        }
        float m2 = 0.0f;
        if (a.w_post || a.gate_kind == MOE_GATE_TOKEN) {
            sum = block_sum(sum, s_buf, 1);
            if (a.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0)
                static_cast<float *>(a.dgate)[t] = sum;
            if (a.w_post)
                m2 = sum * inv_h * gate * r_h * r_h;
        }
        const float f = r_h * gate;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u >= units)
                continue;
            float h[VEC];
            unpack<T, VEC>(in.at(t, 0, i), h);
#pragma unroll
            for (int c = 0; c < VEC; ++c)
                h[c] = fmaf(v[i][c], f, -h[c] * m2);
            static_cast<V *>(a.dh)[row + u] = pack<T, VEC>(h);
        }
        in.next(t);
        __syncthreads();  // the row's shared sums have been read
    }
    float *p = a.part + (int64_t)blockIdx.x * 2 * a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = threadIdx.x + i * blockDim.x;
        if (u >= units)
            continue;
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            p[u * VEC + c] = c_post[i][c];
            p[a.H + u * VEC + c] = c_pre[i][c];
        }
    }
}

// The blocks' partial rows added up: 32 strided sums of a column (few loads after one another: with 8
// it took 10.7 us for 304 partial rows of 4096), then those in order.
template <typename T>
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *__restrict__ part, int nblocks, const NormArgs a,
                                                         float *dw_post, float *dw_pre, float *dgate)
{
    __shared__ float s[32][33];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float acc = 0.0f;
    if (c < a.H)
#pragma unroll 10
        for (int b = w; b < nblocks; b += 32)
            acc += part[((int64_t)b * 2 + blockIdx.y) * a.H + c];
    s[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < a.H) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            sum += s[i][lane];
        if (blockIdx.y == 1) {
            if (dw_pre)
                dw_pre[c] = sum;
        } else {
            const bool ch = a.gate_kind == MOE_GATE_CHANNEL;
            sum *= a.scale;
            if (dw_post)
                dw_post[c] = ch ? row_to_f(static_cast<const T *>(a.gate)[c]) * sum : sum;
            if (ch)
                dgate[c] = (a.w_post ? row_to_f(static_cast<const T *>(a.w_post)[c]) + a.offset : 1.0f) * sum;
        }
    }
}

int row_size(int row_type)
{
    return row_type == MOE_ROW_FP32 ? 4 : row_type == MOE_ROW_BF16 || row_type == MOE_ROW_FP16 ? 2 : 0;
}

int to_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Blocks of the backward, one partial row each: as many as an SM's registers hold of rows this wide
// (at most eight an SM: the partial rows stay below 10 MB), with four rows each where that leaves
// every SM a block.
int bwd_blocks(int64_t T, int H)
{
    const int64_t n = (int64_t)152 * 8192 / H;
    const int64_t most = n < 152 ? 152 : n > 1216 ? 1216 : n;
    const int64_t some = T < 152 ? T : T / 4 < 152 ? 152 : T / 4;
    return (int)(some < most ? some : most);
}

constexpr int kRingBytes = 224 * 1024;  // shared memory of an SM for the rings of its blocks

template <typename T, int VEC, int NV, bool RING>
cudaError_t run_ring(NormArgs a, bool bwd, int threads, int per_sm, cudaStream_t st)
{
    const bool full = a.gate_kind == MOE_GATE_FULL;
    auto kern = bwd ? (full ? norm_bwd_kernel<T, VEC, NV, RING, true> : norm_bwd_kernel<T, VEC, NV, RING, false>)
                    : (full ? norm_kernel<T, VEC, NV, RING, true> : norm_kernel<T, VEC, NV, RING, false>);
    size_t smem = 0;
    if (RING) {
        smem = (size_t)kSlots * (bwd ? 4 : 2) * a.H * sizeof(T);
        const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (err != cudaSuccess)
            return err;
    }
    const int64_t most = bwd ? bwd_blocks(a.T, a.H) : (int64_t)152 * per_sm;
    return launch_kernel(true, kern, dim3((unsigned)(a.T < most ? a.T : most)), dim3(threads), smem, st, a);
}

template <typename T, int VEC, int NV>
cudaError_t run(NormArgs a, bool bwd, cudaStream_t st)
{
    const int units = a.H / VEC;
    const int threads = ((units + NV - 1) / NV + 31) / 32 * 32;
    if (threads > kMaxThreads)
        return cudaErrorInvalidValue;
    // Copied ahead wherever the rows are whole 16-byte pieces and two of them fit.
    int per_sm = (bwd || NV > 1 ? 512 : 1024) / threads;  // (by registers: up to 128 and 64 a thread)
    const int64_t slot = (int64_t)(bwd ? 4 : 2) * a.H * sizeof(T);
    while (per_sm > 1 && per_sm * kSlots * slot > kRingBytes)
        --per_sm;
    if (VEC * sizeof(T) == 16) {
        if (kSlots * slot <= kRingBytes)
            return run_ring<T, VEC, NV, VEC * sizeof(T) == 16>(a, bwd, threads, per_sm, st);
    }
    return run_ring<T, VEC, NV, false>(a, bwd, threads, 16, st);
}

// Pieces a thread holds.  Up to 256 threads have one each: a row of 4096 bf16 elements is as fast in 256
// threads as in 512 (forward 48.1 / 48.5 us for 8192 rows, backward 103 / 105), and single elements are
// faster (8192 rows of 401: 17.8 us, 23.9 with 512 threads).
template <typename T, int VEC>
cudaError_t run_nv(const NormArgs &a, bool bwd, cudaStream_t st)
{
    const int units = a.H / VEC;
    if (units <= 256)
        return run<T, VEC, 1>(a, bwd, st);
    if (units <= (VEC == 1 ? 512 : 2 * kMaxThreads))
        return run<T, VEC, 2>(a, bwd, st);
    if constexpr (VEC * 4 * kMaxThreads >= kMaxH) {
        return run<T, VEC, 4>(a, bwd, st);
    } else {
        if (units <= 4 * kMaxThreads)
            return run<T, VEC, 4>(a, bwd, st);
        if constexpr (VEC * 8 * kMaxThreads >= kMaxH) {
            return run<T, VEC, 8>(a, bwd, st);
        } else {
            if (units <= 8 * kMaxThreads)
                return run<T, VEC, 8>(a, bwd, st);
            return run<T, VEC, 32>(a, bwd, st);
        }
    }
}

template <typename T, int VEC>
cudaError_t run_wide(const NormArgs &a, bool bwd, bool wide, cudaStream_t st)
{
    return wide ? run_nv<T, VEC>(a, bwd, st) : run_nv<T, 1>(a, bwd, st);
}

cudaError_t run_type(int row_type, const NormArgs &a, bool bwd, bool wide, cudaStream_t st)
{
    switch (row_type) {
    case MOE_ROW_BF16: return run_wide<__nv_bfloat16, 8>(a, bwd, wide, st);
    case MOE_ROW_FP16: return run_wide<__half, 8>(a, bwd, wide, st);
    default: return run_wide<float, 4>(a, bwd, wide, st);
    }
}

int check_norm(int row_type, int64_t T, int H, int gate_kind, const void *gate)
{
    if (row_size(row_type) == 0 || T < 0 || H <= 0 || gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL ||
        (gate_kind != MOE_GATE_NONE) != (gate != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (H > kMaxH || T > INT32_MAX)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int moe_block_norm(int row_type, const void *h, const void *residual, const void *gate, int gate_kind,
                   const void *w_post, const void *w_pre, int64_t T, int H, float scale, float weight_offset,
                   float eps, void *y, void *z, float *rstd_h, float *rstd_y, void *stream)
{
    const int rc = check_norm(row_type, T, H, gate_kind, gate);
    if (rc != MOE_OK)
        return rc;
    const int es = row_size(row_type);
    if (!h || !residual || !y || (w_pre != nullptr) != (z != nullptr))
        return MOE_ERR_INVALID_ARG;
    const uintptr_t rows = reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(residual) |
                           reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(z) |
                           reinterpret_cast<uintptr_t>(w_post) | reinterpret_cast<uintptr_t>(w_pre) |
                           (gate_kind == MOE_GATE_TOKEN ? 0 : reinterpret_cast<uintptr_t>(gate));
    if ((rows | reinterpret_cast<uintptr_t>(gate)) & (es - 1))
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    NormArgs a = {};
    a.h = h, a.residual = residual, a.gate = gate, a.w_post = w_post, a.w_pre = w_pre, a.gate_kind = gate_kind;
    a.T = T, a.H = H, a.scale = scale, a.offset = weight_offset, a.eps = eps, a.y = y, a.z = z;
    a.r_h = rstd_h, a.r_y = rstd_y;
    const bool wide = ((rows | (uintptr_t)((int64_t)H * es)) & 15) == 0;
    return to_status(run_type(row_type, a, false, wide, static_cast<cudaStream_t>(stream)));
}

size_t moe_block_norm_workspace_size(int64_t T, int H)
{
    if (T < 0 || H <= 0 || H > kMaxH)
        return 0;
    return (size_t)(T > 0 ? bwd_blocks(T, H) : 1) * 2 * H * sizeof(float);
}

int moe_block_norm_backward(int row_type, const void *h, const void *residual, const void *gate, int gate_kind,
                            const void *w_post, const void *w_pre, const float *rstd_h, const float *rstd_y,
                            const void *dy, const void *dz, int64_t T, int H, float scale, float weight_offset,
                            void *d_residual, void *dh, void *dgate, float *dw_post, float *dw_pre, void *ws,
                            size_t ws_bytes, void *stream)
{
    const int rc = check_norm(row_type, T, H, gate_kind, gate);
    if (rc != MOE_OK)
        return rc;
    const int es = row_size(row_type);
    if (!h || !d_residual || !dh || !ws || (w_post && (!rstd_h || !dw_post)) ||
        (w_pre && (!rstd_y || !dw_pre || !dz || !residual)) || (!w_pre && (dz || !dy)) ||
        (gate_kind != MOE_GATE_NONE) != (dgate != nullptr))
        return MOE_ERR_INVALID_ARG;
    const bool row_gate = gate_kind == MOE_GATE_TOKEN;
    const uintptr_t rows = reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(residual) |
                           reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(dz) |
                           reinterpret_cast<uintptr_t>(d_residual) | reinterpret_cast<uintptr_t>(dh) |
                           reinterpret_cast<uintptr_t>(w_post) | reinterpret_cast<uintptr_t>(w_pre) |
                           (row_gate ? 0 : reinterpret_cast<uintptr_t>(gate)) |
                           (gate_kind == MOE_GATE_FULL ? reinterpret_cast<uintptr_t>(dgate) : 0);
    if (((rows | reinterpret_cast<uintptr_t>(gate)) & (es - 1)) ||
        ((reinterpret_cast<uintptr_t>(ws) | reinterpret_cast<uintptr_t>(dw_post) |
          reinterpret_cast<uintptr_t>(dw_pre) | (gate_kind == MOE_GATE_FULL ? 0 : reinterpret_cast<uintptr_t>(dgate))) &
         3))
        return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe_block_norm_workspace_size(T, H))
        return MOE_ERR_WORKSPACE;
    const auto st = static_cast<cudaStream_t>(stream);
    NormArgs a = {};
    a.h = h, a.residual = residual, a.gate = gate, a.w_post = w_post, a.w_pre = w_pre;
    a.gate_kind = gate_kind, a.T = T, a.H = H, a.scale = scale, a.offset = weight_offset;
    a.r_h = const_cast<float *>(rstd_h), a.r_y = const_cast<float *>(rstd_y), a.dy = dy, a.dz = dz;
    a.dres = d_residual, a.dh = dh, a.dgate = dgate, a.part = static_cast<float *>(ws);
    const bool wide = ((rows | (uintptr_t)((int64_t)H * es)) & 15) == 0;
    cudaError_t err = cudaSuccess;
    const int nblocks = bwd_blocks(T, H);
    if (T > 0)
        err = run_type(row_type, a, true, wide, st);
    if (err != cudaSuccess)
        return MOE_ERR_CUDA;
    // (T = 0: no partial rows, every sum is zero)
    auto reduce = row_type == MOE_ROW_BF16   ? norm_reduce_kernel<__nv_bfloat16>
                  : row_type == MOE_ROW_FP16 ? norm_reduce_kernel<__half>
                                             : norm_reduce_kernel<float>;
    return to_status(launch_kernel(true, reduce, dim3((H + 31) / 32, 2), dim3(1024), 0, st,
                                   static_cast<const float *>(a.part), nblocks, a, dw_post, dw_pre,
                                   gate_kind == MOE_GATE_CHANNEL ? static_cast<float *>(dgate) : nullptr));
}

}  // extern "C"
