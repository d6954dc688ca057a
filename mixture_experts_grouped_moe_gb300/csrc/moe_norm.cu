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
// Bound by HBM: the forward reads h and the residual and writes y and z once each, the backward
// reads h, the residual, dy and dz and writes d residual and dh once each.  A row stays in one block's
// registers between its passes (a row needs its own two sums before its results), so nothing is
// read twice.  All sums are fp32.  z is computed from y before y's rounding, and the backward forms
// the same unrounded y again from h and the residual: reading the rounded y instead would cost the
// same bytes and leave the sums over the rows off by bf16's 2^-9.  The column sums (dw, per-column
// dgate) are
// kept in registers over the rows that a block walks and written as one partial row per block;
// a second launch adds the partial rows in order, so the gradients are bitwise reproducible.
#include "moe_internal.h"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxH = 16384;

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
    float *part;  // [blocks][3][H]: dw_post, dw_pre, dgate (per column)
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

// Gate of element c of the piece (row t, piece u); gate pieces are loaded once per row or column.
template <typename T, int VEC>
__device__ __forceinline__ float gate_of(const NormArgs &a, float row_gate, const Piece<T, VEC> &g, int c)
{
    return a.gate_kind == MOE_GATE_NONE || a.gate_kind == MOE_GATE_TOKEN ? row_gate : row_to_f(g.e[c]);
}

template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> gate_piece(const NormArgs &a, int64_t t, int units, int u)
{
    using V = Piece<T, VEC>;
    if (a.gate_kind == MOE_GATE_CHANNEL)
        return static_cast<const V *>(a.gate)[u];
    if (a.gate_kind == MOE_GATE_FULL)
        return static_cast<const V *>(a.gate)[t * units + u];
    return V{};
}

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormArgs a)
{
    using V = Piece<T, VEC>;
    __shared__ float s_buf[2][kMaxWarps];
    const int units = a.H / VEC;
    const float inv_h = 1.0f / (float)a.H;
    pdl_wait();
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const V *hr = static_cast<const V *>(a.h) + t * units;
        const V *rr = static_cast<const V *>(a.residual) + t * units;
        V h[NV], r[NV];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u < units) {
                h[i] = hr[u];
                r[i] = rr[u];
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (threadIdx.x + i * blockDim.x < units)
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    const float f = row_to_f(h[i].e[c]);
                    sum = fmaf(f, f, sum);
                }
        const float row_gate = a.gate_kind == MOE_GATE_TOKEN ? row_to_f(static_cast<const T *>(a.gate)[t]) : 1.0f;
        float r_h = 1.0f;
        if (a.w_post)
            r_h = rsqrtf(fmaf(block_sum(sum, s_buf, 0), inv_h, a.eps));
        float y[NV][VEC];
        float ysum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u >= units)
                continue;
            const V w = a.w_post ? static_cast<const V *>(a.w_post)[u] : V{};
            const V g = gate_piece<T, VEC>(a, t, units, u);
            V o;
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                float n = row_to_f(h[i].e[c]);
                if (a.w_post)
                    n = n * r_h * (row_to_f(w.e[c]) + a.offset);
                y[i][c] = fmaf(a.scale * gate_of<T, VEC>(a, row_gate, g, c), n, row_to_f(r[i].e[c]));
                ysum = fmaf(y[i][c], y[i][c], ysum);
                o.e[c] = row_from_f<T>(y[i][c]);
            }
            static_cast<V *>(a.y)[t * units + u] = o;
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
                const V w = static_cast<const V *>(a.w_pre)[u];
                V o;
#pragma unroll
                for (int c = 0; c < VEC; ++c)
                    o.e[c] = row_from_f<T>(y[i][c] * r_y * (row_to_f(w.e[c]) + a.offset));
                static_cast<V *>(a.z)[t * units + u] = o;
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

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const NormArgs a)
{
    using V = Piece<T, VEC>;
    __shared__ float s_buf[2][kMaxWarps];
    __shared__ float s_gate[kMaxWarps];
    const int units = a.H / VEC;
    const float inv_h = 1.0f / (float)a.H;
    float c_post[NV][VEC], c_pre[NV][VEC], c_gate[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c)
            c_post[i][c] = c_pre[i][c] = c_gate[i][c] = 0.0f;
    pdl_wait();
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * units;
        V h[NV], r[NV], dy[NV], dz[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u < units) {
                h[i] = static_cast<const V *>(a.h)[row + u];
                dy[i] = a.dy ? static_cast<const V *>(a.dy)[row + u] : piece_zero<T, VEC>();
                if (a.w_pre) {
                    r[i] = static_cast<const V *>(a.residual)[row + u];
                    dz[i] = static_cast<const V *>(a.dz)[row + u];
                }
            }
        }
        const float r_h = a.w_post ? a.r_h[t] : 1.0f;
        const float row_gate = a.gate_kind == MOE_GATE_TOKEN ? row_to_f(static_cast<const T *>(a.gate)[t]) : 1.0f;
        float r_y = 0.0f, m1 = 0.0f;
        float yh[NV][VEC];  // y * r_y, from the same operations as the forward's y
        if (a.w_pre) {
            r_y = a.r_y[t];
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int u = threadIdx.x + i * blockDim.x;
                if (u >= units)
                    continue;
                const V w = static_cast<const V *>(a.w_pre)[u];
                const V wo = a.w_post ? static_cast<const V *>(a.w_post)[u] : V{};
                const V g = gate_piece<T, VEC>(a, t, units, u);
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    float n = row_to_f(h[i].e[c]);
                    if (a.w_post)
                        n = n * r_h * (row_to_f(wo.e[c]) + a.offset);
                    yh[i][c] = fmaf(a.scale * gate_of<T, VEC>(a, row_gate, g, c), n, row_to_f(r[i].e[c])) * r_y;
                    const float d = row_to_f(dz[i].e[c]);
                    c_pre[i][c] = fmaf(d, yh[i][c], c_pre[i][c]);
                    sum = fmaf(d * (row_to_f(w.e[c]) + a.offset), yh[i][c], sum);
                }
            }
            m1 = block_sum(sum, s_buf, 0) * inv_h;
        }
        float v[NV][VEC];
        float sum = 0.0f, gsum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u >= units)
                continue;
            const V wi = a.w_pre ? static_cast<const V *>(a.w_pre)[u] : V{};
            const V wo = a.w_post ? static_cast<const V *>(a.w_post)[u] : V{};
            const V g = gate_piece<T, VEC>(a, t, units, u);
            V o, dg;
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                float D = row_to_f(dy[i].e[c]);
                if (a.w_pre)
                    D += r_y * (row_to_f(dz[i].e[c]) * (row_to_f(wi.e[c]) + a.offset) - yh[i][c] * m1);
                o.e[c] = row_from_f<T>(D);
                const float hh = row_to_f(h[i].e[c]) * r_h;
                const float w = a.w_post ? row_to_f(wo.e[c]) + a.offset : 1.0f;
                const float dn = a.scale * gate_of<T, VEC>(a, row_gate, g, c) * D;
                const float ge = a.scale * hh * w * D;
                c_post[i][c] = fmaf(dn, hh, c_post[i][c]);
                if (a.gate_kind == MOE_GATE_CHANNEL)
                    c_gate[i][c] += ge;
                gsum += ge;
                dg.e[c] = row_from_f<T>(ge);
                v[i][c] = dn * w;
                sum = fmaf(v[i][c], hh, sum);
            }
            static_cast<V *>(a.dres)[row + u] = o;
            if (a.gate_kind == MOE_GATE_FULL)
                static_cast<V *>(a.dgate)[row + u] = dg;
        }
        float m2 = 0.0f;
        if (a.w_post)
            m2 = block_sum(sum, s_buf, 1) * inv_h;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u >= units)
                continue;
            V o;
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float hh = row_to_f(h[i].e[c]) * r_h;
                o.e[c] = row_from_f<T>(a.w_post ? r_h * (v[i][c] - hh * m2) : v[i][c]);
            }
            static_cast<V *>(a.dh)[row + u] = o;
        }
        if (a.gate_kind == MOE_GATE_TOKEN) {
            gsum = warp_sum(gsum);
            if ((threadIdx.x & 31) == 0)
                s_gate[threadIdx.x >> 5] = gsum;
            __syncthreads();
            if (threadIdx.x == 0) {
                float s = 0.0f;
                for (int i = 0; i < (int)(blockDim.x >> 5); ++i)
                    s += s_gate[i];
                static_cast<float *>(a.dgate)[t] = s;
            }
        }
        __syncthreads();  // the row's shared sums have been read
    }
    float *p = a.part + (int64_t)blockIdx.x * 3 * a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = threadIdx.x + i * blockDim.x;
        if (u >= units)
            continue;
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            p[u * VEC + c] = c_post[i][c];
            p[a.H + u * VEC + c] = c_pre[i][c];
            p[2 * a.H + u * VEC + c] = c_gate[i][c];
        }
    }
}

// out[c] = sum over the blocks' partial rows: 8 strided sums of a column, then added in order.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float *__restrict__ part, int nblocks, int H,
                                                         float *dw_post, float *dw_pre, float *dgate)
{
    __shared__ float s[8][33];
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float *out = blockIdx.y == 0 ? dw_post : blockIdx.y == 1 ? dw_pre : dgate;
    if (!out)
        return;
    float acc = 0.0f;
    if (c < H)
        for (int b = w; b < nblocks; b += 8)
            acc += part[((int64_t)b * 3 + blockIdx.y) * H + c];
    s[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < H) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum += s[i][lane];
        out[c] = sum;
    }
}

int row_size(int row_type)
{
    return row_type == MOE_ROW_FP32 ? 4 : row_type == MOE_ROW_BF16 || row_type == MOE_ROW_FP16 ? 2 : 0;
}

int to_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Partial rows of the backward: at most two blocks per SM (304 on 152 SMs).
constexpr int kBwdBlocks = 304;

template <typename T, int VEC, int NV>
cudaError_t run(const NormArgs &a, bool bwd, cudaStream_t st)
{
    const int units = a.H / VEC;
    int threads = ((units + NV - 1) / NV + 31) / 32 * 32;
    if (threads > kMaxThreads)
        return cudaErrorInvalidValue;
    if (bwd) {
        const int grid = (int)(a.T < kBwdBlocks ? a.T : kBwdBlocks);
        return launch_kernel(false, norm_bwd_kernel<T, VEC, NV>, dim3(grid), dim3(threads), 0, st, a);
    }
    const int64_t grid = a.T < 152 * 16 ? a.T : 152 * 16;
    return launch_kernel(false, norm_kernel<T, VEC, NV>, dim3((unsigned)grid), dim3(threads), 0, st, a);
}

// Pieces a thread holds: the fewest that cover the row with at most kMaxThreads threads.
template <typename T, int VEC>
cudaError_t run_nv(const NormArgs &a, bool bwd, cudaStream_t st)
{
    const int units = a.H / VEC;
    if (units <= 256)
        return run<T, VEC, 1>(a, bwd, st);
    if (units <= 2 * 256)
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
    return (size_t)(T < kBwdBlocks ? (T > 0 ? T : 1) : kBwdBlocks) * 3 * H * sizeof(float);
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
    const int nblocks = (int)(T < kBwdBlocks ? T : kBwdBlocks);
    if (T > 0)
        err = run_type(row_type, a, true, wide, st);
    if (err != cudaSuccess)
        return MOE_ERR_CUDA;
    // T = 0: no partial rows, every sum is zero
    float *dg = gate_kind == MOE_GATE_CHANNEL ? static_cast<float *>(dgate) : nullptr;
    return to_status(launch_kernel(false, norm_reduce_kernel, dim3((H + 31) / 32, 3), dim3(256), 0, st,
                                   static_cast<const float *>(a.part), nblocks, H, w_post ? dw_post : nullptr,
                                   w_pre ? dw_pre : nullptr, dg));
}

}  // extern "C"
