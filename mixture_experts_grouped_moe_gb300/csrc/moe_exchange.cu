// The token exchange of the MoE layer as operators of their own: rows of x to the experts' sorted
// order and back with the top-k weights applied (the token reorder and the weighted combine of the
// AITER walk-through, sections 3 and 3.1), and the gradients of both.
//
//   permute            xs[pos(t,j)] = x[t]                       pos(t,j) = slot_pos[t*k + j]
//   permute (FP8)      the same rows as e4m3 codes with a scale per 1x128 group
//   unpermute          out[t] = sum_j w[t,j] ys[pos(t,j)]
//   unpermute backward dys[pos(t,j)] = w[t,j] dout[t],  dw[t,j] = dout[t] . ys[pos(t,j)]
//   permute backward   dx[t] = sum_j dxs[pos(t,j)]               (unpermute with unit weights)
//
// Every pass is bound by HBM and walks the tokens, not the sorted positions: a token's own row is
// read or written once however its k copies fall in expert order, and every sum over j runs in
// ascending j in fp32, so results do not depend on scheduling (no atomics).  A position outside
// [0, P) -- the -1 of a slot left out by the sort -- is skipped: it receives nothing and adds
// nothing, so a token whose slots are all left out gives a zero row.
//
// The padding rows of the sorted order (sorted_ids[p] >= T*k, p < num_tokens_post_padded) are
// zeroed by extra blocks of the same launch when asked for.
#include <cuda_fp8.h>

#include "moe_internal.h"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxK = 32;
constexpr int kUnits = 4;  // pieces a lane moves per item

struct RowArgs {
    const void *src;          // token rows: x or dout (unpermute: unused)
    int64_t ld_src;           // elements
    const int32_t *slot_pos;  // [T][k]
    const int32_t *sorted_ids;
    const int32_t *npp;
    const float *wts;         // [T][k] or null
    int T, k, H;
    int64_t P;
    const void *ys;           // sorted rows read [P][H]
    void *dst;                // sorted rows written [P][H], or token rows (unpermute)
    int64_t ld_dst;
    uint8_t *q;               // FP8 codes [P][H]
    float *s;                 // FP8 scales [H/128][P]
    float *dw;                // [T][k]
    int64_t token_blocks;     // blocks that walk tokens
    int64_t pad_blocks;       // blocks before them that zero padding rows (first, so that both run at once)
};

// Lane j < k of the warp gets the position of the token's slot j (-1 for none).
__device__ __forceinline__ int lane_pos(const RowArgs &a, int64_t t, int lane)
{
    int pos = -1;
    if (lane < a.k) {
        pos = __ldg(a.slot_pos + t * a.k + lane);
        if (pos < 0 || pos >= a.P)
            pos = -1;
    }
    return pos;
}

// Zero the padding rows: an item is 32 sorted positions and one segment of the row; `units` pieces
// of type P per row, `seg` pieces per segment.
template <typename V>
__device__ __forceinline__ void zero_padding(const int32_t *sorted_ids, int64_t npp, int S, int64_t units, int seg,
                                             V *rows, const V &zero, int64_t item, int64_t nitems, int lane,
                                             float *scales = nullptr, int64_t P = 0)
{
    const int64_t nseg = (units + seg - 1) / seg;
    const int64_t total = (npp + 31) / 32 * nseg;
    for (; item < total; item += nitems) {
        const int64_t p0 = item / nseg * 32;
        const int64_t u0 = item % nseg * seg;
        const int64_t u1 = u0 + seg < units ? u0 + seg : units;
        const bool pad = p0 + lane < npp && sorted_ids[p0 + lane] >= S;
        unsigned m = __ballot_sync(0xffffffffu, pad);
        while (m) {
            const int b = __ffs(m) - 1;
            m &= m - 1;
            V *row = rows + (p0 + b) * units;
            for (int64_t u = u0 + lane; u < u1; u += 32)
                row[u] = zero;
        }
        if (scales && pad)  // a zero group's scale is 1 (16 codes a piece, 8 pieces a group)
            for (int64_t g = u0 / 8; g < u1 / 8; ++g)
                scales[g * P + p0 + lane] = 1.0f;
    }
}

// A warp moves one segment (32 lanes x kUnits pieces) of one token's row to its k positions.  HBM: 8192 rows of
// 4096 bf16, top-2, with the sort 40.7 us (73 % of the copy rate).  Rows on 4-byte boundaries only (4098
// elements) move in words, 45.8 us; odd ones (4097) in elements, 60.1.
template <typename V>
__global__ void __launch_bounds__(kThreads) permute_kernel(const RowArgs a, int64_t units, int64_t ld_units, V zero)
{
    const int lane = threadIdx.x & 31;
    const int64_t warp = (blockIdx.x - a.pad_blocks) * kWarps + (threadIdx.x >> 5);
    constexpr int seg = 32 * kUnits;
    V *dst = static_cast<V *>(a.dst);
    pdl_wait();
    pdl_trigger();
    if (warp < 0) {
        const int64_t npp = *a.npp;
        zero_padding(a.sorted_ids, npp < a.P ? npp : a.P, a.T * a.k, units, seg, dst, zero,
                     warp + a.pad_blocks * kWarps, a.pad_blocks * kWarps, lane);
        return;
    }
    const int64_t nseg = (units + seg - 1) / seg;
    const int64_t total = nseg * a.T;
    for (int64_t item = warp; item < total; item += a.token_blocks * kWarps) {
        const int64_t t = item / nseg;
        const int64_t u0 = item % nseg * seg + lane;
        const int pos = lane_pos(a, t, lane);
        const V *src = static_cast<const V *>(a.src) + t * ld_units;
        V v[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            if (u0 + 32 * i < units)
                v[i] = src[u0 + 32 * i];
        for (int j = 0; j < a.k; ++j) {
            const int p = __shfl_sync(0xffffffffu, pos, j);
            if (p < 0)
                continue;
            V *row = dst + (int64_t)p * units;
#pragma unroll
            for (int i = 0; i < kUnits; ++i)
                if (u0 + 32 * i < units)
                    row[u0 + 32 * i] = v[i];
        }
    }
}

// A warp quantises 512 columns of one token's row (a group of 128 columns on 8 lanes, 16 columns
// per lane), once, and writes the codes and scales to the token's k positions.  The next item's loads
// are issued before this one is encoded.  Bound by instruction issue (68 % of the slots): 8192 x 4096, top-2,
// 30 us after the sort's 7.4 (3.9 TB/s); 44 us for both with a division an element and the loads in line.
__global__ void __launch_bounds__(kThreads, 4) permute_fp8_kernel(const RowArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t warp = (blockIdx.x - a.pad_blocks) * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    const int64_t units = a.H / 16;
    if (warp < 0) {
        const int64_t npp = *a.npp;
        zero_padding(a.sorted_ids, npp < a.P ? npp : a.P, a.T * a.k, units, 32 * kUnits,
                     reinterpret_cast<uint4 *>(a.q), make_uint4(0, 0, 0, 0), warp + a.pad_blocks * kWarps,
                     a.pad_blocks * kWarps, lane, a.s, a.P);
        return;
    }
    const int nseg = (int)((units + 31) / 32);
    const int64_t step = a.token_blocks * kWarps;
    int64_t t = warp / nseg;
    int seg = (int)(warp % nseg);
    const int64_t step_t = step / nseg;
    const int step_seg = (int)(step % nseg);
    uint4 raw[2] = {};
    int pos = -1;
    auto load = [&]() {
        if (t >= a.T)
            return;
        const int64_t u = (int64_t)seg * 32 + lane;
        pos = lane_pos(a, t, lane);
        if (u < units) {
            const uint4 *src =
                reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.src) + t * a.ld_src) + 2 * u;
            raw[0] = __ldg(src);
            raw[1] = __ldg(src + 1);
        }
    };
    load();
    while (t < a.T) {
        const int64_t u = (int64_t)seg * 32 + lane;
        const uint32_t w8[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
        const int cur = pos;
        t += step_t;
        seg += step_seg;
        if (seg >= nseg) {
            seg -= nseg;
            ++t;
        }
        load();
        float f[16];
        float amax = 0.0f;
        if (u < units) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                unpack_word(w8[i], f[2 * i], f[2 * i + 1], __nv_bfloat16{});
                amax = fmaxf(amax, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
            }
        }
#pragma unroll
        for (int d = 4; d >= 1; d >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        const float sc = amax > 0.0f ? amax / 448.0f : 1.0f;
        uint32_t w[4];
        if (u < units) {
            divide16(f, sc);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo =
                    __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi =
                    __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
                w[i] = lo | (hi << 16);
            }
        }
        for (int j = 0; j < a.k; ++j) {
            const int p = __shfl_sync(0xffffffffu, cur, j);
            if (p < 0 || u >= units)
                continue;
            *reinterpret_cast<uint4 *>(a.q + (int64_t)p * a.H + 16 * u) = make_uint4(w[0], w[1], w[2], w[3]);
            if ((u & 7) == 0)
                a.s[u / 8 * a.P + p] = sc;
        }
    }
}

// A warp sums one segment of a token's k rows, their loads all in flight.  HBM: 8192 x 4096 bf16, top-2, 35 us
// (84 % of the copy rate), 4096 x 7168, top-8, 87 us (89 %).  Rows that do not start and end on 16 bytes go
// by elements: 8192 x 4097 takes 102 us.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) unpermute_kernel(const RowArgs a, int64_t units, int64_t ld_units)
{
    using V = Piece<T, VEC>;
    constexpr int U = 2;
    constexpr int seg = 32 * U;
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    const int64_t nseg = (units + seg - 1) / seg;
    const int64_t total = nseg * a.T;
    const V *ys = static_cast<const V *>(a.ys);
    for (int64_t item = warp; item < total; item += (int64_t)gridDim.x * kWarps) {
        const int64_t t = item / nseg;
        const int64_t u0 = item % nseg * seg + lane;
        const int pos = lane_pos(a, t, lane);
        const float wt = a.wts && lane < a.k ? __ldg(a.wts + t * a.k + lane) : 1.0f;
        float acc[U][VEC];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int c = 0; c < VEC; ++c)
                acc[i][c] = 0.0f;
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) {
            const int p = __shfl_sync(0xffffffffu, pos, j);
            const float w = __shfl_sync(0xffffffffu, wt, j);
            if (p < 0)
                continue;
            const V *row = ys + (int64_t)p * units;
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (u0 + 32 * i < units) {
                    float f[VEC];
                    unpack<T, VEC>(row[u0 + 32 * i], f);
#pragma unroll
                    for (int c = 0; c < VEC; ++c)
                        acc[i][c] = fmaf(w, f[c], acc[i][c]);
                }
        }
        V *out = static_cast<V *>(a.dst) + t * ld_units;
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (u0 + 32 * i < units)
                out[u0 + 32 * i] = pack<T, VEC>(acc[i]);
    }
}

// WPT warps per token: they hold a chunk of dout's row in registers, and for each slot read the
// row's chunk of ys, add to the slot's dot product and write the weighted row.  A warp's partial
// dot products live in its own row of s_dot; the token's warps are summed in order at the end.  HBM: 76 % of
// its nominal throughput at 7168 columns, top-8.
template <typename T, int VEC, int WPT>
__global__ void __launch_bounds__(kThreads, 4) unpermute_bwd_kernel(const RowArgs a, int64_t units, int64_t ld_units)
{
    using V = Piece<T, VEC>;
    constexpr int TPB = kWarps / WPT;  // tokens a block works on at once
    constexpr int chunk = 32 * WPT * kUnits;
    __shared__ float s_dot[kWarps][kMaxK];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int wt_in = w % WPT, tok = w / WPT;
    V *dys = static_cast<V *>(a.dst);
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x < a.pad_blocks) {
        const int64_t npp = *a.npp;
        zero_padding(a.sorted_ids, npp < a.P ? npp : a.P, a.T * a.k, units, 32 * kUnits, dys, piece_zero<T, VEC>(),
                     (int64_t)blockIdx.x * kWarps + w, a.pad_blocks * kWarps, lane);
        return;
    }
    const V *ys = static_cast<const V *>(a.ys);
    for (int64_t t0 = (blockIdx.x - a.pad_blocks) * TPB; t0 < a.T; t0 += a.token_blocks * TPB) {
        const int64_t t = t0 + tok;
        s_dot[w][lane] = 0.0f;
        __syncwarp();
        if (t < a.T) {
            const int pos = lane_pos(a, t, lane);
            const float wl = a.wts && lane < a.k ? __ldg(a.wts + t * a.k + lane) : 1.0f;
            const V *src = static_cast<const V *>(a.src) + t * ld_units;
            for (int64_t c0 = 0; c0 < units; c0 += chunk) {
                const int64_t u0 = c0 + wt_in * 32 + lane;
                V d[kUnits];
#pragma unroll
                for (int i = 0; i < kUnits; ++i)
                    if (u0 + 32 * WPT * i < units)
                        d[i] = src[u0 + 32 * WPT * i];
                for (int j = 0; j < a.k; ++j) {
                    const int p = __shfl_sync(0xffffffffu, pos, j);
                    const float wj = __shfl_sync(0xffffffffu, wl, j);
                    if (p < 0)
                        continue;
                    const V *yr = ys + (int64_t)p * units;
                    V *dr = dys + (int64_t)p * units;
                    V y[kUnits];
#pragma unroll
                    for (int i = 0; i < kUnits; ++i)
                        if (u0 + 32 * WPT * i < units)
                            y[i] = yr[u0 + 32 * WPT * i];
                    float dot = 0.0f;
#pragma unroll
                    for (int i = 0; i < kUnits; ++i)
                        if (u0 + 32 * WPT * i < units) {
                            float df[VEC], yf[VEC];
                            unpack<T, VEC>(d[i], df);
                            unpack<T, VEC>(y[i], yf);
#pragma unroll
                            for (int c = 0; c < VEC; ++c) {
                                dot = fmaf(df[c], yf[c], dot);
                                df[c] *= wj;
                            }
                            dr[u0 + 32 * WPT * i] = pack<T, VEC>(df);
                        }
                    dot = warp_sum(dot);
                    if (lane == 0)
                        s_dot[w][j] += dot;
                }
            }
        }
        __syncthreads();
        if (t < a.T && wt_in == 0 && lane < a.k) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < WPT; ++i)
                sum += s_dot[w + i][lane];
            a.dw[t * a.k + lane] = sum;
        }
        __syncthreads();
    }
}

int blocks_for(int64_t warps)
{
    const int64_t b = (warps + kWarps - 1) / kWarps;
    return (int)(b < 1 ? 1 : b < 152 * 64 ? b : 152 * 64);
}

// Extra blocks that zero padding rows (an item: 32 positions x one segment of the row).
int pad_blocks(bool zero, int64_t P, int64_t units, int seg)
{
    return zero && P > 0 ? blocks_for((P + 31) / 32 * ((units + seg - 1) / seg)) : 0;
}

int row_size(int row_type)
{
    return row_type == MOE_ROW_FP32 ? 4 : row_type == MOE_ROW_BF16 || row_type == MOE_ROW_FP16 ? 2 : 0;
}

int to_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

template <typename V>
cudaError_t run_permute(RowArgs &a, int64_t row_bytes, int es, bool zero, cudaStream_t st)
{
    const int64_t units = row_bytes / sizeof(V);
    const int seg = 32 * kUnits;
    a.token_blocks = blocks_for((units + seg - 1) / seg * a.T);
    a.pad_blocks = pad_blocks(zero, a.P, units, seg);
    const int grid = (int)(a.token_blocks + a.pad_blocks);
    return launch_kernel(true, permute_kernel<V>, dim3(grid), dim3(kThreads), 0, st, a, units,
                         a.ld_src * es / (int64_t)sizeof(V), V{});
}

template <typename T, int VEC>
cudaError_t run_unpermute(const RowArgs &a, cudaStream_t st)
{
    const int64_t units = a.H / VEC;
    const int grid = blocks_for((units + 63) / 64 * a.T);
    return launch_kernel(true, unpermute_kernel<T, VEC>, dim3(grid), dim3(kThreads), 0, st, a, units,
                         a.ld_dst / VEC);
}

template <typename T, int VEC, int WPT>
cudaError_t run_bwd_w(RowArgs &a, bool zero, cudaStream_t st)
{
    const int64_t units = a.H / VEC;
    a.token_blocks = blocks_for((int64_t)a.T * WPT);
    a.pad_blocks = pad_blocks(zero, a.P, units, 32 * kUnits);
    const int grid = (int)(a.token_blocks + a.pad_blocks);
    return launch_kernel(true, unpermute_bwd_kernel<T, VEC, WPT>, dim3(grid), dim3(kThreads), 0, st, a, units,
                         a.ld_src / VEC);
}

template <typename T, int VEC>
cudaError_t run_bwd(RowArgs &a, bool zero, cudaStream_t st)
{
    // As many warps a token as its row fills with kUnits pieces a lane (both gradients of 8192 tokens, top-2:
    // 1024 columns 26.6 us with one warp a token, 56.6 with eight; 2048 columns 47.0 with two, 70.3 with eight).
    const int64_t units = a.H / VEC;
    if (units <= 32 * kUnits)
        return run_bwd_w<T, VEC, 1>(a, zero, st);
    if (units <= 64 * kUnits)
        return run_bwd_w<T, VEC, 2>(a, zero, st);
    return run_bwd_w<T, VEC, 8>(a, zero, st);
}

// Shape checks shared by the entries: MOE_OK or a negative status.
int check_exchange(int row_type, int T, int k, int H, int64_t P, int64_t ld)
{
    if (row_size(row_type) == 0 || T < 0 || k <= 0 || H <= 0 || P < 0 || ld < H)
        return MOE_ERR_INVALID_ARG;
    if (k > kMaxK || (int64_t)T * k > (int64_t)1 << 30 || P > INT32_MAX)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

// left_out: where the slots left out are counted (a routing with such slots is then no error), or null.
static int sort_with_map(const int32_t *topk_ids, const float *topk_weights, int T, int k, int E, int block_m,
                         int32_t *sorted_ids, float *sorted_weights, int32_t *sorted_expert_ids,
                         int32_t *num_tokens_post_padded, int32_t *expert_counts, int32_t *slot_pos,
                         int32_t *left_out, void *ws, size_t ws_bytes, void *stream)
{
    if (T < 0 || k <= 0 || E <= 0 || block_m <= 0)
        return MOE_ERR_INVALID_ARG;
    if (E > 1024 || k > E || (int64_t)T * k > (int64_t)1 << 30 ||
        (int64_t)T * k + (int64_t)E * block_m - k > INT32_MAX)  // (positions are int32)
        return MOE_ERR_UNSUPPORTED;
    if (!topk_ids || !topk_weights || !sorted_ids || !sorted_weights || !sorted_expert_ids ||
        !num_tokens_post_padded || !slot_pos || !ws)
        return MOE_ERR_INVALID_ARG;
    const size_t need = moe_align_sort_workspace_size(T, k, E);
    if (ws_bytes < need)
        return MOE_ERR_WORKSPACE;
    SortOut so = {};
    so.sorted_ids = sorted_ids;
    so.sorted_weights = sorted_weights;
    so.sorted_expert_ids = sorted_expert_ids;
    so.num_post_padded = num_tokens_post_padded;
    so.expert_counts = expert_counts;
    so.slot_pos = slot_pos;
    so.left_out = left_out;
    // as moe_align_sort lays its scratch out: chunk histograms, then the E + 1 padded offsets
    so.expert_offsets = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + need - (size_t)(E + 1) * 4);
    return to_status(launch_align_sort(topk_ids, topk_weights, T, k, E, block_m, so, ws, true, true,
                                       static_cast<cudaStream_t>(stream)));
}

extern "C" {

int moe_align_sort_map(const int32_t *topk_ids, const float *topk_weights, int T, int k, int E, int block_m,
                       int32_t *sorted_ids, float *sorted_weights, int32_t *sorted_expert_ids,
                       int32_t *num_tokens_post_padded, int32_t *expert_counts, int32_t *slot_pos, void *ws,
                       size_t ws_bytes, void *stream)
{
    return sort_with_map(topk_ids, topk_weights, T, k, E, block_m, sorted_ids, sorted_weights, sorted_expert_ids,
                         num_tokens_post_padded, expert_counts, slot_pos, nullptr, ws, ws_bytes, stream);
}

int moe_align_sort_drop(const int32_t *topk_ids, const float *topk_weights, int T, int k, int E, int block_m,
                        int32_t *sorted_ids, float *sorted_weights, int32_t *sorted_expert_ids,
                        int32_t *num_tokens_post_padded, int32_t *expert_counts, int32_t *slot_pos,
                        int32_t *num_left_out, void *ws, size_t ws_bytes, void *stream)
{
    if (!num_left_out)
        return MOE_ERR_INVALID_ARG;
    return sort_with_map(topk_ids, topk_weights, T, k, E, block_m, sorted_ids, sorted_weights, sorted_expert_ids,
                         num_tokens_post_padded, expert_counts, slot_pos, num_left_out, ws, ws_bytes, stream);
}

int moe_permute(int row_type, const void *x, int64_t ld_x, const int32_t *slot_pos, const int32_t *sorted_ids,
                const int32_t *num_tokens_post_padded, int T, int k, int H, int64_t P, int zero_padding, void *xs,
                void *stream)
{
    const int rc = check_exchange(row_type, T, k, H, P, ld_x);
    if (rc != MOE_OK)
        return rc;
    const int es = row_size(row_type);
    if (zero_padding < 0 || zero_padding > 1 || !x || !slot_pos || !xs ||
        (zero_padding && (!sorted_ids || !num_tokens_post_padded)) ||
        ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(xs)) & (es - 1)))
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    RowArgs a = {};
    a.src = x, a.ld_src = ld_x, a.slot_pos = slot_pos, a.sorted_ids = sorted_ids, a.npp = num_tokens_post_padded;
    a.T = T, a.k = k, a.H = H, a.P = P, a.dst = xs;
    const int64_t row = (int64_t)H * es, pitch = ld_x * es;
    const auto st = static_cast<cudaStream_t>(stream);
    const uintptr_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(xs) | (uintptr_t)row |
                           (uintptr_t)pitch;
    if ((bits & 15) == 0)
        return to_status(run_permute<uint4>(a, row, es, zero_padding, st));
    if ((bits & 3) == 0)
        return to_status(run_permute<uint32_t>(a, row, es, zero_padding, st));
    return to_status(run_permute<uint16_t>(a, row, es, zero_padding, st));
}

int moe_permute_fp8(const void *x, int64_t ld_x, const int32_t *slot_pos, const int32_t *sorted_ids,
                    const int32_t *num_tokens_post_padded, int T, int k, int H, int64_t P, int zero_padding,
                    uint8_t *q, float *s, void *stream)
{
    const int rc = check_exchange(MOE_ROW_BF16, T, k, H, P, ld_x);
    if (rc != MOE_OK)
        return rc;
    if (zero_padding < 0 || zero_padding > 1 || !x || !slot_pos || !q || !s ||
        (zero_padding && (!sorted_ids || !num_tokens_post_padded)))
        return MOE_ERR_INVALID_ARG;
    if (H % 128 != 0 || ld_x % 8 != 0)
        return MOE_ERR_UNSUPPORTED;
    if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(q)) & 15) ||
        (reinterpret_cast<uintptr_t>(s) & 3))
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    RowArgs a = {};
    a.src = x, a.ld_src = ld_x, a.slot_pos = slot_pos, a.sorted_ids = sorted_ids, a.npp = num_tokens_post_padded;
    a.T = T, a.k = k, a.H = H, a.P = P, a.q = q, a.s = s;
    const int64_t blocks = blocks_for((H / 16 + 31) / 32 * (int64_t)T);
    // As many blocks as are resident, whose loads pipeline (8192 x 4096: 38.4 us, 41.6 with a block an item).
    a.token_blocks = blocks < 152 * 4 ? blocks : 152 * 4;
    a.pad_blocks = pad_blocks(zero_padding, P, H / 16, 32 * kUnits);
    const int grid = (int)(a.token_blocks + a.pad_blocks);
    return to_status(launch_kernel(true, permute_fp8_kernel, dim3(grid), dim3(kThreads), 0,
                                   static_cast<cudaStream_t>(stream), a));
}

int moe_unpermute(int row_type, const void *ys, const int32_t *slot_pos, const float *topk_weights, int T, int k,
                  int H, int64_t P, void *out, int64_t ld_out, void *stream)
{
    const int rc = check_exchange(row_type, T, k, H, P, ld_out);
    if (rc != MOE_OK)
        return rc;
    const int es = row_size(row_type);
    if (!ys || !slot_pos || !out || ((reinterpret_cast<uintptr_t>(ys) | reinterpret_cast<uintptr_t>(out)) & (es - 1)))
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    RowArgs a = {};
    a.slot_pos = slot_pos, a.wts = topk_weights, a.T = T, a.k = k, a.H = H, a.P = P, a.ys = ys, a.dst = out;
    a.ld_dst = ld_out;
    const auto st = static_cast<cudaStream_t>(stream);
    const bool wide = rows_aligned16(out, ld_out * es, (int64_t)H * es) && rows_aligned16(ys, 0, 0);
    switch (row_type) {
    case MOE_ROW_BF16:
        return to_status(wide ? run_unpermute<__nv_bfloat16, 8>(a, st) : run_unpermute<__nv_bfloat16, 1>(a, st));
    case MOE_ROW_FP16: return to_status(wide ? run_unpermute<__half, 8>(a, st) : run_unpermute<__half, 1>(a, st));
    default: return to_status(wide ? run_unpermute<float, 4>(a, st) : run_unpermute<float, 1>(a, st));
    }
}

int moe_permute_backward(int row_type, const void *dxs, const int32_t *slot_pos, int T, int k, int H, int64_t P,
                         void *dx, int64_t ld_dx, void *stream)
{
    return moe_unpermute(row_type, dxs, slot_pos, nullptr, T, k, H, P, dx, ld_dx, stream);
}

int moe_unpermute_backward(int row_type, const void *dout, int64_t ld_dout, const void *ys, const int32_t *slot_pos,
                           const float *topk_weights, const int32_t *sorted_ids,
                           const int32_t *num_tokens_post_padded, int T, int k, int H, int64_t P, int zero_padding,
                           void *dys, float *dweights, void *stream)
{
    const int rc = check_exchange(row_type, T, k, H, P, ld_dout);
    if (rc != MOE_OK)
        return rc;
    const int es = row_size(row_type);
    if (zero_padding < 0 || zero_padding > 1 || !dout || !ys || !slot_pos || !dys || !dweights ||
        (zero_padding && (!sorted_ids || !num_tokens_post_padded)) ||
        ((reinterpret_cast<uintptr_t>(ys) | reinterpret_cast<uintptr_t>(dout) | reinterpret_cast<uintptr_t>(dys)) &
         (es - 1)))
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    RowArgs a = {};
    a.src = dout, a.ld_src = ld_dout, a.slot_pos = slot_pos, a.sorted_ids = sorted_ids;
    a.npp = num_tokens_post_padded, a.wts = topk_weights, a.T = T, a.k = k, a.H = H, a.P = P, a.ys = ys;
    a.dst = dys, a.dw = dweights;
    const auto st = static_cast<cudaStream_t>(stream);
    const bool z = zero_padding != 0;
    const bool wide = rows_aligned16(dout, ld_dout * es, (int64_t)H * es) && rows_aligned16(ys, 0, 0) &&
                      rows_aligned16(dys, 0, 0);
    switch (row_type) {
    case MOE_ROW_BF16:
        return to_status(wide ? run_bwd<__nv_bfloat16, 8>(a, z, st) : run_bwd<__nv_bfloat16, 1>(a, z, st));
    case MOE_ROW_FP16: return to_status(wide ? run_bwd<__half, 8>(a, z, st) : run_bwd<__half, 1>(a, z, st));
    default: return to_status(wide ? run_bwd<float, 4>(a, z, st) : run_bwd<float, 1>(a, z, st));
    }
}

}  // extern "C"
