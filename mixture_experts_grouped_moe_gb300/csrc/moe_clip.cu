// The 2-norm of all elements of many tensors, and their clipping to it:
//   norm = sqrt(sum g^2),   out = g * min(1, max_norm / (norm + eps))
// for bf16, fp16 and fp32 tensors together, of any sizes.  Bound by memory: every element is read for the norm,
// and once more to be scaled and written.  The tensors' addresses travel as kernel parameters, so a call needs no
// table in device memory and can be captured into a graph.
//
// A block takes chunks of 32 KB (eight 16-byte loads a thread in flight).  A thread squares and adds its 32 or
// 64 values of a chunk in fp32, where squares overflow above 2^64 and lose bits below 2^-63: a sum outside
// [2^-100, 2^120] is formed again in 64 bits from the values, which are still in registers (inside, what a small
// square loses is below 2^-149 and so nothing against the sum).  Everything above a thread's chunk is summed in 64
// bits in a fixed order: results are bitwise reproducible.
//
// 5.6 GB of fp32 in 2.48 ms (6.8 TB/s, the copy rate), 134 MB in 68 us (the norm alone 26; tensors off 16-byte
// boundaries, scaled element by element, 227), 60 tensors of up to 6000 elements in 9.7 replayed from a graph and 30
// called, all of it the host's.
#include "moe_internal.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 8;                              // 16-byte loads of a thread and chunk
constexpr int kChunkBytes = kThreads * kLoads * 16;    // 32 KB
constexpr int kMaxTensors = 512;                       // of one launch
constexpr int kBlocks = 152 * 8;                       // most blocks of a launch
constexpr int kResident = 152 * 2;                     // blocks that run at once

// Blocks of a launch: those that run at once, or, where each of four times as many has 8 chunks or more, so many, which
// even out unequal speeds (us with 304 / 1216: 67 MB fp32 35.2 / 44.3, 134 MB 67.7 / 74.0, 268 MB 130 / 132, 537 MB
// 252 / 248, 4.3 GB 1922 / 1886).
unsigned blocks_for(int64_t chunks)
{
    if (chunks >= 8 * kBlocks)
        return kBlocks;
    return (unsigned)(chunks < kResident ? (chunks ? chunks : 1) : kResident);
}

struct Tensors {
    int n;
    int64_t chunks;
    const void *g[kMaxTensors];
    void *out[kMaxTensors];
    int64_t numel[kMaxTensors];
    int64_t first[kMaxTensors + 1];  // first chunk of each tensor
    uint8_t type[kMaxTensors];
    uint8_t wide[kMaxTensors];       // on 16-byte boundaries
};
static_assert(sizeof(Tensors) <= 30000, "kernel parameters hold 32764 bytes");

__device__ __forceinline__ int per_chunk(int type) { return type == MOE_ROW_FP32 ? kChunkBytes / 4 : kChunkBytes / 2; }

// The square sum of n values held by one thread.
template <int N>
__device__ __forceinline__ double squares(const float (&f)[N])
{
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i)
        s[i & 3] = fmaf(f[i], f[i], s[i & 3]);
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    if (sum >= 0x1p-100f && sum <= 0x1p120f)
        return sum;
    bool zero = true;  // (gradients of unused weights are whole chunks of zeros)
#pragma unroll
    for (int i = 0; i < N; ++i)
        zero = zero && f[i] == 0.0f;
    if (zero)
        return 0.0;
    double d = 0.0;
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
        float v = f[0];
#pragma unroll
        for (int j = 1; j < N; ++j)
            v = i == j ? f[j] : v;
        d = fma((double)v, (double)v, d);
    }
    return d;
}

// This thread's part of one chunk (32 or 64 values; those past the end are zero).
template <typename T>
__device__ __forceinline__ double chunk_squares(const T *g, int64_t left, bool wide)
{
    constexpr int V = 16 / (int)sizeof(T), kN = kLoads * V;
    float f[kN];
    if (wide) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int64_t e = ((int64_t)i * kThreads + threadIdx.x) * V;
            Piece<T, V> p = piece_zero<T, V>();
            if (e + V <= left)
                p.w = __ldg(reinterpret_cast<const uint4 *>(g + e));
            float v[V];
            unpack(p, v);
            if (e < left && e + V > left) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[j] = e + j < left ? row_to_f(g[e + j]) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < V; ++j)
                f[i * V + j] = v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int64_t e = (int64_t)i * kThreads + threadIdx.x;
            f[i] = e < left ? row_to_f(g[e]) : 0.0f;
        }
    }
    return squares(f);
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *g, T *out, int64_t left, bool wide, float k)
{
    constexpr int V = 16 / (int)sizeof(T);
    if (wide) {
        Piece<T, V> p[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int64_t e = ((int64_t)i * kThreads + threadIdx.x) * V;
            if (e + V <= left)
                p[i].w = *reinterpret_cast<const uint4 *>(g + e);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int64_t e = ((int64_t)i * kThreads + threadIdx.x) * V;
            if (e + V <= left) {
                float v[V];
                unpack(p[i], v);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[j] *= k;
                *reinterpret_cast<uint4 *>(out + e) = pack<T, V>(v).w;
            } else {
                for (int j = 0; j < V && e + j < left; ++j)
                    out[e + j] = row_from_f<T>(row_to_f(g[e + j]) * k);
            }
        }
    } else {
#pragma unroll 8
        for (int i = 0; i < kLoads * V; ++i) {
            const int64_t e = (int64_t)i * kThreads + threadIdx.x;
            if (e < left)
                out[e] = row_from_f<T>(row_to_f(g[e]) * k);
        }
    }
}

// Sum over the block in a fixed order; valid in thread 0.
__device__ __forceinline__ double block_sum(double v, double *warp_sums)
{
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) == 0)
        warp_sums[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (int i = 0; i < kThreads / 32; ++i)
            s += warp_sums[i];
    return s;
}

__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Tensors t, double *part)
{
    __shared__ double warp_sums[kThreads / 32];
    pdl_wait();
    pdl_trigger();
    double sum = 0.0;
    int i = 0;
    for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        while (c >= t.first[i + 1])
            ++i;
        const int64_t at = (c - t.first[i]) * per_chunk(t.type[i]), left = t.numel[i] - at;
        const bool wide = t.wide[i];
        switch (t.type[i]) {
        case MOE_ROW_BF16: sum += chunk_squares(static_cast<const __nv_bfloat16 *>(t.g[i]) + at, left, wide); break;
        case MOE_ROW_FP16: sum += chunk_squares(static_cast<const __half *>(t.g[i]) + at, left, wide); break;
        default: sum += chunk_squares(static_cast<const float *>(t.g[i]) + at, left, wide);
        }
    }
    sum = block_sum(sum, warp_sums);
    if (threadIdx.x == 0)
        part[blockIdx.x] = sum;
}

// The norm from the launches' partial sums: every block forms it alike.  Valid in all threads.
__device__ __forceinline__ float norm_of(const double *part, int parts, double *warp_sums, float *shared_norm)
{
    double v = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads)
        v += part[i];
    v = block_sum(v, warp_sums);
    if (threadIdx.x == 0)
        *shared_norm = (float)sqrt(v);
    __syncthreads();
    return *shared_norm;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double *part, int parts, float *norm)
{
    __shared__ double warp_sums[kThreads / 32];
    __shared__ float shared_norm;
    pdl_wait();
    pdl_trigger();
    const float v = norm_of(part, parts, warp_sums, &shared_norm);
    if (threadIdx.x == 0)
        *norm = v;
}

// The chunks in falling order: those that the norm read last are still in L2.
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Tensors t, const double *part,
                                                         int parts, float max_norm, float eps, float *norm)
{
    __shared__ double warp_sums[kThreads / 32];
    __shared__ float shared_norm;
    pdl_wait();
    pdl_trigger();
    const float v = norm_of(part, parts, warp_sums, &shared_norm);
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *norm = v;
    const float ratio = max_norm / (v + eps);
    const float k = ratio >= 1.0f ? 1.0f : ratio;  // (a NaN stays one)
    int i = t.n - 1;
    for (int64_t c = t.chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        while (c < t.first[i])
            --i;
        if (k == 1.0f && t.g[i] == t.out[i])
            continue;  // nothing changes
        const int64_t at = (c - t.first[i]) * per_chunk(t.type[i]), left = t.numel[i] - at;
        const bool wide = t.wide[i];
        switch (t.type[i]) {
        case MOE_ROW_BF16:
            chunk_scale(static_cast<const __nv_bfloat16 *>(t.g[i]) + at, static_cast<__nv_bfloat16 *>(t.out[i]) + at,
                        left, wide, k);
            break;
        case MOE_ROW_FP16:
            chunk_scale(static_cast<const __half *>(t.g[i]) + at, static_cast<__half *>(t.out[i]) + at, left, wide, k);
            break;
        default:
            chunk_scale(static_cast<const float *>(t.g[i]) + at, static_cast<float *>(t.out[i]) + at, left, wide, k);
        }
    }
}

bool off(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// Tensors [from, from + count) of the call.
void collect(Tensors &t, int from, int count, const int *types, const void *const *g, void *const *out,
             const int64_t *numel)
{
    t.n = count;
    t.chunks = 0;
    for (int j = 0; j < count; ++j) {
        const int i = from + j;
        const int es = types[i] == MOE_ROW_FP32 ? 4 : 2;
        void *o = out ? out[i] : nullptr;
        t.g[j] = g[i], t.out[j] = o, t.numel[j] = numel[i];
        t.type[j] = (uint8_t)types[i];
        t.wide[j] = !off(g[i], 16) && !off(o, 16);
        t.first[j] = t.chunks;
        t.chunks += (numel[i] * es + kChunkBytes - 1) / kChunkBytes;
    }
    t.first[count] = t.chunks;
}

int check(int n, const int *types, const void *const *g, void *const *out, bool scaled, const int64_t *numel,
          const float *norm, const void *ws, size_t ws_bytes)
{
    if (n < 0 || (n && (!types || !g || !numel || (scaled && !out))) || !norm || !ws || off(norm, 4) || off(ws, 8))
        return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        if (types[i] < 0 || types[i] > MOE_ROW_FP32 || numel[i] < 0 || (numel[i] && (!g[i] || (scaled && !out[i]))))
            return MOE_ERR_INVALID_ARG;
        const int es = types[i] == MOE_ROW_FP32 ? 4 : 2;
        if (off(g[i], es) || (scaled && off(out[i], es)))
            return MOE_ERR_INVALID_ARG;
        if (numel[i] > 1ll << 40)
            return MOE_ERR_UNSUPPORTED;
    }
    if (n > 1 << 16)
        return MOE_ERR_UNSUPPORTED;
    if (ws_bytes < MOE_CLIP_WS_BYTES(n))
        return MOE_ERR_WORKSPACE;
    return MOE_OK;
}

int run(int n, const int *types, const void *const *g, void *const *out, bool scaled, const int64_t *numel,
        float max_norm, float eps, float *norm, void *ws, cudaStream_t st)
{
    static_assert(MOE_CLIP_WS_BYTES(1) >= kBlocks * 8 && MOE_CLIP_WS_BYTES(kMaxTensors + 1) >= 2 * kBlocks * 8,
                  "one double for each block of each launch");
    double *part = static_cast<double *>(ws);
    Tensors t;
    int parts = 0;
    for (int from = 0; from < n; from += kMaxTensors) {
        collect(t, from, n - from < kMaxTensors ? n - from : kMaxTensors, types, g, out, numel);
        if (launch_kernel(true, squares_kernel, dim3(blocks_for(t.chunks)), dim3(kThreads), 0, st, t, part + parts) != cudaSuccess)
            return MOE_ERR_CUDA;
        parts += (int)blocks_for(t.chunks);
    }
    if (!scaled || n == 0)
        return launch_kernel(true, norm_kernel, dim3(1), dim3(kThreads), 0, st, (const double *)part, parts, norm) ==
                       cudaSuccess
                   ? MOE_OK
                   : MOE_ERR_CUDA;
    for (int from = (n - 1) / kMaxTensors * kMaxTensors; from >= 0; from -= kMaxTensors) {
        collect(t, from, n - from < kMaxTensors ? n - from : kMaxTensors, types, g, out, numel);
        if (launch_kernel(true, scale_kernel, dim3(blocks_for(t.chunks)), dim3(kThreads), 0, st, t, (const double *)part, parts,
                          max_norm, eps, norm) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_grad_norm(int n, const int *types, const void *const *grads, const int64_t *numel, float *norm, void *ws,
                  size_t ws_bytes, void *stream)
{
    const int rc = check(n, types, grads, nullptr, false, numel, norm, ws, ws_bytes);
    return rc != MOE_OK ? rc
                        : run(n, types, grads, nullptr, false, numel, 0.0f, 0.0f, norm, ws,
                              static_cast<cudaStream_t>(stream));
}

int moe_clip_gradients(int n, const int *types, const void *const *grads, void *const *out, const int64_t *numel,
                       float max_norm, float eps, float *norm, void *ws, size_t ws_bytes, void *stream)
{
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f))
        return MOE_ERR_INVALID_ARG;
    const int rc = check(n, types, grads, out, true, numel, norm, ws, ws_bytes);
    return rc != MOE_OK ? rc
                        : run(n, types, grads, out, true, numel, max_norm, eps, norm, ws,
                              static_cast<cudaStream_t>(stream));
}

}  // extern "C"
