// Rows of bf16, fp16 or fp32 elements for the operators around the layer (token exchange, norms):
// element conversion (arithmetic is fp32) and the aligned pieces a thread loads and stores at once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace moe {

__device__ __forceinline__ float row_to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float row_to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float row_to_f(float v) { return v; }
template <typename T>
__device__ __forceinline__ T row_from_f(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 row_from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half row_from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float row_from_f<float>(float v) { return v; }

// VEC consecutive elements, moved by one load or store (VEC * sizeof(T) of 2, 4 or 16 bytes).
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Piece {
    T e[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> piece_zero()
{
    Piece<T, VEC> p;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        p.e[i] = row_from_f<T>(0.0f);
    return p;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Whether rows of `row_bytes` at pitch `pitch_bytes` from p start and end on 16-byte boundaries.
inline bool rows_aligned16(const void *p, int64_t pitch_bytes, int64_t row_bytes)
{
    return ((reinterpret_cast<uintptr_t>(p) | (uint64_t)pitch_bytes | (uint64_t)row_bytes) & 15) == 0;
}

}  // namespace moe
