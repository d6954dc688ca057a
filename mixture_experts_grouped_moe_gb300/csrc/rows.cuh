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

// VEC consecutive elements, moved by one load or store: 16 bytes, or one element.  (The 16 bytes are
// kept as words: as an array of elements the compiler moves them one by one.)
template <typename T, int VEC>
struct Piece {
    static_assert(VEC * sizeof(T) == 16, "16 bytes, or one element");
    uint4 w;
};
template <typename T>
struct Piece<T, 1> {
    T e;
};

__device__ __forceinline__ void unpack_word(uint32_t w, float &lo, float &hi, __nv_bfloat16)
{
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack_word(uint32_t w, float &lo, float &hi, __half)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    lo = f.x, hi = f.y;
}
__device__ __forceinline__ uint32_t pack_word(float lo, float hi, __nv_bfloat16)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t pack_word(float lo, float hi, __half)
{
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Piece<T, VEC> &p, float (&f)[VEC])
{
    if constexpr (VEC == 1) {
        f[0] = row_to_f(p.e);
    } else if constexpr (sizeof(T) == 4) {
        f[0] = __uint_as_float(p.w.x), f[1] = __uint_as_float(p.w.y);
        f[2] = __uint_as_float(p.w.z), f[3] = __uint_as_float(p.w.w);
    } else {
        unpack_word(p.w.x, f[0], f[1], T{});
        unpack_word(p.w.y, f[2], f[3], T{});
        unpack_word(p.w.z, f[4], f[5], T{});
        unpack_word(p.w.w, f[6], f[7], T{});
    }
}

// Each element rounded to nearest even.
template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> pack(const float (&f)[VEC])
{
    Piece<T, VEC> p;
    if constexpr (VEC == 1) {
        p.e = row_from_f<T>(f[0]);
    } else if constexpr (sizeof(T) == 4) {
        p.w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
        p.w = make_uint4(pack_word(f[0], f[1], T{}), pack_word(f[2], f[3], T{}), pack_word(f[4], f[5], T{}),
                         pack_word(f[6], f[7], T{}));
    }
    return p;
}

template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> piece_zero()
{
    Piece<T, VEC> p;
    if constexpr (VEC == 1)
        p.e = row_from_f<T>(0.0f);
    else
        p.w = make_uint4(0, 0, 0, 0);
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

// v / sc for many v by one divisor, correctly rounded: q = fma(fma(-q0, sc, v), r, q0) with q0 = v r and r
// = 1 / sc correctly rounded (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990), three instructions instead of a division.  It needs the remainder
// v - q0 sc to be exact, which holds for every quotient that does not encode to zero (|q| >= 2^-11) while
// sc >= 2^-90; other divisors take the division.
__device__ __forceinline__ void divide16(float (&f)[16], float sc)
{
    if (sc >= 0x1p-90f && sc <= 0x1p120f) {
        const float r = 1.0f / sc;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float q0 = f[i] * r;
            f[i] = fmaf(fmaf(-q0, sc, f[i]), r, q0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            f[i] /= sc;
    }
}

}  // namespace moe
