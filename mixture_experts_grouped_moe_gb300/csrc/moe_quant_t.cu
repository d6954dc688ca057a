// Transposing FP8 quantiser: the operands of a block-scaled FP8 weight gradient, whose products run
// along the tokens.  For each column c of X and each 128 rows r it takes scale = amax / 448 (1 for an
// all-zero group) and codes e4m3(v / scale) (round to nearest even, saturating), as the row
// quantiser does along a row, and stores q[c][r] and s[r/128][c].  Rows may be gathered through the
// sort's sorted_ids (row p is token sorted_ids[p] / k of X, zero for padding), so the experts' order
// needs no copy of X.
//
// Two bytes read and one written per element.  A block turns 128 rows x 64 columns in shared memory; eight
// threads share a pair of columns, 16 rows each in registers between the maximum and the codes, and store 16
// codes a column at once (128 bytes of a column by its eight threads).  A row is 33 words, so row and pair r
// and p lie in bank r + p: the threads start their rows rotated by 4 * (sub / 2), which spreads a warp's loads
// over all banks.
// Bound by the latency of a block's loads, barrier and stores, so by the blocks that are resident: 8192 x 14336
// in 109 us (3.2 TB/s) with five an SM (48 registers), 143 with the three of 78 registers, 143 with seven.
#include <cuda_fp8.h>

#include "moe_internal.h"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kCols = 64;
constexpr int kPitch = kCols + 2;  // 33 words: consecutive rows fall on consecutive banks

__global__ void __launch_bounds__(256, 5) quant_t_kernel(const __nv_bfloat16 *__restrict__ X, int64_t ld,
                                                     const int32_t *__restrict__ sorted_ids, int S, int k,
                                                     const int32_t *__restrict__ nrows, int64_t R, int64_t ld_q,
                                                     int C, uint8_t *__restrict__ q, float *__restrict__ s)
{
    __shared__ __align__(16) uint16_t tile[128 * kPitch];
    pdl_wait();
    pdl_trigger();
    int64_t rows = R;
    if (nrows) {
        const int64_t n = *nrows;
        rows = n < 0 ? 0 : n < R ? n : R;
    }
    const int c0 = blockIdx.x * kCols;
    for (int64_t r0 = (int64_t)blockIdx.y * 128; r0 < rows; r0 += (int64_t)gridDim.y * 128) {
        __syncthreads();  // the previous tile has been read
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rr = threadIdx.x / 8 + 32 * i, cc = threadIdx.x % 8 * 8;
            const int64_t r = r0 + rr;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows && c0 + cc < C) {
                int64_t src = r;
                if (sorted_ids) {
                    const int slot = sorted_ids[r];
                    src = (unsigned)slot < (unsigned)S ? slot / k : -1;
                }
                if (src >= 0)
                    v = __ldg(reinterpret_cast<const uint4 *>(X + src * ld + c0 + cc));
            }
            uint32_t *d = reinterpret_cast<uint32_t *>(tile + rr * kPitch + cc);
            d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
        }
        __syncthreads();
        const int pair = threadIdx.x / 8, sub = threadIdx.x % 8, turn = sub / 2;
        __nv_bfloat162 v[16];  // rows sub * 16 + (i + 4 turn) % 16 of the two columns
        __nv_bfloat162 top = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int row = sub * 16 + ((i + 4 * turn) & 15);
            v[i] = reinterpret_cast<const __nv_bfloat162 *>(tile)[row * (kPitch / 2) + pair];
            top = __hmax2(top, __habs2(v[i]));
        }
#pragma unroll
        for (int d = 1; d <= 4; d <<= 1)
            top = __hmax2(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (c0 + 2 * pair >= C)  // (C is even)
            continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t c = c0 + 2 * pair + h;
            const float amax = h ? __high2float(top) : __low2float(top);
            const float sc = amax > 0.0f ? amax / 448.0f : 1.0f;
            float f[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                f[i] = h ? __high2float(v[i]) : __low2float(v[i]);
            divide16(f, sc);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo =
                    __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi =
                    __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
                w[i] = lo | (hi << 16);
            }
            // word i holds rows 4 ((i + turn) % 4) on: turn them back
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = turn & 1 ? w[(i + 3) & 3] : w[i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = turn & 2 ? x[(i + 2) & 3] : x[i];
            *reinterpret_cast<uint4 *>(q + c * ld_q + r0 + sub * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            if (sub == 0)
                s[r0 / 128 * C + c] = sc;
        }
    }
}

}  // namespace

}  // namespace moe

extern "C" int moe_quantize_fp8_act_t(const void *X, int64_t ld_x, int64_t R, int C, const int32_t *sorted_ids, int S,
                                      int k, const int32_t *num_rows, uint8_t *q, int64_t ld_q, float *s,
                                      void *stream)
{
    using namespace moe;
    if (R < 0 || C <= 0 || ld_x < C || !X || !q || !s || ld_q < (R + 127) / 128 * 128 ||
        (sorted_ids && (S < 0 || k <= 0)))
        return MOE_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(q)) & 15) ||
        (reinterpret_cast<uintptr_t>(s) & 3))
        return MOE_ERR_INVALID_ARG;
    if (C % 8 != 0 || ld_x % 8 != 0 || ld_q % 16 != 0 || R > INT32_MAX)
        return MOE_ERR_UNSUPPORTED;
    if (R == 0)
        return MOE_OK;
    const int64_t nb = (R + 127) / 128;
    const cudaError_t err =
        launch_kernel(true, quant_t_kernel, dim3((C + kCols - 1) / kCols, (unsigned)(nb < 65535 ? nb : 65535)),
                      dim3(256), 0, static_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16 *>(X), ld_x,
                      sorted_ids, S, k, num_rows, R, ld_q, C, q, s);
    return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
