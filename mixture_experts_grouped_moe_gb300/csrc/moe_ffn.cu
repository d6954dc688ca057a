// The gated feed-forward block that every token passes (a shared expert, a dense layer), 16-bit rows:
//   h = act(x Wg^T) * (x Wu^T),   out = add + h Wd^T
// and its gradients
//   dh = dout Wd,  dg = dh u act'(g),  du = dh act(g),
//   dx = [dg | du] Wgu,  dWgu = [dg | du]^T x,  dWd = dout^T h.
// Products of dense_gemm.cuh in four launches (the three gradients in one; fp16 has one more, for the scale); the
// activation and its gradient are epilogues, and every matrix is read as it lies.  h, and in the backward [dg | du], are
// rounded to the rows' type between the products (they are operands of 16-bit MMAs): errors of half a step an element,
// independent ones, that a sum over I or T averages.  In fp16, whose smallest step is 2^-24, [dg | du] is scaled by a
// power of two first.
//
// 4096 tokens through 7168 x 2048, forward and gradients: 675-700 us replayed from a graph, 710-735 called in a row,
// where the board's power bounds it (1.60 and 1.50 PFLOP/s); forward alone see dense_gemm.cuh and, for few tokens,
// dense_few.cuh.
#include "dense_few.cuh"

namespace moe {
namespace {

using namespace dense;

// The status word; at byte 64 the inverse of the factor of d gate | d up, at 512 the parts of the largest |dout|.
constexpr int64_t kHead = 1024;
static_assert(512 + kMost * sizeof(unsigned) <= kHead, "");

int64_t up1k(int64_t v) { return (v + 1023) / 1024 * 1024; }

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

bool bad_sizes(int64_t T, int H, int I)
{
    return H % 8 != 0 || I % 8 != 0 || H > 1 << 20 || I > 1 << 20 || T > 1 << 30;
}

// Whether T rows of H 16-bit elements at `a`, lda apart, and at `b`, ldb apart, have bytes in common, except as the
// same rows.  Rows that lie between one another's in a wider buffer do not.
bool overlaps(const void *a, int64_t lda, const void *b, int64_t ldb, int64_t T, int H)
{
    const intptr_t d = reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a);  // (a multiple of 16)
    const int64_t last_a = (T - 1) * lda, last_b = (T - 1) * ldb, off = d / 2;
    if (T <= 1)
        return off != 0 && off < H && off > -H;
    if (off >= last_a + H || off + last_b + H <= 0)
        return false;
    if (lda == ldb) {
        const int64_t m = (off % lda + lda) % lda;
        return off != 0 && (m < H || m + H > lda);
    }
    for (int64_t i = 0; i < T; ++i) {  // (different pitches in one buffer: row by row)
        // rows j of a with |j lda - at| < H
        const int64_t at = off + i * ldb;
        const int64_t low = at - H < 0 ? 0 : (at - H) / lda + 1;
        if (low < T && low * lda < at + H)
            return true;
    }
    return false;
}

int to_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// The largest finite |dout| of the rows that fall to each of kMost blocks, as bits.  1 << lg threads share a row, and
// each has four rows in flight: 4096 x 7168 (58 MB) in 18 us.
constexpr int kMostThreads = 1024;
__global__ void __launch_bounds__(kMostThreads) most_kernel(const uint4 *dout, int64_t ld, int64_t T, int pieces,
                                                            int lg, unsigned *most)
{
    __shared__ unsigned warps[kMostThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & ((1 << lg) - 1);
    const int64_t step = (int64_t)kMost * (kMostThreads >> lg);
    unsigned m = 0;
    const auto look = [&](unsigned w) {
        const unsigned lo = w & 0x7fffu, hi = w >> 16 & 0x7fffu;
        m = max(m, lo < 0x7c00u ? lo : 0u);  // (not an infinity or a NaN)
        m = max(m, hi < 0x7c00u ? hi : 0u);
    };
    for (int64_t row = (int64_t)blockIdx.x * (kMostThreads >> lg) + (threadIdx.x >> lg); row < T; row += 4 * step)
        for (int i = lane; i < pieces; i += 1 << lg) {
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = row + j * step < T ? dout[(row + j * step) * ld + i] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                look(w[j].x), look(w[j].y), look(w[j].z), look(w[j].w);
        }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0)
        warps[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kMostThreads / 32; ++i)
            m = max(m, warps[i]);
        most[blockIdx.x] = m;
    }
}

template <class TE>
cudaError_t forward(const Args &base, const void *x, int64_t ld_x, const void *Wgu, const void *Wd, const void *add,
                    int64_t ld_add, int64_t T, int H, int I, int act, void *gu, void *h, void *out, int64_t ld_out,
                    cudaStream_t st)
{
    Args gated = base, down = base;
    gated.act = act, gated.h = h, gated.gu = gu;
    product(gated, T, I, H, 0, x, ld_x, Wgu, H);
    Product &q = product(down, T, H, I, 0, h, I, Wd, I);
    q.d = out, q.ld_d = ld_out, q.add = add, q.ld_add = ld_add;
    const bool few = T <= kFewMost<kGated>;
    const cudaError_t err = few ? launch_few<kGated, TE>(gated, false, st) : launch<kGated, TE>(gated, st);
    if (err != cudaSuccess)
        return err;
    // (the kernel before it waits for whatever wrote W_down, and lets this one start only then)
    return few ? launch_few<kStore, TE>(down, true, st) : launch_store<TE>(down, st);
}

template <class TE>
cudaError_t backward(const Args &base, const void *x, int64_t ld_x, const void *Wgu, const void *Wd, const void *gu,
                     const void *h, const void *dout, int64_t ld_dout, int64_t T, int H, int I, int act, void *dx,
                     int64_t ld_dx, bool f32, bool accumulate, void *dWgu, void *dWd, void *dgu,
                     cudaStream_t st)
{
    const int64_t I2 = 2 * (int64_t)I;
    float *back = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(base.status) + 64);
    if (dx || dWgu) {
        Args a = base;
        a.act = act, a.gu = const_cast<void *>(gu), a.dgu = dgu, a.back = back;
        if (kScaledGrad<TE>) {
            unsigned *most = reinterpret_cast<unsigned *>(reinterpret_cast<uint8_t *>(base.status) + 512);
            int lg = 0;
            while (lg < 9 && 1 << lg < H / 8)
                ++lg;
            const cudaError_t err =
                launch_kernel(true, most_kernel, dim3(kMost), dim3(kMostThreads), 0, st,
                              static_cast<const uint4 *>(dout), ld_dout / 8, T, H / 8, lg, most);
            if (err != cudaSuccess)
                return err;
            a.most = most;
        }
        product(a, T, I, H, 1, dout, ld_dout, Wd, I);
        const cudaError_t err = launch<kGatedBwd, TE>(a, st);
        if (err != cudaSuccess)
            return err;
    }
    Args a = base;
    if (dx) {
        Product &p = product(a, T, H, (int)I2, 1, dgu, I2, Wgu, H);
        p.d = dx, p.ld_d = ld_dx;
        p.scale = kScaledGrad<TE> ? back : nullptr;
    }
    const auto wgrad = [&](Product &p, void *dW) {
        p.d = dW, p.ld_d = p.N, p.d_f32 = f32;
        if (accumulate)
            p.add = dW, p.ld_add = p.N;
    };
    if (dWgu) {
        Product &p = product(a, I2, H, (int)T, 2, dgu, I2, x, ld_x);
        p.scale = kScaledGrad<TE> ? back : nullptr;
        wgrad(p, dWgu);
    }
    if (dWd)
        wgrad(product(a, H, I, (int)T, 2, dout, ld_dout, h, I), dWd);
    return a.n ? launch_store<TE>(a, st) : cudaSuccess;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_ffn_workspace_size(int64_t T, int H, int I, int training)
{
    if (T < 0 || H <= 0 || I <= 0 || training < 0 || training > 1 || bad_sizes(T, H, I))
        return 0;
    return (size_t)(kHead + up1k(T * I * 2 * (training ? 2 : 1)));
}

int moe_ffn(int row_type, int act, const void *x, int64_t ld_x, const void *W_gate_up, const void *W_down,
            const void *add, int64_t ld_add, int64_t T, int H, int I, void *gu, void *h, void *out, int64_t ld_out,
            void *ws, size_t ws_bytes, void *stream)
{
    if (T < 0 || H <= 0 || I <= 0 || act < 0 || act > MOE_ACT_RELU || !x || !W_gate_up || !W_down || !out || !ws ||
        ld_x < H || ld_out < H || (add && ld_add < H) || row_type < 0 || row_type > MOE_ROW_FP32 || (gu && !h))
        return MOE_ERR_INVALID_ARG;
    if (off16(x) || off16(W_gate_up) || off16(W_down) || off16(add) || off16(gu) || off16(h) || off16(out) ||
        off16(ws))
        return MOE_ERR_INVALID_ARG;
    if (row_type == MOE_ROW_FP32 || bad_sizes(T, H, I) || ld_x % 8 != 0 || ld_out % 8 != 0 ||
        (add && ld_add % 8 != 0) || ld_x > 1ll << 36 || ld_out > 1ll << 36 || ld_add > 1ll << 36)
        return MOE_ERR_UNSUPPORTED;
    if (ws_bytes < kHead + (h ? 0 : (size_t)up1k(T * I * 2)))
        return MOE_ERR_WORKSPACE;
    if (T == 0)
        return MOE_OK;
    if (add && overlaps(add, ld_add, out, ld_out, T, H))
        return MOE_ERR_INVALID_ARG;
    uint8_t *at = static_cast<uint8_t *>(ws);
    Args base = {};
    base.status = reinterpret_cast<int *>(at);
    if (!h)
        h = at + kHead;
    const auto st = static_cast<cudaStream_t>(stream);
    const auto go = row_type == MOE_ROW_BF16 ? forward<__nv_bfloat16> : forward<__half>;
    return to_status(go(base, x, ld_x, W_gate_up, W_down, add, ld_add, T, H, I, act, gu, h, out, ld_out, st));
}

int moe_ffn_backward(int row_type, int act, const void *x, int64_t ld_x, const void *W_gate_up, const void *W_down,
                     const void *gu, const void *h, const void *dout, int64_t ld_dout, int64_t T, int H, int I,
                     void *dx, int64_t ld_dx, int grad_type, int accumulate, void *dW_gate_up, void *dW_down, void *ws,
                     size_t ws_bytes, void *stream)
{
    if (T < 0 || H <= 0 || I <= 0 || act < 0 || act > MOE_ACT_RELU || !x || !W_gate_up || !W_down || !gu || !h ||
        !dout || !ws || ld_x < H || ld_dout < H || (dx && ld_dx < H) || row_type < 0 || row_type > MOE_ROW_FP32 ||
        accumulate < 0 || accumulate > 1 || (grad_type != row_type && grad_type != MOE_ROW_FP32))
        return MOE_ERR_INVALID_ARG;
    if (off16(x) || off16(W_gate_up) || off16(W_down) || off16(gu) || off16(h) || off16(dout) || off16(dx) ||
        off16(dW_gate_up) || off16(dW_down) || off16(ws))
        return MOE_ERR_INVALID_ARG;
    if (row_type == MOE_ROW_FP32 || bad_sizes(T, H, I) || ld_x % 8 != 0 || ld_dout % 8 != 0 ||
        (dx && ld_dx % 8 != 0) || ld_x > 1ll << 36 || ld_dout > 1ll << 36 || ld_dx > 1ll << 36)
        return MOE_ERR_UNSUPPORTED;
    if (ws_bytes < moe_ffn_workspace_size(T, H, I, 1))
        return MOE_ERR_WORKSPACE;
    const auto st = static_cast<cudaStream_t>(stream);
    if (T == 0) {  // no tokens: gradients of zero
        const size_t es = grad_type == MOE_ROW_FP32 ? 4 : 2, n = (size_t)H * I * es;
        cudaError_t err = cudaSuccess;
        if (!accumulate && dW_gate_up)
            err = cudaMemsetAsync(dW_gate_up, 0, 2 * n, st);
        if (!accumulate && dW_down && err == cudaSuccess)
            err = cudaMemsetAsync(dW_down, 0, n, st);
        return to_status(err);
    }
    uint8_t *at = static_cast<uint8_t *>(ws);
    Args base = {};
    base.status = reinterpret_cast<int *>(at);
    void *dgu = at + kHead;
    const auto go = row_type == MOE_ROW_BF16 ? backward<__nv_bfloat16> : backward<__half>;
    return to_status(go(base, x, ld_x, W_gate_up, W_down, gu, h, dout, ld_dout, T, H, I, act, dx, ld_dx,
                        grad_type == MOE_ROW_FP32, accumulate != 0, dW_gate_up, dW_down, dgu, st));
}

}  // extern "C"
