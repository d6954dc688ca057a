// Softmax cross entropy over a vocabulary straight from the hidden states, without keeping the logits:
//   l = x W^T,  lse_t = log sum_v exp l_tv,  loss_t = lse_t - l_t,target
// (0 where the target is outside [0, V): a row left out), and for the gradient dloss_t of each row's loss
//   dl_tv = dloss_t (exp(l_tv - lse_t) - [v = target]),  dx = dl W,  dW = dl^T x.
//
// Forward: one product whose epilogue keeps, of each 256-column tile's logits, every row's maximum and sum of
// exponentials (fp32, from the unrounded accumulators) and the target's logit; a warp a row then joins the
// tiles' pairs in a fixed order.  Backward, a piece of the vocabulary at a time: the logits are computed once
// more and leave as dl, rounded to 16 bits, which both gradients' products read; dx is summed over the pieces
// in fp32.  8 T V H operations against 6 that the gradients cannot do without: keeping fp32 logits from the forward
// would take 4 T V bytes.  (Loss and gradients in one call, whose dloss is known beforehand, could go by chunks of rows
// and keep a chunk's logits alone.)
//
// dl is scaled by a power of two to at most 2^15 (the largest finite |dloss| to [2^14, 2^15)) and the gradients
// by its inverse: a mean over many rows makes dl too small for fp16 otherwise (its smallest step, 2^-24, is then
// at most 2^-38 of the largest row's factor).
//
// Bound by the tensor pipe and in a row by the board's power: 4096 x 4096 x 32000 forward and backward 2.47-2.53 ms
// replayed from a graph, 2.67-2.78 called in a row (1.72 and 1.57 PFLOP/s with the repeated logits, 1.29 and 1.18
// without); by memory for few rows: 16 rows 48 us for 262 MB.
#include "dense_few.cuh"

namespace moe {
namespace {

using namespace dense;

constexpr int64_t kHead = 1024;  // status word; at byte 64 dl's factor and its inverse

int64_t up1k(int64_t v) { return (v + 1023) / 1024 * 1024; }
int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }

bool off(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

int to_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// A row's loss from its tiles' (maximum, sum) pairs: a warp a row.
__global__ void __launch_bounds__(256) finish_kernel(const float2 *stats, const float *target_logit,
                                                     const int32_t *targets, int64_t T, int tiles, int V, float *loss,
                                                     float *lse)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= T)
        return;
    float m = -INFINITY, s = 0.0f;
#pragma unroll 4
    for (int i = lane; i < tiles; i += 32) {
        const float2 f = stats[row * tiles + i];
        const float top = fmaxf(m, f.x), base = top == -INFINITY ? 0.0f : top;
        s = s * expf(m - base) + f.y * expf(f.x - base);
        m = top;
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, d), s2 = __shfl_xor_sync(0xffffffffu, s, d);
        const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.0f : top;
        // both lanes of a pair compute the same sum: the one of the lower lane first
        const float a = s * expf(m - base), b = s2 * expf(m2 - base);
        s = a + b;
        m = top;
    }
    if (lane == 0) {
        const float v = m + logf(s);
        const int t = targets[row];
        lse[row] = v;
        loss[row] = t >= 0 && t < V ? v - target_logit[row] : 0.0f;
    }
}

// What the backward needs before its products.  Block 0: the factor of dl, a power of two, from the largest finite
// |dloss| of the rows that count.  The others: x with zeros in the rows left out, so that whatever they hold (padding
// may be a NaN) adds nothing to dW.
__global__ void __launch_bounds__(512) prepare_kernel(const float *dloss, const int32_t *targets, int64_t T, int V,
                                                      float *factor, const uint4 *x, int64_t ld, int pieces,
                                                      uint4 *out)
{
    __shared__ float most[16];
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x > 0) {
        for (int64_t row = blockIdx.x - 1; row < T; row += gridDim.x - 1) {
            const int t = targets[row];
            const bool counts = t >= 0 && t < V;
            for (int i = threadIdx.x; i < pieces; i += 512)
                out[row * pieces + i] = counts ? x[row * ld + i] : make_uint4(0, 0, 0, 0);
        }
        return;
    }
    float m = 0.0f;
    for (int64_t i = threadIdx.x; i < T; i += 512) {
        const int t = targets[i];
        const float v = fabsf(dloss[i]);
        if (t >= 0 && t < V && v <= 3.4028235e38f)  // (not a NaN or an infinity)
            m = fmaxf(m, v);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0)
        most[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 16; ++i)
            m = fmaxf(m, most[i]);
        // 2^(14 - e) with m in [2^e, 2^(e+1)); both it and its inverse stay normal numbers
        int e = m > 0.0f ? ilogbf(m) : 0;
        e = e < -100 ? -100 : e;
        factor[0] = ldexpf(1.0f, 14 - e);
        factor[1] = ldexpf(1.0f, e - 14);
    }
}

bool bad_sizes(int64_t T, int H, int V) { return H % 8 != 0 || H > 1 << 20 || V > 1 << 24 || T > 1 << 30; }

// (maximum, sum) pairs that the forward may keep, whichever way it goes: two for a row of each 256-column tile (few
// rows: one of each 128-column tile).  Where K is split, up to eight of each 128 columns, but not more than kMostSplit
// tiles have of 256 rows with eight a row (few rows: than 32 of them have of the CTAs that run at once).  It grows with
// T and with V, so that a workspace serves smaller batches too.
int64_t pairs_of(int64_t T, int V)
{
    const int64_t whole = 2 * T * (((int64_t)V + 255) / 256), split = 8 * T * (((int64_t)V + 127) / 128);
    constexpr int64_t kMostPairs = kMostSplit * 256 * 8;
    static_assert(kMostPairs >= kFewMost<kLse> * 304, "few rows: 304 CTAs on 152 SMs");
    const int64_t most = split < kMostPairs ? split : kMostPairs;
    return whole > most ? whole : most;
}

// Byte offsets of the workspace (forward: stats and target logits; backward: dl of a piece, kept rows, dx's sum).
struct Forward {
    int64_t stats, own, total;
    Forward(int64_t T, int V)
    {
        stats = kHead;
        own = stats + up1k(pairs_of(T, V) * 8);
        total = own + up1k(T * 4);
    }
};
struct Backward {
    int64_t dl, rows, sum, total;
    Backward(int64_t T, int H, int V, int piece)
    {
        const int64_t pitch = up64(piece < V ? piece : V);
        dl = kHead;
        rows = dl + up1k(T * pitch * 2);
        sum = rows + up1k(T * H * 2);
        total = sum + (piece < V ? up1k(T * H * 4) : 0);
    }
};

template <class TE>
cudaError_t forward(const Args &base, const void *x, int64_t ld_x, const void *W, const int32_t *targets, int64_t T,
                    int H, int V, float2 *stats, float *own, float *loss, float *lse, cudaStream_t st)
{
    Args a = base;
    product(a, T, V, H, 0, x, ld_x, W, H);
    a.V = V;
    a.targets = targets, a.stats = stats, a.target_logit = own;
    const cudaError_t err = T <= kFewMost<kLse>   ? launch_few<kLse, TE>(a, false, st)
                            : H > 64 * kPart      ? launch<kLseLong, TE>(a, st)
                                                  : launch<kLse, TE>(a, st);
    if (err != cudaSuccess)
        return err;
    return launch_kernel(true, finish_kernel, dim3((unsigned)((T + 7) / 8)), dim3(256), 0, st, (const float2 *)stats,
                         (const float *)own, targets, T, a.pairs, V, loss, lse);
}

template <class TE>
cudaError_t backward(const Args &base, const void *x, int64_t ld_x, const void *W, const int32_t *targets,
                     const float *lse, const float *dloss, int64_t T, int H, int V, int piece, void *dx,
                     int64_t ld_dx, bool f32, bool accumulate, void *dW, uint8_t *ws, cudaStream_t st)
{
    const Backward L(T, H, V, piece);
    float *factor = reinterpret_cast<float *>(ws + 64);
    float *sum = reinterpret_cast<float *>(ws + L.sum);
    void *dl = ws + L.dl;
    const int64_t pitch = up64(piece < V ? piece : V);
    // (152 SMs x 4 blocks for the rows; dx alone reads x as it is)
    const int64_t blocks = !dW ? 0 : T < 608 ? T : 608;
    cudaError_t err = launch_kernel(true, prepare_kernel, dim3((unsigned)(1 + blocks)), dim3(512), 0, st, dloss, targets,
                                    T, V, factor, static_cast<const uint4 *>(x), ld_x / 8, H / 8,
                                    reinterpret_cast<uint4 *>(ws + L.rows));
    if (err != cudaSuccess)
        return err;
    const int es = f32 ? 4 : 2;
    for (int64_t v0 = 0; v0 < V; v0 += piece) {
        const int n = (int)(V - v0 < piece ? V - v0 : piece);
        const uint8_t *Wp = static_cast<const uint8_t *>(W) + v0 * H * 2;
        Args a = base;
        Product &p = product(a, T, n, H, 0, x, ld_x, Wp, H);
        a.targets = targets, a.lse = lse, a.dloss = dloss, a.dscale = factor, a.v0 = (int)v0, a.V = V;
        p.d = dl, p.ld_d = pitch;
        if ((err = H > 64 * kPart ? launch<kDlogitsLong, TE>(a, st) : launch<kDlogits, TE>(a, st)) != cudaSuccess)
            return err;
        a = base;
        if (dx) {  // the sum over the pieces, scaled back and rounded with the last one
            const bool last = v0 + n == V;
            Product &q = product(a, T, H, n, 1, dl, pitch, Wp, H);
            q.acc_in = v0 ? sum : nullptr;
            q.d = last ? dx : sum, q.ld_d = last ? ld_dx : H, q.d_f32 = !last;
            q.scale = last ? factor + 1 : nullptr;
        }
        if (dW) {
            Product &q = product(a, n, H, (int)T, 2, dl, pitch, ws + L.rows, H);
            q.d = static_cast<uint8_t *>(dW) + v0 * H * es, q.ld_d = H, q.d_f32 = f32;
            q.scale = factor + 1;
            if (accumulate)
                q.add = q.d, q.ld_add = H;
        }
        if (a.n && (err = launch_store<TE>(a, st)) != cudaSuccess)
            return err;
    }
    return err;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_vocab_loss_workspace_size(int64_t T, int H, int V, int piece)
{
    if (T < 0 || H <= 0 || V <= 0 || piece < 0 || bad_sizes(T, H, V) || (piece && piece % 64 != 0))
        return 0;
    const int64_t f = Forward(T, V).total;
    if (!piece)
        return (size_t)f;
    const int64_t b = Backward(T, H, V, piece).total;
    return (size_t)(f > b ? f : b);
}

int moe_vocab_loss(int row_type, const void *x, int64_t ld_x, const void *W, const int32_t *targets, int64_t T, int H,
                   int V, float *loss, float *lse, void *ws, size_t ws_bytes, void *stream)
{
    if (T < 0 || H <= 0 || V <= 0 || !x || !W || !targets || !loss || !lse || !ws || ld_x < H || row_type < 0 ||
        row_type > MOE_ROW_FP32)
        return MOE_ERR_INVALID_ARG;
    if (off(x, 16) || off(W, 16) || off(targets, 4) || off(loss, 4) || off(lse, 4) || off(ws, 16))
        return MOE_ERR_INVALID_ARG;
    if (row_type == MOE_ROW_FP32 || bad_sizes(T, H, V) || ld_x % 8 != 0 || ld_x > 1ll << 36)
        return MOE_ERR_UNSUPPORTED;
    const Forward L(T, V);
    if (ws_bytes < (size_t)L.total)
        return MOE_ERR_WORKSPACE;
    if (T == 0)
        return MOE_OK;
    uint8_t *at = static_cast<uint8_t *>(ws);
    Args base = {};
    base.status = reinterpret_cast<int *>(at);
    const auto go = row_type == MOE_ROW_BF16 ? forward<__nv_bfloat16> : forward<__half>;
    return to_status(go(base, x, ld_x, W, targets, T, H, V, reinterpret_cast<float2 *>(at + L.stats),
                        reinterpret_cast<float *>(at + L.own), loss, lse, static_cast<cudaStream_t>(stream)));
}

int moe_vocab_loss_backward(int row_type, const void *x, int64_t ld_x, const void *W, const int32_t *targets,
                            const float *lse, const float *dloss, int64_t T, int H, int V, int piece, void *dx,
                            int64_t ld_dx, int grad_type, int accumulate, void *dW, void *ws, size_t ws_bytes,
                            void *stream)
{
    if (T < 0 || H <= 0 || V <= 0 || piece <= 0 || !x || !W || !targets || !lse || !dloss || !ws || ld_x < H ||
        (dx && ld_dx < H) || row_type < 0 || row_type > MOE_ROW_FP32 || accumulate < 0 || accumulate > 1 ||
        (grad_type != row_type && grad_type != MOE_ROW_FP32))
        return MOE_ERR_INVALID_ARG;
    if (off(x, 16) || off(W, 16) || off(targets, 4) || off(lse, 4) || off(dloss, 4) || off(dx, 16) || off(dW, 16) ||
        off(ws, 16))
        return MOE_ERR_INVALID_ARG;
    if (row_type == MOE_ROW_FP32 || bad_sizes(T, H, V) || piece % 64 != 0 || ld_x % 8 != 0 ||
        (dx && ld_dx % 8 != 0) || ld_x > 1ll << 36 || ld_dx > 1ll << 36)
        return MOE_ERR_UNSUPPORTED;
    if (ws_bytes < (size_t)Backward(T, H, V, piece).total)
        return MOE_ERR_WORKSPACE;
    const auto st = static_cast<cudaStream_t>(stream);
    if (T == 0) {  // no rows: a gradient of zero
        if (!dW || accumulate)
            return MOE_OK;
        return to_status(cudaMemsetAsync(dW, 0, (size_t)V * H * (grad_type == MOE_ROW_FP32 ? 4 : 2), st));
    }
    uint8_t *at = static_cast<uint8_t *>(ws);
    Args base = {};
    base.status = reinterpret_cast<int *>(at);
    const auto go = row_type == MOE_ROW_BF16 ? backward<__nv_bfloat16> : backward<__half>;
    return to_status(go(base, x, ld_x, W, targets, lse, dloss, T, H, V, piece, dx, ld_dx, grad_type == MOE_ROW_FP32,
                        accumulate != 0, dW, at, st));
}

}  // extern "C"
