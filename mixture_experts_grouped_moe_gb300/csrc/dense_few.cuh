// Dense products of few rows (T <= 128 tokens): streaming the weights.  The operands are swapped: 128 weight rows
// are the MMA's M side and the tokens, rounded up to NP = 16, 32, 64 or 128, its N side, so that nothing is padded
// to 256 rows and a stage of the pipeline is nearly all weights.  A gated tile holds 64 gate rows and the matching
// 64 up rows, so that both products of a column end in one CTA.
//
// A CTA does one tile, or, with few tiles, 1/S of a tile's K: the S <= 8 CTAs of a cluster add their fp32 parts
// through distributed shared memory (each gets the parts of 128/S rows, adds them in ascending order and applies
// the epilogue).  Two CTAs fit an SM (about 100 KB each, up to 64 tokens), so that up to 304 tiles or parts stream
// at once, and a kernel that follows in the same call starts while this one still runs: it brings its first
// stages of weights before it waits for the tokens (griddepcontrol.wait).
//
// Bound by memory: while it streams, 6.9 TB/s; a gated block's two products for 32 tokens, 4096 x 14336 (352 MB), 60-62
// us, for one token, 7168 x 2048 (88 MB), 21.4.  One deep CTA an SM took 84 us for the first, a split of the second
// product in 4 parts instead of 8 74, rings of 3 stages 69, loads in groups of 2 or 4 blocks 69 and 74.
#pragma once

#include "dense_gemm.cuh"

namespace moe {
namespace dense {

// The most tokens that go this way (us here / by pair tiles: 80 tokens through 4096 x 14336 82 / 94, through 1024 x
// 4096 16.4 / 22.0, 128 through 7168 x 2048 29.2 / 39.8).  Logits up to 32: their epilogue takes a warp a token
// (4096 x 32000: 16 rows 49, 64 rows 62 / 55, 128 rows 107 / 54).
template <int MODE>
constexpr int64_t kFewMost = MODE == kLse ? 32 : 128;
constexpr int kFewThreads = 192;

template <int NP>
constexpr int kFewStageBytes = 16384 + NP * 128;
template <int NP>
constexpr int kFewStages = NP == 16 ? 5 : NP == 32 ? 4 : NP == 64 ? 3 : 4;

// Logits are summed in parts of K here too, at no cost.
template <int MODE>
constexpr bool kFewInParts = MODE == kLse;

template <int NP>
struct __align__(1024) FewSmem {
    uint8_t stage[kFewStages<NP>][kFewStageBytes<NP>];
    float red[128 * NP];  // [S][NP][128 / S]: every CTA's part of the rows that this one finishes
    uint64_t full[kFewStages<NP>];
    uint64_t empty[kFewStages<NP>];
    uint64_t done[2];     // the accumulator (of a part of K) is complete
    uint64_t read[2];     // and has been read
    uint32_t tmem_base;
    int abort;
};
template <int NP>
constexpr size_t kFewSmemBytes = sizeof(FewSmem<NP>) + 1024;
static_assert(2 * (kFewSmemBytes<16> + 1024) <= 228 * 1024 && 2 * (kFewSmemBytes<32> + 1024) <= 228 * 1024 &&
                  2 * (kFewSmemBytes<64> + 1024) <= 228 * 1024 && kFewSmemBytes<128> <= 227 * 1024,
              "two CTAs an SM up to 64 tokens");

// p[0].tm_a: tokens in boxes of 64 x NP; tm_b: weights in boxes of 64 x (gated 64, else 128); M tokens, N
// features, S CTAs a tile.  early: the weights may be read before what precedes the kernel has ended.
template <int MODE, class TE, int NP>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const __grid_constant__ Args a, int early)
{
    using SmemT = FewSmem<NP>;
    constexpr int kS = kFewStages<NP>;
    constexpr int kTile = MODE == kGated ? 64 : 128;  // features of a tile
    constexpr int kColumns = kFewInParts<MODE> ? 2 * NP : NP < 32 ? 32 : NP;  // of TMEM
    extern __shared__ uint8_t smem_raw[];
    SmemT &sm = *reinterpret_cast<SmemT *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Product &p = a.p[0];
    const int S = a.S;
    const int rank = blockIdx.x % S, tile = blockIdx.x / S;
    volatile int *abort_flag = &sm.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kS; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.done[i], 1);
            mbar_init(&sm.read[i], 4);
        }
        sm.abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&p.tm_a);
        tma_prefetch_desc(&p.tm_b);
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, kColumns);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // every CTA of the cluster has started before any of them writes to another's shared memory
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const uint32_t tmem_base = sm.tmem_base;
    const int nkb = (p.K + 63) / 64;
    const int kb0 = (int)((int64_t)nkb * rank / S), kb1 = (int)((int64_t)nkb * (rank + 1) / S);
    bool ok = true;
    int targets = -1;  // logits: those of this warp's tokens, one a lane

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
            const auto weights = [&](int s, int kb) {
                mbar_arrive_expect_tx(&sm.full[s], kFewStageBytes<NP>);
                tma_load_2d(sm.stage[s], &p.tm_b, kb * 64, tile * kTile, &sm.full[s], once);
                if (MODE == kGated)
                    tma_load_2d(sm.stage[s] + 8192, &p.tm_b, kb * 64, p.N + tile * kTile, &sm.full[s], once);
            };
            const auto tokens = [&](int s, int kb) {
                tma_load_2d(sm.stage[s] + 16384, &p.tm_a, kb * 64, 0, &sm.full[s], keep);
            };
            const int pre = early ? min(kS, kb1 - kb0) : 0;
            for (int i = 0; i < pre; ++i)
                weights(i, kb0 + i);
            pdl_wait();
            for (int i = 0; i < pre; ++i)
                tokens(i, kb0 + i);
            int s = pre % kS;
            uint32_t ph = pre / kS;
            for (int kb = kb0 + pre; kb < kb1; ++kb) {
                if (!mbar_wait(&sm.empty[s], ph ^ 1, a.status, abort_flag)) {
                    // copies in flight: a bounded moment for them to land
                    const unsigned long long t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < 20000000ull) {
                    }
                    break;
                }
                weights(s, kb);
                tokens(s, kb);
                if (++s == kS) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // (the tokens come after this wait: the limit of the waits below counts from here, not from a start that
            // may be long before the end of what precedes the kernel)
            pdl_wait();
            const uint32_t type = std::is_same<TE, __nv_bfloat16>::value ? 1u : 0u;
            const uint32_t idesc = make_idesc(type, type, 128, NP);
            int s = 0, acc = 0;
            uint32_t ph = 0;
            const int part = kFewInParts<MODE> ? kPart : kb1 - kb0;
            bool fine = true;
            for (int k0 = kb0, n = 0; fine && k0 < kb1; k0 += part, ++n) {
                acc = kFewInParts<MODE> ? n & 1 : 0;
                // (two parts go ahead; the third waits until the first has been read)
                if (n >= 2 && !mbar_wait(&sm.read[acc], (n / 2 - 1) & 1, a.status, abort_flag))
                    break;
                tc_fence_after();
                const int k1 = min(k0 + part, kb1);
                for (int kb = k0; kb < k1; ++kb) {
                    if (!mbar_wait(&sm.full[s], ph, a.status, abort_flag)) {
                        fine = false;
                        break;
                    }
                    tc_fence_after();
                    const uint8_t *w = sm.stage[s], *x = sm.stage[s] + 16384;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16(tmem_base + acc * NP, smem_desc_sw128(w + kk * 32), smem_desc_sw128(x + kk * 32),
                                 idesc, (kb > k0 || kk > 0) ? 1u : 0u);
                    mma_commit(&sm.empty[s]);
                    if (++s == kS) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                mma_commit(&sm.done[acc]);
            }
        }
    } else {
        pdl_wait();
        pdl_trigger();
        const int q = warp & 3;
        const int r = q * 32 + lane;  // weight row
        if (MODE == kLse && warp - 2 + 4 * lane < (int)p.M)
            targets = a.targets[warp - 2 + 4 * lane];
        const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16);
        constexpr int kC = NP < 32 ? 16 : 32;
        float sums[kFewInParts<MODE> ? NP : 1];
        if constexpr (kFewInParts<MODE>) {
            for (int k0 = kb0, n = 0; k0 < kb1; k0 += kPart, ++n) {
                ok = mbar_wait(&sm.done[n & 1], (n / 2) & 1, a.status, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after();
                float f[kC];
                static_assert(kC == NP, "one load");
                if constexpr (kC == 16)
                    tmem_ld16(tacc + (n & 1) * NP, f);
                else
                    tmem_ld32(tacc + (n & 1) * NP, f);
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    sums[i] = n == 0 ? f[i] : sums[i] + f[i];
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.read[n & 1]);
            }
        } else {
            ok = mbar_wait(&sm.done[0], 0, a.status, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        }
        // rows that a CTA of the cluster finishes: 128 / S consecutive ones, gated as many gate rows and up rows
        const int own = 128 / S;
        int owner, local;
        if (MODE == kGated) {
            const int half = own / 2;
            owner = r % 64 / half;
            local = r / 64 * half + r % half;
        } else {
            owner = r / own;
            local = r % own;
        }
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        const uint32_t dst = cluster_map(sm.red, owner) + (uint32_t)((rank * NP * own + local) * 4);
#pragma unroll 1
        for (int c = 0; c < NP; c += kC) {
            float v[kC];
            if constexpr (kFewInParts<MODE>) {
#pragma unroll
                for (int i = 0; i < kC; ++i)
                    v[i] = sums[i];
            } else if constexpr (kC == 16)
                tmem_ld16(tacc + c, v);
            else
                tmem_ld32(tacc + c, v);
#pragma unroll
            for (int i = 0; i < kC; ++i)
                if (c + i < p.M)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + (uint32_t)((c + i) * own * 4)),
                                 "f"(v[i])
                                 : "memory");
        }
        tc_fence_before();
    }
    __syncwarp();
    if (warp < 2)
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    cluster_sync();  // every part has arrived; (S = 1: the block's own barrier)
    if (warp >= 2 && ok) {
        // An item is 8 consecutive features of a token: 16-byte loads and stores (element by element, with the
        // loads of `add` one after the other, this took 3 to 14 us).
        const int own = 128 / S;
        const auto sum8 = [&](int col, int local, float(&v)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = 0.0f;
            for (int s = 0; s < S; ++s) {
                const float4 *part = reinterpret_cast<const float4 *>(sm.red + (s * NP + col) * own + local);
                const float4 f = part[0], g = part[1];
                v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
                v[4] += g.x, v[5] += g.y, v[6] += g.z, v[7] += g.w;
            }
        };
        if (MODE == kGated) {
            const int half = own / 2, groups = half / 8, f0 = tile * 64 + rank * half;
            for (int e = threadIdx.x - 64; e < groups * (int)p.M; e += 128) {
                const int i = e % groups * 8, col = e / groups, f = f0 + i;
                if (f >= p.N)
                    continue;
                float g[8], u[8], h[8];
                sum8(col, i, g);
                sum8(col, half + i, u);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    h[j] = g[j];
                gate(a.act, h, u);
                store8(static_cast<TE *>(a.h) + (int64_t)col * p.N + f, h);
                if (a.gu) {
                    TE *kept = static_cast<TE *>(a.gu) + (int64_t)col * 2 * p.N + f;
                    store8(kept, g);
                    store8(kept + p.N, u);
                }
            }
        } else if (MODE == kStore) {
            const int groups = own / 8, f0 = tile * 128 + rank * own;
            for (int e = threadIdx.x - 64; e < groups * (int)p.M; e += 128) {
                const int i = e % groups * 8, col = e / groups, f = f0 + i;
                if (f >= p.N)
                    continue;
                float v[8], add[8] = {};
                if (p.add)
                    load8(static_cast<const TE *>(p.add) + col * p.ld_add + f, add);
                sum8(col, i, v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] += add[j];
                store8(static_cast<TE *>(p.d) + col * p.ld_d + f, v);
            }
        } else {
            // logits: a warp a token, its maximum and sum of exponentials over the rows finished here
            const int f0 = tile * 128 + rank * own;
            for (int col = warp - 2; col < (int)p.M; col += 4) {
                const int target = __shfl_sync(0xffffffffu, targets, col / 4);
                float v[4], m = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = lane + 32 * j;
                    v[j] = -INFINITY;
                    if (i < own && f0 + i < p.N) {
                        v[j] = 0.0f;
                        for (int s = 0; s < S; ++s)
                            v[j] += sm.red[(s * NP + col) * own + i];
                        if (f0 + i == target)
                            a.target_logit[col] = v[j];
                    }
                    m = fmaxf(m, v[j]);
                }
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1)
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                const float base = m == -INFINITY ? 0.0f : m * kLog2e;
                float s = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s += exp2_fast(fmaf(v[j], kLog2e, -base));
                s = warp_sum(s);
                if (lane == 0)
                    a.stats[(int64_t)col * a.pairs + tile * S + rank] = make_float2(m, s);
            }
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem_base, kColumns);
}

// ------------------------------------------------------------------- host

// CTAs that share a tile: doubled while all parts run at once (`slots`) and each keeps at least four blocks of K (us
// for one token through 7168 x 2048 with 1, 2, 4, 8 parts in the first product and 4 in the second: 42.0, 28.1, 22.0,
// 21.1; 32 tokens through 4096 x 14336 with 1, 2, 4, 8 in the second: 126, 90, 74, 68).
inline int few_split(int64_t tiles, int K, int slots)
{
    int S = 1;
    while (S < 8 && tiles * 2 * S <= slots && (K + 63) / 64 / (2 * S) >= 4)
        S *= 2;
    return S;
}

template <int MODE, class TE, int NP>
cudaError_t launch_few_np(Args &a, bool early, cudaStream_t st)
{
    constexpr int kTile = MODE == kGated ? 64 : 128;
    auto kern = few_kernel<MODE, TE, NP>;
    const int sms = num_sms_current_device();
    if (sms <= 0)
        return cudaErrorInvalidConfiguration;
    Product &p = a.p[0];
    p.tiles_n = (p.N + kTile - 1) / kTile;
    p.tiles_m = 1;
    a.S = few_split(p.tiles_n, p.K, sms * (NP <= 64 ? 2 : 1));
    a.pairs = p.tiles_n * a.S;
    const int64_t w_rows = MODE == kGated ? 2 * (int64_t)p.N : p.N;
    if (!encode_tmap_2d_pitched(&p.tm_a, p.A, 2, p.K, p.M, p.ld_a, 64, NP) ||
        !encode_tmap_2d_pitched(&p.tm_b, p.B, 2, p.K, w_rows, p.ld_b, 64, kTile))
        return cudaErrorInvalidValue;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewSmemBytes<NP>);
    if (err != cudaSuccess)
        return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.tiles_n * a.S));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = kFewSmemBytes<NP>;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a, early ? 1 : 0);
}

// The product p[0] of M <= kFewMost<MODE> tokens (A) with weights (B).
template <int MODE, class TE>
cudaError_t launch_few(Args &a, bool early, cudaStream_t st)
{
    const int64_t T = a.p[0].M;
    if constexpr (kFewMost<MODE> > 32)
        if (T > 32)
            return T <= 64 ? launch_few_np<MODE, TE, 64>(a, early, st) : launch_few_np<MODE, TE, 128>(a, early, st);
    return T <= 16 ? launch_few_np<MODE, TE, 16>(a, early, st) : launch_few_np<MODE, TE, 32>(a, early, st);
}

}  // namespace dense
}  // namespace moe
