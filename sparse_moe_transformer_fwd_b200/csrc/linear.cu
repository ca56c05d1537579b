// Block-scaled e4m3 matrix product for few rows of activations:
//   out[t, n] = sum_kb s_a[t, kb] s_w[n / 128, kb] * (sum_{i in kb} a[t, i] w[n, i])  (+ residual[t, n])
// with a [T, K] codes in 1x128 tiles and w [N, K] codes in 128x128 blocks
// ("DeepSeek-R1" (aguasto.com), "Quantization": blockwise FP8), each 128-wide
// K block accumulated by the tensor core and added in binary32, as in the
// grouped expert GEMMs.
//
// Up to 64 tokens the product reads each weight byte for at most 128 FLOP, so
// it is bound by HBM: N*K bytes of weights.  The weights are therefore the M
// operand of the MMA (128 rows of W a tile, tokens the N operand: 16, 32 or 64
// columns), and what is split over the SMs is the weight stream itself: its
// (tile, K block) pairs are numbered tile by tile and every CTA takes an equal,
// contiguous share, whatever N and K are.  A tile that several CTAs share is
// finished by whichever of them is last: each stores its binary32 partial sums
// in the workspace and counts itself in; the last one adds them in K order, so
// the result does not depend on timing.
//   warp 0      TMA producer: two K blocks a stage (two 16 KB boxes of W, two
//               boxes of activations)
//   warp 1      TMEM allocator and MMA issuer: a stage's two K blocks go to two
//               adjacent accumulators of one of NBUF TMEM buffers
//   warp 2      scales of each K block, copied to a ring in shared memory with
//               cp.async (rows past T: zeros)
//   warps 4-7   epilogue: thread = weight row; adds each accumulator, times its
//               scale product, to the token sums in registers
// Every wait is bounded; on expiry the block records MOE_ERR_TIMEOUT, counts
// itself in on its tiles without adding (so the counters return to zero),
// drains its loads and MMAs, frees its TMEM and exits.
#include "common.cuh"
#include "kernels.h"
#include "quant_math.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int LS_THREADS = 256;
constexpr int W_BYTES = 128 * 128;  // one tile of weights
constexpr int NBUF = 4;             // TMEM buffers of two accumulators
constexpr int SC_RING = 8;          // scale slots (two K blocks each)

template <int NT>
struct LinearSmem {
    static constexpr int X_BYTES = NT * 128;
    static constexpr int STAGES = NT == 16 ? 6 : (NT == 32 ? 5 : 4);
    alignas(1024) uint8_t w[STAGES][2][W_BYTES];
    alignas(1024) uint8_t x[STAGES][2][X_BYTES];
    struct alignas(16) Scales {
        float x[2][NT];
        float w[2];
        float pad[2];
    } sc[SC_RING];
    uint64_t full[STAGES], empty[STAGES];
    uint64_t sfull[SC_RING], sempty[SC_RING];
    uint64_t tfull[NBUF], tempty[NBUF];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
    int last;
};

struct LinearParams {
    const float *a_scales, *w_scales;
    const uint16_t *residual;  // bf16 [T, N] or NULL
    void *out;                 // [T, N] bf16, or binary32 (out_f32)
    float *partial;            // [gridDim.x][2][NT][128]
    int *counters;             // [tiles], zero between launches
    int *status;
    int T, N, KB, tiles;
    int out_f32;
    int w_rowmajor;
};

// K blocks [first, first + count) of one tile: a CTA's share of that tile.
struct Segment {
    int tile, kb0, nk;
};

// The share [u0, u1) of CTA c among G: (tile, K block) pairs in tile order.
__device__ __forceinline__ long long share_begin(long long U, int c, int G) { return U * c / G; }
// The CTA whose share holds pair u.
__device__ __forceinline__ int share_of(long long U, long long u, int G) {
    return static_cast<int>(((u + 1) * G + U - 1) / U) - 1;
}

__device__ __forceinline__ float bf16_f(uint16_t v) {
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ void store_out(const LinearParams &p, size_t at, float v, float res) {
    if (p.residual) v = __fadd_rn(v, res);
    if (p.out_f32) static_cast<float *>(p.out)[at] = v;
    else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(v);
}

// Finishes a shared tile: the sums of its `shares` CTAs c0, c0 + 1, ... added
// in that (K) order.  Warp q takes tokens q, q + 4, ..., lane l rows 4l .. 4l
// + 3, and the loads of eight shares (or as many tokens) are in flight
// together: one load at a time cost 0.5 us a share (6 us at one token, K =
// 7168, N = 2112, against 3 us for the whole weight stream).
template <int NT>
__device__ __forceinline__ void add_shares(const LinearParams &p, long long U, int tile, int c0, int shares,
                                           int q, int lane) {
    const int KB = p.KB, G = gridDim.x;
    // Every share but the first one's begins on this tile: its first segment,
    // slot 0.  The first CTA's is its last segment unless it began here too.
    const int slot0 = share_begin(U, c0, G) / KB == tile ? 0 : 1;
    const float4 *base = reinterpret_cast<const float4 *>(p.partial) + static_cast<size_t>(c0) * 2 * NT * 32 + lane;
    const int n0 = tile * 128 + lane * 4;
    for (int t = q; t < p.T; t += 4) {
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        uint16_t res[4] = {0, 0, 0, 0};
        const size_t at = static_cast<size_t>(t) * p.N + n0;
        if (p.residual)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n0 + i < p.N) res[i] = p.residual[at + i];
        for (int c = 0; c < shares; c += 8) {
            float4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < shares)
                    v[i] = __ldcg(base + (static_cast<size_t>(c + i) * 2 + (c + i == 0 ? slot0 : 0)) * NT * 32 + t * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (c + i >= shares) break;
                acc.x = __fadd_rn(acc.x, v[i].x);
                acc.y = __fadd_rn(acc.y, v[i].y);
                acc.z = __fadd_rn(acc.z, v[i].z);
                acc.w = __fadd_rn(acc.w, v[i].w);
            }
        }
        const float f[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n0 + i < p.N) store_out(p, at + i, f[i], bf16_f(res[i]));
    }
}

template <int NT>
__global__ void __launch_bounds__(LS_THREADS, 1)
linear_stream_kernel(const __grid_constant__ CUtensorMap tmap_x,
                     const __grid_constant__ CUtensorMap tmap_w, const LinearParams p) {
    using S = LinearSmem<NT>;
    constexpr int STAGES = S::STAGES;
    constexpr int TMEM_COLS = NBUF * 2 * NT;  // 128, 256 or 512
    extern __shared__ uint8_t smem_raw[];
    S &s = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int KB = p.KB;
    const long long U = static_cast<long long>(p.tiles) * KB;
    const long long u0 = share_begin(U, blockIdx.x, gridDim.x), u1 = share_begin(U, blockIdx.x + 1, gridDim.x);

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < SC_RING; ++i) {
            mbar_init(&s.sfull[i], 32);
            mbar_init(&s.sempty[i], 4);
        }
        for (int i = 0; i < NBUF; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 4);
        }
        mbar_init(&s.mma_done, 1);
        s.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&tmap_x);
        prefetch_tmap(&tmap_w);
    }
    if (warp == 1) {
        tmem_alloc(&s.tmem_base, TMEM_COLS);
        tmem_relinquish();
    }
    pdl_wait_and_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = s.tmem_base;
    volatile int *abort = &s.abort;

    auto next_segment = [&](long long &u, Segment &g) {
        if (u >= u1) return false;
        g.tile = static_cast<int>(u / KB);
        g.kb0 = static_cast<int>(u - static_cast<long long>(g.tile) * KB);
        g.nk = static_cast<int>(min(static_cast<long long>(KB - g.kb0), u1 - u));
        u += g.nk;
        return true;
    };

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, armed = 0, armed_phase = 0;
            bool ok = true;
            long long u = u0;
            Segment g;
            while (ok && next_segment(u, g)) {
                for (int kb = g.kb0; kb < g.kb0 + g.nk; kb += 2) {
                    const int n = min(2, g.kb0 + g.nk - kb);
                    if (!mbar_wait(&s.empty[stage], phase ^ 1, abort, p.status)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&s.full[stage], n * (W_BYTES + S::X_BYTES));
                    for (int j = 0; j < n; ++j) {
                        if (p.w_rowmajor)
                            tma_load_2d(s.w[stage][j], &tmap_w, (kb + j) * 128, g.tile * 128, &s.full[stage]);
                        else
                            tma_load_2d(s.w[stage][j], &tmap_w, 0, (g.tile * KB + kb + j) * 128, &s.full[stage]);
                        tma_load_2d(s.x[stage][j], &tmap_x, (kb + j) * 128, 0, &s.full[stage]);
                    }
                    armed |= 1u << stage;
                    armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // drain: every load issued has landed before the block exits
            const long long t0 = clock64();
            for (int i = 0; i < STAGES; ++i) {
                if (!(armed >> i & 1)) continue;
                while (!mbar_try_wait(&s.full[i], armed_phase >> i & 1)) {
                    if (clock64() - t0 > kWaitBudgetCycles) {
                        set_status(p.status, MOE_ERR_TIMEOUT);
                        break;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = instr_desc<true>(128, NT);
            int stage = 0, tb = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true;
            long long u = u0;
            Segment g;
            while (ok && next_segment(u, g)) {
                for (int i = 0; i < g.nk; i += 2) {
                    const int n = min(2, g.nk - i);
                    if (!mbar_wait(&s.tempty[tb], tphase ^ 1, abort, p.status) ||
                        !mbar_wait(&s.full[stage], phase, abort, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    for (int j = 0; j < n; ++j) {
                        const uint32_t d = tmem_base + (2 * tb + j) * NT;
                        const uint64_t wd = smem_desc_sw128(smem_u32(s.w[stage][j]));
                        const uint64_t xd = smem_desc_sw128(smem_u32(s.x[stage][j]));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) tc_mma<true>(d, wd + 2 * kk, xd + 2 * kk, idesc, kk != 0);
                    }
                    tc_commit(&s.empty[stage]);
                    tc_commit(&s.tfull[tb]);
                    if (++tb == NBUF) {
                        tb = 0;
                        tphase ^= 1;
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // all MMAs issued are complete before TMEM is freed
            tc_commit(&s.mma_done);
            const long long t0 = clock64();
            while (!mbar_try_wait(&s.mma_done, 0)) {
                if (clock64() - t0 > kWaitBudgetCycles) {
                    set_status(p.status, MOE_ERR_TIMEOUT);
                    break;
                }
            }
        }
    } else if (warp == 2) {
        // lane l copies the scales of tokens l, l + 32 (of both K blocks) and
        // lanes 0, 1 the weights' (their barrier counts 32 arrivals, one a
        // lane, each made when that lane's copies have landed)
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        long long u = u0;
        Segment g;
        while (ok && next_segment(u, g)) {
            for (int kb = g.kb0; kb < g.kb0 + g.nk; kb += 2) {
                const int n = min(2, g.kb0 + g.nk - kb);
                int go = 1;
                if (lane == 0) go = mbar_wait(&s.sempty[slot], phase ^ 1, abort, p.status) ? 1 : 0;
                if (__shfl_sync(0xffffffffu, go, 0) == 0) {
                    ok = false;
                    break;
                }
                for (int j = 0; j < n; ++j) {
                    for (int t = lane; t < NT; t += 32) {
                        const bool in = t < p.T;
                        cp_async4(&s.sc[slot].x[j][t],
                                  p.a_scales + (in ? static_cast<size_t>(t) * KB + kb + j : 0), in);
                    }
                }
                if (lane < n)
                    cp_async4(&s.sc[slot].w[lane], p.w_scales + static_cast<size_t>(g.tile) * KB + kb + lane, true);
                cp_async_mbar_arrive(&s.sfull[slot]);
                if (++slot == SC_RING) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        cp_async_wait_all();
    } else if (warp >= 4) {
        const int q = warp & 3;
        const int r = q * 32 + lane;  // weight row of the tile
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        int tb = 0, slot = 0;
        uint32_t tphase = 0, sphase = 0;
        bool ok = true, first = true;
        long long u = u0;
        Segment g;
        while (next_segment(u, g)) {
            float acc[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[i] = 0.0f;
            for (int i = 0; i < g.nk && ok; i += 2) {
                const bool both = i + 1 < g.nk;
                const bool ready = mbar_wait(&s.sfull[slot], sphase, abort, p.status) &&
                                   mbar_wait(&s.tfull[tb], tphase, abort, p.status);
                if (!__all_sync(0xffffffffu, ready)) {  // the loads below are warp-wide
                    ok = false;
                    break;
                }
                tc_fence_after();
                const auto &sc = s.sc[slot];
#pragma unroll
                for (int c = 0; c < 2 * NT; c += 32) {
                    float v[32];
                    tmem_ld32(lane_base + 2 * tb * NT + c, v);
                    tmem_wait_ld(v);
                    // 32 columns: both K blocks' 16 tokens, or 32 tokens of one
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const int j = (c + e) / NT, t = (c + e) % NT;
                        if (j == 0 || both) {
                            const float4 sx = *reinterpret_cast<const float4 *>(&sc.x[j][t]);
                            const float sw = sc.w[j];
                            acc[t] = __fmaf_rn(v[e], __fmul_rn(sx.x, sw), acc[t]);
                            acc[t + 1] = __fmaf_rn(v[e + 1], __fmul_rn(sx.y, sw), acc[t + 1]);
                            acc[t + 2] = __fmaf_rn(v[e + 2], __fmul_rn(sx.z, sw), acc[t + 2]);
                            acc[t + 3] = __fmaf_rn(v[e + 3], __fmul_rn(sx.w, sw), acc[t + 3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s.tempty[tb]);
                    mbar_arrive(&s.sempty[slot]);
                }
                if (++tb == NBUF) {
                    tb = 0;
                    tphase ^= 1;
                }
                if (++slot == SC_RING) {
                    slot = 0;
                    sphase ^= 1;
                }
            }
            if (g.nk == KB) {
                const int n = g.tile * 128 + r;
                if (ok && n < p.N) {
#pragma unroll
                    for (int t0 = 0; t0 < NT; t0 += 16) {
                        float res[16];
#pragma unroll
                        for (int t = 0; t < 16; ++t)
                            res[t] = p.residual && t0 + t < p.T
                                         ? bf16_f(p.residual[static_cast<size_t>(t0 + t) * p.N + n]) : 0.0f;
#pragma unroll
                        for (int t = 0; t < 16; ++t)
                            if (t0 + t < p.T) store_out(p, static_cast<size_t>(t0 + t) * p.N + n, acc[t0 + t], res[t]);
                    }
                }
            } else {
                // shared tile: partial sums to the workspace, [token][128 rows];
                // the last CTA adds them all, its own among them, in K order
                const long long tu = static_cast<long long>(g.tile) * KB;
                const int c0 = share_of(U, tu, gridDim.x), shares = share_of(U, tu + KB - 1, gridDim.x) - c0 + 1;
                float *mine = p.partial + (static_cast<size_t>(blockIdx.x) * 2 + (first ? 0 : 1)) * NT * 128 + r;
                if (ok) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        if (t < p.T) mine[t * 128] = acc[t];
                }
                __threadfence();
                named_bar_sync(1, 128);
                if (threadIdx.x == 128) {
                    const int last = atomicAdd(p.counters + g.tile, 1) == shares - 1;
                    if (last) p.counters[g.tile] = 0;  // everyone has counted: zero for the next launch
                    s.last = last;
                }
                named_bar_sync(1, 128);
                if (ok && s.last) {
                    __threadfence();
                    add_shares<NT>(p, U, g.tile, c0, shares, q, lane);
                }
                named_bar_sync(1, 128);  // s.last is rewritten by the next shared tile
            }
            first = false;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// x [rows, K] bf16 (behind the pre-norm, with rstd set) -> codes and scales of
// its 1x128 tiles, 16 lanes a tile (tile_scale has the arithmetic).
__global__ void __launch_bounds__(256)
linear_quant_kernel(const uint16_t *__restrict__ x, int rows, int K, PreNorm pn, int ue,
                    uint8_t *__restrict__ a, float *__restrict__ a_scales) {
    pdl_wait_and_trigger();
    const int KB = K / 128, l16 = threadIdx.x % 16;
    const long long tiles = static_cast<long long>(rows) * KB;
    const long long step = static_cast<long long>(gridDim.x) * 16;
    // both halves of a warp stay in the loop together (the shuffles below)
    for (long long i0 = static_cast<long long>(blockIdx.x) * 16 + (threadIdx.x / 32) * 2; i0 < tiles; i0 += step) {
        const long long i = i0 + (threadIdx.x / 16 & 1);
        const bool in = i < tiles;
        const int t = in ? static_cast<int>(i / KB) : 0;
        const int c = (in ? static_cast<int>(i - static_cast<long long>(t) * KB) : 0) * 128 + l16 * 8;
        float v[8];
        load_x8(x, t, c, K, pn, v);
        uint2 code;
        const float sc = quant_tile8(v, ue, &code);
        if (!in) continue;
        *reinterpret_cast<uint2 *>(a + static_cast<size_t>(t) * K + c) = code;
        if (l16 == 0) a_scales[i] = sc;
    }
}

// out[t, n] = sum of the ksplit binary32 planes [ksplit][T][ldp] in order
// (+ residual), in bf16 or binary32; one thread per 8 columns, whole 16-byte
// vectors where N is a multiple of 8.
__global__ void __launch_bounds__(128)
linear_finish_kernel(const float *__restrict__ partial, int ksplit, int T, int N, int ldp,
                     const uint16_t *__restrict__ residual, void *__restrict__ out, int out_f32) {
    const int t = blockIdx.x;
    const int n0 = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
    pdl_wait_and_trigger();
    if (n0 >= N) return;
    const size_t plane = static_cast<size_t>(T) * ldp;
    const float *src = partial + static_cast<size_t>(t) * ldp + n0;
    float f[8];
    {
        const float4 a = __ldcg(reinterpret_cast<const float4 *>(src));
        const float4 b = __ldcg(reinterpret_cast<const float4 *>(src + 4));
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    for (int k = 1; k < ksplit; ++k) {
        const float4 a = __ldcg(reinterpret_cast<const float4 *>(src + k * plane));
        const float4 b = __ldcg(reinterpret_cast<const float4 *>(src + k * plane + 4));
        const float g[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __fadd_rn(f[i], g[i]);
    }
    const size_t at = static_cast<size_t>(t) * N + n0;
    if (N % 8 == 0) {
        if (residual) {
            const uint4 h = *reinterpret_cast<const uint4 *>(residual + at);
            const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __fadd_rn(f[2 * i], bf16_lo(w[i]));
                f[2 * i + 1] = __fadd_rn(f[2 * i + 1], bf16_hi(w[i]));
            }
        }
        if (out_f32) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
            o[0] = make_float4(f[0], f[1], f[2], f[3]);
            o[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) =
                make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                           pack_bf16x2(f[6], f[7]));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (n0 + i >= N) break;
        if (residual) f[i] = __fadd_rn(f[i], __uint_as_float(static_cast<uint32_t>(residual[at + i]) << 16));
        if (out_f32) static_cast<float *>(out)[at + i] = f[i];
        else static_cast<__nv_bfloat16 *>(out)[at + i] = __float2bfloat16_rn(f[i]);
    }
}

template <int NT>
cudaError_t launch_stream_t(const LinearStreamArgs &g, cudaStream_t st) {
    CUtensorMap mx, mw;
    const int tiles = (g.N + 127) / 128, KB = g.K / 128;
    if (!make_map_2d(&mx, g.a, true, g.K, g.T, NT)) return cudaErrorInvalidValue;
    if (g.w_rowmajor ? !make_map_2d(&mw, g.w, true, g.K, g.N) : !make_map_2d(&mw, g.w, true, 128, tiles * KB * 128))
        return cudaErrorInvalidValue;
    constexpr size_t smem = sizeof(LinearSmem<NT>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory budget of one CTA");
    static DeviceConfigured configured{};
    if (first_use_on_device(configured)) {
        const cudaError_t e = cudaFuncSetAttribute(linear_stream_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        mark_used_on_device(configured);
    }
    LinearParams p{};
    p.a_scales = g.a_scales;
    p.w_scales = g.w_scales;
    p.residual = g.residual;
    p.out = g.out;
    p.partial = g.partial;
    p.counters = g.counters;
    p.status = g.status;
    p.T = g.T;
    p.N = g.N;
    p.KB = KB;
    p.tiles = tiles;
    p.out_f32 = g.out_f32;
    p.w_rowmajor = g.w_rowmajor;
    const long long units = static_cast<long long>(tiles) * KB;
    const int grid = static_cast<int>(std::min<long long>(units, std::min(num_sms(), kLinearMaxCtas)));
    return launch_pdl(linear_stream_kernel<NT>, dim3(grid), dim3(LS_THREADS), smem, st, mx, mw, p);
}

}  // namespace

cudaError_t launch_linear_stream(const LinearStreamArgs &g, cudaStream_t st, int *launches) {
    if (g.T < 1 || g.T > kLinearStreamRows) return cudaErrorInvalidValue;
    mark_launch(st, *launches, "linear_stream");
    LAUNCH_OR_RETURN(g.T <= 16 ? launch_stream_t<16>(g, st)
                               : (g.T <= 32 ? launch_stream_t<32>(g, st) : launch_stream_t<64>(g, st)));
    ++*launches;
    return cudaGetLastError();
}

cudaError_t launch_linear_quant(const uint16_t *x, int rows, int K, PreNorm pn, bool ue8m0, uint8_t *a,
                                float *a_scales, cudaStream_t st, int *launches) {
    mark_launch(st, *launches, "linear_quant");
    const long long want = (static_cast<long long>(rows) * (K / 128) + 15) / 16;
    const int grid = static_cast<int>(std::min<long long>(want, num_sms() * 16LL));
    LAUNCH_OR_RETURN(launch_pdl(linear_quant_kernel, dim3(grid), dim3(256), 0, st, x, rows, K, pn, ue8m0 ? 1 : 0, a,
                                a_scales));
    ++*launches;
    return cudaGetLastError();
}

cudaError_t launch_linear_finish(const float *partial, int ksplit, int T, int N, int ldp,
                                 const uint16_t *residual, void *out, int out_f32, cudaStream_t st,
                                 int *launches) {
    if (ksplit < 1 || ldp % 8 || ldp < N) return cudaErrorInvalidValue;
    mark_launch(st, *launches, "linear_finish");
    const dim3 grid(T, (N + 1023) / 1024);
    LAUNCH_OR_RETURN(launch_pdl(linear_finish_kernel, grid, dim3(128), 0, st, partial, ksplit, T, N, ldp,
                                residual, out, out_f32));
    ++*launches;
    return cudaGetLastError();
}

}  // namespace moe
