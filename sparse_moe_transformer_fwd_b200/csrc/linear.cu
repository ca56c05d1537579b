// Block-scaled e4m3 matrix product for few rows of activations:
//   out[t, n] = sum_kb s_a[t, kb] s_w[n / 128, kb] * (sum_{i in kb} a[t, i] w[n, i])  (+ residual[t, n])
// with a [T, K] codes in 1x128 tiles and w [N, K] codes in 128x128 blocks
// ("DeepSeek-R1" (aguasto.com), "Quantization": blockwise FP8), each 128-wide
// K block accumulated by the tensor core and added in binary32, as in the
// grouped expert GEMMs.
//
// Few tokens read each weight byte for few FLOP, so the product is bound by
// HBM: N*K bytes of weights.  The weights are therefore the M operand of the MMA
// (128 rows of W a tile, tokens the N operand: 16, 32 or 64 columns; more tokens
// take several groups of columns, tiles of their own that read the same weights
// from L2 at about the same time).  A CTA's first tile is its own number, then
// it takes the next free one (HBM serves some SMs faster: of 7168 x 64007 in
// equal shares the first CTA ended after 58 us, the last after 76).  The tiles
// past the last whole round (all of them, where there are fewer than SMs) are
// cut into equal parts of K, as many as pay (linear_plan).  The parts' binary32
// sums are added in K order, so the result does not depend on timing: where all
// tiles are cut, in 3 to 16 parts, a tile's CTAs are one cluster that exchanges
// them through shared memory (1 us); else they go to the workspace and a second
// kernel adds them (2 us; a tile's last CTA alone took 13 with 64 tokens, and 10
// with its own part kept in registers).
//   warp 0      TMA producer: a stage is two K blocks (two 16 KB boxes of W, two
//               boxes of activations)
//   warp 1      TMEM allocator and MMA issuer: a stage's K blocks go to adjacent
//               accumulators; a stage is one wait and one commit
//   warps 2-3   scales of a K block each, copied to a ring in shared memory with
//               cp.async (rows past T: zeros)
//   warps 4-7   epilogue: 32 weight rows a warp; adds each accumulator, times its
//               scale product, to the sums in registers
//   warps 8-12  (at most 16 tokens of bf16 input, short shares) quantise the
//               stage's 1x128 tiles of x straight into the operand's swizzled
//               rows; every CTA does it for the K blocks it reads, which costs
//               less than a launch that writes the codes first
// Measured (one B200, CUDA graph): 1 token, 7168 x 2112 7.7 us, of which start
// and end take 4.5; 7 tokens, 7168 x 64007 75 us (6.1 TB/s); 64 tokens, 16384 x
// 7168 29.6 us (one token 25), 30.7 with a residual.
// Every wait is bounded; on expiry the block records MOE_ERR_TIMEOUT, drains its
// loads and MMAs, frees its TMEM and exits; the last CTA out zeroes the item
// counter.  (A cluster's barrier has no limit of its own: every CTA reaches it,
// since its other waits end.)
#include "common.cuh"
#include "kernels.h"
#include "quant_math.cuh"

#include <algorithm>
#include <cstring>
#include <mutex>

namespace moe {
namespace {

constexpr int W_BYTES = 128 * 128;  // one tile of weights
constexpr int SC_RING = 8;          // scale slots (two K blocks each)
constexpr int QUEUE = 4;            // work items between the producer and the other roles
constexpr int XQ_WARPS = 5;         // warps that quantise x
constexpr int MAX_CLUSTER = 16;     // parts that a cluster adds

template <int NT>
struct LinearSmem {
    static constexpr int X_BYTES = NT * 128;
    static constexpr int STAGES = NT == 16 ? 6 : (NT == 32 ? 5 : 4);
    static constexpr int TMEM_COLS = NT == 16 ? 256 : 512;  // two accumulators a stage
    static_assert(STAGES * 2 * NT <= TMEM_COLS, "accumulators of the ring's stages");
    alignas(1024) uint8_t w[STAGES][2][W_BYTES];
    alignas(1024) uint8_t x[STAGES][2][X_BYTES];
    // the cluster's sums for this CTA's share of the tile, [part][share] (64
    // columns: in the ring, once every CTA is through with its own)
    static constexpr bool SUMS_IN_RING = NT == 64;
    static constexpr int SUMS = NT * 64 + MAX_CLUSTER;
    alignas(16) float2 sums[SUMS_IN_RING ? 2 : SUMS];
    static_assert(SUMS * 8 <= static_cast<int>(sizeof(w)), "the sums in the ring");
    struct alignas(16) Scales {
        float x[2][NT];
        float w[2];
        float pad[2];
    } sc[SC_RING];
    uint64_t full[STAGES];  // operands landed, and the accumulators drained (4 warps)
    uint64_t done[STAGES];  // MMAs done: accumulators to read, operands to overwrite
    uint64_t sfull[SC_RING], sempty[SC_RING];
    int queue[QUEUE];
    uint64_t qfull[QUEUE], qempty[QUEUE];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
};

struct LinearParams {
    const uint16_t *x;         // [T, K] bf16, quantised here (with XQ)
    const float *a_scales, *w_scales;
    const uint16_t *residual;  // bf16 [T, N] or NULL
    void *out;                 // [T, N] bf16, or binary32 (out_f32)
    float *partial;            // [rest * parts][NT][128]
    LinearCounters *counters;  // zero between launches
    int *status;
    int T, N, KB;
    int groups;   // of NT tokens: tile = (128 rows of W) * groups + group
    int whole;    // tiles worked on whole: the first ones
    int rest;     // tiles after them
    int parts;    // parts of K of each of those
    int cluster;  // a tile's parts are one cluster, which adds them (else a kernel after this one)
    uint32_t share, per_share;  // of the tile's (2 tokens, row) pieces each CTA of the cluster adds; ceil(2^32 / share)
    int out_f32;
    int w_rowmajor;
    int ue;       // power-of-two scales (with XQ)
    int early_w;  // W may be read ahead of the kernel before this one
};

// K blocks kb0 .. kb0 + nk - 1 of one tile: 128 rows of W from n0, NT tokens from t0.
struct Segment {
    int tile, n0, t0, kb0, nk;
    int part;  // of the cut tiles' parts, all of them
};

__device__ __forceinline__ float bf16_f(uint16_t v) {
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
// Where a tile's sums go.
struct LinearOut {
    const uint16_t *residual;
    void *out;
    int T, N, f32;
    __device__ __forceinline__ void store(size_t at, float v, float res) const {
        if (residual) v = __fadd_rn(v, res);
        if (f32) static_cast<float *>(out)[at] = v;
        else static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
    }
};

// Four rows n0 .. n0 + 3 of token t: the sums of `parts` CTAs added in that (K)
// order, eight loads in flight (one at a time cost 0.5 us each).  partial: the
// first part's piece, the next NT * 128 values on.
template <int NT>
__device__ __forceinline__ void add_parts(const float4 *partial, int parts, const LinearOut &o, int t, int n0) {
    const size_t at = static_cast<size_t>(t) * o.N + n0;
    const bool vec = o.N % 4 == 0;  // whole 8- or 16-byte pieces (n0 is a multiple of 4)
    float res[4] = {};
    if (o.residual) {
        if (vec && n0 < o.N) {
            const uint2 w = *reinterpret_cast<const uint2 *>(o.residual + at);
            res[0] = bf16_lo(w.x), res[1] = bf16_hi(w.x), res[2] = bf16_lo(w.y), res[3] = bf16_hi(w.y);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n0 + i < o.N) res[i] = bf16_f(o.residual[at + i]);
        }
    }
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int c = 0; c < parts; c += 8) {
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = c + i < parts ? __ldcg(partial + (c + i) * (NT * 32)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            acc.x = __fadd_rn(acc.x, v[i].x);
            acc.y = __fadd_rn(acc.y, v[i].y);
            acc.z = __fadd_rn(acc.z, v[i].z);
            acc.w = __fadd_rn(acc.w, v[i].w);
        }
    }
    float f[4] = {acc.x, acc.y, acc.z, acc.w};
    if (!vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n0 + i < o.N) o.store(at + i, f[i], res[i]);
        return;
    }
    if (n0 >= o.N) return;
    if (o.residual)
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __fadd_rn(f[i], res[i]);
    if (o.f32) *reinterpret_cast<float4 *>(static_cast<float *>(o.out) + at) = make_float4(f[0], f[1], f[2], f[3]);
    else *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(o.out) + at) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

// The parts of all cut tiles, a thread four rows of a token.
template <int NT>
__global__ void __launch_bounds__(256)
linear_sum_kernel(const float *__restrict__ partial, int first_tile, int rest, int parts, int groups, const LinearOut o) {
    pdl_wait_and_trigger();
    const int i = blockIdx.x * 256 + threadIdx.x;  // (tile, token of its group, four rows)
    const int lane = i & 31, t = (i >> 5) % NT, tile = (i >> 5) / NT;
    const int row = (first_tile + tile) / groups, token = (first_tile + tile - row * groups) * NT + t;
    if (tile >= rest || token >= o.T) return;
    add_parts<NT>(reinterpret_cast<const float4 *>(partial) + (static_cast<size_t>(tile) * parts * NT + t) * 32 + lane, parts, o,
                  token, row * 128 + lane * 4);
}

// The cluster's barrier, per thread, and another CTA's copy of a shared address.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t cta, const float2 &v) {
    uint32_t remote;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(cta));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(v.x), "f"(v.y) : "memory");
}

// 8 x GROUPS accumulator columns of 16 rows: value 4 g + 2 i + j of a lane is
// row lane / 4 + 8 i, column 8 g + 2 (lane % 4) + j.  A lane so holds four rows
// of a quarter of the tokens, and reads only those tokens' scales: with a row
// and every token to each lane the reads of 64 tokens' scales took 512 of a
// stage's 1300 clk of shared memory.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, float (&v)[32]) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// Four groups, into v[16 HALF] on.
template <int HALF>
__device__ __forceinline__ void tmem_ld_rows16_half(uint32_t taddr, float (&v)[32]) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v) + 16 * HALF;
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

template <int NT, bool XQ>
constexpr int ls_threads() { return (XQ ? 8 + XQ_WARPS : 8) * 32; }

// NT token columns; XQ: x is given in bf16 and quantised here
template <int NT, bool XQ>
__global__ void __launch_bounds__((ls_threads<NT, XQ>()), 1)
linear_stream_kernel(const __grid_constant__ CUtensorMap tmap_x,
                     const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ LinearParams p) {
    static_assert(!XQ || NT == 16, "x is quantised here for at most 16 tokens");
    using S = LinearSmem<NT>;
    constexpr int STAGES = S::STAGES;
    extern __shared__ uint8_t smem_raw[];
    S &s = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int KB = p.KB;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&s.full[i], 1 + 4 + (XQ ? XQ_WARPS : 0));
            mbar_init(&s.done[i], 1);
        }
        for (int i = 0; i < SC_RING; ++i) {
            mbar_init(&s.sfull[i], 64 + (XQ ? XQ_WARPS : 0));
            mbar_init(&s.sempty[i], 4);
        }
        for (int i = 0; i < QUEUE; ++i) {
            mbar_init(&s.qfull[i], 1);
            mbar_init(&s.qempty[i], 7 + (XQ ? XQ_WARPS : 0));  // MMA, scales, epilogue, quantisers
        }
        mbar_init(&s.mma_done, 1);
        s.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&tmap_x);
        prefetch_tmap(&tmap_w);
    }
    if (warp == 1) {
        tmem_alloc(&s.tmem_base, S::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, s.tmem_base, 0);
    volatile int *abort = &s.abort;
    float2 *sums = S::SUMS_IN_RING ? reinterpret_cast<float2 *>(s.w) : s.sums;
    // The kernel before this one has finished when this returns; the producer
    // alone may read W ahead of it (early_w).
    if (!(warp == 0 && p.early_w)) pdl_wait();
    pdl_trigger();
    // Cluster barriers: the first when every CTA may be written to, the second
    // when the sums have arrived.
    if (p.cluster && !S::SUMS_IN_RING) cluster_arrive();

    const int items = p.whole + p.rest * p.parts;
    auto decode = [&](int id, Segment &g) {
        if (id < 0 || id >= items) return false;
        if (id < p.whole) {
            g.tile = id;
            g.kb0 = 0;
            g.nk = KB;
            g.part = -1;
        } else {
            g.part = id - p.whole;
            const int tile = g.part / p.parts, k = g.part - tile * p.parts;
            g.tile = p.whole + tile;
            g.kb0 = k * KB / p.parts;
            g.nk = (k + 1) * KB / p.parts - g.kb0;
        }
        const int row = NT == 64 ? g.tile / p.groups : g.tile;  // 16 and 32 columns hold the whole batch
        g.n0 = row * 128;
        g.t0 = NT == 64 ? (g.tile - row * p.groups) * NT : 0;
        return true;
    };
    // A role's items (whole warps): the CTA's number, then what the producer hands
    // on; in turn where there are less than two rounds of whole tiles, which end
    // before taking them evens anything out (24576 x 1536: 10.8 us, taken 12.1).
    const bool taken = p.whole >= 2 * static_cast<int>(gridDim.x);
    struct Taken {
        int n = 0, slot = 0;
        uint32_t phase = 0;
    };
    auto next_segment = [&](Taken &q, Segment &g) {
        if (q.n == 0 || !taken) return decode(blockIdx.x + q.n++ * gridDim.x, g);
        const bool got = __all_sync(0xffffffffu, mbar_wait(&s.qfull[q.slot], q.phase, abort, p.status));
        const int id = got ? s.queue[q.slot] : -1;
        __syncwarp();
        if (got && lane == 0) mbar_arrive(&s.qempty[q.slot]);
        if (++q.slot == QUEUE) {
            q.slot = 0;
            q.phase ^= 1;
        }
        return decode(id, g);
    };

    if (warp == 0) {
        // One lane: coordinates advance by constants (every instruction of this
        // loop costs a lone thread about five clocks).
        if (lane == 0) {
            const uint32_t w_base = smem_u32(s.w[0][0]), x_base = smem_u32(s.x[0][0]), f_base = smem_u32(&s.full[0]);
            const uint64_t policy = l2_evict_normal();
            const int x_bytes = min(p.T, NT) * 128;
            int stage = 0;
            uint32_t phase = 0, armed = 0, armed_phase = 0;
            bool ok = true, waited = !p.early_w;
            int first_x[STAGES], first_t[STAGES], first_n[STAGES], behind = 0;  // stages whose activations wait for the kernel before
            auto load_x = [&](int st, int x0, int t0, int n) {
                for (int j = 0; j < n; ++j)
                    tma_load_2d_policy(x_base + (2 * st + j) * S::X_BYTES, &tmap_x, x0 + j * 128, t0, f_base + st * 8, policy);
            };
            auto catch_up = [&] {
                pdl_wait();
                waited = true;
                for (int i = 0; i < behind; ++i) load_x(i, first_x[i], NT == 64 ? first_t[i] : 0, first_n[i]);
            };
            // the next free item is asked for while the one before is loaded, and
            // handed on once known
            int id = blockIdx.x, slot = 0;
            uint32_t qphase = 0;
            auto hand_on = [&](int v) {
                if (!mbar_wait(&s.qempty[slot], qphase ^ 1, abort, p.status)) return false;
                s.queue[slot] = v;
                mbar_arrive(&s.qfull[slot]);
                if (++slot == QUEUE) {
                    slot = 0;
                    qphase ^= 1;
                }
                return true;
            };
            Segment g;
            while (ok && decode(id, g)) {
                int next = id + gridDim.x;
                const bool ask = taken && waited;  // (the launch before may hold the counter until then)
                if (ask) next = gridDim.x + atomicAdd(&p.counters->next, 1);
                int wx = p.w_rowmajor ? g.kb0 * 128 : 0, wy = p.w_rowmajor ? g.n0 : g.n0 * KB + g.kb0 * 128;
                const int dx = p.w_rowmajor ? 128 : 0, dy = p.w_rowmajor ? 0 : 128;
                int xx = g.kb0 * 128;
                for (int left = g.nk; left > 0; left -= 2) {
                    if (!waited && behind == STAGES) catch_up();
                    if (!mbar_wait(&s.done[stage], phase ^ 1, abort, p.status)) {
                        ok = false;
                        break;
                    }
                    const int n = min(2, left);
                    const uint32_t bar = f_base + stage * 8, w = w_base + stage * 2 * W_BYTES;
                    mbar_arrive_expect_tx(&s.full[stage], n * (W_BYTES + (XQ ? 0 : x_bytes)));
                    tma_load_2d_policy(w, &tmap_w, wx, wy, bar, policy);
                    if (n == 2) tma_load_2d_policy(w + W_BYTES, &tmap_w, wx + dx, wy + dy, bar, policy);
                    if constexpr (!XQ) {
                        if (waited) load_x(stage, xx, g.t0, n);
                        else first_x[behind] = xx, first_t[behind] = NT == 64 ? g.t0 : 0, first_n[behind] = n, ++behind;  // the ring's first round: slot = behind
                    }
                    wx += 2 * dx, wy += 2 * dy, xx += 2 * 128;
                    armed |= 1u << stage;
                    armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (taken && !ask) {
                    if (!waited) catch_up();
                    next = gridDim.x + atomicAdd(&p.counters->next, 1);
                }
                id = next < items ? next : -1;
                if (ok && taken && !hand_on(id)) ok = false;
            }
            if (!waited) catch_up();
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
        constexpr uint32_t idesc = instr_desc<true>(128, NT);
        const uint64_t wd0 = smem_desc_sw128(smem_u32(s.w[0][0])), xd0 = smem_desc_sw128(smem_u32(s.x[0][0]));
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        Taken item;
        Segment g;
        while (ok && next_segment(item, g)) {
            for (int left = g.nk; left > 0; left -= 2) {
                if (!__all_sync(0xffffffffu, mbar_wait(&s.full[stage], phase, abort, p.status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + 2 * stage * NT;
                const uint64_t wd = wd0 + stage * (2 * W_BYTES >> 4), xd = xd0 + stage * (2 * S::X_BYTES >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) tc_mma<true>(d, wd + 2 * kk, xd + 2 * kk, idesc, kk != 0);
                    if (left > 1)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma<true>(d + NT, wd + (W_BYTES >> 4) + 2 * kk, xd + (S::X_BYTES >> 4) + 2 * kk, idesc, kk != 0);
                    tc_commit(&s.done[stage]);
                }
                __syncwarp();
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // all MMAs issued are complete before TMEM is freed (the same lane is
        // elected every time, and a commit covers that lane's MMAs)
        if (elect_one()) tc_commit(&s.mma_done);
        __syncwarp();
        const long long t0 = clock64();
        while (!mbar_try_wait(&s.mma_done, 0)) {
            if (clock64() - t0 > kWaitBudgetCycles) {
                set_status(p.status, MOE_ERR_TIMEOUT);
                break;
            }
        }
    } else if (warp == 2 || warp == 3) {
        // Warp 2 + j copies the scales of the stage's K block j: lane l those of
        // tokens l, l + 32, lane 0 the weights' (every lane arrives on the slot's
        // barrier when its copies have landed).
        const int j = warp - 2;
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        Taken item;
        Segment g;
        while (ok && next_segment(item, g)) {
            const float *ws = p.w_scales + static_cast<size_t>(g.n0 / 128) * KB;
            for (int kb = g.kb0 + j; kb - j < g.kb0 + g.nk; kb += 2) {
                if (!__all_sync(0xffffffffu, mbar_wait(&s.sempty[slot], phase ^ 1, abort, p.status))) {
                    ok = false;
                    break;
                }
                if (kb < g.kb0 + g.nk) {
                    if constexpr (!XQ)
#pragma unroll
                        for (int t = lane; t < NT; t += 32)
                            cp_async4(&s.sc[slot].x[j][t], p.a_scales + (g.t0 + t < p.T ? static_cast<size_t>(g.t0 + t) * KB + kb : 0),
                                      g.t0 + t < p.T);
                    if (lane == 0) cp_async4(&s.sc[slot].w[j], ws + kb, true);
                }
                cp_async_mbar_arrive(&s.sfull[slot]);
                if (++slot == SC_RING) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        cp_async_wait_all();
    } else if (XQ && warp >= 8) {
        // Half-warps over the stage's (K block, token) tiles, up to PER each;
        // the next stage's vectors are loaded before this stage's are encoded.
        // Lane l16 of a half writes codes 8 l16 .. 8 l16 + 7 of its token's
        // 128-byte row, 16-byte chunks XOR-swizzled by the row as the TMA does.
        constexpr int HALVES = 2 * XQ_WARPS, PER = (2 * 16 + HALVES - 1) / HALVES;
        const int half = (warp - 8) * 2 + (lane >> 4), l16 = lane & 15, T = p.T;
        Taken item;
        struct Cursor {  // a stage: K blocks i, i + 1 of a segment
            Segment g;
            int i;
            bool more;
        } ahead{{}, 0, false}, at;
        ahead.more = next_segment(item, ahead.g);
        uint4 v[PER], next[PER];
        int block[PER], token[PER];  // of tile half + i * HALVES of any stage
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            block[i] = (half + i * HALVES) / T;
            token[i] = half + i * HALVES - block[i] * T;
        }
        auto load = [&](const Cursor &c, uint4 (&r)[PER]) {
            const int n = c.more ? min(2, c.g.nk - c.i) * T : 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (half + i * HALVES < n)
                    r[i] = __ldg(reinterpret_cast<const uint4 *>(
                        p.x + static_cast<size_t>(token[i]) * (KB * 128) + (c.g.kb0 + c.i + block[i]) * 128 + l16 * 8));
            }
        };
        load(ahead, next);
        int stage = 0, slot = 0;
        uint32_t phase = 0, sphase = 0;
        while (ahead.more) {
            at = ahead;
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = next[i];
            ahead.i += 2;
            if (ahead.i >= ahead.g.nk) {
                ahead.i = 0;
                ahead.more = next_segment(item, ahead.g);
            }
            load(ahead, next);
            const int n = min(2, at.g.nk - at.i) * T;
            if (!__all_sync(0xffffffffu, mbar_wait(&s.sempty[slot], sphase ^ 1, abort, p.status) &&
                                             mbar_wait(&s.done[stage], phase ^ 1, abort, p.status)))
                break;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int tile = half + i * HALVES;
                if ((half & ~1) + i * HALVES >= n) break;  // the whole warp
                float f[8];
                widen8(v[i], f);
                uint2 code;
                const float sc = quant_tile8(f, p.ue, &code);
                if (tile < n) {
                    const int j = block[i], t = token[i];
                    *reinterpret_cast<uint2 *>(s.x[stage][j] + t * 128 + (((l16 >> 1) ^ (t & 7)) << 4) + (l16 & 1) * 8) = code;
                    if (l16 == 0) s.sc[slot].x[j][t] = sc;
                }
            }
            fence_proxy_async_smem();  // the MMA reads the codes
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s.full[stage]);
                mbar_arrive(&s.sfull[slot]);
            }
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1;
            }
            if (++slot == SC_RING) {
                slot = 0;
                sphase ^= 1;
            }
        }
    } else if (warp >= 4 && warp < 8) {
        const int q = warp & 3;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        int stage = 0, slot = 0;
        uint32_t phase = 0, sphase = 0;
        bool ok = true;
        if (lane < STAGES) mbar_arrive(&s.full[lane]);  // the accumulators are free
        __syncwarp();
        Taken item;
        Segment g;
        while (next_segment(item, g)) {
            // the residual's rows into L2 while the tile streams (two lines a token)
            if (const int i = threadIdx.x & 127; p.residual && i < 2 * NT && g.t0 + i / 2 < p.T && g.n0 + (i & 1) * 64 < p.N)
                l2_prefetch_line(p.residual + static_cast<size_t>(g.t0 + i / 2) * p.N + g.n0 + (i & 1) * 64);
            // [token group][16 rows][8 rows]: tokens 8 group + 2 (lane % 4) and the next
            float2 acc[NT / 8][2][2];
#pragma unroll
            for (int i = 0; i < NT / 8; ++i)
                acc[i][0][0] = acc[i][0][1] = acc[i][1][0] = acc[i][1][1] = make_float2(0.0f, 0.0f);
            for (int i = 0; i < g.nk && ok; i += 2) {
                const bool both = i + 1 < g.nk;
                const bool ready = mbar_wait(&s.sfull[slot], sphase, abort, p.status) &&
                                   mbar_wait(&s.done[stage], phase, abort, p.status);
                if (!__all_sync(0xffffffffu, ready)) {  // the loads below are warp-wide
                    ok = false;
                    break;
                }
                tc_fence_after();
                const auto &sc = s.sc[slot];
                const uint32_t base = lane_base + 2 * stage * NT;
                // 8 columns from c on of the stage's accumulators, of rows 0-15 and 16-31
                auto add = [&](int c, const float *lo, const float *hi) {
                    const int j = c / NT, gr = c % NT / 8;
                    if (j == 0 || both) {
                        const float2 sx = *reinterpret_cast<const float2 *>(&sc.x[j][8 * gr + 2 * (lane & 3)]);
                        const float2 f = __fmul2_rn(sx, make_float2(sc.w[j], sc.w[j]));
                        acc[gr][0][0] = __ffma2_rn(make_float2(lo[0], lo[1]), f, acc[gr][0][0]);
                        acc[gr][0][1] = __ffma2_rn(make_float2(lo[2], lo[3]), f, acc[gr][0][1]);
                        acc[gr][1][0] = __ffma2_rn(make_float2(hi[0], hi[1]), f, acc[gr][1][0]);
                        acc[gr][1][1] = __ffma2_rn(make_float2(hi[2], hi[3]), f, acc[gr][1][1]);
                    }
                };
                auto drained = [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.full[stage]);
                };
                if constexpr (NT == 16) {
                    float v[32];
                    tmem_ld_rows16_half<0>(base, v);
                    tmem_ld_rows16_half<1>(base + (16 << 16), v);
                    tmem_wait_ld(v);
                    drained();
#pragma unroll
                    for (int e = 0; e < 4; ++e) add(8 * e, v + 4 * e, v + 16 + 4 * e);
                } else {
#pragma unroll
                    for (int c = 0; c < 2 * NT; c += 64) {
                        float v0[32], v1[32];
                        tmem_ld_rows16(base + c, v0);
                        tmem_ld_rows16(base + c + (16 << 16), v1);
                        tmem_wait_ld(v0, v1);
                        if (c + 64 >= 2 * NT) drained();
#pragma unroll
                        for (int e = 0; e < 8; ++e) add(c + 8 * e, v0 + 4 * e, v1 + 4 * e);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.sempty[slot]);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
                if (++slot == SC_RING) {
                    slot = 0;
                    sphase ^= 1;
                }
            }
            const int T = p.T - g.t0;  // tokens from the group's first on
            const int r = q * 32 + (lane >> 2), t2 = 2 * (lane & 3);
            if (p.cluster) {  // each piece to the CTA of the cluster that adds it
                if (S::SUMS_IN_RING) cluster_arrive();
                cluster_wait();
                const uint32_t at = smem_u32(sums) + (blockIdx.x % p.parts) * p.share * 8;
#pragma unroll
                for (int gr = 0; gr < NT / 8; ++gr) {
                    if (8 * gr >= T) break;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t piece = ((gr * 4 + q) * 4 + e) * 32 + lane, owner = __umulhi(piece, p.per_share);
                        st_cluster(at + (piece - owner * p.share) * 8, owner, acc[gr][e >> 1][e & 1]);
                    }
                }
                cluster_arrive();
                continue;
            }
            if (g.nk != KB) {  // one part of a tile: [token][128 rows] to the workspace
                float *mine = p.partial + static_cast<size_t>(g.part) * NT * 128 + r;
                if (ok) {
#pragma unroll
                    for (int e = 0; e < NT; ++e) {
                        const int t = e / 8 * 8 + t2 + (e & 1);
                        const float2 v = acc[e / 8][e >> 2 & 1][e >> 1 & 1];
                        if (t < T) mine[t * 128 + (e & 6) * 4] = e & 1 ? v.y : v.x;
                    }
                }
                continue;
            }
            if (!ok) continue;
            // (addresses advance by constants: worked out for each of 64 values
            // they took 2.7 us a tile)
            const size_t first = static_cast<size_t>(g.t0 + t2) * p.N + g.n0 + r;
            const int rows = p.N - g.n0 - r;  // e (8 rows on) is a row if 8 e < rows
            auto store = [&](auto *dst, auto &&convert) {
                constexpr int AHEAD = 2;  // token groups whose residuals are in flight together
                const size_t group = static_cast<size_t>(8) * p.N;
#pragma unroll
                for (int g0 = 0; g0 < NT / 8; g0 += AHEAD) {
                    if (8 * g0 >= T) break;
                    float res[AHEAD][2][4] = {};
                    if (p.residual) {
#pragma unroll
                        for (int i = 0; i < 2 * AHEAD; ++i) {
                            const uint16_t *src = p.residual + first + (g0 + i / 2) * group + (i & 1) * p.N;
                            if (8 * (g0 + i / 2) + t2 + (i & 1) < T)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (8 * e < rows) res[i / 2][i & 1][e] = bf16_f(src[8 * e]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2 * AHEAD; ++i) {
                        auto *to = dst + first + (g0 + i / 2) * group + (i & 1) * p.N;
                        if (8 * (g0 + i / 2) + t2 + (i & 1) < T)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 a = acc[g0 + i / 2][e >> 1][e & 1];
                                float v = i & 1 ? a.y : a.x;
                                if (p.residual) v = __fadd_rn(v, res[i / 2][i & 1][e]);
                                if (8 * e < rows) to[8 * e] = convert(v);
                            }
                    }
                }
            };
            if (p.out_f32) store(static_cast<float *>(p.out), [](float v) { return v; });
            else store(static_cast<__nv_bfloat16 *>(p.out), [](float v) { return __float2bfloat16_rn(v); });
        }
    }

    if (p.cluster) {
        if (warp < 4 || warp >= 8) {
            if (S::SUMS_IN_RING) cluster_arrive();
            cluster_wait();
            cluster_arrive();
        }
        cluster_wait();
        Segment g;
        decode(blockIdx.x, g);
        const int rank = blockIdx.x % p.parts;
        const LinearOut out{p.residual, p.out, p.T, p.N, p.out_f32};
        // a piece: [token group][warp][8 rows][lane]; residuals of BATCH pieces in
        // flight together (one at a time, 64 tokens' took 7 us; few tokens have
        // one, and less code to fetch)
        constexpr int BATCH = NT == 64 ? 4 : 1;
        for (uint32_t i0 = threadIdx.x; i0 < p.share; i0 += BATCH * blockDim.x) {
            float res[BATCH][2] = {};
            size_t at[BATCH];
            int have[BATCH];  // tokens of the piece that are stored
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const uint32_t i = i0 + b * blockDim.x;
                const int piece = rank * p.share + i;
                const int n = g.n0 + (piece >> 5 & 15) * 8 + (piece >> 2 & 7), t = g.t0 + (piece >> 9) * 8 + 2 * (piece & 3);
                have[b] = i < p.share && n < p.N ? min(2, min(g.t0 + NT, p.T) - t) : 0;
                at[b] = static_cast<size_t>(t) * p.N + n;
                if (p.residual && have[b] > 0) res[b][0] = bf16_f(p.residual[at[b]]);
                if (p.residual && have[b] > 1) res[b][1] = bf16_f(p.residual[at[b] + p.N]);
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                if (have[b] <= 0) continue;
                float2 f = make_float2(0.0f, 0.0f);
#pragma unroll 4
                for (int k = 0; k < p.parts; ++k) {
                    const float2 v = sums[k * p.share + i0 + b * blockDim.x];
                    f.x = __fadd_rn(f.x, v.x), f.y = __fadd_rn(f.y, v.y);
                }
                out.store(at[b], f.x, res[b][0]);
                if (have[b] > 1) out.store(at[b] + p.N, f.y, res[b][1]);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, S::TMEM_COLS);
    }
    // the last CTA out zeroes the item counter for the next launch
    if (threadIdx.x == 0 && taken) {
        __threadfence();
        if (atomicAdd(&p.counters->exited, 1) == static_cast<int>(gridDim.x) - 1) p.counters->next = p.counters->exited = 0;
    }
}

// x [rows, K] bf16 -> codes and scales of its 1x128 tiles, 16 lanes a tile
// (tile_scale has the arithmetic).
__global__ void __launch_bounds__(256)
linear_quant_kernel(const uint16_t *__restrict__ x, int rows, int K, int ue, uint8_t *__restrict__ a,
                    float *__restrict__ a_scales) {
    pdl_wait_and_trigger();
    const int KB = K / 128, l16 = threadIdx.x % 16;
    const long long tiles = static_cast<long long>(rows) * KB;
    const long long step = static_cast<long long>(gridDim.x) * 16;
    // both halves of a warp stay in the loop together (the shuffles below)
    for (long long i0 = static_cast<long long>(blockIdx.x) * 16 + (threadIdx.x / 32) * 2; i0 < tiles; i0 += step) {
        const long long i = i0 + (threadIdx.x / 16 & 1);
        const bool in = i < tiles;
        float v[8];
        widen8(in ? *reinterpret_cast<const uint4 *>(x + i * 128 + l16 * 8) : make_uint4(0, 0, 0, 0), v);
        uint2 code;
        const float sc = quant_tile8(v, ue, &code);
        if (!in) continue;
        *reinterpret_cast<uint2 *>(a + i * 128 + l16 * 8) = code;
        if (l16 == 0) a_scales[i] = sc;
    }
}

// The same behind the pre-norm, a block a token: x = bf16((h * rstd) * gamma).
// The row is read from shared memory where it fits (its statistics staged it),
// and gamma is on its way meanwhile.
constexpr int PQ_THREADS = 512;
__global__ void __launch_bounds__(PQ_THREADS)
linear_prenorm_quant_kernel(const uint16_t *__restrict__ h, const uint16_t *__restrict__ gamma, int K, float eps, int ue,
                            uint8_t *__restrict__ a, float *__restrict__ a_scales) {
    __shared__ __align__(16) uint16_t chunk[kRstdChunk];
    __shared__ float rstd_sh;
    constexpr int HALVES = PQ_THREADS / 16, AHEAD = kRstdChunk / 128 / HALVES;
    const size_t t = blockIdx.x;
    const uint16_t *row = h + t * K;
    const int KB = K / 128, half = threadIdx.x / 16, l16 = threadIdx.x % 16;
    pdl_wait_and_trigger();
    uint4 g[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (half + i * HALVES < KB) g[i] = __ldg(reinterpret_cast<const uint4 *>(gamma + (half + i * HALVES) * 128 + l16 * 8));
    const float rstd = block_rstd(row, K, eps, chunk, &rstd_sh);
    const uint16_t *src = K <= kRstdChunk ? chunk : row;
    auto encode = [&](int kb, const uint4 &gv) {  // both halves of a warp (the shuffles)
        float v[8] = {};
        if (kb < KB) prenorm8(*reinterpret_cast<const uint4 *>(src + kb * 128 + l16 * 8), gv, rstd, v);
        uint2 code;
        const float sc = quant_tile8(v, ue, &code);
        if (kb >= KB) return;
        *reinterpret_cast<uint2 *>(a + t * K + kb * 128 + l16 * 8) = code;
        if (l16 == 0) a_scales[t * KB + kb] = sc;
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if ((half & ~1) + i * HALVES < KB) encode(half + i * HALVES, g[i]);
    for (int kb = half + AHEAD * HALVES; (kb & ~1) < KB; kb += HALVES)
        encode(kb, kb < KB ? __ldg(reinterpret_cast<const uint4 *>(gamma + kb * 128 + l16 * 8)) : make_uint4(0, 0, 0, 0));
}

// A tile of the tiled GEMM (tiles numbered column by column): the sums of its
// ksplit ranges [range][128][256] in order (+ residual); a thread takes 8 columns
// of a row, whole 16-byte vectors where N is a multiple of 8.
__global__ void __launch_bounds__(256)
linear_tiles_kernel(const float *__restrict__ partial, int from, int ksplit, int T, int N,
                    const uint16_t *__restrict__ residual, void *__restrict__ out, int out_f32) {
    const int tile = from + blockIdx.x, m_tiles = (T + 127) / 128, nt = tile / m_tiles;
    const int row = blockIdx.y * 8 + threadIdx.x / 32, c = threadIdx.x % 32 * 8;
    const int t = (tile - nt * m_tiles) * 128 + row, n0 = nt * 256 + c;
    pdl_wait_and_trigger();
    if (t >= T || n0 >= N) return;
    const float4 *src = reinterpret_cast<const float4 *>(partial + ((static_cast<size_t>(blockIdx.x) * ksplit * 128 + row) * 256 + c));
    constexpr int PLANE = 128 * 256 / 4, AHEAD = 4;
    float f[8] = {};
    for (int k0 = 0; k0 < ksplit; k0 += AHEAD) {
        float4 a[AHEAD], b[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (k0 + k >= ksplit) break;
            a[k] = __ldcg(src + static_cast<size_t>(k0 + k) * PLANE);
            b[k] = __ldcg(src + static_cast<size_t>(k0 + k) * PLANE + 1);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (k0 + k >= ksplit) break;
            const float g[8] = {a[k].x, a[k].y, a[k].z, a[k].w, b[k].x, b[k].y, b[k].z, b[k].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __fadd_rn(f[i], g[i]);
        }
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
        if (residual) f[i] = __fadd_rn(f[i], bf16_f(residual[at + i]));
        if (out_f32) static_cast<float *>(out)[at + i] = f[i];
        else static_cast<__nv_bfloat16 *>(out)[at + i] = __float2bfloat16_rn(f[i]);
    }
}

template <int NT>
constexpr size_t stream_smem() {
    static_assert(sizeof(LinearSmem<NT>) + 1024 <= 227 * 1024, "shared memory budget of one CTA");
    return sizeof(LinearSmem<NT>) + 1024;
}

template <int NT, bool XQ>
cudaError_t configure_stream() {
    static DeviceConfigured configured{};
    if (!first_use_on_device(configured)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(linear_stream_kernel<NT, XQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(stream_smem<NT>()));
    if (e == cudaSuccess)  // clusters of more than 8
        e = cudaFuncSetAttribute(linear_stream_kernel<NT, XQ>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) mark_used_on_device(configured);
    return e;
}

// [n]: clusters of n CTAs that the current device holds at once (one CTA an SM,
// a cluster within one of the device's groups of SMs: 33 of 4, 22 of 6, 15 of 9,
// 7 of 16 on one B200); asked once for each device.
struct ClusterRoom {
    int n[MAX_CLUSTER + 1];
};
const ClusterRoom &cluster_room() {
    static const ClusterRoom none{};
    static ClusterRoom known[64];
    static std::once_flag asked[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || configure_stream<16, false>() != cudaSuccess) return none;
    std::call_once(asked[dev], [dev] {
        for (int n = 2; n <= MAX_CLUSTER; ++n) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(n);
            cfg.blockDim = dim3(ls_threads<16, false>());
            cfg.dynamicSmemBytes = stream_smem<16>();
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim = {static_cast<unsigned>(n), 1, 1};
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&known[dev].n[n], linear_stream_kernel<16, false>, &cfg) != cudaSuccess) {
                cudaGetLastError();
                known[dev].n[n] = 0;
            }
        }
    });
    return known[dev];
}

template <int NT, bool XQ>
cudaError_t launch_stream_t(const LinearStreamArgs &g, cudaStream_t st, int *launches) {
    CUtensorMap mx, mw;
    const int rows = (g.N + 127) / 128, KB = g.K / 128, groups = (g.T + NT - 1) / NT, tiles = rows * groups;
    std::memset(&mx, 0, sizeof mx);
    // boxes of the tokens there are: rows past the array, which TMA fills with
    // zeros, cost 0.5 us at one token of 7168 x 7168 (columns past T hold anything)
    const int box = std::min(g.T, NT);
    if (!XQ && !make_map_2d(&mx, g.a, true, g.K, g.T, box)) return cudaErrorInvalidValue;
    if (g.w_rowmajor ? !make_map_2d(&mw, g.w, true, g.K, g.N) : !make_map_2d(&mw, g.w, true, 128, rows * KB * 128))
        return cudaErrorInvalidValue;
    {
        const cudaError_t e = configure_stream<NT, XQ>();
        if (e != cudaSuccess) return e;
    }
    LinearParams p{};
    p.x = g.x;
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
    const LinearPlan plan = linear_plan(g.T, tiles, KB);
    p.groups = groups;
    p.whole = plan.whole;
    p.rest = plan.rest;
    p.parts = plan.parts;
    p.cluster = plan.cluster;
    p.share = (static_cast<uint32_t>((std::min(g.T, NT) + 7) / 8) * 512 + plan.parts - 1) / plan.parts;
    p.per_share = static_cast<uint32_t>(((1ull << 32) + p.share - 1) / p.share);
    p.out_f32 = g.out_f32;
    p.w_rowmajor = g.w_rowmajor;
    p.ue = g.ue8m0;
    p.early_w = g.early_w;
    mark_launch(st, *launches, "linear_stream");
    const auto kernel = linear_stream_kernel<NT, XQ>;
    constexpr int threads = ls_threads<NT, XQ>();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = stream_smem<NT>();
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(plan.parts), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = plan.cluster ? 2 : 1;
    LAUNCH_OR_RETURN(cudaLaunchKernelEx(&cfg, kernel, mx, mw, p));
    ++*launches;
    if (plan.parts == 1 || plan.cluster) return cudaSuccess;
    mark_launch(st, *launches, "linear_sum");
    const LinearOut out{g.residual, g.out, g.T, g.N, g.out_f32};
    LAUNCH_OR_RETURN(launch_pdl(linear_sum_kernel<NT>, dim3(plan.rest * NT / 8), dim3(256), 0, st, g.partial, plan.whole,
                                plan.rest, plan.parts, groups, out));
    ++*launches;
    return cudaSuccess;
}

}  // namespace

// One CTA a SM.  The rest tiles are cut into the number of parts that ends
// first, by measured costs: a CTA alone streams a K block of a tile in 0.15 us
// (0.2 with 32 columns, 0.34 with 64: 3 and 6 KB more of activations) and stores
// a whole one in 0.2 (0.3, 1); storing and adding parts takes 2 us, and 1 in clusters (not of two, which sit on one
// pair of SMs: 64 tokens, 16384 x 7168 in 112 CTAs 36.7 us so and 32.8 spread
// out with the second kernel).  Parts of all tiles together (equal shares of the
// whole stream, two cut tiles a CTA) took 7 us longer for one token at 1536 x
// 24576 and 3 at 7168 x 2112.
LinearPlan linear_plan(int T, int tiles, int KB) {
    const int most = std::min(num_sms(), kLinearMaxCtas);
    LinearPlan p;
    p.whole = tiles / most * most;
    p.rest = tiles - p.whole;
    p.parts = 1;
    p.cluster = false;
    const float block = T <= 16 ? 0.15f : (T <= 32 ? 0.2f : 0.34f);
    const float store = T <= 16 ? 0.2f : (T <= 32 ? 0.3f : 1.0f);
    p.us = block * KB + store;
    const ClusterRoom &room = cluster_room();
    for (int k = 2; p.rest && k <= std::min(most / p.rest, KB); ++k) {
        const bool cluster = !p.whole && k > 2 && k <= MAX_CLUSTER && room.n[k] >= p.rest;
        const float t = block * ((KB + k - 1) / k) + (cluster ? 1.0f : 2.0f);
        if (t < p.us) p.us = t, p.parts = k, p.cluster = cluster;
    }
    if (!p.rest) p.us = 0.0f;
    p.us += (block * KB + store) * (p.whole / most);
    p.grid = p.whole ? most : p.rest * p.parts;
    return p;
}

cudaError_t launch_linear_stream(const LinearStreamArgs &g, cudaStream_t st, int *launches) {
    if (g.T < 1 || g.T > (g.x ? kLinearQuantRows : kLinearStreamRows)) return cudaErrorInvalidValue;
    cudaError_t e;
    if (g.x) e = launch_stream_t<16, true>(g, st, launches);
    else if (g.T <= 16) e = launch_stream_t<16, false>(g, st, launches);
    else if (g.T <= 32) e = launch_stream_t<32, false>(g, st, launches);
    else e = launch_stream_t<64, false>(g, st, launches);
    LAUNCH_OR_RETURN(e);
    return cudaGetLastError();
}

cudaError_t launch_linear_quant(const uint16_t *x, int rows, int K, bool ue8m0, uint8_t *a, float *a_scales,
                                cudaStream_t st, int *launches) {
    mark_launch(st, *launches, "linear_quant");
    const long long want = (static_cast<long long>(rows) * (K / 128) + 15) / 16;
    const int grid = static_cast<int>(std::min<long long>(want, num_sms() * 16LL));
    LAUNCH_OR_RETURN(launch_pdl(linear_quant_kernel, dim3(grid), dim3(256), 0, st, x, rows, K, ue8m0 ? 1 : 0, a, a_scales));
    ++*launches;
    return cudaGetLastError();
}

cudaError_t launch_linear_prenorm_quant(const uint16_t *h, const uint16_t *gamma, int rows, int K, float eps, bool ue8m0,
                                        uint8_t *a, float *a_scales, cudaStream_t st, int *launches) {
    mark_launch(st, *launches, "linear_prenorm_quant");
    LAUNCH_OR_RETURN(launch_pdl(linear_prenorm_quant_kernel, dim3(rows), dim3(PQ_THREADS), 0, st, h, gamma, K, eps, ue8m0 ? 1 : 0, a,
                                a_scales));
    ++*launches;
    return cudaGetLastError();
}

cudaError_t launch_linear_tiles(const float *partial, int from, int tiles, int ksplit, int T, int N,
                                const uint16_t *residual, void *out, int out_f32, cudaStream_t st,
                                int *launches) {
    if (ksplit < 1 || from >= tiles) return cudaErrorInvalidValue;
    mark_launch(st, *launches, "linear_tiles");
    LAUNCH_OR_RETURN(launch_pdl(linear_tiles_kernel, dim3(tiles - from, 16), dim3(256), 0, st, partial, from, ksplit, T, N,
                                residual, out, out_f32));
    ++*launches;
    return cudaGetLastError();
}

}  // namespace moe
