// The whole MoE layer for a few tokens in one launch ("DeepSeek-R1"
// architecture card: 256 routed experts, 8 active per token, 1 shared expert).
//
// For at most 16 tokens the layer reads the weights of the experts that the
// tokens meet (44 MB an expert at d 7168, d_expert 2048) and little else, so
// it is bound by that many bytes of HBM: 61 us at one token by the measured rate
// of a copy, 6.5 TB/s (a stream that only reads is faster: 7.5 below).  What
// stands above that in separate kernels is the chain between them (router, top-k,
// permutation, quantisation, two GEMMs, combine) and the router itself, whose
// logits are sequential chains of d fused multiply-adds (20 us at d = 7168).
// This kernel runs all of it on one persistent CTA per SM, so that weights
// stream while everything else is worked out:
//   1. every CTA quantises its share of x and computes its experts' logits
//      roughly (order of summation left free).  Once all have (one grid
//      barrier), each CTA finds the experts that the rough logits select and
//      starts on their gate/up products, for all tokens at once (the tokens
//      are the MMA's 16 columns whether they chose the expert or not, so an
//      expert's H does not depend on who chose it).
//   2. meanwhile four warps run the exact logit chains, in the order that
//      moe_route defines, and select from them.  An expert that the rough
//      logits missed is appended to the work; one that they took in vain has
//      cost its time.  So routing is moe_route's, bit for bit.
//   3. down products of the experts selected, in two parts of K, each begun as
//      soon as that expert's H is complete (warp 9 watches the counts, so that no
//      item pays the L2 round trip); its weights are loaded ahead of that.
//   4. the epilogue warps of all CTAs add the experts' rows with their gates, in
//      rank order, each 128-column block once its products are counted.
// Work items are 128 features of one expert (gate and up rows, all of K) and
// 128 output columns of one expert (half of K); weights are the M operand of
// the MMA.  Items are numbered and taken from a counter.
//   warp 0      TMA producer: takes the items and hands them on by a queue; two
//               weight tiles a stage (gate and up rows of one K block, or two K
//               blocks of the down product) and the tokens' columns
//   warp 1      TMEM allocator and MMA issuer (two accumulators of 16 columns
//               in every stage of the operands' ring)
//   warp 2      the stage's scales (e4m3), copied ahead with cp.async
//   warp 3      tells the other CTAs of finished items
//   warps 4-7   epilogue: thread = weight row
//   warps 8-11  exact routing: 8-10 copy the operands, 11 runs the chains; then
//               warp 9 watches for complete experts' H
// Measured (one B200, 7168 / 2048, 256 experts of which 8 and a shared one, CUDA
// graph): e4m3, 1 token 71 us (HBM from 11 us on), 3 tokens 168 us, 16 tokens 605
// us (7.5 TB/s); bf16, 2048 / 1408, 64 experts of which 6, 5 tokens 67 to 74 us; two
// tokens of bf16 512 / 256, 16 experts, 16.7 us, where the chain of steps bounds it.
// The kernel is launched cooperatively (all CTAs resident), since CTAs wait for
// one another.  Every wait is bounded: on expiry the CTA records
// MOE_ERR_TIMEOUT, sets an abort word that ends the others' waits, drains what
// it has in flight, frees its TMEM and exits; the last CTA to exit zeroes every
// counter, so the workspace serves the next call.
#include "common.cuh"
#include "kernels.h"
#include "quant_math.cuh"
#include "route_math.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int FT = kFewTokens;  // MMA columns
constexpr int FEW_THREADS = 384;
constexpr int FEW_STAGES = 5;
constexpr int W_BYTES = 128 * 128;
constexpr int X_BYTES = FT * 128;
constexpr int SC_RING = 8;
constexpr int TMEM_COLS = 256;  // two accumulators of 16 columns a stage
static_assert(FEW_STAGES * 2 * FT <= TMEM_COLS, "accumulators of the ring's stages");
constexpr int MAIN_THREADS = 256;   // warps 0-7
constexpr int ROUTE_THREADS = 128;  // warps 8-11
constexpr int MAX_K = 32;
constexpr int SIGNALS = 4;
constexpr int QUEUE = 4;  // work items between the producer and the other roles
// Exact logits: chunks of RC columns of the router rows and tokens of one pass
// (RC_ROWS in all) in a ring of RC_BUFS in shared memory; rows are padded by 16
// bytes, so that lanes on different rows read different banks.
constexpr int RC = 128, RC_ROWS = 18, RC_BUFS = 7, RC_LD = RC + 8;
static_assert(FT == 16, "a stage's two accumulators are one 32-column TMEM load");

struct FewSmem {
    alignas(1024) uint8_t w[FEW_STAGES][2][W_BYTES];
    alignas(1024) uint8_t x[FEW_STAGES][2][X_BYTES];
    struct alignas(16) Scales {
        float x[2][FT];
        float w[2];
        float pad[2];
    } sc[SC_RING];
    alignas(16) uint16_t chunk[RC_BUFS][RC_ROWS][RC_LD];
    float amax[4][FT];
    float gate[FT][MAX_K];
    uint16_t sel[FT][MAX_K];       // exact selection
    uint16_t list[kFewMaxList];    // experts worked on: shared, predicted, missed
    uint16_t used[kFewMaxList];    // positions in list of the experts selected
    uint32_t rough_set[32], exact_set[32];
    int8_t rank[FT];
    int n_rough, n_list, n_used;
    uint64_t full[FEW_STAGES];  // operands landed, and the accumulators drained (4 warps)
    uint64_t done[FEW_STAGES];  // MMAs done: accumulators to read, operands to overwrite
    uint64_t sfull[SC_RING], sempty[SC_RING];
    int queue[QUEUE];
    uint64_t qfull[QUEUE], qempty[QUEUE];
    // finished items between the epilogue and warp 3
    int *sig_count[SIGNALS];
    int sig_add[SIGNALS];
    uint64_t sig_full[SIGNALS], sig_free[SIGNALS];
    uint8_t h_ready[kFewMaxList + 7];  // [list position] the expert's H is complete
    uint64_t selected, routed;  // the rough selection; the exact one
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
    int last;
};
static_assert(sizeof(FewSmem) + 1024 <= 227 * 1024, "shared memory budget of one CTA");

struct FewParams {
    const uint16_t *x;         // [T, d]
    const uint16_t *residual;  // [T, d] added to out, or NULL
    const uint16_t *w_router;
    const float *bias;
    const uint8_t *w13, *w2;
    const float *w13_scales, *w2_scales;
    uint16_t *out;
    int32_t *idx_out;        // [T, k]
    float *gates_out;        // [T, k]
    uint8_t *xq;             // [T, d] codes (fp8)
    float *xs;               // [d/128][16]
    float *rough, *scores;   // [T, E]
    void *h;                 // [list][16][de]
    float *hs;               // [list][de/128][16]
    float *y;                // [2][T][k + n_shared][d] binary32: a part of the product each
    FewCounters *ctr;
    int *status;
    int T, d, E, k, de, n_shared;
    float routed_scale;
    int ue, w_rowmajor;
    int inject_fault;  // 1: the exact routing waits for one block more than there are
};

__device__ __forceinline__ int ld_acquire(const int *p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void red_release(int *p, int v) {
    asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ int add_acq_rel(int *p, int v) {
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}
// generic-proxy writes to global memory before, async-proxy (TMA) reads after
__device__ __forceinline__ void fence_proxy_async_global() {
    asm volatile("fence.proxy.async.global;" ::: "memory");
}

// Waits until *p reaches `want`; false on abort or when the budget runs out
// (which aborts every CTA of the launch).
__device__ __forceinline__ bool wait_count(const int *p, int want, const FewParams &q, volatile int *abort) {
    if (ld_acquire(p) >= want) return true;
    const long long t0 = clock64();
    while (true) {
        if (ld_acquire(p) >= want) return true;
        if (*abort) return false;
        if (ld_acquire(&q.ctr->abort)) {
            *abort = 1;
            return false;
        }
        if (clock64() - t0 > kWaitBudgetCycles) {
            *abort = 1;
            atomicExch(&q.ctr->abort, 1);
            set_status(q.status, MOE_ERR_TIMEOUT);
            return false;
        }
    }
}
// The same for an mbarrier of this CTA; a CTA that gives up ends the others'
// waits too.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const FewParams &q, volatile int *abort) {
    if (mbar_wait(bar, parity, abort, q.status)) return true;
    atomicExch(&q.ctr->abort, 1);
    return false;
}

struct Item {
    bool down;
    int pos;     // position in the list
    int expert;  // weight slot
    int blk;     // 128-feature block of H, or 128-column block of the output
    int q0, stages;  // its stages: q0 .. q0 + stages - 1 (gate/up: all)
    int used, part;  // down: index of the expert among those selected, part of the product
};

// warp_topk's choice, by integers of the same order as the selection values (two
// warp reductions a round, not five shuffles of three values).  A NaN, which only
// the bias can bring in, is ordered by its bits there and not at all in warp_topk;
// here each round still takes another expert.
template <int PER_LANE>
__device__ __forceinline__ void topk_keys(const float *row, const float *bias, int E, int k, int lane, int &my_e,
                                          float &my_s) {
    float s[PER_LANE];
    uint32_t key[PER_LANE];
#pragma unroll
    for (int m = 0; m < PER_LANE; ++m) {
        const int e = lane + 32 * m;
        s[m] = e < E ? __ldcg(row + e) : 0.0f;
        key[m] = e < E ? __float_as_uint(__ldg(bias + e)) : 0u;
    }
#pragma unroll
    for (int m = 0; m < PER_LANE; ++m) {
        const uint32_t b = __float_as_uint(__fadd_rn(s[m], __uint_as_float(key[m])));
        // 0: taken or none; a real key is at least 1
        key[m] = lane + 32 * m < E ? max(b >> 31 ? ~b : b | 0x80000000u, 1u) : 0u;
    }
    my_e = 0;
    my_s = 0.0f;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
        int at = 0;
        float bs = 0.0f;
#pragma unroll
        for (int m = 0; m < PER_LANE; ++m)
            if (key[m] > best) best = key[m], at = m, bs = s[m];
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(lane + 32 * at) : 0xffffffffu);
        const float es = __shfl_sync(0xffffffffu, bs, e & 31);
#pragma unroll
        for (int m = 0; m < PER_LANE; ++m)
            if (static_cast<uint32_t>(lane + 32 * m) == e) key[m] = 0;
        if (lane == j) {
            my_e = static_cast<int>(e);
            my_s = es;
        }
    }
}
// Not inlined: the rough selection brings its code into the instruction cache,
// from which the weight stream keeps everything away, before the exact one
// runs it.
__device__ __noinline__ void topk_any(const float *row, const float *bias, int E, int k, int lane, int &e, float &s) {
    if (E <= 256) topk_keys<8>(row, bias, E, k, lane, e, s);
    else topk_keys<kMaxPerLane>(row, bias, E, k, lane, e, s);
}

// One warp appends the set bits of `set` that `without` lacks, in ascending
// order, to `list` from position n on; returns the new length.
__device__ __noinline__ int append_set(const uint32_t *set, const uint32_t *without, uint16_t *list, int n, int lane) {
    const uint32_t m = set[lane] & (without ? ~without[lane] : 0xffffffffu);
    int before = __popc(m);
    const int mine = before;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, before, off);
        if (lane >= off) before += o;
    }
    int at = n + before - mine;
    for (uint32_t b = m; b; b &= b - 1) list[at++] = static_cast<uint16_t>(32 * lane + __ffs(b) - 1);
    return n + __shfl_sync(0xffffffffu, before, 31);
}

template <bool FP8>
__global__ void __launch_bounds__(FEW_THREADS, 1)
moe_few_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w13,
               const __grid_constant__ CUtensorMap tmap_h, const __grid_constant__ CUtensorMap tmap_w2,
               const FewParams p) {
    extern __shared__ uint8_t smem_raw[];
    FewSmem &s = *reinterpret_cast<FewSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int G = gridDim.x, cta = blockIdx.x;
    const int T = p.T, d = p.d, E = p.E, k = p.k, de = p.de;
    constexpr int KE = FP8 ? 128 : 64;  // elements of a 128-byte K block
    const int KB1 = d / KE, KB2 = de / KE;
    const int nf = de / 128, nd = d / 128;
    volatile int *abort = &s.abort;

    if (tid == 0) {
        for (int i = 0; i < FEW_STAGES; ++i) {
            mbar_init(&s.full[i], 1 + 4);
            mbar_init(&s.done[i], 1);
        }
        for (int i = 0; i < SC_RING; ++i) {
            mbar_init(&s.sfull[i], 32);
            mbar_init(&s.sempty[i], 4);
        }
        for (int i = 0; i < QUEUE; ++i) {
            mbar_init(&s.qfull[i], 1);
            mbar_init(&s.qempty[i], FP8 ? 6 : 5);  // MMA, scales, four epilogue warps
        }
        for (int i = 0; i < SIGNALS; ++i) {
            mbar_init(&s.sig_full[i], 128);
            mbar_init(&s.sig_free[i], 1);
        }
        mbar_init(&s.selected, 1);
        mbar_init(&s.routed, 1);
        mbar_init(&s.mma_done, 1);
        s.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&tmap_x);
        prefetch_tmap(&tmap_w13);
        prefetch_tmap(&tmap_h);
        prefetch_tmap(&tmap_w2);
    }
    if (tid < 32) s.rough_set[tid] = s.exact_set[tid] = 0;
    for (int i = tid; i < static_cast<int>(sizeof s.h_ready) / 4; i += FEW_THREADS) reinterpret_cast<uint32_t *>(s.h_ready)[i] = 0;
    __syncthreads();

    // --------------- 1. x, rough logits, rough selection (warps 0-7; the exact
    // logits run in warps 8-11 meanwhile)
    bool ready = true;
    uint32_t tmem_base = 0;
    if (warp < 8) {
        if (warp == 1) {
            tmem_alloc(&s.tmem_base, TMEM_COLS);
            tmem_relinquish();
        }
        if constexpr (FP8) {
            // half-warps over the (token, 128-column) tiles of all CTAs
            const int half = cta * (MAIN_THREADS / 16) + tid / 16, l16 = tid % 16;
            for (int i0 = half & ~1; i0 < T * nd; i0 += G * (MAIN_THREADS / 16)) {
                const int i = i0 + (half & 1);
                const bool in = i < T * nd;
                const int t = in ? i / nd : 0, kb = in ? i % nd : 0, c = kb * 128 + l16 * 8;
                float v[8];
                widen8(*reinterpret_cast<const uint4 *>(p.x + static_cast<size_t>(t) * d + c), v);
                uint2 code;
                const float sc = quant_tile8(v, p.ue, &code);
                if (in) {
                    *reinterpret_cast<uint2 *>(p.xq + static_cast<size_t>(t) * d + c) = code;
                    if (l16 == 0) p.xs[kb * FT + t] = sc;
                }
            }
        }
        // rough logits of experts cta, cta + G, ..., two at a time: a thread holds
        // a few columns of both rows and goes through the tokens, the next
        // token's loads in flight.  (The code is short because it runs once:
        // unrolled over tokens as well it took 4 us for one token, most of
        // them instruction fetches.)
        const int ne = E > cta ? (E - 1 - cta) / G + 1 : 0;
        constexpr int NV = 4;
        float(*part)[2 * FT] = reinterpret_cast<float(*)[2 * FT]>(s.sc);  // [warp][token][expert]
        static_assert(sizeof s.sc >= MAIN_THREADS / 32 * 2 * FT * 4, "partial sums of the rough logits");
        for (int e0 = 0; e0 < ne; e0 += 2) {
            float mine = 0.0f;  // lane 2t + j: this warp's sum of (token t, expert j)
            for (int v0 = tid; v0 < (d / 8 + MAIN_THREADS - 1) / MAIN_THREADS * MAIN_THREADS; v0 += NV * MAIN_THREADS) {
                const uint4 *w0 = reinterpret_cast<const uint4 *>(p.w_router + static_cast<size_t>(cta + e0 * G) * d);
                const uint4 *w1 = reinterpret_cast<const uint4 *>(p.w_router + static_cast<size_t>(cta + min(e0 + 1, ne - 1) * G) * d);
                const uint4 *xr = reinterpret_cast<const uint4 *>(p.x);
                uint4 a0[NV], a1[NV], b[NV];
#pragma unroll
                for (int c = 0; c < NV; ++c) {
                    const int v = v0 + c * MAIN_THREADS;
                    a0[c] = a1[c] = b[c] = make_uint4(0, 0, 0, 0);
                    if (v < d / 8) a0[c] = __ldg(w0 + v), a1[c] = __ldg(w1 + v), b[c] = __ldg(xr + v);
                }
#pragma unroll 1
                for (int t = 0; t < T; ++t) {
                    float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
                    for (int c = 0; c < NV; ++c) {
                        const int v = v0 + c * MAIN_THREADS;
                        const uint32_t xv[4] = {b[c].x, b[c].y, b[c].z, b[c].w}, u[4] = {a0[c].x, a0[c].y, a0[c].z, a0[c].w},
                                       w[4] = {a1[c].x, a1[c].y, a1[c].z, a1[c].w};
                        if (t + 1 < T && v < d / 8) b[c] = __ldg(xr + (t + 1) * (d / 8) + v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            l0 = fmaf(bf16_lo(u[i]), bf16_lo(xv[i]), l0);
                            l1 = fmaf(bf16_lo(w[i]), bf16_lo(xv[i]), l1);
                            l0 = fmaf(bf16_hi(u[i]), bf16_hi(xv[i]), l0);
                            l1 = fmaf(bf16_hi(w[i]), bf16_hi(xv[i]), l1);
                        }
                    }
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) {
                        l0 += __shfl_xor_sync(0xffffffffu, l0, off);
                        l1 += __shfl_xor_sync(0xffffffffu, l1, off);
                    }
                    if (lane == 2 * t) mine += l0;
                    if (lane == 2 * t + 1) mine += l1;
                }
            }
            part[warp][lane] = mine;
            named_bar_sync(3, MAIN_THREADS);
            if (tid < 2 * T && e0 + (tid & 1) < ne) {
                float l = 0.0f;
#pragma unroll
                for (int w = 0; w < MAIN_THREADS / 32; ++w) l += part[w][tid];
                p.rough[static_cast<size_t>(tid >> 1) * E + cta + (e0 + (tid & 1)) * G] = __fdividef(1.0f, 1.0f + __expf(-l));
            }
            if (e0 + 2 < ne) named_bar_sync(3, MAIN_THREADS);
        }
        // The shared expert's weights are needed whatever the routing: into L2
        // while it is found.
        if (tid == 96 && p.n_shared) {
            const size_t es = FP8 ? 1 : 2, b13 = static_cast<size_t>(2) * de * d * es, b2 = static_cast<size_t>(d) * de * es;
            for (size_t o = static_cast<size_t>(cta) * W_BYTES; o < b13; o += static_cast<size_t>(G) * W_BYTES)
                l2_prefetch(p.w13 + E * b13 + o, static_cast<uint32_t>(min(b13 - o, static_cast<size_t>(W_BYTES))));
            for (size_t o = static_cast<size_t>(cta) * W_BYTES; o < b2; o += static_cast<size_t>(G) * W_BYTES)
                l2_prefetch(p.w2 + E * b2 + o, static_cast<uint32_t>(min(b2 - o, static_cast<size_t>(W_BYTES))));
        }
        fence_proxy_async_global();  // the codes of x are read by TMA
        named_bar_sync(3, MAIN_THREADS);
        if (tid == 0) {
            red_release(&p.ctr->prepared, 1);
            wait_count(&p.ctr->prepared, G, p, abort);
            fence_proxy_async_global();
        }
        named_bar_sync(3, MAIN_THREADS);
        ready = !s.abort;  // without x and the rough selection no work is done
        ready = __all_sync(0xffffffffu, ready);
        if (ready)
            for (int t = warp; t < T; t += MAIN_THREADS / 32) {
                int e;
                float sc;
                topk_any(p.rough + static_cast<size_t>(t) * E, p.bias, E, k, lane, e, sc);
                if (lane < k) atomicOr(&s.rough_set[e >> 5], 1u << (e & 31));
            }
        tc_fence_before();
        named_bar_sync(3, MAIN_THREADS);
        tc_fence_after();
        if (warp == 0) {
            if (lane == 0 && p.n_shared) s.list[0] = static_cast<uint16_t>(E);
            const int n = append_set(s.rough_set, nullptr, s.list, p.n_shared, lane);
            __syncwarp();
            if (lane == 0) {
                s.n_rough = s.n_list = n;
                mbar_arrive(&s.selected);
            }
        }
        named_bar_sync(3, MAIN_THREADS);
        tmem_base = __shfl_sync(0xffffffffu, s.tmem_base, 0);
    }
    const int gu_rough = warp < 8 ? s.n_rough * nf : 0;  // gate/up items of the rough selection

    // Work items, numbered: gate/up of the list (all of K), then the down
    // products of the experts selected, in parts of half their K where that is
    // four stages or more (a part's sums go to rows of their own).  A CTA's first
    // is its own number, then it takes the next free one: CTAs that HBM serves
    // faster do more (gate/up of one token ends between 38 and 53 us).  The
    // producer takes it while it loads the one before and hands it to the other
    // roles by a queue.  An item only waits for items of lower number, and a CTA
    // holds one ahead only of a lower one, so the waits end.
    const int S2 = (KB2 + 1) / 2, P2 = S2 >= 4 ? 2 : 1;
    bool routed = false;
    auto decode = [&](int id, Item &it) {
        if (id < 0) return false;
        if (id >= gu_rough && !routed) {
            if (!wait_bar(&s.routed, 0, p, abort)) return false;
            routed = true;
        }
        const int gu = routed ? s.n_list * nf : gu_rough;
        it.down = id >= gu;
        if (!it.down) {
            it.pos = id / nf;
            it.blk = id - it.pos * nf;
            it.q0 = 0;
            it.stages = KB1;
        } else {
            const int item = (id - gu) / P2;
            it.used = item / nd;
            if (it.used >= s.n_used) return false;
            it.part = id - gu - item * P2;
            it.pos = s.used[it.used];
            it.blk = item - it.used * nd;
            it.q0 = it.part * S2 / P2;
            it.stages = (it.part + 1) * S2 / P2 - it.q0;
        }
        it.expert = s.list[it.pos];
        return true;
    };
    // H of list position pos is complete: told by warp 9, whose polling keeps
    // the L2 round trip (1.5 us under the weight stream) out of every item.
    auto wait_h = [&](int pos) {
        volatile uint8_t *flag = &s.h_ready[pos];
        const long long t0 = clock64();
        while (!*flag) {
            if (*abort) return false;
            if (clock64() - t0 > kWaitBudgetCycles) {
                *abort = 1;
                atomicExch(&p.ctr->abort, 1);
                set_status(p.status, MOE_ERR_TIMEOUT);
                return false;
            }
        }
        __threadfence_block();
        return true;
    };
    // the other roles' side of the queue (whole warps)
    struct Taken {
        int slot;
        uint32_t phase;
    };
    auto take = [&](Taken &q, Item &it) {
        const bool got = __all_sync(0xffffffffu, ready && wait_bar(&s.qfull[q.slot], q.phase, p, abort));
        const int id = got ? s.queue[q.slot] : -1;
        __syncwarp();
        if (got && lane == 0) mbar_arrive(&s.qempty[q.slot]);
        if (++q.slot == QUEUE) {
            q.slot = 0;
            q.phase ^= 1;
        }
        return __all_sync(0xffffffffu, decode(id, it));
    };

    if (warp == 0) {
        // ------------------------------------------------------- producer
        // One lane; coordinates advance by constants, since every instruction
        // of this loop costs a lone thread about five clocks (address arithmetic
        // in it held a stage to 1130 clk; a stage of HBM takes 1190, one of L2
        // 470).
        if (lane == 0) {
            const uint32_t w_base = smem_u32(s.w[0][0]), x_base = smem_u32(s.x[0][0]), f_base = smem_u32(&s.full[0]);
            const uint64_t once = l2_evict_first(), keep = l2_evict_normal();  // a weight is read once
            const int x_bytes = T * 128;  // boxes of the tokens there are (the other columns hold anything)
            int stage = 0;
            uint32_t phase = 0, armed = 0, armed_phase = 0;
            bool ok = true;
            Item it;
            int slot = 0, id = cta;
            uint32_t qphase = 0;
            auto publish = [&](int v) {
                if (!wait_bar(&s.qempty[slot], qphase ^ 1, p, abort)) return false;
                s.queue[slot] = v;
                mbar_arrive(&s.qfull[slot]);
                if (++slot == QUEUE) {
                    slot = 0;
                    qphase ^= 1;
                }
                return true;
            };
            while (ok && ready && decode(id, it)) {
                if (!publish(id)) {
                    ok = false;
                    break;
                }
                id = G + atomicAdd(&p.ctr->next, 1);  // in flight while this item is loaded
                // tiles a and b of a stage: gate and up rows of one K block, or
                // two K blocks of the same rows
                const CUtensorMap *wm = it.down ? &tmap_w2 : &tmap_w13, *xm = it.down ? &tmap_h : &tmap_x;
                const int per = it.down ? 2 : 1;  // K blocks a stage
                const long long band = it.down ? static_cast<long long>(it.expert) * nd + it.blk
                                               : static_cast<long long>(it.expert) * 2 * nf + it.blk;
                const int kb = per * it.q0, KB = it.down ? KB2 : KB1;
                int ax, ay, bx, by, dx, dy;
                if (p.w_rowmajor) {
                    ax = kb * KE, ay = static_cast<int>(band * 128);
                    bx = it.down ? ax + KE : ax, by = it.down ? ay : ay + nf * 128;
                    dx = per * KE, dy = 0;
                } else {
                    ax = bx = 0, ay = static_cast<int>((band * KB + kb) * 128);
                    by = it.down ? ay + 128 : ay + nf * KB1 * 128;
                    dx = 0, dy = per * 128;
                }
                const int xy = it.down ? it.pos * FT : 0, last = it.q0 + it.stages - 1;
                const bool odd = it.down && 2 * last + 1 == KB2;  // the last stage holds one K block
                int xx = kb * KE;
                // H is loaded once the expert's H is complete; the weights of the
                // ring's stages go ahead of that
                bool have_x = !it.down;
                int deferred = 0;
                auto load_x = [&](int st, int x0, bool two) {
                    tma_load_2d_policy(x_base + st * 2 * X_BYTES, xm, x0, xy, f_base + st * 8, keep);
                    if (two) tma_load_2d_policy(x_base + st * 2 * X_BYTES + X_BYTES, xm, x0 + KE, xy, f_base + st * 8, keep);
                };
                auto flush = [&](bool short_last) {  // the last `deferred` stages issued wait for their tokens
                    have_x = wait_h(it.pos);
                    fence_proxy_async_global();
                    // (given up: whatever H holds, so that the drain below ends)
                    for (; deferred > 0; --deferred)
                        load_x((stage - deferred + FEW_STAGES) % FEW_STAGES, xx - deferred * 2 * KE, deferred > 1 || !short_last);
                    return have_x;
                };
                volatile uint8_t *h_flag = &s.h_ready[it.pos];
                for (int q = it.q0; q <= last; ++q) {
                    if (!have_x && (deferred == FEW_STAGES || *h_flag) && !flush(false)) {
                        ok = false;
                        break;
                    }
                    if (!wait_bar(&s.done[stage], phase ^ 1, p, abort)) {
                        ok = false;
                        break;
                    }
                    const bool one = odd && q == last;
                    const uint32_t bar = f_base + stage * 8, w = w_base + stage * 2 * W_BYTES;
                    mbar_arrive_expect_tx(&s.full[stage], one ? W_BYTES + x_bytes : 2 * W_BYTES + per * x_bytes);
                    tma_load_2d_policy(w, wm, ax, ay, bar, once);
                    if (!one) tma_load_2d_policy(w + W_BYTES, wm, bx, by, bar, once);
                    if (have_x) load_x(stage, xx, it.down && !one);
                    else ++deferred;
                    ax += dx, ay += dy, bx += dx, by += dy, xx += per * KE;
                    armed |= 1u << stage;
                    armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == FEW_STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (deferred > 0 && !flush(ok && odd)) ok = false;
            }
            if (ok && ready) publish(-1);
            const long long t0 = clock64();
            for (int st = 0; st < FEW_STAGES; ++st) {
                if (!(armed >> st & 1)) continue;
                while (!mbar_try_wait(&s.full[st], armed_phase >> st & 1)) {
                    if (clock64() - t0 > kWaitBudgetCycles) {
                        set_status(p.status, MOE_ERR_TIMEOUT);
                        break;
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        // One wait and one commit a stage, the warp together: with separate
        // barriers for operands and accumulators on both sides, and one lane
        // issuing, a stage took 1340 clk here, which held the whole stream to
        // 6.4 TB/s; the eight MMAs themselves take 330.
        constexpr uint32_t idesc = instr_desc<FP8>(128, FT);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        Taken taken{0, 0};
        Item it;
        const uint64_t wd0 = smem_desc_sw128(smem_u32(s.w[0][0])), xd0 = smem_desc_sw128(smem_u32(s.x[0][0]));
        while (ok && take(taken, it)) {
            // both tiles of a gate/up stage take the same tokens
            const uint64_t x_step = it.down ? X_BYTES >> 4 : 0;
            for (int q = it.q0; q < it.q0 + it.stages; ++q) {
                if (!__all_sync(0xffffffffu, wait_bar(&s.full[stage], phase, p, abort))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t dt = tmem_base + 2 * stage * FT;
                const uint64_t wd = wd0 + stage * (2 * W_BYTES >> 4), xd = xd0 + stage * (2 * X_BYTES >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) tc_mma<FP8>(dt, wd + 2 * kk, xd + 2 * kk, idesc, kk != 0);
                    if (!it.down || 2 * q + 1 < KB2)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma<FP8>(dt + FT, wd + (W_BYTES >> 4) + 2 * kk, xd + x_step + 2 * kk, idesc, kk != 0);
                    tc_commit(&s.done[stage]);
                }
                __syncwarp();
                if (++stage == FEW_STAGES) {
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
    } else if (warp == 2) {
        // --------------------------------------------------------- scales
        // lanes 0-3: the first tile's token scales (16 bytes each), 4-7 the
        // second's, 8 and 9 the tiles' weight scales.  The token scales bypass
        // L1 (other CTAs wrote them during this launch).
        if constexpr (FP8) {
            int slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            Taken taken{0, 0};
            Item it;
            while (ok && take(taken, it)) {
                if (it.down && !__all_sync(0xffffffffu, wait_h(it.pos))) break;
                for (int q = it.q0; q < it.q0 + it.stages; ++q) {
                    if (!__all_sync(0xffffffffu, wait_bar(&s.sempty[slot], phase ^ 1, p, abort))) {
                        ok = false;
                        break;
                    }
                    const int n = it.down ? min(2, KB2 - 2 * q) : 2;
                    if (lane < 8) {
                        const int j = lane >> 2;
                        const float *src = it.down ? p.hs + (static_cast<size_t>(it.pos) * KB2 + min(2 * q + j, KB2 - 1)) * FT
                                                   : p.xs + q * FT;
                        cp_async16(&s.sc[slot].x[j][4 * (lane & 3)], src + 4 * (lane & 3), true);
                    } else if (lane < 8 + n) {
                        const int j = lane - 8;
                        const float *src = it.down
                            ? p.w2_scales + (static_cast<size_t>(it.expert) * nd + it.blk) * KB2 + 2 * q + j
                            : p.w13_scales + (static_cast<size_t>(it.expert) * 2 * nf + j * nf + it.blk) * KB1 + q;
                        cp_async4(&s.sc[slot].w[j], src, true);
                    }
                    cp_async_mbar_arrive(&s.sfull[slot]);
                    if (++slot == SC_RING) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
            cp_async_wait_all();
        }
    } else if (warp == 3) {
        // -------------------------------------------------------- signals
        // The release to the other CTAs waits for the item's stores to arrive
        // (1 to 2 us under the weight stream): here, not in the epilogue.
        int slot = 0;
        uint32_t phase = 0;
        while (ready && __all_sync(0xffffffffu, wait_bar(&s.sig_full[slot], phase, p, abort))) {
            int *count = s.sig_count[slot];
            if (!count) break;
            if (lane == 0) {
                red_release(count, s.sig_add[slot]);
                mbar_arrive(&s.sig_free[slot]);
            }
            if (++slot == SIGNALS) {
                slot = 0;
                phase ^= 1;
            }
        }
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------- epilogue
        const int q4 = warp & 3, r = q4 * 32 + lane, etid = tid - 128;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q4 * 32) << 16);
        int stage = 0, slot = 0;
        uint32_t phase = 0, sphase = 0;
        bool ok = true;
        Taken taken{0, 0};
        Item it;
        if (lane < FEW_STAGES) mbar_arrive(&s.full[lane]);  // the accumulators are free
        __syncwarp();
        int sig = 0;
        uint32_t sig_phase = 0;
        // *count += add once the stores that all four warps have made arrive
        auto signal = [&](int *count, int add) {
            bool free = true;
            if (etid == 0) {
                free = wait_bar(&s.sig_free[sig], sig_phase ^ 1, p, abort);
                s.sig_count[sig] = count;
                s.sig_add[sig] = add;
            }
            __syncwarp();
            if (free) mbar_arrive(&s.sig_full[sig]);
            if (++sig == SIGNALS) {
                sig = 0;
                sig_phase ^= 1;
            }
        };
        // the four warps agree on every step that has a barrier of theirs
        auto all_ok = [&](bool mine) {
            int all;
            __syncwarp();
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
                         "bar.red.and.pred q, 1, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                         : "=r"(all) : "r"(mine ? 1 : 0) : "memory");
            return all != 0;
        };
        while (true) {
            if (!all_ok(take(taken, it))) break;
            float acc0[FT], acc1[FT];
#pragma unroll
            for (int t = 0; t < FT; ++t) acc0[t] = acc1[t] = 0.0f;
            for (int q = it.q0; q < it.q0 + it.stages; ++q) {
                bool go = true;
                if constexpr (FP8) go = wait_bar(&s.sfull[slot], sphase, p, abort);
                go = go && wait_bar(&s.done[stage], phase, p, abort);
                if (!__all_sync(0xffffffffu, go)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const bool both = !it.down || 2 * q + 1 < KB2;
                float v[32];
                tmem_ld32(lane_base + 2 * stage * FT, v);
                tmem_wait_ld(v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.full[stage]);
                if constexpr (FP8) {
                    const auto &sc = s.sc[slot];
                    const float w0 = sc.w[0], w1 = sc.w[1];
#pragma unroll
                    for (int t = 0; t < FT; t += 4) {
                        const float4 x0 = *reinterpret_cast<const float4 *>(&sc.x[0][t]);
                        acc0[t] = __fmaf_rn(v[t], __fmul_rn(x0.x, w0), acc0[t]);
                        acc0[t + 1] = __fmaf_rn(v[t + 1], __fmul_rn(x0.y, w0), acc0[t + 1]);
                        acc0[t + 2] = __fmaf_rn(v[t + 2], __fmul_rn(x0.z, w0), acc0[t + 2]);
                        acc0[t + 3] = __fmaf_rn(v[t + 3], __fmul_rn(x0.w, w0), acc0[t + 3]);
                        if (both) {
                            const float4 x1 = *reinterpret_cast<const float4 *>(&sc.x[1][t]);
                            acc1[t] = __fmaf_rn(v[FT + t], __fmul_rn(x1.x, w1), acc1[t]);
                            acc1[t + 1] = __fmaf_rn(v[FT + t + 1], __fmul_rn(x1.y, w1), acc1[t + 1]);
                            acc1[t + 2] = __fmaf_rn(v[FT + t + 2], __fmul_rn(x1.z, w1), acc1[t + 2]);
                            acc1[t + 3] = __fmaf_rn(v[FT + t + 3], __fmul_rn(x1.w, w1), acc1[t + 3]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.sempty[slot]);
                    if (++slot == SC_RING) {
                        slot = 0;
                        sphase ^= 1;
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < FT; ++t) {
                        acc0[t] = __fadd_rn(acc0[t], v[t]);
                        if (both) acc1[t] = __fadd_rn(acc1[t], v[FT + t]);
                    }
                }
                if (++stage == FEW_STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!all_ok(ok)) break;
            if (!it.down) {
                // H = silu(G) U of feature blk*128 + r, every token; then its
                // 1x128 tile's codes (the tile is this CTA's 128 rows)
                float h[FT];
#pragma unroll
                for (int t = 0; t < FT; ++t) h[t] = __fdividef(acc0[t], 1.0f + __expf(-acc0[t])) * acc1[t];
                const size_t row = static_cast<size_t>(it.pos) * FT;
                if constexpr (FP8) {
#pragma unroll
                    for (int t = 0; t < FT; ++t) {
                        float m = fabsf(h[t]);
#pragma unroll
                        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                        if (lane == 0) s.amax[q4][t] = m;
                    }
                    named_bar_sync(1, 128);
#pragma unroll
                    for (int t = 0; t < FT; ++t) {
                        if (t >= T) break;
                        const float m = fmaxf(fmaxf(s.amax[0][t], s.amax[1][t]), fmaxf(s.amax[2][t], s.amax[3][t]));
                        float inv;
                        const float sc = tile_scale(m, p.ue, &inv);
                        static_cast<uint8_t *>(p.h)[(row + t) * de + it.blk * 128 + r] =
                            static_cast<uint8_t>(e4m3x2(__fmul_rn(h[t], inv), 0.0f));
                        if (r == 0) p.hs[(static_cast<size_t>(it.pos) * KB2 + it.blk) * FT + t] = sc;
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < FT; ++t)
                        if (t < T)
                            static_cast<__nv_bfloat16 *>(p.h)[(row + t) * de + it.blk * 128 + r] = __float2bfloat16_rn(h[t]);
                }
                fence_proxy_async_global();  // H is read by TMA
                signal(&p.ctr->h_done[it.pos], 1);
                continue;
            }
            // Y rows of the tokens that chose this expert (binary32: few rows),
            // apart for each part of the product
            const int kk = k + p.n_shared;
            const size_t part_rows = static_cast<size_t>(T) * kk * d;
            if (etid < FT) {
                int rank = -1;
                if (it.expert == E) rank = k;
                else if (etid < T)
                    for (int j = k - 1; j >= 0; --j)
                        if (s.sel[etid][j] == it.expert) rank = j;
                s.rank[etid] = static_cast<int8_t>(rank);
            }
            named_bar_sync(1, 128);
#pragma unroll
            for (int t = 0; t < FT; ++t) {
                if (t >= T) break;
                const int j = s.rank[t];
                if (j >= 0)
                    p.y[it.part * part_rows + (static_cast<size_t>(t) * kk + j) * d + it.blk * 128 + r] = __fadd_rn(acc0[t], acc1[t]);
            }
            signal(&p.ctr->col_done[it.blk], it.stages);
        }
        signal(nullptr, 0);
        // ------------------------------------------------------- combine
        // out = sum_j g_j Y_j (rank order) + shared (+ residual): the (token,
        // 128-column) pieces over the warps of all CTAs, each when every
        // expert's stages of its columns are counted (the last CTA to count
        // doing a whole column block left 16 CTAs with three or four each, 10
        // us at one token).  Lane l takes columns 4l .. 4l + 3.
        if (ready && ok && __all_sync(0xffffffffu, wait_bar(&s.routed, 0, p, abort))) {
            const int kk = k + p.n_shared;
            const size_t part_rows = static_cast<size_t>(T) * kk * d;
            for (int piece = q4 * G + cta; piece < T * nd; piece += 4 * G) {
                const int t = piece / nd, blk = piece - t * nd;
                if (!__all_sync(0xffffffffu, wait_count(&p.ctr->col_done[blk], s.n_used * S2, p, abort))) break;
                const int c = blk * 128 + lane * 4;
                const float4 *yr = reinterpret_cast<const float4 *>(p.y + static_cast<size_t>(t) * kk * d + c);
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                constexpr int BATCH = 5;  // ranks whose loads are in flight together
                for (int j0 = 0; j0 < kk; j0 += BATCH) {
                    float4 v[BATCH], v1[BATCH];
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) {
                        if (j0 + j >= kk) break;
                        const float4 *src = yr + static_cast<size_t>(j0 + j) * (d / 4);
                        v[j] = __ldcg(src);
                        v1[j] = P2 > 1 ? __ldcg(src + part_rows / 4) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) {
                        if (j0 + j >= kk) break;
                        const float g = j0 + j < k ? s.gate[t][j0 + j] : 1.0f;
                        acc.x = __fmaf_rn(g, __fadd_rn(v[j].x, v1[j].x), acc.x);
                        acc.y = __fmaf_rn(g, __fadd_rn(v[j].y, v1[j].y), acc.y);
                        acc.z = __fmaf_rn(g, __fadd_rn(v[j].z, v1[j].z), acc.z);
                        acc.w = __fmaf_rn(g, __fadd_rn(v[j].w, v1[j].w), acc.w);
                    }
                }
                const size_t at = static_cast<size_t>(t) * d + c;
                if (p.residual) {
                    const uint2 res = *reinterpret_cast<const uint2 *>(p.residual + at);
                    acc.x = __fadd_rn(acc.x, bf16_lo(res.x));
                    acc.y = __fadd_rn(acc.y, bf16_hi(res.x));
                    acc.z = __fadd_rn(acc.z, bf16_lo(res.y));
                    acc.w = __fadd_rn(acc.w, bf16_hi(res.y));
                }
                *reinterpret_cast<uint2 *>(p.out + at) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
            }
        }
    } else if (warp >= 8) {
        // -------------------------------------------------- exact routing
        // One lane a (token, expert) logit: sequential fused multiply-adds over
        // d.  The operands come through a ring in shared memory: read straight
        // from L2, under the load of the weight stream, they took 100 us at d =
        // 7168 (a chain needs 15); and 45 us with the copies issued by the
        // warp that runs the chains.
        const int rt = tid - 256, rw = warp - 8;
        const int ne = E > cta ? (E - 1 - cta) / G + 1 : 0;
        const int per_pass = min(RC_ROWS - T, 32 / T);  // experts a pass: a warp's lanes
        for (int e0 = 0; e0 < ne; e0 += per_pass) {
            const int n = min(per_pass, ne - e0), rows = n + T;
            auto load_chunk = [&](int c) {  // rows 0 .. n - 1: router, then the tokens
                for (int v = rt; v < rows * (RC / 8); v += ROUTE_THREADS - 32) {
                    const int row = v / (RC / 8), col = v % (RC / 8) * 8;
                    const uint16_t *src = row < n ? p.w_router + static_cast<size_t>(cta + (e0 + row) * G) * d
                                                  : p.x + static_cast<size_t>(row - n) * d;
                    cp_async16(&s.chunk[c % RC_BUFS][row][col], src + c * RC + col, true);
                }
            };
            const int nc = d / RC;
            if (rw < 3) {  // three warps copy, chunk after chunk; the fourth has its scheduler nearly to itself
#pragma unroll
                for (int c = 0; c < RC_BUFS - 1; ++c) {
                    if (c < nc) load_chunk(c);
                    cp_async_commit();
                }
                for (int c = 0; c < nc; ++c) {
                    cp_async_wait<RC_BUFS - 2>();
                    named_bar_sync(2, ROUTE_THREADS);  // chunk c landed; chunk c - 1 is done with
                    if (c + RC_BUFS - 1 < nc) load_chunk(c + RC_BUFS - 1);
                    cp_async_commit();
                }
                cp_async_wait<0>();
                named_bar_sync(2, ROUTE_THREADS);  // the ring is free for the next pass
                continue;
            }
            const bool mine = lane < n * T;
            const int t = mine ? lane % T : 0, ei = mine ? lane / T : 0;
            float l = 0.0f;
            for (int c = 0; c < nc; ++c) {
                named_bar_sync(2, ROUTE_THREADS);
                const uint4 *wr = reinterpret_cast<const uint4 *>(s.chunk[c % RC_BUFS][ei]);
                const uint4 *xr = reinterpret_cast<const uint4 *>(s.chunk[c % RC_BUFS][n + t]);
                // operands two vectors ahead of the chain (a 3-slot register ring)
                constexpr int NV = RC / 8, PD = 2;
                uint4 av[PD + 1], bv[PD + 1];
#pragma unroll
                for (int v = 0; v < PD; ++v) av[v] = wr[v], bv[v] = xr[v];
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    if (v + PD < NV) av[(v + PD) % (PD + 1)] = wr[v + PD], bv[(v + PD) % (PD + 1)] = xr[v + PD];
                    const uint4 a = av[v % (PD + 1)], b = bv[v % (PD + 1)];
                    l = __fmaf_rn(bf16_lo(b.x), bf16_lo(a.x), l);
                    l = __fmaf_rn(bf16_hi(b.x), bf16_hi(a.x), l);
                    l = __fmaf_rn(bf16_lo(b.y), bf16_lo(a.y), l);
                    l = __fmaf_rn(bf16_hi(b.y), bf16_hi(a.y), l);
                    l = __fmaf_rn(bf16_lo(b.z), bf16_lo(a.z), l);
                    l = __fmaf_rn(bf16_hi(b.z), bf16_hi(a.z), l);
                    l = __fmaf_rn(bf16_lo(b.w), bf16_lo(a.w), l);
                    l = __fmaf_rn(bf16_hi(b.w), bf16_hi(a.w), l);
                }
            }
            named_bar_sync(2, ROUTE_THREADS);
            if (mine) p.scores[static_cast<size_t>(t) * E + cta + (e0 + ei) * G] = sigmoid_cw(l, exp_consts());
        }
        named_bar_sync(2, ROUTE_THREADS);
        if (rt == 0) {
            red_release(&p.ctr->scored, 1);
            wait_count(&p.ctr->scored, G + p.inject_fault, p, abort);
        }
        named_bar_sync(2, ROUTE_THREADS);
        if (!*abort) {
            for (int t = rw; t < T; t += 4) {
                int e;
                float sc;
                topk_any(p.scores + static_cast<size_t>(t) * E, p.bias, E, k, lane, e, sc);
                const float g = warp_gate(sc, k, p.routed_scale);
                if (lane < k) {
                    s.sel[t][lane] = static_cast<uint16_t>(e);
                    s.gate[t][lane] = g;
                    atomicOr(&s.exact_set[e >> 5], 1u << (e & 31));
                    if (cta == 0) {
                        p.idx_out[static_cast<size_t>(t) * k + lane] = e;
                        p.gates_out[static_cast<size_t>(t) * k + lane] = g;
                    }
                }
            }
        }
        named_bar_sync(2, ROUTE_THREADS);
        if (rw == 0 && __all_sync(0xffffffffu, wait_bar(&s.selected, 0, p, abort)) && !*abort) {
            const int n = append_set(s.exact_set, s.rough_set, s.list, s.n_rough, lane);
            __syncwarp();
            // positions of the selected experts, in list order
            int n_used = 0;
            for (int j0 = 0; j0 < n; j0 += 32) {
                const int j = j0 + lane;
                const int e = j < n ? s.list[j] : 0;
                const bool use = j < n && (e == E || (s.exact_set[e >> 5] >> (e & 31) & 1));
                const uint32_t m = __ballot_sync(0xffffffffu, use);
                if (use) s.used[n_used + __popc(m & ((1u << lane) - 1))] = static_cast<uint16_t>(j);
                n_used += __popc(m);
            }
            __syncwarp();
            if (lane == 0) {
                s.n_list = n;
                s.n_used = n_used;
                mbar_arrive(&s.routed);
            }
        }
        if (rw == 1 && __all_sync(0xffffffffu, wait_bar(&s.routed, 0, p, abort))) {
            // watch the list's experts until every H is complete
            const long long t0 = clock64();
            bool all = false;
            while (!all && !*abort) {
                all = true;
                for (int pos = lane; pos < s.n_list; pos += 32) {
                    if (s.h_ready[pos]) continue;
                    if (ld_acquire(&p.ctr->h_done[pos]) >= nf) {
                        __threadfence_block();
                        *static_cast<volatile uint8_t *>(&s.h_ready[pos]) = 1;
                    } else {
                        all = false;
                    }
                }
                all = __all_sync(0xffffffffu, all);
                if (!all && (ld_acquire(&p.ctr->abort) || clock64() - t0 > kWaitBudgetCycles)) break;
            }
        }
    }

    // ------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
    if (tid == 0) s.last = add_acq_rel(&p.ctr->exited, 1) == G - 1;
    __syncthreads();
    if (s.last) {  // nobody waits any more: every counter back to zero
        int *c = reinterpret_cast<int *>(p.ctr);
        for (int j = tid; j < static_cast<int>(sizeof(FewCounters) / sizeof(int)); j += FEW_THREADS) c[j] = 0;
    }
}

// Pre-norm of the few tokens, a block each: x = bf16((h * rstd) * gamma).
__global__ void __launch_bounds__(256)
few_prenorm_kernel(const uint16_t *__restrict__ h, const uint16_t *__restrict__ gamma, int d, float eps,
                   uint16_t *__restrict__ xn) {
    __shared__ __align__(16) uint16_t chunk[kRstdChunk];
    __shared__ float rstd_sh;
    const uint16_t *row = h + static_cast<size_t>(blockIdx.x) * d;
    pdl_wait_and_trigger();
    const float rstd = block_rstd(row, d, eps, chunk, &rstd_sh);
    for (int v = threadIdx.x; v < d / 8; v += blockDim.x) {
        float x[8];
        prenorm8(reinterpret_cast<const uint4 *>(row)[v], reinterpret_cast<const uint4 *>(gamma)[v], rstd, x);
        reinterpret_cast<uint4 *>(xn + static_cast<size_t>(blockIdx.x) * d)[v] =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
}

}  // namespace

cudaError_t launch_few_prenorm(const uint16_t *h, const uint16_t *gamma, int T, int d, float eps, uint16_t *xn,
                               cudaStream_t st, int *launches) {
    mark_launch(st, *launches, "few_prenorm");
    LAUNCH_OR_RETURN(launch_pdl(few_prenorm_kernel, dim3(T), dim3(256), 0, st, h, gamma, d, eps, xn));
    ++*launches;
    return cudaGetLastError();
}

cudaError_t launch_few(const FewArgs &g, cudaStream_t st, int *launches) {
    const moe_shape &s = *g.shape;
    const bool fp8 = s.precision != MOE_BF16;
    const int slots = s.n_experts + s.n_shared;
    const int es = fp8 ? 1 : 2;
    const bool rm = s.weight_layout == MOE_LAYOUT_ROWMAJOR;
    CUtensorMap mx, m13, mh, m2;
    const long long rows13 = static_cast<long long>(slots) * 2 * s.d_expert, rows2 = static_cast<long long>(slots) * s.d_model;
    const long long t13 = rm ? rows13 : rows13 * s.d_model * es / 128, t2 = rm ? rows2 : rows2 * s.d_expert * es / 128;
    if (t13 >= (1LL << 31) || t2 >= (1LL << 31)) return cudaErrorInvalidValue;
    const int per = 128 / es;
    const void *xop = fp8 ? static_cast<const void *>(g.xq) : g.x;
    if (!make_map_2d(&mx, xop, fp8, s.d_model, s.T, s.T) ||
        !make_map_2d(&mh, g.h, fp8, s.d_expert, g.list_rows * FT, s.T) ||
        !make_map_2d(&m13, g.w13, fp8, rm ? s.d_model : per, static_cast<int>(t13)) ||
        !make_map_2d(&m2, g.w2, fp8, rm ? s.d_expert : per, static_cast<int>(t2)))
        return cudaErrorInvalidValue;
    FewParams p{};
    p.x = g.x;
    p.residual = g.residual;
    p.w_router = g.w_router;
    p.bias = g.bias;
    p.w13 = static_cast<const uint8_t *>(g.w13);
    p.w2 = static_cast<const uint8_t *>(g.w2);
    p.w13_scales = g.w13_scales;
    p.w2_scales = g.w2_scales;
    p.out = g.out;
    p.idx_out = g.idx;
    p.gates_out = g.gates;
    p.xq = g.xq;
    p.xs = g.xs;
    p.rough = g.rough;
    p.scores = g.scores;
    p.h = g.h;
    p.hs = g.hs;
    p.y = g.y;
    p.ctr = g.counters;
    p.status = g.status;
    p.T = s.T;
    p.d = s.d_model;
    p.E = s.n_experts;
    p.k = s.top_k;
    p.de = s.d_expert;
    p.n_shared = s.n_shared;
    p.routed_scale = s.routed_scale;
    p.ue = s.precision == MOE_FP8_UE8M0;
    p.w_rowmajor = rm;
    p.inject_fault = g.inject_fault;
    const size_t smem = sizeof(FewSmem) + 1024;
    static DeviceConfigured configured{};
    if (first_use_on_device(configured)) {
        cudaError_t e = cudaFuncSetAttribute(moe_few_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(moe_few_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        mark_used_on_device(configured);
    }
    mark_launch(st, *launches, "moe_few");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms());
    cfg.blockDim = dim3(FEW_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // CTAs wait for one another: all resident, or no launch
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    LAUNCH_OR_RETURN(fp8 ? cudaLaunchKernelEx(&cfg, moe_few_kernel<true>, mx, m13, mh, m2, p)
                         : cudaLaunchKernelEx(&cfg, moe_few_kernel<false>, mx, m13, mh, m2, p));
    ++*launches;
    return cudaGetLastError();
}

}  // namespace moe
