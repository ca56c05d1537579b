// Arithmetic of the router shared by its kernels: the sigmoid, the pre-norm of
// an input vector, and the top-k selection and gates of one token by one warp
// ("DeepSeek v3 and R1 Model Architecture", section "Local Balanced Routing to
// Experts").
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moe {

// ------------------------------------------------- exp / sigmoid (binary32)
// Constants derived from their definitions: ln 2 split into a head with the
// low 12 significand bits cleared (so n * head is exact for |n| < 2^12) and
// a tail; Taylor coefficients 1/i! rounded to binary32.
constexpr double kLn2 = 0.693147180559945309417232121458176568;
constexpr double kLog2e = 1.442695040888963407359924681001892137;

struct ExpConsts {
    float log2e, ln2_hi, ln2_lo, c[8];
};

__device__ __forceinline__ ExpConsts exp_consts() {
    ExpConsts k;
    k.log2e = static_cast<float>(kLog2e);
    k.ln2_hi = __uint_as_float(__float_as_uint(static_cast<float>(kLn2)) & 0xfffff000u);
    k.ln2_lo = static_cast<float>(kLn2 - static_cast<double>(k.ln2_hi));
    double f = 1.0;
    for (int i = 0; i < 8; ++i) {
        if (i) f *= i;
        k.c[i] = static_cast<float>(1.0 / f);
    }
    return k;
}

// 8 bf16 x values (one 16-byte vector) of token t at absolute column c0:
// the input itself, or the pre-norm of the residual stream h.
__device__ __forceinline__ uint4 x_vec(uint4 raw, const PreNorm &pn, int t, int c0) {
    if (!pn.gamma) return raw;
    const float r = pn.rstd[t];
    const uint4 gr = *reinterpret_cast<const uint4 *>(pn.gamma + c0);
    const uint32_t h4[4] = {raw.x, raw.y, raw.z, raw.w}, g4[4] = {gr.x, gr.y, gr.z, gr.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = pack_bf16x2(prenorm_elem(bf16_lo(h4[i]), r, bf16_lo(g4[i])),
                           prenorm_elem(bf16_hi(h4[i]), r, bf16_hi(g4[i])));
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ float sigmoid_cw(float l, const ExpConsts &k) {
    float y = -l;
    y = fminf(fmaxf(y, -87.0f), 87.0f);
    float n = rintf(__fmul_rn(y, k.log2e));
    float r = __fmaf_rn(-n, k.ln2_hi, y);
    r = __fmaf_rn(-n, k.ln2_lo, r);
    float p = k.c[7];
#pragma unroll
    for (int i = 6; i >= 0; --i) p = __fmaf_rn(p, r, k.c[i]);
    // 2^n with n in [-126, 126]: exact scaling of a normal result
    float e = __fmul_rn(p, __int_as_float((static_cast<int>(n) + 127) << 23));
    return __fdiv_rn(1.0f, __fadd_rn(1.0f, e));
}

constexpr int kMaxPerLane = 32;  // experts a lane of warp_topk holds: E <= 1024

// Top-k of one token's E affinities by one warp: sel = s + bias, k rounds of a
// warp arg-max under (sel desc, expert asc).  Lane j < k returns its rank-j
// choice in e and that expert's affinity in s.
template <int PER_LANE>
__device__ __forceinline__ void warp_topk(const float *srow, const float *bias, int E, int k, int lane,
                                          int &my_e, float &my_s) {
    float s[PER_LANE], sel[PER_LANE];
    uint32_t taken = 0;
#pragma unroll
    for (int m = 0; m < PER_LANE; ++m) {
        const int e = lane + 32 * m;
        if (e < E) {
            s[m] = srow[e];
            sel[m] = __fadd_rn(s[m], bias[e]);
        } else {
            s[m] = 0.0f;
            sel[m] = 0.0f;
            taken |= 1u << m;
        }
    }
    my_s = 0.0f;  // lane j keeps the affinity of its rank-j choice
    my_e = 0;
    for (int j = 0; j < k; ++j) {
        // best untaken expert of this lane (lowest index among equals: e grows with m)
        float bv = 0.0f;
        int be = 0x7fffffff;
        float bs = 0.0f;
#pragma unroll
        for (int m = 0; m < PER_LANE; ++m) {
            if (taken & (1u << m)) continue;
            const int e = lane + 32 * m;
            if (be == 0x7fffffff || sel[m] > bv) {
                bv = sel[m];
                be = e;
                bs = s[m];
            }
        }
        // warp arg-max under (sel desc, expert asc); lanes without candidates carry e = INT_MAX
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, off);
            const int oe = __shfl_xor_sync(0xffffffffu, be, off);
            const float os = __shfl_xor_sync(0xffffffffu, bs, off);
            const bool other_better =
                (oe != 0x7fffffff) && (be == 0x7fffffff || ov > bv || (ov == bv && oe < be));
            if (other_better) {
                bv = ov;
                be = oe;
                bs = os;
            }
        }
        if ((be & 31) == lane) taken |= 1u << (be >> 5);
        if (lane == j) {
            my_s = bs;
            my_e = be;
        }
    }
}

// Gate of lane j's rank-j choice: g_j = s_j / S * routed_scale, S the binary32
// sum of the selected s in rank order.
__device__ __forceinline__ float warp_gate(float my_s, int k, float routed_scale) {
    float S = 0.0f;
    for (int j = 0; j < k; ++j) S = __fadd_rn(S, __shfl_sync(0xffffffffu, my_s, j));
    return __fmul_rn(__fdiv_rn(my_s, S), routed_scale);
}

}  // namespace moe
