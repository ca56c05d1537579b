// Quantisation of activations by the kernels that read them (linear.cu,
// few.cu): the input vector, pre-normed or not, and its 1x128 tile's codes and
// scale ("DeepSeek-R1" (aguasto.com), "Quantization": blockwise FP8).
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moe {

// Scale and factor of a 1x128 activation tile in the calls that quantise on
// the way to a product (moe_linear, moe_forward_few): scale = amax * (1/448)
// and *inv = 448 * (1/amax), each operation a correctly rounded binary32 one.
// One reciprocal serves both where fp8_block_quant divides twice (a tile is
// quantised again by every CTA that reads it); either value is within an ulp
// of the quotient, so only an element at a border of two codes can differ.
// The factor of a tile below 448 / FLT_MAX is held at FLT_MAX (no code is NaN
// for 0 * inf); an all-zero tile gets scale 1 and factor 0; ue: power-of-two
// scale (ue8m0_scale).  An infinite amax gives factor 0, so the infinity's code
// is NaN and the row's results are, with either scale (ue8m0_scale alone would
// make it 448 * 2^120).
__device__ __forceinline__ float tile_scale(float amax, bool ue, float *inv) {
    if (amax == 0.0f) {
        *inv = 0.0f;
        return 1.0f;
    }
    if (ue) {
        const float sc = ue8m0_scale(amax, inv);
        if (isinf(amax)) *inv = 0.0f;
        return sc;
    }
    *inv = fminf(__fmul_rn(__frcp_rn(amax), 448.0f), 3.402823466e38f);
    return __fmul_rn(amax, static_cast<float>(1.0 / 448.0));
}

// Eight consecutive bf16 columns, widened.
__device__ __forceinline__ void widen8(const uint4 &raw, float (&v)[8]) {
    const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(r[i]);
        v[2 * i + 1] = bf16_hi(r[i]);
    }
}

// A 1x128 tile held by 16 lanes, 8 values each: this lane's codes, and the
// tile's scale.
__device__ __forceinline__ float quant_tile8(const float (&v)[8], bool ue, uint2 *code) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float inv;
    const float sc = tile_scale(m, ue, &inv);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(__fmul_rn(v[2 * i], inv), __fmul_rn(v[2 * i + 1], inv));
    *code = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    return sc;
}

// 1 / sqrt(mean of the squares of a row + eps) as rstd_kernel defines it: lane l
// of one warp sums the squares of columns l mod 32 in order, five butterfly
// rounds add the lanes.  The block stages the row in shared memory for that
// warp (chunk: kRstdChunk columns; d a multiple of 128): 1 us at d = 7168,
// where the warp's own loads from L2 take ten.  Every thread returns it; the
// row's last chunk stays in `chunk`.
constexpr int kRstdChunk = 8192;
__device__ __forceinline__ float block_rstd(const uint16_t *row, int d, float eps, uint16_t *chunk, float *shared) {
    float acc = 0.0f;
    for (int c = 0; c < d; c += kRstdChunk) {
        const int n = min(kRstdChunk, d - c);
        for (int v = threadIdx.x; v < n / 8; v += blockDim.x)
            reinterpret_cast<uint4 *>(chunk)[v] = reinterpret_cast<const uint4 *>(row + c)[v];
        __syncthreads();
        if (threadIdx.x < 32) {
#pragma unroll 8
            for (int i = threadIdx.x; i < n; i += 32) {
                const float v = __uint_as_float(static_cast<uint32_t>(chunk[i]) << 16);
                acc = __fmaf_rn(v, v, acc);
            }
        }
        if (c + kRstdChunk < d) __syncthreads();
    }
    if (threadIdx.x < 32) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, off));
        if (threadIdx.x == 0)
            *shared = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(acc, static_cast<float>(d)), eps)));
    }
    __syncthreads();
    return *shared;
}

// Eight pre-normed columns.
__device__ __forceinline__ void prenorm8(const uint4 &raw, const uint4 &graw, float rstd, float (&v)[8]) {
    const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w}, g[4] = {graw.x, graw.y, graw.z, graw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = prenorm_elem(bf16_lo(r[i]), rstd, bf16_lo(g[i]));
        v[2 * i + 1] = prenorm_elem(bf16_hi(r[i]), rstd, bf16_hi(g[i]));
    }
}

}  // namespace moe
