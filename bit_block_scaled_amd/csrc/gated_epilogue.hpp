// Device code the gated feed-forward kernels share after their products:
// 8-bit checkpoints of a 32-column block, reading them back, output stores.
#pragma once

#include "bbs_device.hpp"
#include "gated.hpp"

namespace bbs {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// A transposed 32 x 32 product block: lane l holds row l % 32 and columns
// 8 (v / 4) + 4 (l / 32) + v % 4, so lanes l and l ^ 32 hold a row's 32
// columns between them, i.e. one MXFP8 block of a checkpoint.

__device__ __forceinline__ void scale16(f32x16 &v, float s) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= s;
}

// MXFP8 codes of the lane's 16 values (word q: columns 8 q + 4 (l / 32)) and
// the block's E8M0 byte, as the quantizer's MXFP8 copy to nearest.
__device__ __forceinline__ uint32_t checkpoint16(const f32x16 &v, uint32_t (&w)[4]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(v[i]));
    a = fmaxf(a, __shfl_xor(a, 32, 64));
    const uint32_t byte = e8m0_byte(a);
    const float scale = e8m0_cvt_scale(byte);
    // byte 0 (2^-127) is converted at 2^-126 after doubling
    const float twice = byte ? 1.0f : 2.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        w[q] = e4m3_rne4_scaled(v[4 * q] * twice, v[4 * q + 1] * twice, v[4 * q + 2] * twice,
                                v[4 * q + 3] * twice, scale);
    return byte;
}

// Into row m, block at column n of an M x N checkpoint, with the words exchanged
// between lanes l and l ^ 32 first: lane half h then holds the block's columns
// 16 h .. 16 h + 15 and stores them at once.  N is a multiple of 32, so a block
// is wholly in or out.  Every lane of the wave takes part.
__device__ __forceinline__ void store_checkpoint16(const uint32_t (&w)[4], uint32_t byte, uint8_t *codes,
                                                   uint8_t *scales, int64_t N, bool row_in, int64_t m,
                                                   int64_t n, int half) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    if (!row_in || n >= N) return;
    *reinterpret_cast<uint4 *>(codes + m * N + n + 16 * half) = make_uint4(a[0], a[1], b[0], b[1]);
    if (half == 0) scales[m * (N / 32) + n / 32] = (uint8_t)byte;
}

template <bool BF16_OUT>
__device__ __forceinline__ void store4(void *base, int64_t at, float y0, float y1, float y2, float y3) {
    if (BF16_OUT)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + at) =
            make_uint2(pk_bf16(y0, y1), pk_bf16(y2, y3));
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(base) + at) = make_float4(y0, y1, y2, y3);
}

// 2^(byte - 127), an FP32 subnormal for byte 0.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Four E4M3 codes of a word times 2^(byte - 127).  The conversion takes its
// scale from the exponent field alone, so byte 0 (2^-127) needs no other
// encoding (measured over every code).
__device__ __forceinline__ void decode4(uint32_t w, uint32_t byte, float (&v)[4]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const float scale = __uint_as_float(byte << 23);
    const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)w, scale, false);
    const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)w, scale, true);
    v[0] = lo[0];
    v[1] = lo[1];
    v[2] = hi[0];
    v[3] = hi[1];
}

// Four consecutive columns of one row through the gated activation's backward
// pass: dgate = dh u act'(g), dup = dh act(g).  g_word, u_word: their
// checkpoint codes; g_byte, u_byte: the block scales.
template <int ACT, bool BF16_OUT>
__device__ __forceinline__ void gated_grad4(const float (&dh)[4], uint32_t g_word, uint32_t g_byte,
                                            uint32_t u_word, uint32_t u_byte, float (&dg)[4], float (&du)[4]) {
    float g[4], u[4];
    decode4(g_word, g_byte, g);
    decode4(u_word, u_byte, u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float slope;
        const float a = gate_act_grad<ACT, BF16_OUT>(g[e], slope);
        dg[e] = dh[e] * u[e] * slope;
        du[e] = dh[e] * a;
    }
}

// Eight consecutive outputs.
template <bool BF16_OUT>
__device__ __forceinline__ void store8(void *base, int64_t at, const float (&a)[4], const float (&b)[4]) {
    if (BF16_OUT) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at) =
            make_uint4(pk_bf16(a[0], a[1]), pk_bf16(a[2], a[3]), pk_bf16(b[0], b[1]), pk_bf16(b[2], b[3]));
    } else {
        store4<false>(base, at, a[0], a[1], a[2], a[3]);
        store4<false>(base, at + 4, b[0], b[1], b[2], b[3]);
    }
}

}  // namespace bbs
