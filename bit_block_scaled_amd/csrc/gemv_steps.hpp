// Steps of the products of a few BF16 tokens with 4-bit weights (gfx950), shared
// by the matrix-vector and the expert kernels: loads of a wave's share of the
// weights and their products by matrix instructions.
#pragma once

#include "bbs_device.hpp"
#include "gated_epilogue.hpp"

namespace bbs {
namespace gemv {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    return __builtin_amdgcn_cvt_scalef32_f32_fp8((int)byte, 1.0f, 0);
}

// B bytes from p, which may lie at any address.
template <int B>
__device__ __forceinline__ uint32_t load_bytes(const uint8_t *p) {
    uint32_t v = 0;
    __builtin_memcpy(&v, p, B);
    return v;
}

// Value n of an array of FP32 values or BF16 patterns.
__device__ __forceinline__ float value_at(const void *p, int64_t n, int bf16) {
    return bf16 ? bf16_to_f32(static_cast<const uint16_t *>(p)[n]) : static_cast<const float *>(p)[n];
}

// Layout of the block scales.
constexpr int kRows16 = 0;       // NVFP4, one E4M3 byte per 16 weights of a row
constexpr int kTiles16 = 1;      // NVFP4, one E4M3 byte per 16 x 16 weights
constexpr int kRows32 = 2;       // MXFP4, one E8M0 byte per 32 weights of a row

// ---------------------------------------------------------------------------
// Up to four tokens: v_mfma_f32_4x4x4_16b_bf16, sixteen independent 4 x 4 x 4
// products.  Lane 4b + i feeds product b: token i's activations and weight row
// i's codes at the same four K values, and receives column i (its own row) for
// the four tokens.  So a lane that holds 16 consecutive codes of one row needs
// four chained instructions to sum its scale block for four tokens, and one
// FMA a token to scale the sum: 0.5 conversions and T / 16 FMAs a weight, and
// no cross-lane work before the end of K.
//
// A wave's step is 512 K values of 4 R rows: lane 4b + i reads 16 bytes (32
// codes) of rows i, 4 + i, ... at K offset 32 b.
// ---------------------------------------------------------------------------
constexpr int kStepK = 512;

template <int NM, int R>
struct Step {
    uint4 w[NM][R];          // 32 codes
    uint32_t s[NM][R];       // two E4M3 bytes or one E8M0 byte
    uint4 x[4];              // 32 activations of one token
};

// The lane's places in a step, set once: byte offsets of its rows from the
// workgroup's first row, and its token's activations.
template <int R>
struct Place {
    uint32_t code[R], scale[R];
    const uint16_t *x;
};

template <int SC, int R>
__device__ __forceinline__ Place<R> place_of(const GemvParams &p, int64_t n0) {
    static_assert(4 * R <= 16, "NVFP4 rows are a multiple of 16, and a tile's scale serves 16 rows");
    Place<R> pl;
    const int lane = threadIdx.x & 63, i = lane & 3, b = lane >> 2;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        // MXFP4 has any number of rows: the last one stands in past the end
        const uint32_t row = SC == kRows32 ? (uint32_t)min((int64_t)(4 * r + i), p.N - 1 - n0) : 4 * r + i;
        pl.code[r] = row * (uint32_t)(p.K / 2) + b * 16;
        pl.scale[r] = SC == kRows16   ? row * (uint32_t)(p.K / 16) + b * 2
                      : SC == kRows32 ? row * (uint32_t)(p.K / 32) + b
                                      : b * 2;
    }
    pl.x = p.x + min((int64_t)i, p.T - 1) * p.ldx + b * 32;
    return pl;
}

// TAIL: the step K ends in; a lane then has both its 16-value halves, the
// first, or none.  It loads the halves from wherever they are or, past the
// end, from the row's last one, and clears what does not belong to it: no
// load waits behind a branch.
template <int SC, int NM, int R, bool TAIL>
__device__ __forceinline__ void load_step(Step<NM, R> &st, const GemvParams &p, const Place<R> &pl,
                                          int64_t n0, int64_t step) {
    const int b = (threadIdx.x & 63) >> 2;
    const int64_t k0 = step * kStepK;
    // TAIL: the lane's halves (16-value units from k0) as loaded
    const int left = TAIL ? (int)(p.K - k0) / 16 : 32;
    const int h0 = min(2 * b, left - 1), h1 = min(2 * b + 1, left - 1);
    const bool first = 2 * b < left, second = 2 * b + 1 < left;
#pragma unroll
    for (int w = 0; w < NM; ++w) {
        const GemvParams::Weight &W = w ? p.u : p.w;
        const uint8_t *cb = W.codes + n0 * (p.K / 2) + k0 / 2;
        const uint8_t *sb = W.scales + (SC == kRows16   ? n0 * (p.K / 16) + k0 / 16
                                        : SC == kRows32 ? n0 * (p.K / 32) + k0 / 32
                                                        : n0 / 16 * (p.K / 16) + k0 / 16);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!TAIL) {
                st.w[w][r] = *reinterpret_cast<const uint4 *>(cb + pl.code[r]);
            } else {
                const uint8_t *row = cb + pl.code[r] - 16 * b;
                const uint2 c0 = *reinterpret_cast<const uint2 *>(row + 8 * h0);
                const uint2 c1 = *reinterpret_cast<const uint2 *>(row + 8 * h1);
                st.w[w][r] = make_uint4(first ? c0.x : 0, first ? c0.y : 0, second ? c1.x : 0, second ? c1.y : 0);
            }
            if (SC == kTiles16 && r > 0) {
                st.s[w][r] = st.s[w][0];                 // the workgroup's rows share a tile row
            } else if (SC == kRows32) {
                const uint8_t *s = sb + pl.scale[r];
                st.s[w][r] = load_bytes<1>(TAIL ? s - b + h0 / 2 : s);
            } else if (!TAIL) {
                st.s[w][r] = load_bytes<2>(sb + pl.scale[r]);
            } else {
                const uint8_t *s = sb + pl.scale[r] - 2 * b;
                st.s[w][r] = load_bytes<1>(s + h0) | load_bytes<1>(s + h1) << 8;
            }
        }
    }
    const uint4 *xr = reinterpret_cast<const uint4 *>(pl.x + k0) - 4 * (TAIL ? b : 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (!TAIL) {
            st.x[q] = xr[q];
        } else {
            const uint4 v = xr[2 * (q < 2 ? h0 : h1) + (q & 1)];
            const bool in = q < 2 ? first : second;
            st.x[q] = make_uint4(in ? v.x : 0, in ? v.y : 0, in ? v.z : 0, in ? v.w : 0);
        }
    }
}

__device__ __forceinline__ s16x4 half_of(const uint4 &v, int h) {
    return __builtin_bit_cast(s16x4, h ? make_uint2(v.z, v.w) : make_uint2(v.x, v.y));
}

// Four E2M1 codes (half h of the word) as BF16.
__device__ __forceinline__ s16x4 codes4(uint32_t w, int h) {
    const bf16x2 a = h ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2)
                       : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0);
    const bf16x2 b = h ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3)
                       : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1);
    return __builtin_bit_cast(s16x4, make_uint2(__builtin_bit_cast(uint32_t, a),
                                                __builtin_bit_cast(uint32_t, b)));
}

// TT <= 4 rows of the products are summed: tokens, or the parts of tokens' hidden values.
// What stands in a row that the caller does not need stays in that row's sum.
template <int SC, int NM, int TT, int R>
__device__ __forceinline__ void add_step(float (&acc)[NM][R][TT], const Step<NM, R> &st) {
#pragma unroll
    for (int hb = 0; hb < 2; ++hb)                       // the lane's two 16-value halves
#pragma unroll
        for (int w = 0; w < NM; ++w)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    d = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(half_of(st.x[2 * hb + (q >> 1)], q & 1),
                                                               codes4(word(st.w[w][r], 2 * hb + (q >> 1)), q & 1),
                                                               d, 0, 0, 0);
                const float sc = SC == kRows32 ? e8m0_value(st.s[w][r]) : e4m3_value(st.s[w][r] >> (8 * hb));
#pragma unroll
                for (int t = 0; t < TT; ++t) acc[w][r][t] = __builtin_fmaf(d[t], sc, acc[w][r][t]);
            }
}

// Sum over the sixteen lanes with the same lane % 4.
__device__ __forceinline__ float sum_blocks(float v) {
    v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x124, 0xF, 0xF, false));   // row_ror:4
    v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x128, 0xF, 0xF, false));   // row_ror:8
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// ---------------------------------------------------------------------------
// Five tokens and more: v_mfma_f32_16x16x32_bf16, sixteen weight rows by
// sixteen tokens.  Code x scale is exact in BF16 (at most 6 significant bits
// for E2M1 x E4M3), so the weights are expanded once and serve every token
// tile.  A wave's step is 128 K values of its row tiles: lane 16 g + i reads
// 16 bytes (32 codes) of row i at K offset 32 g, which feed four instructions.
// ---------------------------------------------------------------------------
constexpr int kTileK = 128;

// Eight codes of a word times their block scale, in BF16.
template <int SC>
__device__ __forceinline__ bf16x8 expand8(uint32_t w, float sc) {
    uint32_t o[4];
    if constexpr (SC == kRows32) {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3));
    } else {
        const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
        const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
        const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
        const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
        o[0] = pk_bf16(v0[0] * sc, v0[1] * sc);
        o[1] = pk_bf16(v1[0] * sc, v1[1] * sc);
        o[2] = pk_bf16(v2[0] * sc, v2[1] * sc);
        o[3] = pk_bf16(v3[0] * sc, v3[1] * sc);
    }
    return __builtin_bit_cast(bf16x8, make_uint4(o[0], o[1], o[2], o[3]));
}

template <int NM, int NR>
struct TileWeights {
    uint4 c[NM][NR];
    uint32_t s[NM][NR];                  // two E4M3 bytes or one E8M0 byte
};

template <int NR>
struct TilePlace {
    uint32_t code[NR], scale[NR];        // from the workgroup's first row
};

// TAIL: as for the few-token step, the lane's two 16-value halves are loaded
// from inside K and cleared where they lie past it.
template <int SC, int NM, int NR, bool TAIL, bool SCALES = true>
__device__ __forceinline__ void load_weights(TileWeights<NM, NR> &tw, const GemvParams &p,
                                             const TilePlace<NR> &pl, int64_t n0, int64_t k0) {
    const int g = (threadIdx.x & 63) >> 4;
    const int left = TAIL ? (int)(p.K - k0) / 16 : 8;
    const int h0 = min(2 * g, left - 1), h1 = min(2 * g + 1, left - 1);
    const bool first = 2 * g < left, second = 2 * g + 1 < left;
#pragma unroll
    for (int w = 0; w < NM; ++w) {
        const GemvParams::Weight &W = w ? p.u : p.w;
        const uint8_t *cb = W.codes + n0 * (p.K / 2) + k0 / 2;
        const uint8_t *sb = W.scales + (SC == kRows16   ? n0 * (p.K / 16) + k0 / 16
                                        : SC == kRows32 ? n0 * (p.K / 32) + k0 / 32
                                                        : n0 / 16 * (p.K / 16) + k0 / 16);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            if (!TAIL) {
                tw.c[w][r] = *reinterpret_cast<const uint4 *>(cb + pl.code[r]);
                if (SCALES) tw.s[w][r] = load_bytes<SC == kRows32 ? 1 : 2>(sb + pl.scale[r]);
            } else {
                const uint8_t *row = cb + pl.code[r] - 16 * g;
                const uint2 c0 = *reinterpret_cast<const uint2 *>(row + 8 * h0);
                const uint2 c1 = *reinterpret_cast<const uint2 *>(row + 8 * h1);
                tw.c[w][r] = make_uint4(first ? c0.x : 0, first ? c0.y : 0, second ? c1.x : 0, second ? c1.y : 0);
                if (SC == kRows32) {
                    tw.s[w][r] = load_bytes<1>(sb + pl.scale[r] - g + h0 / 2);
                } else {
                    const uint8_t *s = sb + pl.scale[r] - 2 * g;
                    tw.s[w][r] = load_bytes<1>(s + h0) | load_bytes<1>(s + h1) << 8;
                }
            }
        }
    }
}

// The products of one step; x(t, j): chunk j of the lane's eight activations
// for token tile t.
template <int SC, int NM, int NT, int NR, typename X>
__device__ __forceinline__ void tile_products(f32x4 (&acc)[NM][NR][NT], const TileWeights<NM, NR> &tw, X x) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        bf16x8 xf[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xf[t] = x(t, j);
#pragma unroll
        for (int w = 0; w < NM; ++w)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float sc = SC == kRows32 ? e8m0_value(tw.s[w][r]) : e4m3_value(tw.s[w][r] >> (8 * (j >> 1)));
                const bf16x8 a = expand8<SC>(word(tw.c[w][r], j), sc);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[w][r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, xf[t], acc[w][r][t], 0, 0, 0);
            }
    }
}

}  // namespace gemv
}  // namespace bbs
