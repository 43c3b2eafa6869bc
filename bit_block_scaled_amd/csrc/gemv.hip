// Matrix-vector products with 4-bit weights for a few tokens (gfx950):
//   y[t, n] = s_dec * sum_b scale[n, b] * sum_{k in b} x[t, k] * code[n, k]
// with BF16 activations and NVFP4 (1x16 or 16x16 scales) or MXFP4 weights, and
// the gated form h = act(x Wg^T) * (x Wu^T), which reads both matrices in one
// kernel.
//
// The weights' bytes bound these products: about half a byte a weight, read
// once, against 2 T flops.  Weights go from memory straight to registers, 16
// bytes a lane, with every load of a wave's share in flight at once; the
// waves of a workgroup split K and join their sums through LDS in a fixed
// order, so enough waves are in flight also where N is small.  The matrix
// instructions take the BF16 activations as they are; E2M1 codes are exact in
// BF16, so only the FP32 sums round.
#include <algorithm>

#include "bbs_device.hpp"
#include "gated_epilogue.hpp"

namespace bbs {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

namespace {

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

// Layout of the block scales.
constexpr int kRows16 = 0;       // NVFP4, one E4M3 byte per 16 weights of a row
constexpr int kTiles16 = 1;      // NVFP4, one E4M3 byte per 16 x 16 weights
constexpr int kRows32 = 2;       // MXFP4, one E8M0 byte per 32 weights of a row

// One output from its sums: decode scales, activation, one rounding.  The
// activation and the output type are the same for every lane.
template <int SC, int NM>
__device__ __forceinline__ void finish(const GemvParams &p, int64_t t, int64_t n, const float (&v)[2]) {
    float y = SC == kRows32 ? v[0] : v[0] * p.w.s_dec[0];
    if constexpr (NM == 2) {
        const float u = SC == kRows32 ? v[1] : v[1] * p.u.s_dec[0];
        y = (p.act == kActSilu ? gate_act<kActSilu, false>(y) : gate_act<kActGelu, false>(y)) * u;
    }
    if (p.bf16_out) static_cast<uint16_t *>(p.y)[t * p.ldy + n] = (uint16_t)pk_bf16(y, y);
    else static_cast<float *>(p.y)[t * p.ldy + n] = y;
}

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
//
// Bound by the weights' bytes where there are enough: one token, NVFP4, 4096 x
// 14336 in 7.7 us (33 MB, 4.3 TB/s, partly from the last-level cache), gated 2
// x 14336 x 4096 in 11.3 us (59 MB, 5.2 TB/s); 1536 x 4096 (3.2 MB) takes 3.1
// us, about an empty kernel's time.
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

// TT tokens are computed (1, 2 or 4), those from p.T on are not stored.
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

constexpr int kFewSplit = 8;     // most waves of a workgroup (K splits)

template <int SC, int NM, int TT, int R>
__global__ __launch_bounds__(64 * kFewSplit) void gemv_few_kernel(GemvParams p) {
    constexpr int NO = TT * R * 4;                       // outputs, of NM sums each
    __shared__ float part[kFewSplit][NM * NO];
    const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * (4 * R);
    const int64_t full = p.K / kStepK;
    const Place<R> pl = place_of<SC, R>(p, n0);
    float acc[NM][R][TT] = {};
    int64_t s = wave;
    if (s < full) {
        Step<NM, R> cur, nxt;
        load_step<SC, NM, R, false>(cur, p, pl, n0, s);
        for (; s + nw < full; s += nw) {
            load_step<SC, NM, R, false>(nxt, p, pl, n0, s + nw);
            add_step<SC, NM, TT, R>(acc, cur);
            cur = nxt;
        }
        add_step<SC, NM, TT, R>(acc, cur);
        s += nw;
    }
    if (s == full && p.K % kStepK) {
        Step<NM, R> last;
        load_step<SC, NM, R, true>(last, p, pl, n0, s);
        add_step<SC, NM, TT, R>(acc, last);
    }
#pragma unroll
    for (int w = 0; w < NM; ++w)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const float v = sum_blocks(acc[w][r][t]);
                if (lane < 4) part[wave][w * NO + (t * R + r) * 4 + lane] = v;
            }
    __syncthreads();
    for (int o = threadIdx.x; o < NO; o += blockDim.x) {
        float v[2] = {0.0f, 0.0f};
        for (int k = 0; k < nw; ++k)
#pragma unroll
            for (int w = 0; w < NM; ++w) v[w] += part[k][w * NO + o];
        const int64_t t = o / (R * 4), n = n0 + o % (R * 4);
        if (t < p.T && n < p.N) finish<SC, NM>(p, t, n, v);
    }
}

// ---------------------------------------------------------------------------
// Five tokens and more: v_mfma_f32_16x16x32_bf16, sixteen weight rows by
// sixteen tokens.  Code x scale is exact in BF16 (at most 6 significant bits
// for E2M1 x E4M3), so the weights are expanded once and serve every token
// tile.  A wave's step is 128 K values of its row tiles: lane 16 g + i reads
// 16 bytes (32 codes) of row i at K offset 32 g, which feed four instructions.
//
// The activations of a step go to the wave's own part of LDS (NT x 16 tokens x
// 256 bytes, asynchronous copies of whole token rows): taken straight to
// registers in the instructions' layout every lane would touch another cache
// line, and with 48 tokens those loads took longer than the weights'.  In LDS
// the 16-byte chunk c of token i lies at place c ^ i, so the sixteen lanes of
// one fragment read fall on sixteen different bank groups.
//
// Bound by the latency of a step and the L1 accesses of scattered rows: MXFP4
// 14336 x 4096 (32 MB) takes 15.4 us for 48 tokens in a graph and 16.3 in a
// kernel trace; where it took 16.6, it took 12.8 without the activations' copies
// and 12.1 without the weights' loads.  NVFP4 with 16x16 scales takes 10.0 us for
// up to 16 tokens, with 1x16 scales 12.8.  A step ahead in registers, two steps a
// fetch, twice the waves, activations shared by two row halves and a rotated
// order of K each changed it by less than 5% or made it slower.
// ---------------------------------------------------------------------------
constexpr int kTileK = 128;
constexpr int kTileSplit = 8;    // most waves of a workgroup (K splits)

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

// NT token tiles, NR row tiles of each matrix.
template <int SC, int NM, int NT, int NR>
__global__ __launch_bounds__(64 * kTileSplit) void gemv_tile_kernel(GemvParams p) {
    constexpr int NO = NR * NT * 256;                     // sums of one matrix
    // the waves' activations, then their sums [wave][matrix][row tile][token tile][lane][4]
    extern __shared__ __align__(16) uint8_t tile_lds[];
    const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NR);
    const int t0 = NR == 4 ? 0 : blockIdx.y * (16 * NT);  // the workgroup's first token (tile_shape)
    TilePlace<NR> pl;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const uint32_t row = (uint32_t)min((int64_t)(16 * r + i), p.N - 1 - n0);
        pl.code[r] = row * (uint32_t)(p.K / 2) + 16 * g;
        pl.scale[r] = SC == kRows16   ? row * (uint32_t)(p.K / 16) + 2 * g
                      : SC == kRows32 ? row * (uint32_t)(p.K / 32) + g
                                      : row / 16 * (uint32_t)(p.K / 16) + 2 * g;
    }
    // copy q of a step: tokens 4 q .. 4 q + 3, lane l the chunk that belongs at
    // place l % 16 of token 4 q + l / 16
    uint8_t *const xl = tile_lds + wave * (NT * 4096);
    const uint16_t *src[4 * NT];
#pragma unroll
    for (int q = 0; q < 4 * NT; ++q) {
        const int t = 4 * q + g;
        src[q] = p.x + min((int64_t)(t0 + t), p.T - 1) * p.ldx + 8 * (i ^ (t & 15));
    }
    f32x4 acc[NM][NR][NT];
#pragma unroll
    for (int w = 0; w < NM; ++w)
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[w][r][t] = f32x4{0, 0, 0, 0};

    const int64_t full = p.K / kTileK;
    TileWeights<NM, NR> tw;
    const auto step = [&](int64_t k0) {
        // the wave's reads of the step before are done
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int q = 0; q < 4 * NT; ++q) copy_lds16(src[q] + k0, xl + q * 1024);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        tile_products<SC, NM, NT, NR>(acc, tw, [&](int t, int j) {
            return *reinterpret_cast<const bf16x8 *>(xl + (16 * t + i) * 256 + 16 * ((4 * g + j) ^ i));
        });
    };
    int64_t at = 0;                                       // steps done by all waves
    // Runs of steps of one wave, whose row scales come with one load of 16
    // bytes a row: a load for every step touches the same lines again for a
    // byte or two a lane (48 tokens, MXFP4 14336 x 4096: 16.6 us against 19.0;
    // gated, 16 tokens, NVFP4: 20.8 against 22.8).  NVFP4's runs are half as
    // long and lose elsewhere (64 tokens, 4096 x 14336: 30.6 against 29.4; 16
    // tokens, 14336 x 4096: 13.1 against 12.8; gated, 40 tokens, 4096 x 8192:
    // 22.3 against 20.9), and rows that do not begin at four bytes make such
    // loads slow (gated, 13 tokens, 1552 x 4112: 9.0 against 7.0).
    constexpr int kRun = SC == kRows32 ? 4 : 2;
    if constexpr (SC == kRows32 || (SC == kRows16 && NM == 2 && NR == 2)) {
        const int64_t runs = p.K % (SC == kRows32 ? 128 : 64) ? 0 : full;
        for (; at + kRun * nw <= runs; at += kRun * nw) {
            const int64_t k0 = (at + kRun * wave) * kTileK;
            uint4 sv[NM][NR];
#pragma unroll
            for (int w = 0; w < NM; ++w)
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const uint8_t *row = (w ? p.u : p.w).scales + (n0 * p.K + k0) / (SC == kRows32 ? 32 : 16) +
                                         (pl.scale[r] - (SC == kRows32 ? g : 2 * g));
                    __builtin_memcpy(&sv[w][r], row, 16);
                }
#pragma unroll
            for (int q = 0; q < kRun; ++q) {
                load_weights<SC, NM, NR, false, false>(tw, p, pl, n0, k0 + q * kTileK);
#pragma unroll
                for (int w = 0; w < NM; ++w)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        if (SC == kRows32) tw.s[w][r] = word(sv[w][r], q) >> (8 * g) & 0xff;
                        else tw.s[w][r] = word(sv[w][r], 2 * q + (g >> 1)) >> (16 * (g & 1)) & 0xffff;
                step(k0 + q * kTileK);
            }
        }
    }
    for (at += wave; at < full; at += nw) {
        load_weights<SC, NM, NR, false>(tw, p, pl, n0, at * kTileK);
        step(at * kTileK);
    }
    if (full % nw == wave && p.K % kTileK) {
        const int64_t k0 = full * kTileK;
        load_weights<SC, NM, NR, true>(tw, p, pl, n0, k0);
        const int left = (int)(p.K - k0) / 8;             // chunks of a token inside K
        tile_products<SC, NM, NT, NR>(acc, tw, [&](int t, int j) {
            const uint4 v = *reinterpret_cast<const uint4 *>(
                p.x + min((int64_t)(t0 + 16 * t + i), p.T - 1) * p.ldx + k0 + 8 * min(4 * g + j, left - 1));
            const bool in = 4 * g + j < left;
            return __builtin_bit_cast(bf16x8, make_uint4(in ? v.x : 0, in ? v.y : 0, in ? v.z : 0, in ? v.w : 0));
        });
    }
    __syncthreads();                                      // the activations' place is reused
    float *const part = reinterpret_cast<float *>(tile_lds);
    // lane 16 g + i holds token i of a token tile and rows 4 g .. 4 g + 3
#pragma unroll
    for (int w = 0; w < NM; ++w)
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                *reinterpret_cast<f32x4 *>(part + (wave * NM + w) * NO + (r * NT + t) * 256 + lane * 4) = acc[w][r][t];
    __syncthreads();
    for (int o = threadIdx.x; o < NO; o += blockDim.x) {
        float v[2] = {0.0f, 0.0f};
        for (int s = 0; s < nw; ++s)
#pragma unroll
            for (int w = 0; w < NM; ++w) v[w] += part[(s * NM + w) * NO + o];
        // consecutive o: rows 4 g + v of one token
        const int tile = o >> 8, l = (o >> 2) & 63;
        const int64_t t = t0 + (tile % NT) * 16 + (l & 15);
        const int64_t n = n0 + (tile / NT) * 16 + (l >> 4) * 4 + (o & 3);
        if (t < p.T && n < p.N) finish<SC, NM>(p, t, n, v);
    }
}

// ---------------------------------------------------------------------------
// Launch rules
// ---------------------------------------------------------------------------
template <int SC, int NM, int TT, int R>
hipError_t few(const GemvParams &p, hipStream_t s) {
    const int64_t steps = (p.K + kStepK - 1) / kStepK;
    // two steps a wave, both loaded before the first is used: one token, 4096
    // x 14336: 8.1 us with 8 waves, 9.3 with 4, 8.2 with 16; 1536 x 4096: 3.2
    // us with 4 waves, 3.1 with 8, 4.6 with 1
    const int64_t waves = std::min<int64_t>((steps + 1) / 2, kFewSplit);
    const dim3 grid((unsigned)((p.N + 4 * R - 1) / (4 * R)));
    hipLaunchKernelGGL((gemv_few_kernel<SC, NM, TT, R>), grid, dim3((unsigned)(64 * waves)), 0, s, p);
    return hipGetLastError();
}

template <int SC, int NM, int NT, int NR>
hipError_t tile(const GemvParams &p, hipStream_t s) {
    const int64_t steps = (p.K + kTileK - 1) / kTileK;
    const int64_t waves = std::min<int64_t>(steps, kTileSplit);
    const dim3 grid((unsigned)((p.N + 16 * NR - 1) / (16 * NR)), (unsigned)((p.T + 16 * NT - 1) / (16 * NT)));
    // a wave's activations, then its sums
    constexpr size_t wave_bytes = (size_t)NT * 1024 * (NM * NR > 4 ? NM * NR : 4);
    static const bool attr_set = [] {
        (void)hipFuncSetAttribute(reinterpret_cast<const void *>(&gemv_tile_kernel<SC, NM, NT, NR>),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, (int)(kTileSplit * wave_bytes));
        return true;
    }();
    (void)attr_set;
    hipLaunchKernelGGL((gemv_tile_kernel<SC, NM, NT, NR>), grid, dim3((unsigned)(64 * waves)),
                       waves * wave_bytes, s, p);
    return hipGetLastError();
}

// Rows of a workgroup, over both matrices of the gated form: 16 from 4096 rows
// of a matrix on, which is one workgroup for each of 256 CUs and two in the
// gated form, and 8 below.
//   1 token, 4096 x 14336: 8.1 us with 16 rows, 8.4 with 8
//   1 token, 1536 x 4096: 3.2 us with 8 rows, 3.7 with 16, 3.4 with 4
// Gated, between one and two workgroups of 16 a CU, the number of rows and K
// decide: 2064 x 1024 3.2 us with 8 rows, 3.5 with 16; 3008 x 4096 5.2 and 5.8;
// 2048 x 4096 4.4 and 4.4; 4080 x 8192 10.0 and 8.6.
template <int SC, int NM, int TT>
hipError_t few_rows(const GemvParams &p, hipStream_t s) {
    return p.N >= 4096 ? few<SC, NM, TT, 4 / NM>(p, s) : few<SC, NM, TT, 2 / NM>(p, s);
}

// Row tiles and token tiles of a workgroup.  Each workgroup reads its tokens'
// activations once for all its rows and its rows once for all its tokens, and
// more than one workgroup a CU means a second round or less LDS for each.
//
// So as few row tiles as keep the grid within the CUs, four over both matrices
// at most, and then all the tokens (us, NVFP4, K 4096):
//   tokens x rows   16 rows   32 rows   64 rows
//   16 x 4608       9.4       7.9                  (288 tiles of 16)
//   64 x 5120       18        14.4      15.3       (320)
//   16 x 8192       9.9       8.5       12.3       (512)
//   40 x 8192       18        12.9      18.4
//   48 x 14336                22.8      19.6       (896; MXFP4: 16.6 with 64 rows)
// With short K and one token tile the second row tile costs more than the
// second round (16 x 4112 x 1568: 4.2 and 4.5 us; 16 x 6144 x 2048: 6.1 and 5.4).
//
// One row tile leaves room for fewer tokens in a workgroup: as many token
// tiles as keep the grid within the CUs (64 tokens, 1536 x 4096: 6.8 us with
// two, 9.4 with four, 8.8 with one; 512 x 2048: 4.0 with one, 6.2 with four; 24
// tokens, 4096 x 4096: 7.2 with two, 9.2 with one).  Where that is all four
// (for one MXFP4 matrix, whose expansion is cheaper, also three), two of each
// read fewer activations (64 tokens, 4096 x 14336: 26.8 us against 29.3,
// MXFP4 20.4 against 26.6; 48 tokens 26.1 against 24.4, MXFP4 19.8 and 22.0).
template <int SC, int NM>
hipError_t tile_shape(const GemvParams &p, hipStream_t s) {
    const int64_t rows = (p.N + 15) / 16, tiles = (p.T + 15) / 16, cus = device_cus(s);
    if (rows > 2 * cus && NM == 1) {
        if (tiles == 1) return tile<SC, NM, 1, 4 / NM>(p, s);
        if (tiles == 2) return tile<SC, NM, 2, 4 / NM>(p, s);
        if (tiles == 3) return tile<SC, NM, 3, 4 / NM>(p, s);
        return tile<SC, NM, 4, 4 / NM>(p, s);
    }
    if (rows > cus && (rows > 2 * cus || tiles > 1 || p.K >= 2048)) {
        if (tiles == 1) return tile<SC, NM, 1, 2>(p, s);
        if (tiles == 2) return tile<SC, NM, 2, 2>(p, s);
        if (tiles == 3) return tile<SC, NM, 3, 2>(p, s);
        return tile<SC, NM, 4, 2>(p, s);
    }
    constexpr int kMost = SC == kRows32 && NM == 1 ? 2 : 3;
    int64_t nt = 1;
    while (nt < tiles && rows * ((tiles + nt - 1) / nt) > cus) ++nt;
    if (nt > kMost) return tile<SC, NM, 2, 2>(p, s);
    if (nt == 1) return tile<SC, NM, 1, 1>(p, s);
    if (nt == 2) return tile<SC, NM, 2, 1>(p, s);
    return tile<SC, NM, kMost, 1>(p, s);
}

// Up to four tokens take the 4x4x4 form (three, 14336 x 4096: 11.3 us against
// 12.4), more the 16x16x32 form (six, 1536 x 4096: 4.5 us against 4.9; eight,
// 14336 x 4096: 10.1 against 19.5).
template <int SC, int NM>
hipError_t run(const GemvParams &p, hipStream_t s) {
    if (p.T == 1) return few_rows<SC, NM, 1>(p, s);
    if (p.T == 2) return few_rows<SC, NM, 2>(p, s);
    if (p.T <= 4) return few_rows<SC, NM, 4>(p, s);
    return tile_shape<SC, NM>(p, s);
}

template <int SC>
hipError_t by_act(const GemvParams &p, hipStream_t s) {
    return p.act < 0 ? run<SC, 1>(p, s) : run<SC, 2>(p, s);
}

}  // namespace

// A launch has fewer than 2^32 threads a dimension (more are cut off without an
// error), and the kernels take up to 64 a row: more than 2^25 rows go in parts.
hipError_t launch_gemv(const GemvParams &p, bool mxfp4, hipStream_t s) {
    constexpr int64_t kRows = (int64_t)1 << 25;
    GemvParams q = p;
    for (int64_t n = 0; n < p.N; n += kRows) {
        q.N = std::min(kRows, p.N - n);
        q.y = static_cast<uint8_t *>(p.y) + n * (p.bf16_out ? 2 : 4);
        for (auto w : {&GemvParams::w, &GemvParams::u}) {
            if (p.act < 0 && w == &GemvParams::u) continue;
            (q.*w).codes = (p.*w).codes + n * (p.K / 2);
            (q.*w).scales = (p.*w).scales + (mxfp4 ? n * (p.K / 32) : (p.tile2d ? n / 16 : n) * (p.K / 16));
        }
        const hipError_t e = mxfp4      ? by_act<kRows32>(q, s)
                             : p.tile2d ? by_act<kTiles16>(q, s)
                                        : by_act<kRows16>(q, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace bbs
