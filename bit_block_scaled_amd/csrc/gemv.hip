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
#include <type_traits>

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

// One output from its sums: decode scales, activation, one rounding.
template <bool MX, int ACT, bool BF16_OUT>
__device__ __forceinline__ void finish(const GemvParams &p, int64_t t, int64_t n, float v0, float v1) {
    float y = MX ? v0 : v0 * p.s_dec[0][0];
    if constexpr (ACT >= 0) y = gate_act<ACT>(y) * (MX ? v1 : v1 * p.s_dec[1][0]);
    if (BF16_OUT) static_cast<uint16_t *>(p.y)[t * p.ldy + n] = (uint16_t)pk_bf16(y, y);
    else static_cast<float *>(p.y)[t * p.ldy + n] = y;
}

// ---------------------------------------------------------------------------
// Up to eight tokens: v_mfma_f32_4x4x4_16b_bf16, sixteen independent 4 x 4 x 4
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

template <bool MX, int NM, int NG, int R>
struct Step {
    uint4 w[NM][R];          // 32 codes
    uint32_t s[NM][R];       // two E4M3 bytes or one E8M0 byte
    uint4 x[NG][4];          // 32 activations of one token
};

template <bool MX, int NM, int NG, int R>
__device__ __forceinline__ void load_step(Step<MX, NM, NG, R> &st, const GemvParams &p, int64_t n0,
                                          int64_t step) {
    const int lane = threadIdx.x & 63, i = lane & 3;
    const int64_t k = step * kStepK + (lane >> 2) * 32;
    // K is a multiple of 16: a lane has both its 16-value halves, the first, or none
    const bool first = k < p.K, second = k + 16 < p.K;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < NM; ++w)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t n = min(n0 + 4 * r + i, p.N - 1);
            const uint8_t *c = p.codes[w] + n * (p.K / 2) + k / 2;
            st.w[w][r] = zero;
            st.s[w][r] = 0;
            if (second) st.w[w][r] = *reinterpret_cast<const uint4 *>(c);
            else if (first) {
                const uint2 h = *reinterpret_cast<const uint2 *>(c);
                st.w[w][r].x = h.x;
                st.w[w][r].y = h.y;
            }
            if (MX) {
                if (first) st.s[w][r] = load_bytes<1>(p.scales[w] + n * (p.K / 32) + k / 32);
            } else {
                const uint8_t *s = p.scales[w] + (p.tile2d ? n / 16 : n) * (p.K / 16) + k / 16;
                if (second) st.s[w][r] = load_bytes<2>(s);
                else if (first) st.s[w][r] = load_bytes<1>(s);
            }
        }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const uint4 *xr = reinterpret_cast<const uint4 *>(p.x + min((int64_t)(4 * g + i), p.T - 1) * p.ldx + k);
#pragma unroll
        for (int q = 0; q < 4; ++q) st.x[g][q] = (q < 2 ? first : second) ? xr[q] : zero;
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

// TT tokens are computed (1, 2, 4 or 8), those from p.T on are not stored.
template <bool MX, int NM, int TT, int R>
__device__ __forceinline__ void add_step(float (&acc)[NM][R][TT],
                                         const Step<MX, NM, (TT + 3) / 4, R> &st) {
    constexpr int NG = (TT + 3) / 4, NT = TT < 4 ? TT : 4;
#pragma unroll
    for (int hb = 0; hb < 2; ++hb)                       // the lane's two 16-value halves
#pragma unroll
        for (int w = 0; w < NM; ++w)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                s16x4 cw[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) cw[q] = codes4(word(st.w[w][r], 2 * hb + (q >> 1)), q & 1);
                const uint32_t sb = MX ? st.s[w][r] : (st.s[w][r] >> (8 * hb)) & 0xFFu;
                const float sc = MX ? e8m0_value(sb) : e4m3_value(sb);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        d = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(half_of(st.x[g][2 * hb + (q >> 1)], q & 1),
                                                                   cw[q], d, 0, 0, 0);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        acc[w][r][4 * g + t] = __builtin_fmaf(d[t], sc, acc[w][r][4 * g + t]);
                }
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

constexpr int kMaxSplit = 16;            // waves of a workgroup (K splits)

template <bool MX, int ACT, bool BF16_OUT, int TT, int R>
__global__ __launch_bounds__(64 * kMaxSplit) void gemv_few_kernel(GemvParams p) {
    constexpr int NM = ACT >= 0 ? 2 : 1, NG = (TT + 3) / 4, NS = NM * R * TT * 4;
    __shared__ float part[kMaxSplit][NS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * (4 * R);
    const int64_t steps = (p.K + kStepK - 1) / kStepK;
    float acc[NM][R][TT] = {};
    for (int64_t s = wave; s < steps; s += 2 * nw) {
        Step<MX, NM, NG, R> a, b;
        load_step<MX, NM, NG, R>(a, p, n0, s);
        if (s + nw < steps) {
            load_step<MX, NM, NG, R>(b, p, n0, s + nw);
            add_step<MX, NM, TT, R>(acc, a);
            add_step<MX, NM, TT, R>(acc, b);
        } else {
            add_step<MX, NM, TT, R>(acc, a);
        }
    }
#pragma unroll
    for (int w = 0; w < NM; ++w)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const float v = sum_blocks(acc[w][r][t]);
                if (lane < 4) part[wave][((w * TT + t) * R + r) * 4 + lane] = v;
            }
    __syncthreads();
    constexpr int NO = TT * R * 4;       // outputs, of NM sums each
    for (int o = threadIdx.x; o < NO; o += blockDim.x) {
        float v[2] = {0.0f, 0.0f};
        for (int k = 0; k < nw; ++k)
#pragma unroll
            for (int w = 0; w < NM; ++w) v[w] += part[k][w * NO + o];
        const int64_t t = o / (R * 4), n = n0 + o % (R * 4);
        if (t < p.T && n < p.N) finish<MX, ACT, BF16_OUT>(p, t, n, v[0], v[1]);
    }
}

// ---------------------------------------------------------------------------
// Nine tokens and more: v_mfma_f32_16x16x32_bf16, sixteen weight rows by
// sixteen tokens.  Code x scale is exact in BF16 (at most 6 significant bits
// for E2M1 x E4M3), so the weights are expanded once and serve every token
// tile.  A wave's step is 256 K values: lane 16 g + i reads 32 bytes (64
// codes) of row i and 64 activations of token i at K offset 64 g, which feed
// eight instructions.
// ---------------------------------------------------------------------------
constexpr int kTileK = 256;
constexpr int kTileSplit = 8;

template <bool MX>
__device__ __forceinline__ bf16x8 expand8(uint32_t w, float sc) {
    uint32_t o[4];
    if constexpr (MX) {
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

// NT token tiles, NR row tiles of each matrix.
template <bool MX, int ACT, bool BF16_OUT, int NT, int NR>
__global__ __launch_bounds__(64 * kTileSplit) void gemv_tile_kernel(GemvParams p) {
    constexpr int NM = ACT >= 0 ? 2 : 1;
    constexpr int NO = NR * NT * 256;                     // sums of one matrix
    extern __shared__ __align__(16) float tile_part[];    // [wave][matrix][row tile][token tile][lane][4]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
    const int i = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NR);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    f32x4 acc[NM][NR][NT];
#pragma unroll
    for (int w = 0; w < NM; ++w)
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[w][r][t] = f32x4{0, 0, 0, 0};

    for (int64_t k = (int64_t)wave * kTileK + 64 * g; k - 64 * g < p.K; k += (int64_t)nw * kTileK) {
        // the lane's 16-value blocks that lie inside K: 4, or fewer at the end
        const int64_t left = (p.K - k) / 16;
        const int nb = left < 0 ? 0 : left > 4 ? 4 : (int)left;
        uint4 cw[NM][NR][2], xv[NT][8];
        uint32_t sw[NM][NR];
#pragma unroll
        for (int w = 0; w < NM; ++w)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const int64_t n = min(n0 + 16 * r + i, p.N - 1);
                const uint8_t *c = p.codes[w] + n * (p.K / 2) + k / 2;
                const uint8_t *s = MX ? p.scales[w] + n * (p.K / 32) + k / 32
                                      : p.scales[w] + (p.tile2d ? n / 16 : n) * (p.K / 16) + k / 16;
                cw[w][r][0] = cw[w][r][1] = zero;
                sw[w][r] = 0;
                if (nb == 4) {
                    cw[w][r][0] = reinterpret_cast<const uint4 *>(c)[0];
                    cw[w][r][1] = reinterpret_cast<const uint4 *>(c)[1];
                    sw[w][r] = MX ? load_bytes<2>(s) : load_bytes<4>(s);
                } else {
#pragma unroll
                    for (int b = 0; b < 3; ++b)
                        if (b < nb) {
                            const uint2 h = reinterpret_cast<const uint2 *>(c)[b];
                            if (b & 1) cw[w][r][b >> 1].z = h.x, cw[w][r][b >> 1].w = h.y;
                            else cw[w][r][b >> 1].x = h.x, cw[w][r][b >> 1].y = h.y;
                            if (!MX) sw[w][r] |= load_bytes<1>(s + b) << (8 * b);
                            else if (!(b & 1)) sw[w][r] |= load_bytes<1>(s + b / 2) << (4 * b);
                        }
                }
            }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint4 *xr = reinterpret_cast<const uint4 *>(p.x + min((int64_t)(16 * t + i), p.T - 1) * p.ldx + k);
#pragma unroll
            for (int q = 0; q < 8; ++q) xv[t][q] = q < 2 * nb ? xr[q] : zero;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
            for (int w = 0; w < NM; ++w)
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const uint32_t sb = (sw[w][r] >> (8 * (MX ? q >> 2 : q >> 1))) & 0xFFu;
                    const bf16x8 a = expand8<MX>(word(cw[w][r][q >> 2], q & 3),
                                                 MX ? e8m0_value(sb) : e4m3_value(sb));
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        acc[w][r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            a, __builtin_bit_cast(bf16x8, xv[t][q]), acc[w][r][t], 0, 0, 0);
                }
    }
    // lane 16 g + i holds token i of a token tile and rows 4 g .. 4 g + 3
#pragma unroll
    for (int w = 0; w < NM; ++w)
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                *reinterpret_cast<f32x4 *>(tile_part + (wave * NM + w) * NO + (r * NT + t) * 256 + lane * 4) =
                    acc[w][r][t];
    __syncthreads();
    for (int o = threadIdx.x; o < NO; o += blockDim.x) {
        float v[2] = {0.0f, 0.0f};
        for (int s = 0; s < nw; ++s)
#pragma unroll
            for (int w = 0; w < NM; ++w) v[w] += tile_part[(s * NM + w) * NO + o];
        // consecutive o: rows 4 g + v of one token
        const int tile = o >> 8, l = (o >> 2) & 63;
        const int64_t t = (tile % NT) * 16 + (l & 15);
        const int64_t n = n0 + (tile / NT) * 16 + (l >> 4) * 4 + (o & 3);
        if (t < p.T && n < p.N) finish<MX, ACT, BF16_OUT>(p, t, n, v[0], v[1]);
    }
}

// ---------------------------------------------------------------------------
// Launch rules
// ---------------------------------------------------------------------------

template <bool MX, int ACT, bool BF16_OUT, int TT, int R>
hipError_t few(const GemvParams &p, hipStream_t s) {
    const int64_t steps = (p.K + kStepK - 1) / kStepK;
    // two steps a wave: both are loaded before the first is used
    const int64_t waves = steps <= 1 ? 1 : steps >= 2 * kMaxSplit ? kMaxSplit : (steps + 1) / 2;
    const dim3 grid((unsigned)((p.N + 4 * R - 1) / (4 * R)));
    hipLaunchKernelGGL((gemv_few_kernel<MX, ACT, BF16_OUT, TT, R>), grid, dim3((unsigned)(64 * waves)), 0, s, p);
    return hipGetLastError();
}

template <bool MX, int ACT, bool BF16_OUT, int NT, int NR>
hipError_t tile(const GemvParams &p, hipStream_t s) {
    constexpr int NM = ACT >= 0 ? 2 : 1;
    const int64_t steps = (p.K + kTileK - 1) / kTileK;
    const int64_t waves = steps >= kTileSplit ? kTileSplit : steps;
    const dim3 grid((unsigned)((p.N + 16 * NR - 1) / (16 * NR)));
    constexpr size_t wave_bytes = (size_t)NM * NR * NT * 1024;
    static const bool attr_set = [] {
        (void)hipFuncSetAttribute(
            reinterpret_cast<const void *>(&gemv_tile_kernel<MX, ACT, BF16_OUT, NT, NR>),
            hipFuncAttributeMaxDynamicSharedMemorySize, (int)(kTileSplit * wave_bytes));
        return true;
    }();
    (void)attr_set;
    hipLaunchKernelGGL((gemv_tile_kernel<MX, ACT, BF16_OUT, NT, NR>), grid, dim3((unsigned)(64 * waves)),
                       waves * wave_bytes, s, p);
    return hipGetLastError();
}

template <bool MX, int ACT, bool BF16_OUT>
hipError_t run(const GemvParams &p, hipStream_t s) {
    // rows of a workgroup: fewer for the gated form, which reads two matrices
    constexpr int R = ACT >= 0 ? 2 : 4;
    if (p.T <= 8) {
        if (p.T == 1) return few<MX, ACT, BF16_OUT, 1, R>(p, s);
        if (p.T == 2) return few<MX, ACT, BF16_OUT, 2, R>(p, s);
        if (p.T <= 4) return few<MX, ACT, BF16_OUT, 4, R>(p, s);
        return few<MX, ACT, BF16_OUT, 8, R>(p, s);
    }
    constexpr int NR = ACT >= 0 ? 1 : 2;
    if (p.T <= 16) return tile<MX, ACT, BF16_OUT, 1, NR>(p, s);
    if (p.T <= 32) return tile<MX, ACT, BF16_OUT, 2, NR>(p, s);
    if (p.T <= 48) return tile<MX, ACT, BF16_OUT, 3, NR>(p, s);
    return tile<MX, ACT, BF16_OUT, 4, NR>(p, s);
}

}  // namespace

hipError_t launch_gemv(const GemvParams &p, bool mxfp4, int act, bool bf16_out, hipStream_t s) {
    auto pick = [&](auto mx, auto a) {
        constexpr bool MX = decltype(mx)::value;
        constexpr int ACT = decltype(a)::value;
        return bf16_out ? run<MX, ACT, true>(p, s) : run<MX, ACT, false>(p, s);
    };
    auto by_act = [&](auto mx) {
        if (act == kActSilu) return pick(mx, std::integral_constant<int, kActSilu>{});
        if (act == kActGelu) return pick(mx, std::integral_constant<int, kActGelu>{});
        return pick(mx, std::integral_constant<int, -1>{});
    };
    return mxfp4 ? by_act(std::true_type{}) : by_act(std::false_type{});
}

}  // namespace bbs
