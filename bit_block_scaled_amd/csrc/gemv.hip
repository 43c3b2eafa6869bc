// Matrix-vector products with 4-bit weights for a few tokens (gfx950):
// y[t, n] = s_dec * sum_b scale[n, b] * sum_{k in b} x[t, k] * code[n, k],
// BF16 activations, NVFP4 (1x16 or 16x16 scales) or MXFP4 weights, and the
// gated form h = act(x Wg^T) * (x Wu^T).
#include "bbs_device.hpp"
#include "gated_epilogue.hpp"

namespace bbs {

namespace {

constexpr int kTok = 4;              // tokens per pass over a weight row

// One wave per weight row (row pair of the gated form); the lanes stride
// over the row's blocks and the wave's sums are added at the end.
template <bool MX, int ACT, bool BF16_OUT>
__global__ __launch_bounds__(256) void gemv_kernel(GemvParams p) {
    constexpr int NM = ACT >= 0 ? 2 : 1;
    constexpr int B = MX ? 32 : 16;
    const int lane = threadIdx.x & 63;
    const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (n >= p.N) return;
    const int64_t t0 = (int64_t)blockIdx.y * kTok;
    float acc[NM][kTok] = {};
    for (int64_t b = lane; b < p.K / B; b += 64) {
#pragma unroll
        for (int w = 0; w < NM; ++w) {
            const int64_t sr = (!MX && p.tile2d) ? n / 16 : n;
            const uint32_t sb = p.scales[w][sr * (p.K / B) + b];
            const float sc = MX ? e8m0_value(sb) : e4m3_pos_value(sb);
            const uint32_t *cw = reinterpret_cast<const uint32_t *>(p.codes[w] + n * (p.K / 2) + b * (B / 2));
#pragma unroll
            for (int tt = 0; tt < kTok; ++tt) {
                if (t0 + tt >= p.T) break;
                const uint32_t *xr = reinterpret_cast<const uint32_t *>(p.x + (t0 + tt) * p.ldx + b * B);
                float s = 0.0f;
                for (int j = 0; j < B / 2; ++j) {
                    const uint32_t c = cw[j / 4] >> (8 * (j % 4)), x = xr[j];
                    s = __builtin_fmaf(bf16_to_f32(x & 0xFFFFu), e2m1_value(c & 15u), s);
                    s = __builtin_fmaf(bf16_to_f32(x >> 16), e2m1_value((c >> 4) & 15u), s);
                }
                acc[w][tt] = __builtin_fmaf(s, sc, acc[w][tt]);
            }
        }
    }
#pragma unroll
    for (int tt = 0; tt < kTok; ++tt) {
        float v[NM];
#pragma unroll
        for (int w = 0; w < NM; ++w) {
            v[w] = acc[w][tt];
            for (int o = 32; o > 0; o >>= 1) v[w] += __shfl_xor(v[w], o, 64);
            if (!MX) v[w] *= p.s_dec[w][0];
        }
        float y = v[0];
        if constexpr (ACT >= 0) y = gate_act<ACT>(v[0]) * v[NM - 1];
        const int64_t t = t0 + tt;
        if (lane == 0 && t < p.T) {
            if (BF16_OUT) static_cast<uint16_t *>(p.y)[t * p.ldy + n] = (uint16_t)pk_bf16(y, y);
            else static_cast<float *>(p.y)[t * p.ldy + n] = y;
        }
    }
}

template <bool MX, int ACT>
hipError_t run(const GemvParams &p, bool bf16_out, hipStream_t s) {
    const dim3 grid((unsigned)((p.N + 3) / 4), (unsigned)((p.T + kTok - 1) / kTok));
    if (bf16_out) hipLaunchKernelGGL((gemv_kernel<MX, ACT, true>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((gemv_kernel<MX, ACT, false>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemv(const GemvParams &p, bool mxfp4, int act, bool bf16_out, hipStream_t s) {
    if (act < 0) return mxfp4 ? run<true, -1>(p, bf16_out, s) : run<false, -1>(p, bf16_out, s);
    if (act == kActGelu)
        return mxfp4 ? run<true, kActGelu>(p, bf16_out, s) : run<false, kActGelu>(p, bf16_out, s);
    return mxfp4 ? run<true, kActSilu>(p, bf16_out, s) : run<false, kActSilu>(p, bf16_out, s);
}

}  // namespace bbs
