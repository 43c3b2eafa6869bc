// The gated activation of a feed-forward block and the parameter blocks of
// the operators built on it: h = act(g) * u with g = x Wg^T, u = x Wu^T.
//
// Both activations are g * sigma(z): SiLU with z = g, and GELU in its tanh
// form with z = 2 sqrt(2/pi) (g + 0.044715 g^3), because
// (1 + tanh(z / 2)) / 2 = sigma(z).  The derivative is
// sigma(z) + g sigma(z) (1 - sigma(z)) dz/dg.
#pragma once

#include "bbs_kernels.hpp"

namespace bbs {

constexpr int kActSilu = 0, kActGelu = 1, kActNone = 2;

// Forward: NVFP4 operands (b = the gate weights, u = the up weights of the
// same shape and layout), output h, optional MXFP8 checkpoints of g and u.
struct GatedParams {
    Fp4View a, b, u;
    int64_t M, N, K;               // N = rows of b and of u
    void *h;
    int64_t ldh;
    uint8_t *g_codes, *g_scales, *u_codes, *u_scales;   // all null without checkpoints
};

// Backward through the down projection and the gated activation: MXFP8
// operands dY (M x K) and the transposed down weights (N x K).
struct GatedBwdParams {
    Mx8GemmParams mm;              // mm.c = dgate, mm.ldc its row stride
    const uint8_t *g_codes, *g_scales, *u_codes, *u_scales;
    void *du;
};

// A few tokens (rows of x, BF16) times one or two 4-bit weight matrices.
struct GemvParams {
    const uint16_t *x;
    int64_t T, ldx;
    struct Weight {
        const uint8_t *codes, *scales;
        const float *s_dec;        // null for MXFP4
    } w, u;                        // u: the up weights of the gated form
    int64_t N, K;
    int tile2d;
    void *y;
    int64_t ldy;
    int bf16_out;
    int act;                       // < 0: one matrix, y = x W^T; else the gated form of the two
    // one matrix: y = epi_act(x W^T + bias) + r
    const void *bias;              // N values, or null
    int bias_bf16;
    int epi_act;
    const void *r;                 // residual of y's type, or null
    int64_t ldr;
};

hipError_t launch_gated_gemm(const GatedParams &p, int act, bool bf16_out, hipStream_t s);
// The large-tile kernel (K % 128 == 0, 16-byte aligned codes, 8-byte aligned scales).
hipError_t launch_gated_gemm_big(const GatedParams &p, int act, bool bf16_out, hipStream_t s);
// The same for the backward pass (any K, K and N below 2^24).
hipError_t launch_gated_bwd_big(const GatedBwdParams &p, int act, bool bf16_out, hipStream_t s);
hipError_t launch_gated_bwd(const GatedBwdParams &p, int act, bool bf16_out, hipStream_t s);
hipError_t launch_gemv(const GemvParams &p, bool mxfp4, hipStream_t s);

// e^-z within a few FP32 ulp for every z: the product with log2 e is carried
// in two parts (the hardware exponential rounds to one ulp), so the relative
// error does not grow with |z|.  Infinite for z < -89, 0 for z > 104.
__device__ __forceinline__ float exp_neg(float z) {
    const float w = -__builtin_amdgcn_fmed3f(z, -104.0f, 104.0f);
    constexpr float kL = 1.44269502e+00f;                 // log2 e rounded to FP32
    constexpr float kLlo = 1.92596299e-08f;               // log2 e - kL
    const float t = w * kL;
    const float lo = __builtin_fmaf(w, kLlo, __builtin_fmaf(w, kL, -t));
    return __builtin_amdgcn_exp2f(t) * __builtin_fmaf(lo, 0.693147182f, 1.0f);
}

template <int ACT>
__device__ __forceinline__ float gate_z(float g) {
    if (ACT == kActSilu) return g;
    return 1.5957691216f * __builtin_fmaf(0.044715f * (g * g), g, g);
}

// act(g) = g sigma(z), sigma(z) = 1 / (1 + e^-z).  TO_BF16: the result is
// rounded to BF16, and the exponent's product with log2 e may round once: the
// relative error of e^-z is then |z| 2^-24 at most, far below half a BF16 step
// wherever e^-z matters beside 1 or the result is not negligible.
template <int ACT, bool TO_BF16>
__device__ __forceinline__ float gate_act(float g) {
    const float z = gate_z<ACT>(g);
    const float e = TO_BF16 ? __builtin_amdgcn_exp2f(z * -1.44269502f) : exp_neg(z);
    return g * __builtin_amdgcn_rcpf(1.0f + e);
}

// act(g) and its derivative s + g s (1 - s) dz/dg for every finite g, with 1 - s
// taken as e^-z s, which does not cancel for large z.  Where e^-z overflows
// (z < -88.7) s is 0, and so are both results; the minimum keeps s e^-z from
// being 0 times infinity there.  GELU's dz/dg grows as g^2 beside a factor
// that is 0 from |g| = 12 on, and is held to |g| <= 16, so that it stays finite.
template <int ACT, bool TO_BF16>
__device__ __forceinline__ float gate_act_grad(float g, float &slope) {
    const float z = gate_z<ACT>(g);
    const float e = TO_BF16 ? __builtin_amdgcn_exp2f(z * -1.44269502f) : exp_neg(z);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    const float a = g * s;
    const float r = a * (s * fminf(e, 3.0e38f));
    if (ACT == kActSilu) {
        slope = s + r;
    } else {
        const float h = __builtin_amdgcn_fmed3f(g, -16.0f, 16.0f);
        slope = __builtin_fmaf(r, 1.5957691216f * __builtin_fmaf(0.134145f * h, h, 1.0f), s);
    }
    return a;
}

}  // namespace bbs
