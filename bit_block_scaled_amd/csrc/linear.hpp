// A linear layer's product with what stands around it, y = act(A W^T + b) + r,
// and the backward pass of the bias and the activation: parameter blocks,
// launchers and the arithmetic the kernels share.
#pragma once

#include "gated_epilogue.hpp"

namespace bbs {

struct LinearParams {
    Fp4View a, b;                      // b: the weights, N rows
    int64_t M, N, K;
    void *c;
    int64_t ldc;
    const void *bias;                  // N values, or null
    int bias_bf16;
    int act;
    const void *r;                     // residual of c's type, or null (may be c itself)
    int64_t ldr;
    uint8_t *z_codes, *z_scales;       // MXFP8 checkpoint of z = A W^T + b, or null
};

// Most row ranges whose column sums the backward pass keeps apart.
constexpr int kBiasParts = 64;

struct BiasActBwdParams {
    const uint16_t *dy;
    int64_t M, N, ldy;
    const uint8_t *z_codes, *z_scales; // unused without an activation
    int act;
    uint16_t *dz;                      // or null
    int64_t ldz;
    void *db;                          // or null
    int db_bf16;
    float *part;                       // parts x N sums
};

hipError_t launch_linear(const LinearParams &p, bool bf16_out, hipStream_t s);
// The large-tile kernel (K % 128 == 0, 16-byte aligned codes, 8-byte aligned scales).
hipError_t launch_linear_big(const LinearParams &p, bool bf16_out, hipStream_t s);
hipError_t launch_bias_act_bwd(const BiasActBwdParams &p, hipStream_t s);

// act is the same for every lane, so it is chosen once for NV values.
template <bool TO_BF16, int NV, typename V>
__device__ __forceinline__ void act_all(V &v, int act) {
    if (act == kActSilu) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = gate_act<kActSilu, TO_BF16>(v[i]);
    } else if (act == kActGelu) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = gate_act<kActGelu, TO_BF16>(v[i]);
    }
}

}  // namespace bbs
