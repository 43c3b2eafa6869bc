// A mixture-of-experts layer for a few tokens: parameter block and launcher.
#pragma once

#include "gated.hpp"

namespace bbs {

constexpr int kMoeSlots = 32;          // most experts a token chooses
constexpr int kMoeExperts = 1024;

// One token's share of an expert: the pair (row of h) that holds it and its weight.
struct MoeEntry {
    int32_t pair;
    float weight;
};

struct MoeParams {
    const uint16_t *x;                 // T x K
    int64_t T, ldx;
    const int32_t *ids;                // T x k
    const float *weights;              // T x k, or null (1)
    int k, E;
    GemvParams::Weight g, u, d;        // stacked: E x F rows of K (g: the gated form), E x N rows of F
    int64_t K, F, N;
    int tile2d, gated, act;
    const void *r;                     // residual of y's type, or null
    int64_t ldr;
    void *y;                           // T x N
    int64_t ldy;
    int bf16_out;
    uint8_t *ws;                       // moe_ws_bytes
};

// Bytes of workspace: the routing and the hidden values.
inline int64_t moe_slots(int64_t T, int64_t k, int64_t E) { return T * k < E ? T * k : E; }
inline int64_t moe_plan_bytes(int64_t T, int64_t k, int64_t E) {
    return (moe_slots(T, k, E) * (8 + T * (int64_t)sizeof(MoeEntry)) + 15) / 16 * 16;
}
inline int64_t moe_ws_bytes(int64_t T, int64_t k, int64_t E, int64_t F) {
    return moe_plan_bytes(T, k, E) + 3 * T * k * F * 2;
}

hipError_t launch_moe(const MoeParams &p, bool mxfp4, hipStream_t s);

}  // namespace bbs
