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
    uint8_t *ws;                       // moe_ws_bytes; the hidden values first
    float *part;                       // in ws, behind them: outputs of a range of a pair
};

// ---------------------------------------------------------------------------
// The tile kernels' shapes
// ---------------------------------------------------------------------------
// Two waves a SIMD, with 256 registers each.  Three (168 registers) were slower: 16
// tokens, MXFP4, 118.6 us against 113.7; 64 tokens, NVFP4, 281 against 186, with 75
// registers in scratch memory in the down projection.
constexpr int kMoeTileWaves = 8;
constexpr int kMoeStep = 512;                                      // K values of a step
constexpr int kMoeLds = 160 * 1024;                                // of a CU

// How a tile kernel divides its K: ranges of `range` values (a multiple of a step where
// there are several), of which `rows` (32, 16, 8 or 4) rows fit LDS.
struct MoeShape {
    int64_t range;
    int ranges, rows;
};

// LDS of a tile kernel: the rows, the waves' sums (for each 16 rows), the units.  The
// lists that lead to the units (12 bytes an expert, 4 a pair: 20 KB at most) lie where
// the rows and sums come, which are 28 KB at least.
__host__ __device__ inline int64_t moe_rows_bytes(const MoeShape &s) {
    return (s.range + kMoeStep - 1) / kMoeStep * s.rows * 1024;
}
__host__ __device__ constexpr int64_t moe_sums_bytes(int tiles) { return kMoeTileWaves * 512 * 4 * tiles; }
inline int64_t moe_units_bytes(int64_t T, int64_t k) { return 16 + T * k * 12; }
inline int64_t moe_tile_lds(int64_t T, int64_t k, const MoeShape &s) {
    return moe_rows_bytes(s) + moe_sums_bytes((s.rows + 15) / 16) + moe_units_bytes(T, k);
}
// Up projection: an activation needs all of K, so the rows are as many as fit (0: too few).
inline MoeShape moe_up_shape(int64_t T, int64_t k, int64_t K) {
    MoeShape s{K, 1, 16};
    while (s.rows >= 4 && moe_tile_lds(T, k, s) > kMoeLds) s.rows /= 2;
    if (s.rows < 4) s.rows = 0;
    return s;
}
// Down projection: two tiles of sixteen rows past eight tokens (the values' parts fill
// the first: 64 tokens, 84.9 us against 88), and as few ranges as leave room for them.
inline MoeShape moe_down_shape(int64_t T, int64_t k, int64_t F) {
    MoeShape s{F, 1, T > 8 ? 32 : 16};
    while (moe_tile_lds(T, k, s) > kMoeLds) {
        ++s.ranges;
        s.range = (F + kMoeStep * s.ranges - 1) / (kMoeStep * s.ranges) * kMoeStep;
    }
    s.ranges = (int)((F + s.range - 1) / s.range);
    return s;
}

// Bytes of workspace: the hidden values, then the routing or the pairs' outputs.
inline int64_t moe_slots(int64_t T, int64_t k, int64_t E) { return T * k < E ? T * k : E; }
inline int64_t moe_hidden_bytes(int64_t T, int64_t k, int64_t F) { return 3 * T * k * F * 2; }
inline int64_t moe_ws_bytes(int64_t T, int64_t k, int64_t E, int64_t F, int64_t N) {
    const int64_t plan = moe_slots(T, k, E) * (8 + T * (int64_t)sizeof(MoeEntry));
    const int64_t part = moe_down_shape(T, k, F).ranges * T * k * N * 4;
    return moe_hidden_bytes(T, k, F) + (plan > part ? plan : part);
}

hipError_t launch_moe(const MoeParams &p, bool mxfp4, hipStream_t s);

}  // namespace bbs
