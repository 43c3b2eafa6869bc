// Gated NVFP4 GEMM, large-tile kernel for K % 128 == 0 (gfx950):
//   g = A Wg^T, u = A Wu^T, h = act(g) * u, optional MXFP8 checkpoints of g, u.
//
// The tile engine's 256 x 256 tile holds 256 rows by 128 columns of both
// products: its B side alternates 32-column blocks of the gate and the up
// weights inside each wave's share (GatedB), so the two accumulators of one
// output sit in the same lane and register place, and the activation, the
// product and the checkpoints are register arithmetic in the epilogue.  A
// checkpoint's 32-block is one accumulator block's row, held by lanes l and
// l ^ 32.  The epilogue of a tile runs while the next tile's first slabs are
// copied, as for the plain outputs.
//
// Bound by the matrix instructions and the expansion beside them, as the plain
// product: 8192 x 14336 x 4096 takes 1.34 ms = 1.44 PFLOP/s (1.40 ms with
// checkpoints, whose 242 MB take 50 us to write at the copy rate); the FP16
// product of a library reaches 1.49 PFLOP/s on the same card.  2048 x 1536 x
// 4096 takes 55 us: 192 half tiles leave a quarter of the CUs idle.
#include "gemm_nvfp4_tiles.hpp"
#include "gated_epilogue.hpp"

namespace bbs {

namespace {

template <int ACT, bool BF16_OUT, int NJ>
__device__ __forceinline__ void gated_epilogue(uint8_t *stage, uint8_t *stage2, const GatedParams &p,
                                               const f32x16 (&acc)[4][NJ], const big::TileRef &t, int wm,
                                               int wn, int lane) {
    constexpr int HJ = NJ / 2, WC = HJ * 32;              // the wave's output columns
    constexpr int ES = BF16_OUT ? 2 : 4, RS = WC * ES + 16;
    constexpr int LPR = WC * ES / 16, RPI = 64 / LPR;     // lanes a row, rows an instruction on read-back
    uint8_t *const buf[2] = {stage + (threadIdx.x >> 6) * (32 * RS), stage2 + (threadIdx.x >> 6) * (32 * RS)};
    const int64_t mw = t.m0 + wm * 128, nw = t.n0 + wn * WC;
    const int half = lane >> 5;
    const float sg = p.b.s_dec[0], su = p.u.s_dec[0];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = mw + i * 32 + (lane & 31);
        const float sa = p.a.s_dec[p.a.sdec_rows ? (m < t.m_end ? m : t.m_end - 1) : 0];
        uint8_t *const row = buf[i & 1] + (lane & 31) * RS;
#pragma unroll
        for (int j = 0; j < HJ; ++j) {
            f32x16 g = acc[i][j], u = acc[i][j + HJ];
            scale16(g, sa * sg);
            scale16(u, sa * su);
            if (p.g_codes) {
                uint32_t w[4];
                const int64_t n = nw + j * 32;
                const uint32_t bg = checkpoint16(g, w);
                store_checkpoint16(w, bg, p.g_codes, p.g_scales, p.N, m < t.m_end, m, n, half);
                const uint32_t bu = checkpoint16(u, w);
                store_checkpoint16(w, bu, p.u_codes, p.u_scales, p.N, m < t.m_end, m, n, half);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = gate_act<ACT, BF16_OUT>(g[4 * q + e]) * u[4 * q + e];
                store4<BF16_OUT>(row, j * 32 + 8 * q + 4 * half, h[0], h[1], h[2], h[3]);
            }
        }
        big::lds_order();
#pragma unroll
        for (int q = 0; q < 32 / RPI; ++q) {
            const int r = q * RPI + lane / LPR, cb = (lane % LPR) * 16;
            const uint4 v = *reinterpret_cast<const uint4 *>(buf[i & 1] + r * RS + cb);
            const int64_t mo = mw + i * 32 + r, n = nw + cb / ES;
            if (mo < t.m_end && n < p.N)
                *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.h) + (mo * p.ldh + n) * ES) = v;
        }
    }
}

template <int ACT, bool BF16_OUT>
__global__ __launch_bounds__(big::NT) void nvfp4_gated_gemm_kernel(GatedParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    big::Smem &sm = *reinterpret_cast<big::Smem *>(smem_raw);
    uint8_t *const stage2 = smem_raw + sizeof(big::Smem);
    constexpr int BF = big::BN / 2;                       // output columns of a tile
    const int64_t tm = (p.M + big::BM - 1) / big::BM, tn = (p.N + BF - 1) / BF;
    // as for the dense GEMM: a last round that fills at most half the
    // workgroups runs as half tiles (64 columns)
    const int64_t total = tm * tn, rem = total % gridDim.x;
    const bool split = rem > 0 && 2 * rem <= gridDim.x;
    const int64_t n_whole = split ? total - rem : total;
    auto tile_at = [&](int64_t tid, big::TileRef &r) {
        const int64_t gsize = big::GROUP_M * tn;
        const int64_t g = tid / gsize, in = tid - g * gsize;
        const int64_t gm = (tm - g * big::GROUP_M) < big::GROUP_M ? (tm - g * big::GROUP_M) : big::GROUP_M;
        r.m0 = (g * big::GROUP_M + in % gm) * big::BM;
        r.m_end = p.M;
        r.n0 = (in / gm) * BF;
        r.g = 0;
    };
    TileWalk walk(n_whole), half_walk(split ? 2 * rem : 0);
    auto next_tile = [&](big::TileRef &r) -> bool {
        int64_t tid;
        if (!walk.take(tid)) return false;
        tile_at(tid, r);
        return true;
    };
    auto next_half = [&](big::TileRef &r) -> bool {
        int64_t h;
        if (!half_walk.take(h)) return false;
        tile_at(n_whole + (h >> 1), r);
        r.n0 += (h & 1) * (BF / 2);
        return true;
    };
    const big::GatedB B{p.b, p.u};
    auto b_side = [B](int) { return B; };
    auto ident = [](int64_t r) { return r; };
    auto finish = [&](uint8_t *stage, const auto &acc, const big::TileRef &t, int wm, int wn, int lane)
                      __attribute__((always_inline)) {
        gated_epilogue<ACT, BF16_OUT>(stage, stage2, p, acc, t, wm, wn, lane);
    };
    if (p.b.tile2d) big::run_tiles<true, 4>(sm, nullptr, nullptr, p.a, p.K, p.N, next_tile, b_side, ident, finish);
    else big::run_tiles<false, 4>(sm, nullptr, nullptr, p.a, p.K, p.N, next_tile, b_side, ident, finish);
    if (split) {
        __syncthreads();      // the last whole tile's epilogue has read its staging rows
        if (p.b.tile2d)
            big::run_tiles<true, 2>(sm, nullptr, nullptr, p.a, p.K, p.N, next_half, b_side, ident, finish);
        else
            big::run_tiles<false, 2>(sm, nullptr, nullptr, p.a, p.K, p.N, next_half, b_side, ident, finish);
    }
}

}  // namespace

hipError_t launch_gated_gemm_big(const GatedParams &p, int act, bool bf16_out, hipStream_t s) {
    const int64_t tiles = ((p.M + big::BM - 1) / big::BM) * ((p.N + big::BN / 2 - 1) / (big::BN / 2));
    const int64_t grid = persistent_grid(2 * tiles, s);
    if (act == kActGelu) {
        if (bf16_out) launch_with_smem<nvfp4_gated_gemm_kernel<kActGelu, true>>(grid, kSmemPlain, p, s);
        else launch_with_smem<nvfp4_gated_gemm_kernel<kActGelu, false>>(grid, kSmemPlain, p, s);
    } else {
        if (bf16_out) launch_with_smem<nvfp4_gated_gemm_kernel<kActSilu, true>>(grid, kSmemPlain, p, s);
        else launch_with_smem<nvfp4_gated_gemm_kernel<kActSilu, false>>(grid, kSmemPlain, p, s);
    }
    return hipGetLastError();
}

}  // namespace bbs
