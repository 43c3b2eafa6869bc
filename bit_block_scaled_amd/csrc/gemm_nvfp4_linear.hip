// NVFP4 product of a linear layer with its epilogue, large-tile kernel for
// K % 128 == 0 (gfx950):
//   z = A W^T + b, c = act(z) + r, optional MXFP8 checkpoint of z.
//
// The tile engine's products stay as they are.  In the epilogue a lane holds,
// of each 32 x 32 block, 16 values of one output row: decode scale and bias
// are one FMA each, the checkpoint's 32-block is that row of the block (held
// by lanes l and l ^ 32), the activation register arithmetic.  The values then
// go through LDS to whole row segments, where the residual, loaded in the same
// segments, is added.  With a residual they are staged in FP32, so that the sum
// rounds once.
#include "gemm_nvfp4_tiles.hpp"
#include "linear.hpp"

namespace bbs {

namespace {

template <bool BF16_OUT, bool RES, int NJ>
__device__ __forceinline__ void linear_epilogue(uint8_t *stage, uint8_t *stage2, const LinearParams &p,
                                                const f32x16 (&acc)[4][NJ], const big::TileRef &t, int wm, int wn,
                                                int lane) {
    constexpr bool HALF = BF16_OUT && !RES;               // staged in BF16
    constexpr int ES = HALF ? 2 : 4;                      // bytes of a staged value
    constexpr int PJ = HALF ? NJ : 2;                     // 32-column blocks of a piece
    constexpr int PC = PJ * 32, RS = PC * ES + 16;        // its columns, its staging row stride
    constexpr int VL = BF16_OUT ? 8 : 4;                  // outputs of a lane on read-back (16 bytes)
    constexpr int LPR = PC / VL, RPI = 64 / LPR;          // lanes a row, rows an instruction
    constexpr int NQ = 32 / RPI;
    uint8_t *const buf[2] = {stage + (threadIdx.x >> 6) * (32 * RS), stage2 + (threadIdx.x >> 6) * (32 * RS)};
    const int64_t mw = t.m0 + wm * 128, nw = t.n0 + wn * (NJ * 32);
    const int half = lane >> 5;
    const float sb = p.b.s_dec[0];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = mw + i * 32 + (lane & 31);
        const float scale = p.a.s_dec[p.a.sdec_rows ? (m < t.m_end ? m : t.m_end - 1) : 0] * sb;
#pragma unroll
        for (int piece = 0; piece < NJ / PJ; ++piece) {
            uint8_t *const b = buf[(i * (NJ / PJ) + piece) & 1];
            uint8_t *const row = b + (lane & 31) * RS;
            const int64_t np = nw + piece * PC;           // the piece's first column
            const int64_t mo = mw + i * 32 + lane / LPR, no = np + (lane % LPR) * VL;
            uint4 res[NQ];
            if constexpr (RES) {
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    const int64_t mr = mo + q * RPI;
                    res[q] = make_uint4(0, 0, 0, 0);
                    if (mr < t.m_end && no < p.N)
                        res[q] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.r) +
                                                                  (mr * p.ldr + no) * (16 / VL));
                }
            }
#pragma unroll
            for (int jj = 0; jj < PJ; ++jj) {
                const int64_t n = np + jj * 32;
                f32x16 v = acc[i][piece * PJ + jj];
                scale16(v, scale);
                if (p.bias) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int64_t nb = n + 8 * g + 4 * half;
                        float bv[4];
                        load_bias4(p.bias, p.bias_bf16, nb < p.N ? nb : 0, bv);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[4 * g + e] = v[4 * g + e] + bv[e];
                    }
                }
                if (p.z_codes) {
                    uint32_t w[4];
                    const uint32_t byte = checkpoint16(v, w);
                    store_checkpoint16(w, byte, p.z_codes, p.z_scales, p.N, m < t.m_end, m, n, half);
                }
                act_all<BF16_OUT, 16>(v, p.act);
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    store4<HALF>(row, jj * 32 + 8 * g + 4 * half, v[4 * g], v[4 * g + 1], v[4 * g + 2],
                                 v[4 * g + 3]);
            }
            big::lds_order();
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const uint8_t *const src = b + (q * RPI + lane / LPR) * RS + (lane % LPR) * (VL * ES);
                uint4 o = *reinterpret_cast<const uint4 *>(src);
                if constexpr (RES) {
                    const uint32_t rw[4] = {res[q].x, res[q].y, res[q].z, res[q].w};
                    if constexpr (BF16_OUT) {
                        const uint4 o2 = *reinterpret_cast<const uint4 *>(src + 16);
                        const uint32_t vw[8] = {o.x, o.y, o.z, o.w, o2.x, o2.y, o2.z, o2.w};
                        uint32_t ow[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            ow[e] = pk_bf16(__uint_as_float(vw[2 * e]) + __uint_as_float(rw[e] << 16),
                                            __uint_as_float(vw[2 * e + 1]) + __uint_as_float(rw[e] & 0xFFFF0000u));
                        o = make_uint4(ow[0], ow[1], ow[2], ow[3]);
                    } else {
                        const uint32_t vw[4] = {o.x, o.y, o.z, o.w};
                        uint32_t ow[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            ow[e] = __float_as_uint(__uint_as_float(vw[e]) + __uint_as_float(rw[e]));
                        o = make_uint4(ow[0], ow[1], ow[2], ow[3]);
                    }
                }
                const int64_t mr = mo + q * RPI;
                if (mr < t.m_end && no < p.N)
                    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.c) + (mr * p.ldc + no) * (16 / VL)) = o;
            }
        }
    }
}

template <bool BF16_OUT, bool RES>
__global__ __launch_bounds__(big::NT) void nvfp4_linear_kernel(LinearParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    big::Smem &sm = *reinterpret_cast<big::Smem *>(smem_raw);
    uint8_t *const stage2 = smem_raw + sizeof(big::Smem);
    const int64_t tm = (p.M + big::BM - 1) / big::BM, tn = (p.N + big::BN - 1) / big::BN;
    // as for the plain product: a last round that fills at most half the
    // workgroups runs as half tiles (128 columns)
    const int64_t total = tm * tn, rem = total % gridDim.x;
    const bool split = rem > 0 && 2 * rem <= gridDim.x;
    const int64_t n_whole = split ? total - rem : total;
    auto tile_at = [&](int64_t tid, big::TileRef &r) {
        const int64_t gsize = big::GROUP_M * tn;
        const int64_t g = tid / gsize, in = tid - g * gsize;
        const int64_t gm = (tm - g * big::GROUP_M) < big::GROUP_M ? (tm - g * big::GROUP_M) : big::GROUP_M;
        r.m0 = (g * big::GROUP_M + in % gm) * big::BM;
        r.m_end = p.M;
        r.n0 = (in / gm) * big::BN;
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
        r.n0 += (h & 1) * (big::BN / 2);
        return true;
    };
    const Fp4View B = p.b;
    auto b_side = [B](int) { return B; };
    auto ident = [](int64_t r) { return r; };
    auto finish = [&](uint8_t *stage, const auto &acc, const big::TileRef &t, int wm, int wn, int lane)
                      __attribute__((always_inline)) {
        linear_epilogue<BF16_OUT, RES>(stage, stage2, p, acc, t, wm, wn, lane);
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

hipError_t launch_linear_big(const LinearParams &p, bool bf16_out, hipStream_t s) {
    const int64_t tiles = ((p.M + big::BM - 1) / big::BM) * ((p.N + big::BN - 1) / big::BN);
    const int64_t grid = persistent_grid(2 * tiles, s);
    if (p.r) {
        if (bf16_out) launch_with_smem<nvfp4_linear_kernel<true, true>>(grid, kSmemPlain, p, s);
        else launch_with_smem<nvfp4_linear_kernel<false, true>>(grid, kSmemPlain, p, s);
    } else {
        if (bf16_out) launch_with_smem<nvfp4_linear_kernel<true, false>>(grid, kSmemPlain, p, s);
        else launch_with_smem<nvfp4_linear_kernel<false, false>>(grid, kSmemPlain, p, s);
    }
    return hipGetLastError();
}

}  // namespace bbs
