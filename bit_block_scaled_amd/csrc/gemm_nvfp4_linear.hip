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
//
// Bound by the products' matrix instructions, and beside them by the epilogue's
// vector ones (22 a value with GELU and a checkpoint), during which a SIMD's only
// wave leaves its matrix unit idle.  Measured, BF16 outputs, replayed from a graph on one
// card (others were up to 5% slower in all of them): 8192 x 4096 x 14336 with bias and
// residual 659 us (1.46 PFLOP/s), the product alone 650; 8192 x 14336 x 4096 alone 663
// us, with bias 673, with bias, GELU and checkpoint 727 (1.32).
#include "gemm_nvfp4_tiles.hpp"
#include "linear.hpp"

namespace bbs {

namespace {

constexpr size_t kSmemLinear = kSmemPlain + 4 * 128 * sizeof(float);    // and a wave's columns of the bias

// Nothing is loaded once the stores have begun but the residual, a piece ahead of
// its use: loads and stores share one counter, so a load's wait is one for the stores
// before it, and with one wave a SIMD nothing else would run meanwhile.
template <bool BF16_OUT, bool RES, int NJ>
__device__ __forceinline__ void linear_epilogue(uint8_t *stage, uint8_t *stage2, float *bias, const LinearParams &p,
                                                const f32x16 (&acc)[4][NJ], const big::TileRef &t, int wm, int wn,
                                                int lane) {
    constexpr bool HALF = BF16_OUT && !RES;               // staged in BF16
    constexpr int ES = HALF ? 2 : 4;                      // bytes of a staged value
    constexpr int PJ = HALF ? NJ : 2;                     // 32-column blocks of a piece
    constexpr int PC = PJ * 32, RS = PC * ES + 16;        // its columns, its staging row stride
    constexpr int VL = BF16_OUT ? 8 : 4;                  // outputs of a lane on read-back (16 bytes)
    constexpr int OS = 16 / VL;                           // bytes of an output
    constexpr int LPR = PC / VL, RPI = 64 / LPR;          // lanes a row, rows an instruction
    constexpr int NQ = 32 / RPI, NP = NJ / PJ;            // instructions a piece, pieces a row block
    const int wave = threadIdx.x >> 6, half = lane >> 5;
    uint8_t *const buf[2] = {stage + wave * (32 * RS), stage2 + wave * (32 * RS)};
    const int64_t mw = t.m0 + wm * 128, nw = t.n0 + wn * (NJ * 32);
    // the lane's first row and column on read-back, and how many are left from there
    const int64_t mo = mw + lane / LPR, no = nw + (lane % LPR) * VL;
    const int rows = (int)min(t.m_end - mo, (int64_t)128), cols = (int)min(p.N - no, (int64_t)(NJ * 32));
    uint8_t *const out = static_cast<uint8_t *>(p.c) + (mo * p.ldc + no) * OS;
    const uint8_t *const from = static_cast<const uint8_t *>(p.r) + (mo * p.ldr + no) * OS;
    auto at = [](int k, int q) { return k / NP * 32 + q * RPI; };       // row from there: piece k, instruction q
    uint4 res[2][RES ? NQ : 1];
    auto load_res = [&](int k) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            res[k & 1][q] = make_uint4(0, 0, 0, 0);
            if (at(k, q) < rows && k % NP * PC < cols)
                res[k & 1][q] = *reinterpret_cast<const uint4 *>(from + (at(k, q) * p.ldr + k % NP * PC) * OS);
        }
    };
    float scale[4];
    const float sb = p.b.s_dec[0];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = mw + i * 32 + (lane & 31);
        scale[i] = p.a.s_dec[p.a.sdec_rows ? (m < t.m_end ? m : t.m_end - 1) : 0] * sb;
    }
    if (p.bias) {
        bias += wave * 128;                               // the wave's columns, two a lane
        const int64_t n = min(nw + 2 * min(lane, NJ * 16 - 1), p.N - 2);
        float2 b;
        if (p.bias_bf16) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.bias) + n);
            b = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
        } else {
            b = *reinterpret_cast<const float2 *>(static_cast<const float *>(p.bias) + n);
        }
        if (lane < NJ * 16) *reinterpret_cast<float2 *>(bias + 2 * lane) = b;
        big::lds_order();
    }
    if constexpr (RES) load_res(0);
#pragma unroll
    for (int k = 0; k < 4 * NP; ++k) {
        const int i = k / NP, piece = k % NP;
        uint8_t *const b = buf[k & 1];
        uint8_t *const row = b + (lane & 31) * RS;
        if constexpr (RES)
            if (k + 1 < 4 * NP) load_res(k + 1);
        const int64_t m = mw + i * 32 + (lane & 31);
#pragma unroll
        for (int jj = 0; jj < PJ; ++jj) {
            f32x16 v = acc[i][piece * PJ + jj];
            // keeps the block in its accumulators until here: read all at once at the
            // epilogue's start they pushed 170 registers into scratch memory, whose
            // reloads wait for the stores
            asm volatile("" : "+a"(v));
            scale16(v, scale[i]);
            if (p.bias) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float4 bv = *reinterpret_cast<const float4 *>(bias + piece * PC + jj * 32 + 8 * g + 4 * half);
                    v[4 * g] += bv.x;
                    v[4 * g + 1] += bv.y;
                    v[4 * g + 2] += bv.z;
                    v[4 * g + 3] += bv.w;
                }
            }
            if (p.z_codes) {
                uint32_t w[4];
                const uint32_t byte = checkpoint16(v, w);
                store_checkpoint16(w, byte, p.z_codes, p.z_scales, p.N, m < t.m_end, m, nw + piece * PC + jj * 32, half);
            }
            act_all<BF16_OUT, 16>(v, p.act);
#pragma unroll
            for (int g = 0; g < 4; ++g)
                store4<HALF>(row, jj * 32 + 8 * g + 4 * half, v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
        }
        big::lds_order();
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const uint8_t *const src = b + (q * RPI + lane / LPR) * RS + (lane % LPR) * (VL * ES);
            uint4 o = *reinterpret_cast<const uint4 *>(src);
            if constexpr (RES) {
                const uint4 r = res[k & 1][q];
                const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
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
            if (at(k, q) < rows && piece * PC < cols)
                *reinterpret_cast<uint4 *>(out + (at(k, q) * p.ldc + piece * PC) * OS) = o;
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <bool BF16_OUT, bool RES>
__global__ __launch_bounds__(big::NT) void nvfp4_linear_kernel(LinearParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    big::Smem &sm = *reinterpret_cast<big::Smem *>(smem_raw);
    uint8_t *const stage2 = smem_raw + sizeof(big::Smem);
    float *const bias = reinterpret_cast<float *>(smem_raw + kSmemPlain);
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
        linear_epilogue<BF16_OUT, RES>(stage, stage2, bias, p, acc, t, wm, wn, lane);
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
        if (bf16_out) launch_with_smem<nvfp4_linear_kernel<true, true>>(grid, kSmemLinear, p, s);
        else launch_with_smem<nvfp4_linear_kernel<false, true>>(grid, kSmemLinear, p, s);
    } else {
        if (bf16_out) launch_with_smem<nvfp4_linear_kernel<true, false>>(grid, kSmemLinear, p, s);
        else launch_with_smem<nvfp4_linear_kernel<false, false>>(grid, kSmemLinear, p, s);
    }
    return hipGetLastError();
}

}  // namespace bbs
