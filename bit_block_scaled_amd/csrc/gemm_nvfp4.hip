// NVFP4 x NVFP4 GEMM, large-tile kernels for K % 128 == 0 (gfx950): the dense
// and grouped products on the tile engine, with plain, quantizing and
// encoding outputs.
#include "gemm_nvfp4_tiles.hpp"

namespace bbs {

// The tile loop with one of the plain or encoding epilogues.
//   scale_of(m, g)         output scale of row m in group g's tile
template <int OUT, bool BT, bool DROP, int NJ, typename Next, typename BView, typename RowMap,
          typename ScaleFn>
__device__ __forceinline__ void run_out(big::Smem &sm, float *tab, const GemmParams &p, Next next_tile,
                                        BView b_view, RowMap a_row, ScaleFn scale_of) {
    auto finish = [&](uint8_t *stage, const f32x16 (&acc)[4][NJ], const big::TileRef &t, int wm, int wn,
                      int lane) __attribute__((always_inline)) {
        const int g = t.g;
        big::epilogue<OUT, DROP, NJ>(stage, tab, acc, t.m0, t.m_end, t.n0, p.N,
                                     [&](int64_t m) { return scale_of(m, g); }, p.c, p.ldc, wm, wn, lane, p.q);
    };
    big::run_tiles<BT, NJ>(sm, tab, OUT == big::OUT_QG ? p.q.gelu_tab : nullptr, p.a, p.K, p.N, next_tile,
                           b_view, a_row, finish);
}

template <int OUT>
__device__ __forceinline__ void dense_body(const GemmParams &p, uint8_t *smem_raw) {
    big::Smem &sm = *reinterpret_cast<big::Smem *>(smem_raw);
    float *tab = reinterpret_cast<float *>(smem_raw + sizeof(big::Smem));
    if ((OUT == big::OUT_Q || OUT == big::OUT_QG) && blockIdx.x == 0 && threadIdx.x == 0)
        p.q.s_dec[0] = 1.0f / p.q.s_enc[0];
    const int64_t tm = (p.M + big::BM - 1) / big::BM, tn = (p.N + big::BN - 1) / big::BN;
    const int64_t total = tm * tn, grid = gridDim.x;
    // A last round of whole tiles that would leave more than half the
    // workgroups idle is run as twice as many 256 x 128 half tiles (plain
    // output modes): every workgroup then takes one half, and the round
    // costs about half a tile instead of a whole one.
    constexpr bool kHalves = OUT == big::OUT_F32 || OUT == big::OUT_BF16;
    const int64_t rem = total % grid;
    const bool split = kHalves && rem > 0 && 2 * rem <= grid;
    const int64_t n_whole = split ? total - rem : total;
    const int64_t M = p.M;
    auto tile_at = [&](int64_t tid, big::TileRef &r) {
        // grouped order: GROUP_M tiles down M, then along N
        const int64_t gsize = big::GROUP_M * tn;
        const int64_t g = tid / gsize, in = tid - g * gsize;
        const int64_t gm = (tm - g * big::GROUP_M) < big::GROUP_M ? (tm - g * big::GROUP_M) : big::GROUP_M;
        r.m0 = (g * big::GROUP_M + in % gm) * big::BM;
        r.m_end = M;
        r.n0 = (in / gm) * big::BN;
        r.g = 0;
    };
    TileWalk walk(n_whole);
    auto next_tile = [&](big::TileRef &r) -> bool {
        int64_t tid;
        if (!walk.take(tid)) return false;
        tile_at(tid, r);
        return true;
    };
    // half h: tile n_whole + h / 2, columns 128 * (h % 2) onwards (both
    // halves of a tile fall in one XCD's contiguous share)
    TileWalk half_walk(split ? 2 * rem : 0);
    auto next_half = [&](big::TileRef &r) -> bool {
        int64_t h;
        if (!half_walk.take(h)) return false;
        tile_at(n_whole + (h >> 1), r);
        r.n0 += (h & 1) * (big::BN / 2);
        return true;
    };
    const Fp4View B = p.b;
    auto b_view = [B](int) { return B; };
    auto ident = [](int64_t r) { return r; };
    const float sb = p.b.s_dec[0];
    auto run = [&](auto scale_of) {
        if (p.b.tile2d)
            run_out<OUT, true, false, 4>(sm, tab, p, next_tile, b_view, ident, scale_of);
        else
            run_out<OUT, false, false, 4>(sm, tab, p, next_tile, b_view, ident, scale_of);
        if constexpr (kHalves) {
            if (split) {
                // the last whole tile's epilogue has read its staging rows
                // before the ring is refilled
                __syncthreads();
                if (p.b.tile2d)
                    run_out<OUT, true, false, 2>(sm, tab, p, next_half, b_view, ident,
                                                        scale_of);
                else
                    run_out<OUT, false, false, 2>(sm, tab, p, next_half, b_view, ident,
                                                         scale_of);
            }
        }
    };
    if (p.a.sdec_rows) {
        const float *sa = p.a.s_dec;
        run([sa, sb](int64_t m, int) { return sa[m] * sb; });
    } else {
        const float out_scale = p.a.s_dec[0] * sb;
        run([out_scale](int64_t, int) { return out_scale; });
    }
}

template <bool BF16_OUT>
__global__ __launch_bounds__(big::NT) void nvfp4_gemm_big_kernel(GemmParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    dense_body<BF16_OUT ? big::OUT_BF16 : big::OUT_F32>(p, smem_raw);
}

template <bool GELU>
__global__ __launch_bounds__(big::NT) void nvfp4_gemm_quant_kernel(GemmParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    dense_body<GELU ? big::OUT_QG : big::OUT_Q>(p, smem_raw);
}

__global__ __launch_bounds__(big::NT) void nvfp4_gemm_s2f6_kernel(GemmParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    dense_body<big::OUT_S2F6>(p, smem_raw);
}

constexpr int kMaxGroupsBig = 1024;

template <int OUT>
__device__ __forceinline__ void grouped_body(const GemmParams &p, uint8_t *smem_raw,
                                             int64_t *tile_start, int64_t *row_start) {
    big::Smem &sm = *reinterpret_cast<big::Smem *>(smem_raw);
    float *tab = reinterpret_cast<float *>(smem_raw + sizeof(big::Smem));
    if ((OUT == big::OUT_Q || OUT == big::OUT_QG) && blockIdx.x == 0 && threadIdx.x == 0)
        p.q.s_dec[0] = 1.0f / p.q.s_enc[0];
    const int64_t n_tiles_n = (p.N + big::BN - 1) / big::BN;
    if (threadIdx.x == 0) {
        int64_t acc = 0, prev = 0;
        for (int g = 0; g <= p.G; ++g) {
            int64_t off = p.group_offsets[g];
            off = off < prev ? prev : off;
            off = off > p.max_rows ? p.max_rows : off;
            row_start[g] = off;
            if (g > 0) acc += ((off - prev + big::BM - 1) / big::BM) * n_tiles_n;
            tile_start[g] = acc;
            prev = off;
        }
    }
    __syncthreads();
    TileWalk walk(tile_start[p.G]);
    const int G = p.G;
    auto next_tile = [&](big::TileRef &r) -> bool {
        int64_t tile;
        if (!walk.take(tile)) return false;
        int g = 0;
        while (g + 1 < G && tile_start[g + 1] <= tile) ++g;
        const int64_t local = tile - tile_start[g];
        const int64_t mt = local / n_tiles_n, nt = local - mt * n_tiles_n;
        r.m0 = row_start[g] + mt * big::BM;
        r.m_end = row_start[g + 1];
        r.n0 = nt * big::BN;
        r.g = g;
        return true;
    };
    const Fp4View B0 = p.b;
    const int64_t b_codes = p.N * (p.K / 2), b_scales = (B0.tile2d ? (p.N / 16) : p.N) * (p.K / 16);
    auto b_view = [B0, b_codes, b_scales](int g) {
        Fp4View B = B0;
        B.codes = B0.codes + (int64_t)g * b_codes;
        B.scales = B0.scales + (int64_t)g * b_scales;
        return B;
    };
    const int32_t *ri = p.row_index;
    const int64_t src_rows = p.a_src_rows;
    auto gather = [ri, src_rows](int64_t r) -> int64_t {
        const int64_t s = ri ? (int64_t)ri[r] : r;
        return (s >= 0 && s < src_rows) ? s : -1;
    };
    const float *sdb = p.b.s_dec;
    auto run = [&](auto scale_of) {
        if (B0.tile2d)
            run_out<OUT, true, true, 4>(sm, tab, p, next_tile, b_view, gather, scale_of);
        else
            run_out<OUT, false, true, 4>(sm, tab, p, next_tile, b_view, gather, scale_of);
    };
    // the output scale of row m: the decode scale of the A row it was
    // computed from times the expert's; 0 for a dropped slot (its copies
    // read A row 0 in place of a row the map misses)
    if (p.a.sdec_rows) {
        const float *sa = p.a.s_dec;
        run([sa, sdb, gather](int64_t m, int g) {
            const int64_t s = gather(m);
            return s < 0 ? 0.0f : sa[s] * sdb[g];
        });
    } else {
        const float sa0 = p.a.s_dec[0];
        run([sa0, sdb, gather](int64_t m, int g) { return gather(m) < 0 ? 0.0f : sa0 * sdb[g]; });
    }
}

template <bool BF16_OUT>
__global__ __launch_bounds__(big::NT) void grouped_nvfp4_gemm_big_kernel(GemmParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ int64_t tile_start[kMaxGroupsBig + 1];
    __shared__ int64_t row_start[kMaxGroupsBig + 1];
    grouped_body<BF16_OUT ? big::OUT_BF16 : big::OUT_F32>(p, smem_raw, tile_start, row_start);
}

template <bool GELU>
__global__ __launch_bounds__(big::NT) void grouped_nvfp4_gemm_quant_kernel(GemmParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ int64_t tile_start[kMaxGroupsBig + 1];
    __shared__ int64_t row_start[kMaxGroupsBig + 1];
    grouped_body<GELU ? big::OUT_QG : big::OUT_Q>(p, smem_raw, tile_start, row_start);
}

__global__ __launch_bounds__(big::NT) void grouped_nvfp4_gemm_s2f6_kernel(GemmParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ int64_t tile_start[kMaxGroupsBig + 1];
    __shared__ int64_t row_start[kMaxGroupsBig + 1];
    grouped_body<big::OUT_S2F6>(p, smem_raw, tile_start, row_start);
}

__global__ void clear_amax_kernel(unsigned *amax) { *amax = 0u; }

static int64_t dense_tiles(const GemmParams &p) {
    return ((p.M + big::BM - 1) / big::BM) * ((p.N + big::BN - 1) / big::BN);
}

constexpr size_t kSmemGelu = sizeof(big::Smem) + kGeluTabSize * sizeof(float);

hipError_t launch_nvfp4_gemm_quant(const GemmParams &p, bool gelu, hipStream_t s) {
    if (p.q.amax) hipLaunchKernelGGL(clear_amax_kernel, dim3(1), dim3(1), 0, s, p.q.amax);
    if (gelu) {
        const hipError_t e = launch_gelu_table(const_cast<float *>(p.q.gelu_tab), s);
        if (e != hipSuccess) return e;
    }
    const int64_t grid = persistent_grid(dense_tiles(p), s);
    if (gelu) launch_with_smem<nvfp4_gemm_quant_kernel<true>>(grid, kSmemGelu, p, s);
    else launch_with_smem<nvfp4_gemm_quant_kernel<false>>(grid, kSmemBig, p, s);
    return hipGetLastError();
}

hipError_t launch_grouped_nvfp4_gemm_quant(const GemmParams &p, bool gelu, hipStream_t s) {
    if (p.G > kMaxGroupsBig) return hipErrorInvalidValue;
    if (p.q.amax) hipLaunchKernelGGL(clear_amax_kernel, dim3(1), dim3(1), 0, s, p.q.amax);
    if (gelu) {
        const hipError_t e = launch_gelu_table(const_cast<float *>(p.q.gelu_tab), s);
        if (e != hipSuccess) return e;
    }
    const int64_t grid = persistent_grid(0, s);
    if (gelu) launch_with_smem<grouped_nvfp4_gemm_quant_kernel<true>>(grid, kSmemGelu, p, s);
    else launch_with_smem<grouped_nvfp4_gemm_quant_kernel<false>>(grid, kSmemBig, p, s);
    return hipGetLastError();
}

hipError_t launch_nvfp4_gemm_s2f6(const GemmParams &p, hipStream_t s) {
    launch_with_smem<nvfp4_gemm_s2f6_kernel>(persistent_grid(dense_tiles(p), s), kSmemBig, p, s);
    return hipGetLastError();
}

hipError_t launch_grouped_nvfp4_gemm_s2f6(const GemmParams &p, hipStream_t s) {
    if (p.G > kMaxGroupsBig) return hipErrorInvalidValue;
    launch_with_smem<grouped_nvfp4_gemm_s2f6_kernel>(persistent_grid(0, s), kSmemBig, p, s);
    return hipGetLastError();
}

hipError_t launch_nvfp4_gemm_big(const GemmParams &p, bool bf16_out, hipStream_t s) {
    // up to two workgroups per tile, so that fewer tiles than CUs run as
    // half tiles
    const int64_t grid = persistent_grid(2 * dense_tiles(p), s);
    if (bf16_out) launch_with_smem<nvfp4_gemm_big_kernel<true>>(grid, kSmemPlain, p, s);
    else launch_with_smem<nvfp4_gemm_big_kernel<false>>(grid, kSmemPlain, p, s);
    return hipGetLastError();
}

hipError_t launch_grouped_nvfp4_gemm_big(const GemmParams &p, bool bf16_out, hipStream_t s) {
    if (p.G > kMaxGroupsBig) return hipErrorInvalidValue;
    const int64_t grid = persistent_grid(0, s);
    if (bf16_out) launch_with_smem<grouped_nvfp4_gemm_big_kernel<true>>(grid, kSmemPlain, p, s);
    else launch_with_smem<grouped_nvfp4_gemm_big_kernel<false>>(grid, kSmemPlain, p, s);
    return hipGetLastError();
}

}  // namespace bbs
