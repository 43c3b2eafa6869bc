// Gated feed-forward operators, small-tile kernels for any K the formats
// allow (gfx950), and the choice between them and the large-tile kernels.
//
//   forward   g = A Wg^T, u = A Wu^T (NVFP4 x NVFP4), h = act(g) * u, and
//             optionally MXFP8 checkpoints of the FP32 g and u
//   backward  dh = dY W (MXFP8 x MXFP8), dg = dh * u * act'(g),
//             du = dh * act(g), with g and u read back from the checkpoints
//
// The forward kernel is the small-tile engine of the NVFP4 products; the backward
// kernel walks K the same way.  There what a copied piece reads past K is
// overwritten by zeros where a code could be NaN.
#include "gemm_nvfp4_small.hpp"
#include "gated_epilogue.hpp"

namespace bbs {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

namespace {

using small::kThreads;
using small::copy_at, small::held, small::join_groups, small::lesser, small::launch, small::run_tile;
using small::GatedSide, small::tile_of, small::tiles_of, small::word_of;

// ---------------------------------------------------------------------------
// Forward: TM rows by 64 columns of both products.
//
// Bound by the expansion of the codes: a wave's 64 x 64 part (TM 128) expands
// four fragments for every four matrix instructions.  528 x 2736 x 1552, BF16:
// 20.9 us on 215 CUs, 2.3 a pair of slabs and 5.5 beside them (on those CUs
// VALU is active 70% of the slabs' time, the matrix units 40%, over half of it
// together); 272 x 1568 x 1184 with checkpoints: 12.5 us.
// Reading the next slab's codes into registers a step ahead, with a ring one
// stage deeper, made it slower by 5%, so it is not the copies' latency.
// ---------------------------------------------------------------------------
template <int TM, int NS, int G, int ACT, bool BF16_OUT>
__global__ __launch_bounds__(kThreads * G, TM == 256 ? 2 : 1) void gated_gemm_kernel(GatedParams p) {
    constexpr int RA = TM / 64;                    // 32-row blocks of a wave
    extern __shared__ __align__(16) uint8_t smem[];
    auto finish = [](const GatedParams &p, const f32x16 (&acc)[RA][2], int64_t mw, int64_t n0, int wn, int lane)
                      __attribute__((always_inline)) {
        const int h = lane >> 5, rl = lane & 31;
        const float sg = p.b.s_dec[0], su = p.u.s_dec[0];
        const int64_t n = n0 + wn * 32 + 16 * h;               // the lane's first column
#pragma unroll
        for (int i = 0; i < RA; ++i) {
            const int64_t m = mw + i * 32 + rl;
            const float sa = p.a.s_dec[p.a.sdec_rows ? (m < p.M ? m : p.M - 1) : 0];
            f32x16 g = acc[i][0], u = acc[i][1];
            scale16(g, sa * sg);
            scale16(u, sa * su);
            const bool in = m < p.M && n < p.N;
            if (p.g_codes) {
                uint32_t wg[4], wu[4];
                const uint32_t bg = checkpoint16(g, wg), bu = checkpoint16(u, wu);
                if (in) {
                    *reinterpret_cast<uint4 *>(p.g_codes + m * p.N + n) = make_uint4(wg[0], wg[1], wg[2], wg[3]);
                    *reinterpret_cast<uint4 *>(p.u_codes + m * p.N + n) = make_uint4(wu[0], wu[1], wu[2], wu[3]);
                    if (h == 0) {
                        p.g_scales[m * (p.N / 32) + n / 32] = (uint8_t)bg;
                        p.u_scales[m * (p.N / 32) + n / 32] = (uint8_t)bu;
                    }
                }
            }
            if (!in) continue;
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
                float y[2][4];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e >> 2][e & 3] = gate_act<ACT, BF16_OUT>(g[4 * q + e]) * u[4 * q + e];
                store8<BF16_OUT>(p.h, m * p.ldh + n + 4 * q, y[0], y[1]);
            }
        }
    };
    run_tile<TM, NS, G, GatedSide>(smem, p, finish);
}

// ---------------------------------------------------------------------------
// Backward: T x T tiles.  The scaled FP8 instruction adds each aligned group of
// eight products on a grid 2^-13 below the group's largest, as in the plain MXFP8
// GEMM: dh is 2e-5 off (relative norm), a hundredth of its BF16 rounding.
// Operand layout as there: lane group g feeds bytes [16g, 16g + 16) and [64 + 16g, 64 + 16g
// + 16) of its row and the scale of the slab's 32-block g.
//
// The product's blocks give lane group g of a wave rows 4 g .. 4 g + 3 of each
// B block, so the B rows are copied in the order that makes those four rows of
// its Q blocks 4 Q consecutive columns (bwd_column): a lane's checkpoint codes
// are then one load an operand and row, taken before the slabs so that they
// are there when the products are, and its outputs whole 16-byte stores.
// (2048 x 4096 x 1536: 28.1 us; with words of four columns, read behind the
// products, 36.9, of which 17 were this epilogue.)
// ---------------------------------------------------------------------------
template <int T>
struct BwdStage {
    uint8_t a[T * 128];              // chunk c of row r at place c ^ ((r >> 1) & 7)
    uint8_t b[T * 128];
    uint32_t sc[2][2 * T];           // the words that hold a row's 4 scale bytes
};

__device__ __forceinline__ int swz8(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// The tile's column in B row r: row 16 j + 4 g + e of a wave's half is its
// column 4 Q g + 4 j + e.
template <int T>
__device__ __forceinline__ int bwd_column(int r) {
    constexpr int H = T / 2, Q = T / 32;
    const int x = r % H;
    return r - x + 4 * Q * (x >> 2 & 3) + 4 * (x >> 4) + (x & 3);
}

template <int T, int NS, int G, int ACT, bool BF16_OUT>
__global__ __launch_bounds__(kThreads * G) void gated_bwd_kernel(GatedBwdParams p) {
    constexpr int AHEAD = NS - 1;
    constexpr int Q = T / 32;                          // 1 KB copies of a wave and operand; MFMA blocks a side
    constexpr int kIssued = 2 * Q + 2;
    extern __shared__ __align__(16) uint8_t smem[];
    const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    BwdStage<T> *const st = reinterpret_cast<BwdStage<T> *>(smem) + grp * NS;
    const Mx8GemmParams &mm = p.mm;
    const int t = threadIdx.x & 255, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    int64_t m0, n0;
    tile_of((uint32_t)((mm.M + T - 1) / T), (uint32_t)((mm.N + T - 1) / T), m0, n0);
    m0 *= T;
    n0 *= T;
    const int64_t nkb = mm.K / 32, nslab = (mm.K + 127) / 128;
    const int tail = (int)(mm.K % 128);

    uint32_t aoff[Q], boff[Q];                         // as in the forward kernel
    const uint8_t *const abase = mm.a_codes + m0 * mm.K, *const bbase = mm.b_codes + n0 * mm.K;
    const uint8_t *const aend = mm.a_codes + mm.M * mm.K - 16, *const bend = mm.b_codes + mm.N * mm.K - 16;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int row = (wave * Q + q) * 8 + (lane >> 3), c = swz8(row, lane & 7);
        aoff[q] = (uint32_t)(min((int64_t)row, mm.M - 1 - m0) * mm.K) + 16 * c;
        boff[q] = (uint32_t)(min((int64_t)bwd_column<T>(row), mm.N - 1 - n0) * mm.K) + 16 * c;
    }
    auto scale_row = [&](int r) -> const uint8_t * {
        return r < T ? mm.a_scales + min(m0 + r, mm.M - 1) * nkb
                     : mm.b_scales + min(n0 + bwd_column<T>(r - T), mm.N - 1) * nkb;
    };
    const int sgroup = min(wave, 2 * T / 64 - 1) * 64;
    const uint8_t *const ssrc = word_of(scale_row(sgroup + lane));
    const uint8_t *const slast = sgroup + lane < T ? word_of(mm.a_scales + mm.M * nkb - 1)
                                                   : word_of(mm.b_scales + mm.N * nkb - 1);
    auto issue = [&](int64_t s, int stage) {
        BwdStage<T> &d = st[stage];
        const int64_t at = s * 128;
        if (s != nslab - 1) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                copy_at(abase + at, aoff[q], d.a + (wave * Q + q) * 1024);
                copy_at(bbase + at, boff[q], d.b + (wave * Q + q) * 1024);
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) copy_lds4(ssrc + s * 4 + 4 * w, &d.sc[w][sgroup]);
        } else {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                copy_at(abase + at, held(aoff[q], aend - (abase + at)), d.a + (wave * Q + q) * 1024);
                copy_at(bbase + at, held(boff[q], bend - (bbase + at)), d.b + (wave * Q + q) * 1024);
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) copy_lds4(lesser(ssrc + s * 4 + 4 * w, slast), &d.sc[w][sgroup]);
        }
    };

    const int kg = lane >> 4, rl = lane & 15;
    int sha[Q], shb[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        sha[i] = (int)(reinterpret_cast<uintptr_t>(scale_row(wm * (T / 2) + i * 16 + rl)) & 3);
        shb[i] = (int)(reinterpret_cast<uintptr_t>(scale_row(T + wn * (T / 2) + i * 16 + rl)) & 3);
    }
    f32x4 acc[Q][Q];
#pragma unroll
    for (int i = 0; i < Q; ++i)
#pragma unroll
        for (int j = 0; j < Q; ++j) acc[i][j] = f32x4{0};

    // the lane's checkpoint codes: 4 Q columns of one row in each row block
    const int64_t n = n0 + wn * (T / 2) + 4 * Q * kg;
    uint32_t gw[Q][Q], uw[Q][Q], gs[Q], us[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const int64_t m = min(m0 + wm * (T / 2) + i * 16 + rl, mm.M - 1), c = min(n, mm.N - 4 * Q);
        __builtin_memcpy(gw[i], __builtin_assume_aligned(p.g_codes + m * mm.N + c, 4 * Q), 4 * Q);
        __builtin_memcpy(uw[i], __builtin_assume_aligned(p.u_codes + m * mm.N + c, 4 * Q), 4 * Q);
        gs[i] = p.g_scales[m * (mm.N / 32) + c / 32];
        us[i] = p.u_scales[m * (mm.N / 32) + c / 32];
    }

    const int64_t own = (nslab - grp + G - 1) / G;       // the group's slabs
    for (int k = 0; k < AHEAD; ++k)
        if (k < own) issue(k * G + grp, k);
    int rd = 0, wr = AHEAD;                              // stages of its slab it and of slab it + AHEAD
    for (int64_t it = 0; it < (nslab + G - 1) / G; ++it) {
        if (it + AHEAD <= own) big::wait_vmcnt<(AHEAD - 1) * kIssued>();    // slab it has landed
        else big::wait_vmcnt<0>();
        __syncthreads();
        const int64_t s = it * G + grp;
        if (it + AHEAD < own) issue(s + AHEAD * G, wr);  // into the stage read before this barrier
        BwdStage<T> &d = st[rd];
        rd = rd + 1 == NS ? 0 : rd + 1;
        wr = wr + 1 == NS ? 0 : wr + 1;
        uint32_t keep = ~0u;
        if (tail && it == (nslab - 1) / G) {
            if (s == nslab - 1) {
                // chunks past K hold other rows' codes: zeros, with scale byte 0
                keep = (1u << (8 * (tail / 32))) - 1;
                const int first = tail / 16, n = 8 - first;
                for (int e = t; e < 2 * T * n; e += kThreads) {
                    const int r = e / n % T, c = first + e % n;
                    *reinterpret_cast<uint4 *>((e < T * n ? d.a : d.b) + r * 128 + 16 * swz8(r, c)) =
                        make_uint4(0, 0, 0, 0);
                }
            }
            __syncthreads();
        }
        if (G > 1 && s >= nslab) continue;
        i32x8 af[Q], bf[Q];
        int sa[Q], sb[Q];
        auto fragment = [&](const uint8_t *side, int r) {
            const uint4 x0 = *reinterpret_cast<const uint4 *>(side + r * 128 + 16 * swz8(r, kg));
            const uint4 x1 = *reinterpret_cast<const uint4 *>(side + r * 128 + 16 * swz8(r, 4 + kg));
            return i32x8{(int)x0.x, (int)x0.y, (int)x0.z, (int)x0.w,
                         (int)x1.x, (int)x1.y, (int)x1.z, (int)x1.w};
        };
        auto scale = [&](int row, int shift) {
            const uint32_t w = __builtin_amdgcn_alignbyte(d.sc[1][row], d.sc[0][row], shift) & keep;
            return (int)((w >> (8 * kg)) & 0xFFu);
        };
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const int ra = wm * (T / 2) + i * 16 + rl, rb = wn * (T / 2) + i * 16 + rl;
            af[i] = fragment(d.a, ra);
            bf[i] = fragment(d.b, rb);
            sa[i] = scale(ra, sha[i]);
            sb[i] = scale(T + rb, shb[i]);
        }
#pragma unroll
        for (int i = 0; i < Q; ++i)
#pragma unroll
            for (int j = 0; j < Q; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[j], af[i], acc[i][j], 0, 0, 0,
                                                                             sb[j], 0, sa[i]);
    }

    join_groups<G>(smem, grp, wave, lane, reinterpret_cast<float(&)[Q * Q * 4]>(acc));
    if (grp) return;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const int64_t m = m0 + wm * (T / 2) + i * 16 + rl;
        if (m >= mm.M || n >= mm.N) continue;
#pragma unroll
        for (int j = 0; j < Q; j += 2) {
            float dg[2][4], du[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float dh[4] = {acc[i][j + k][0], acc[i][j + k][1], acc[i][j + k][2], acc[i][j + k][3]};
                gated_grad4<ACT, BF16_OUT>(dh, gw[i][j + k], gs[i], uw[i][j + k], us[i], dg[k], du[k]);
            }
            store8<BF16_OUT>(mm.c, m * mm.ldc + n + 4 * j, dg[0], dg[1]);
            store8<BF16_OUT>(p.du, m * mm.ldc + n + 4 * j, du[0], du[1]);
        }
    }
}

template <int TM, int NS, int G>
hipError_t fwd(const GatedParams &p, int act, bool bf16_out, hipStream_t s) {
    const int64_t tiles = tiles_of(p.M, p.N, TM, GatedSide::kCols);
    constexpr size_t shm = G * NS * sizeof(small::Stage<TM>);
    if (act == kActGelu)
        return bf16_out ? launch<gated_gemm_kernel<TM, NS, G, kActGelu, true>>(tiles, kThreads * G, shm, p, s)
                        : launch<gated_gemm_kernel<TM, NS, G, kActGelu, false>>(tiles, kThreads * G, shm, p, s);
    return bf16_out ? launch<gated_gemm_kernel<TM, NS, G, kActSilu, true>>(tiles, kThreads * G, shm, p, s)
                    : launch<gated_gemm_kernel<TM, NS, G, kActSilu, false>>(tiles, kThreads * G, shm, p, s);
}

template <int T, int NS, int G>
hipError_t bwd(const GatedBwdParams &p, int act, bool bf16_out, hipStream_t s) {
    const int64_t tiles = tiles_of(p.mm.M, p.mm.N, T, T);
    constexpr size_t shm = G * NS * sizeof(BwdStage<T>);
    if (act == kActGelu)
        return bf16_out ? launch<gated_bwd_kernel<T, NS, G, kActGelu, true>>(tiles, kThreads * G, shm, p, s)
                        : launch<gated_bwd_kernel<T, NS, G, kActGelu, false>>(tiles, kThreads * G, shm, p, s);
    return bf16_out ? launch<gated_bwd_kernel<T, NS, G, kActSilu, true>>(tiles, kThreads * G, shm, p, s)
                    : launch<gated_bwd_kernel<T, NS, G, kActSilu, false>>(tiles, kThreads * G, shm, p, s);
}

}  // namespace

// The choice of tiles, times on 256 CUs.  Large tiles win where they fill the
// CUs; below that the number of CUs reached decides, and where even small
// tiles leave some idle, groups of waves split a tile's slabs.  Two 256-row
// workgroups share a CU (their registers are held to half) and stand in for
// the large tiles where K or the scales' alignment rules those out.
//   rows x F x K        large    256 rows   128 rows, 2 groups   64, 4 groups
//   256 x 4096 x 4096   50 us               38 us                29 us   (256 tiles of 64 rows)
//   512 x 4096 x 2048   31 us               25 us                33 us   (256 of 128)
//   1024 x 4096 x 4096  68 us    71 us      81 us                        (512 of 128)
//   4096 x 4096 x 4096  203 us   246 us     304 us
hipError_t launch_gated_gemm(const GatedParams &p, int act, bool bf16_out, hipStream_t s) {
    auto al8 = [](const void *q) { return reinterpret_cast<uintptr_t>(q) % 8 == 0; };
    const bool large = p.K % 128 == 0 && al8(p.a.scales) && al8(p.b.scales) && al8(p.u.scales);
    const int64_t cus = device_cus(s);
    if (tiles_of(p.M, p.N, 64, GatedSide::kCols) <= cus) return fwd<64, 2, 4>(p, act, bf16_out, s);
    if (tiles_of(p.M, p.N, 128, GatedSide::kCols) <= cus) return fwd<128, 3, 2>(p, act, bf16_out, s);
    if (large) return launch_gated_gemm_big(p, act, bf16_out, s);
    return fwd<256, 2, 1>(p, act, bf16_out, s);
}

// As above:
//   rows x F x K        large    128     128, 2 groups   64      64, 2 groups
//   256 x 4096 x 4096   64 us    41 us   39 us           22 us   22 us    (256 tiles of 64)
//   512 x 4096 x 2048   43 us    27 us   26 us           20 us   23 us    (512 of 64)
//   1024 x 4096 x 4096  66 us    46 us   39 us           66 us   70 us    (256 of 128)
//   2048 x 4096 x 1536  41 us    30 us   43 us           48 us   70 us    (512 of 128)
//   512 x 14336 x 4096  71 us    57 us   98 us          136 us  153 us    (448 of 128)
//   1024 x 10240 x 1536 43 us    41 us                                    (640 of 128)
//   1024 x 10240 x 4096 70 us    87 us                                    (640 of 128)
//   4096 x 8192 x 2048  134 us   145 us                                   (2048 of 128)
// Two small tiles share a CU and one's epilogue runs under the other's slabs,
// so they win as long as one round of them does the work, and with few slabs
// a tile also beyond; on each slab the large tile spends less.  The same holds
// where K is no multiple of 128 (1024 x 10240: 50 and 44 us with K 1504, 89
// and 105 with 4064).
hipError_t launch_gated_bwd(const GatedBwdParams &p, int act, bool bf16_out, hipStream_t s) {
    const Mx8GemmParams &mm = p.mm;
    const int64_t lim = (int64_t)1 << 24;          // the large tiles' row offsets are 32 bits wide
    const int64_t cus = device_cus(s), t64 = tiles_of(mm.M, mm.N, 64, 64), t128 = tiles_of(mm.M, mm.N, 128, 128);
    if (t64 <= cus) return bwd<64, 3, 2>(p, act, bf16_out, s);
    if (t64 <= 2 * cus) return bwd<64, 3, 1>(p, act, bf16_out, s);
    if (t128 <= cus) return bwd<128, 2, 2>(p, act, bf16_out, s);
    const bool large = t128 > 2 * cus && mm.K >= 2048;
    if (large && mm.K < lim && mm.N < lim) return launch_gated_bwd_big(p, act, bf16_out, s);
    return bwd<128, 2, 1>(p, act, bf16_out, s);
}

}  // namespace bbs
