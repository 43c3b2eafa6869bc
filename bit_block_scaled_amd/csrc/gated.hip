// Gated feed-forward operators, small-tile kernels for any K the formats
// allow (gfx950), and the choice between them and the large-tile kernels.
//
//   forward   g = A Wg^T, u = A Wu^T (NVFP4 x NVFP4), h = act(g) * u, and
//             optionally MXFP8 checkpoints of the FP32 g and u
//   backward  dh = dY W (MXFP8 x MXFP8), dg = dh * u * act'(g),
//             du = dh * act(g), with g and u read back from the checkpoints
//
// A workgroup of four waves (2 x 2) walks K in slabs of 128 through a ring of
// LDS stages filled by asynchronous copies, as the large-tile kernels do, but
// with tiles small enough for two or more workgroups a CU: one's arithmetic
// covers another's waits, and a problem of a few hundred rows still reaches
// every CU.
//
// K's last slab may be partial and rows may start at any multiple of 8 bytes
// (codes) or at any byte (scales).  Codes are copied in 16-byte pieces from
// where they are; what a piece reads past K belongs to the next row and is
// cancelled by a zero scale, or overwritten by zeros where a code could be NaN.
// Scales are copied as the aligned words that contain them and shifted into
// place when they are read; the shift is the same in every slab.  No copy
// leaves the operand's own bytes but for the rest of the words at its ends.
#include "gemm_nvfp4_tiles.hpp"
#include "gated_epilogue.hpp"

namespace bbs {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

namespace {

constexpr int kThreads = 256;

// The aligned word at or before p, and the last one an array [p, p + bytes) touches.
__device__ __forceinline__ const uint8_t *word_of(const uint8_t *p) {
    return reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)3);
}
__device__ __forceinline__ const uint8_t *lesser(const uint8_t *a, const uint8_t *b) { return a < b ? a : b; }

// copy_lds16 from base + off, base the same for the wave.  A scalar register
// that a vector instruction wrote may be read by a memory instruction five
// wait states later, which the compiler does not see to in front of an asm.
__device__ __forceinline__ void copy_at(const uint8_t *base, uint32_t off, const void *lds) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    const uint64_t sb = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) << 32 |
                        (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b);
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(sb), "{m0}"(lds_addr(lds))
                 : "memory");
}

// An offset held to at most `last`, which is not negative.
__device__ __forceinline__ uint32_t held(uint32_t off, int64_t last) { return (uint32_t)min((int64_t)off, last); }

// Tile of workgroup b: workgroup b runs on XCD b % 8, so each XCD is given a
// contiguous range of tile ids, and ids walk 8 row tiles down before moving
// along the columns, which keeps operand panels in one XCD's L2.  In 32 bits
// (the launch holds the tiles below 2^24), as 64-bit divisions are long
// (64 x 512 x 512: 8.3 us against 8.6).
__device__ __forceinline__ void tile_of(uint32_t tm, uint32_t tn, int64_t &mt, int64_t &nt) {
    const uint32_t total = tm * tn, x = blockIdx.x % 8, share = total / 8, extra = total % 8;
    const uint32_t id = x * share + (x < extra ? x : extra) + blockIdx.x / 8;
    const uint32_t g = id / (8 * tn), in = id - g * (8 * tn);
    const uint32_t gm = tm - g * 8 < 8 ? tm - g * 8 : 8;
    mt = g * 8 + in % gm;
    nt = in / gm;
}

// Adds the sums of groups 1 .. G - 1 to group 0's, in that order.
template <int G, int NV>
__device__ __forceinline__ void join_groups(uint8_t *smem, int grp, int wave, int lane, float (&v)[NV]) {
    if (G == 1) return;
    __syncthreads();                               // the rings are free
    float *const part = reinterpret_cast<float *>(smem) + (wave * NV) * 64 + lane;
    if (grp) {
#pragma unroll
        for (int i = 0; i < NV; ++i) part[((grp - 1) * 4 * NV + i) * 64] = v[i];
    }
    __syncthreads();
    if (!grp) {
#pragma unroll
        for (int g = 1; g < G; ++g)
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] += part[((g - 1) * 4 * NV + i) * 64];
    }
}

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
constexpr int kBF = 64;

template <int TM>
struct FwdStage {
    uint8_t a[TM * 64];              // 64 code bytes a row and slab, swizzled as big::Stage
    uint8_t b[2 * kBF * 64];
    uint32_t sc[3][TM + 2 * kBF];    // the words that hold a row's 8 scale bytes (A rows, then B rows)
};

// The tile's B rows alternate 32 rows of the gate matrix and the same 32 of the
// up matrix.  The product's blocks give lane half h rows 8 q + 4 h + e of each
// 32, which hold columns 16 h + 4 q + e of the block: a lane's outputs are then
// 16 consecutive columns, and its half of a checkpoint's block one store.
__device__ __forceinline__ int b_column(int r) {
    return 32 * (r >> 6) + 16 * (r >> 2 & 1) + 4 * (r >> 3 & 3) + (r & 3);
}
// Row of the gate matrix' column c (the up matrix' row is 32 further).
__device__ __forceinline__ int b_row(int c) {
    return 64 * (c >> 5) + 8 * (c >> 2 & 3) + 4 * (c >> 4 & 1) + (c & 3);
}

template <int TM, int NS, int G, int ACT, bool BF16_OUT>
__global__ __launch_bounds__(kThreads * G, TM == 256 ? 2 : 1) void gated_gemm_kernel(GatedParams p) {
    constexpr int RA = TM / 64;                    // 32-row blocks of a wave
    constexpr int SG = TM > 128 ? 2 : 1;           // groups of 64 scale rows a wave copies
    constexpr int kIssued = RA + 2 + 3 * SG;       // copies one wave issues a slab
    constexpr int AHEAD = NS - 1;                  // slabs in flight beyond the one consumed
    extern __shared__ __align__(16) uint8_t smem[];
    // four waves a group; group g of G takes slabs g, g + G, ... in its own ring
    const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    FwdStage<TM> *const st = reinterpret_cast<FwdStage<TM> *>(smem) + grp * NS;
    const int t = threadIdx.x & 255, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    int64_t m0, n0;
    tile_of((uint32_t)((p.M + TM - 1) / TM), (uint32_t)((p.N + kBF - 1) / kBF), m0, n0);
    m0 *= TM;
    n0 *= kBF;
    const int64_t kb = p.K / 2, ks = p.K / 16;
    const int64_t nslab = (p.K + 127) / 128;
    const int tail = (int)(p.K % 128);             // K values of a partial last slab, 0: none

    // copy sources (rows past the end are clamped: they feed nothing that is written)
    // as 32-bit offsets (K < 2^25) from the tile's first row, which need no
    // address arithmetic a copy; a wave copies rows of one weight matrix
    uint32_t aoff[RA], boff[2];
    const uint8_t *const abase = p.a.codes + m0 * kb, *const aend = p.a.codes + p.a.rows * kb - 16;
    const uint8_t *const wcodes = (wave & 1 ? p.u : p.b).codes;
    const uint8_t *const bbase = wcodes + n0 * kb, *const bend = wcodes + p.N * kb - 16;
    const int pos = big::swz(lane >> 2, lane & 3);
#pragma unroll
    for (int q = 0; q < RA; ++q)
        aoff[q] = (uint32_t)(min((int64_t)((wave * RA + q) * 16 + (lane >> 2)), p.M - 1 - m0) * kb) + 16 * pos;
#pragma unroll
    for (int q = 0; q < 2; ++q)
        boff[q] = (uint32_t)(min((int64_t)b_column((wave * 2 + q) * 16 + (lane >> 2)), p.N - 1 - n0) * kb) + 16 * pos;
    // scales: the words of a row's bytes, 64 rows a copy (the waves past the
    // last row repeat the last 64)
    auto scale_row = [&](int r) -> const uint8_t * {
        if (r < TM) {
            const int64_t m = min(m0 + r, p.M - 1);
            return p.a.scales + (p.a.tile2d ? m / 16 : m) * ks;
        }
        const Fp4View &W = (((r - TM) >> 5) & 1) ? p.u : p.b;
        const int64_t n = min(n0 + b_column(r - TM), p.N - 1);
        return W.scales + (W.tile2d ? n / 16 : n) * ks;
    };
    int sgroup[SG];
    const uint8_t *ssrc[SG], *slast[SG];
#pragma unroll
    for (int k = 0; k < SG; ++k) {
        sgroup[k] = min(wave * SG + k, (TM + 2 * kBF) / 64 - 1) * 64;
        const int r = sgroup[k] + lane;
        const Fp4View &W = r < TM ? p.a : (((r - TM) >> 5) & 1) ? p.u : p.b;
        const int64_t rows = r < TM ? p.a.rows : p.N;
        ssrc[k] = word_of(scale_row(r));
        slast[k] = word_of(W.scales + (W.tile2d ? rows / 16 : rows) * ks - 1);
    }
    // the last slab's copies are held inside the operands
    auto issue = [&](int64_t s, int stage) {
        FwdStage<TM> &d = st[stage];
        const int64_t at = s * 64;
        if (s != nslab - 1) {
#pragma unroll
            for (int q = 0; q < RA; ++q) copy_at(abase + at, aoff[q], d.a + (wave * RA + q) * 1024);
#pragma unroll
            for (int q = 0; q < 2; ++q) copy_at(bbase + at, boff[q], d.b + (wave * 2 + q) * 1024);
#pragma unroll
            for (int k = 0; k < SG; ++k)
#pragma unroll
                for (int w = 0; w < 3; ++w) copy_lds4(ssrc[k] + s * 8 + 4 * w, &d.sc[w][sgroup[k]]);
        } else {
#pragma unroll
            for (int q = 0; q < RA; ++q) copy_at(abase + at, held(aoff[q], aend - (abase + at)), d.a + (wave * RA + q) * 1024);
#pragma unroll
            for (int q = 0; q < 2; ++q) copy_at(bbase + at, held(boff[q], bend - (bbase + at)), d.b + (wave * 2 + q) * 1024);
#pragma unroll
            for (int k = 0; k < SG; ++k)
#pragma unroll
                for (int w = 0; w < 3; ++w)
                    copy_lds4(lesser(ssrc[k] + s * 8 + 4 * w, slast[k]), &d.sc[w][sgroup[k]]);
        }
    };

    // the lane's fragment rows and the byte shift of their scales
    const int h = lane >> 5, rl = lane & 31;
    int sha[RA], shb[2];
#pragma unroll
    for (int i = 0; i < RA; ++i)
        sha[i] = (int)(reinterpret_cast<uintptr_t>(scale_row(wm * (TM / 2) + i * 32 + rl)) & 3);
#pragma unroll
    for (int j = 0; j < 2; ++j)
        shb[j] = (int)(reinterpret_cast<uintptr_t>(scale_row(TM + wn * 64 + j * 32 + rl)) & 3);

    f32x16 acc[RA][2];
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{0};

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
        FwdStage<TM> &d = st[rd];
        rd = rd + 1 == NS ? 0 : rd + 1;
        wr = wr + 1 == NS ? 0 : wr + 1;
        uint32_t keep[2] = {~0u, ~0u};                   // scale bytes of blocks inside K
        const bool last = tail && s == nslab - 1;
        if (last) {
            const int nb = tail / 16;
            keep[0] = nb >= 4 ? ~0u : (1u << (8 * nb)) - 1;
            keep[1] = nb <= 4 ? 0u : nb >= 8 ? ~0u : (1u << (8 * (nb - 4))) - 1;
        }
        if (tail % 32 && it == (nslab - 1) / G) {
            // an operand's very last row ends in half a piece, which was copied
            // from 8 bytes earlier: move it into place
            const int c = tail / 32;
            const int64_t col = p.N - 1 - n0;
            const int64_t r = t == 0 ? p.a.rows - 1 - m0 : b_row((int)min(col, (int64_t)kBF)) + 32 * (t - 1);
            if (last && (t == 0 ? r < TM : t <= 2 && col < kBF)) {
                uint8_t *piece = (t == 0 ? d.a : d.b) + r * 64 + 16 * big::swz((int)r, c);
                *reinterpret_cast<uint2 *>(piece) = *reinterpret_cast<const uint2 *>(piece + 8);
            }
            __syncthreads();
        }
        if (G > 1 && s >= nslab) continue;
        uint32_t sa[RA][2], sb[2][2];
        auto scales = [&](uint32_t (&o)[2], int row, int shift) {
            const uint32_t w0 = d.sc[0][row], w1 = d.sc[1][row], w2 = d.sc[2][row];
            o[0] = __builtin_amdgcn_alignbyte(w1, w0, shift) & keep[0];
            o[1] = __builtin_amdgcn_alignbyte(w2, w1, shift) & keep[1];
        };
#pragma unroll
        for (int i = 0; i < RA; ++i) scales(sa[i], wm * (TM / 2) + i * 32 + rl, sha[i]);
#pragma unroll
        for (int j = 0; j < 2; ++j) scales(sb[j], TM + wn * 64 + j * 32 + rl, shb[j]);
        uint4 ca[2][RA], cb[2][2];
        f16x2 pa[2][RA], pb[2][2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int i = 0; i < RA; ++i) {
                const int r = wm * (TM / 2) + i * 32 + rl;
                ca[c][i] = *reinterpret_cast<const uint4 *>(d.a + r * 64 + 16 * big::swz(r, 2 * c + h));
                pa[c][i] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sa[i][c] >> (16 * h), 1.0f, false);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = wn * 64 + j * 32 + rl;
                cb[c][j] = *reinterpret_cast<const uint4 *>(d.b + r * 64 + 16 * big::swz(r, 2 * c + h));
                pb[c][j] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sb[j][c] >> (16 * h), 1.0f, false);
            }
        }
        // eight MFMA steps; the operands of step k + 1 are expanded between the
        // MFMAs of step k
        f16x8 af[2][RA], bf[2][2];
        auto expand = [&](int k) __attribute__((always_inline)) {
            const int c = k >> 2, w = k & 3;
#pragma unroll
            for (int i = 0; i < RA; ++i) af[k & 1][i] = big::expand8_f16(big::word(ca[c][i], w), pa[c][i][w >> 1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) bf[k & 1][j] = big::expand8_f16(big::word(cb[c][j], w), pb[c][j][w >> 1]);
        };
        expand(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k < 7) expand(k + 1);
#pragma unroll
            for (int i = 0; i < RA; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bf[k & 1][j], af[k & 1][i], acc[i][j], 0, 0, 0);
#pragma unroll
            for (int m = 0; m < 2 * RA; ++m) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, (RA + 2) * 8 / (2 * RA), 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    join_groups<G>(smem, grp, wave, lane, reinterpret_cast<float(&)[RA * 32]>(acc));
    if (grp) return;
    const float sg = p.b.s_dec[0], su = p.u.s_dec[0];
    const int64_t n = n0 + wn * 32 + 16 * h;               // the lane's first column
#pragma unroll
    for (int i = 0; i < RA; ++i) {
        const int64_t m = m0 + wm * (TM / 2) + i * 32 + rl;
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

// Launch with dynamic LDS; the kernel's limit is raised once per kernel.
template <auto Kernel, typename Params>
hipError_t launch(int64_t tiles, int threads, size_t shm, const Params &p, hipStream_t s) {
    if (tiles * threads > UINT32_MAX) return hipErrorInvalidConfiguration;    // would be cut off
    static const bool attr_set = [shm] {
        (void)hipFuncSetAttribute(reinterpret_cast<const void *>(Kernel),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, (int)shm);
        return true;
    }();
    (void)attr_set;
    hipLaunchKernelGGL(Kernel, dim3((unsigned)tiles), dim3((unsigned)threads), shm, s, p);
    return hipGetLastError();
}

int64_t tiles_of(int64_t M, int64_t N, int tm, int tn) { return ((M + tm - 1) / tm) * ((N + tn - 1) / tn); }

template <int TM, int NS, int G>
hipError_t fwd(const GatedParams &p, int act, bool bf16_out, hipStream_t s) {
    const int64_t tiles = tiles_of(p.M, p.N, TM, kBF);
    constexpr size_t shm = G * NS * sizeof(FwdStage<TM>);
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
    if (tiles_of(p.M, p.N, 64, kBF) <= cus) return fwd<64, 2, 4>(p, act, bf16_out, s);
    if (tiles_of(p.M, p.N, 128, kBF) <= cus) return fwd<128, 3, 2>(p, act, bf16_out, s);
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
