// The small-tile engine of the NVFP4 x NVFP4 products, for any K the format
// allows (gfx950): TM rows of A by 128 rows of the B side a workgroup.
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
// cancelled by a zero scale.  Scales are copied as the aligned words that
// contain them and shifted into place when they are read; the shift is the same
// in every slab.  No copy leaves the operand's own bytes but for the rest of the
// words at its ends.
#pragma once

#include "gemm_nvfp4_tiles.hpp"

namespace bbs {
namespace small {

constexpr int kThreads = 256;
constexpr int kRowsB = 128;          // rows of the B side of a tile

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

// As join_groups for two column blocks of NV values each, of which group 0 receives the
// first one's sums and group 1 the second one's, in v (a: the group's shares of both).
// The same additions in the same order.
template <int G, int NV>
__device__ __forceinline__ void join_blocks(uint8_t *smem, int grp, int wave, int lane, const float (&a)[2][NV],
                                            float (&v)[NV]) {
    __syncthreads();                               // the rings are free
    // block j's shares, of the G - 1 groups that do not own it
    float *const part = reinterpret_cast<float *>(smem) + (wave * NV) * 64 + lane;
    auto at = [&](int j, int g, int i) -> float & { return part[((j * (G - 1) + (g < j ? g : g - 1)) * 4 * NV + i) * 64]; };
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (grp != j) {
#pragma unroll
            for (int i = 0; i < NV; ++i) at(j, grp, i) = a[j][i];
        }
    __syncthreads();
    if (grp == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = a[0][i] + at(0, 1, i);
    } else if (grp == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = at(1, 0, i) + a[1][i];
    }
    if (grp < 2) {
#pragma unroll
        for (int g = 2; g < G; ++g)
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] += at(grp, g, i);
    }
}

template <int TM>
struct Stage {
    uint8_t a[TM * 64];              // 64 code bytes a row and slab, swizzled as big::Stage
    uint8_t b[kRowsB * 64];
    uint32_t sc[3][TM + kRowsB];     // the words that hold a row's 8 scale bytes (A rows, then B rows)
};

// The B side of a tile tells the codes and the scales of the operand of which
// tile row r holds a row (the same for each aligned 32 rows; all operands have
// p.b's scale layout), how many operands there are (kMats) and how many columns of each the tile covers (kCols), which of them row r is (column)
// and where column c of the first one lies (row; the second one's is 32 further).
//
// The product's blocks give lane half h rows 8 q + 4 h + e of each 32, which hold
// columns 16 h + 4 q + e of the block: a lane's outputs are then 16 consecutive
// columns.
__device__ __forceinline__ int column32(int r) { return 16 * (r >> 2 & 1) + 4 * (r >> 3 & 3) + (r & 3); }
__device__ __forceinline__ int row32(int c) { return 8 * (c >> 2 & 3) + 4 * (c >> 4 & 1) + (c & 3); }

// One operand, b.
struct PlainSide {
    static constexpr int kMats = 1, kCols = kRowsB;
    template <typename Params>
    static __device__ __forceinline__ const uint8_t *codes(const Params &p, int) { return p.b.codes; }
    template <typename Params>
    static __device__ __forceinline__ const uint8_t *scales(const Params &p, int) { return p.b.scales; }
    static __device__ __forceinline__ int column(int r) { return (r & ~31) + column32(r); }
    static __device__ __forceinline__ int row(int c) { return (c & ~31) + row32(c); }
};

// Two operands of one shape: 32 rows of the gate matrix b and the same 32 of the
// up matrix u in turn, so that a lane receives both products of an output.
struct GatedSide {
    static constexpr int kMats = 2, kCols = kRowsB / 2;
    template <typename Params>
    static __device__ __forceinline__ const uint8_t *codes(const Params &p, int r) {
        return r >> 5 & 1 ? p.u.codes : p.b.codes;
    }
    template <typename Params>
    static __device__ __forceinline__ const uint8_t *scales(const Params &p, int r) {
        return r >> 5 & 1 ? p.u.scales : p.b.scales;
    }
    static __device__ __forceinline__ int column(int r) { return 32 * (r >> 6) + column32(r); }
    static __device__ __forceinline__ int row(int c) { return 64 * (c >> 5) + row32(c); }
};

// The workgroup's tile of the product of p.a and the side, p.M x p.N over p.K
// (blockDim.x = 256 G, LDS of G NS stages at smem).
// finish(p, acc, m, n0, wn, lane) receives the FP32 sums, without decode scales: in
// acc[i][j] a lane holds row m + 32 i + lane % 32 and, of the tile's 32-column
// block 2 wn + j of B's rows, 16 consecutive columns (column above).  With one operand
// it is finish(p, v, m, n, lane) for a column block at a time: in v[i] a lane holds row
// m + 32 i + lane % 32 and 16 columns from n + 16 (lane / 32) on.  Two groups then finish a
// block each.
template <int TM, int NS, int G, typename Side, typename Params, typename Finish>
__device__ __forceinline__ void run_tile(uint8_t *smem, const Params &p, Finish finish) {
    constexpr int RA = TM / 64;                    // 32-row blocks of a wave
    constexpr int SG = TM > 128 ? 2 : 1;           // groups of 64 scale rows a wave copies
    constexpr int kIssued = RA + 2 + 3 * SG;       // copies one wave issues a slab
    constexpr int AHEAD = NS - 1;                  // slabs in flight beyond the one consumed
    // four waves a group; group g of G takes slabs g, g + G, ... in its own ring
    const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    Stage<TM> *const st = reinterpret_cast<Stage<TM> *>(smem) + grp * NS;
    const int t = threadIdx.x & 255, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    int64_t m0, n0;
    tile_of((uint32_t)((p.M + TM - 1) / TM), (uint32_t)((p.N + Side::kCols - 1) / Side::kCols), m0, n0);
    m0 *= TM;
    n0 *= Side::kCols;
    const int64_t kb = p.K / 2, ks = p.K / 16;
    const int64_t nslab = (p.K + 127) / 128;
    const int tail = (int)(p.K % 128);             // K values of a partial last slab, 0: none

    // copy sources (rows past the end are clamped: they feed nothing that is written)
    // as 32-bit offsets (K < 2^25) from the tile's first row, which need no
    // address arithmetic a copy; a wave copies rows of one weight matrix
    uint32_t aoff[RA], boff[2];
    const uint8_t *const abase = p.a.codes + m0 * kb, *const aend = p.a.codes + p.a.rows * kb - 16;
    const uint8_t *const wcodes = Side::codes(p, wave * 32);
    const uint8_t *const bbase = wcodes + n0 * kb, *const bend = wcodes + p.N * kb - 16;
    const int pos = big::swz(lane >> 2, lane & 3);
#pragma unroll
    for (int q = 0; q < RA; ++q)
        aoff[q] = (uint32_t)(min((int64_t)((wave * RA + q) * 16 + (lane >> 2)), p.M - 1 - m0) * kb) + 16 * pos;
#pragma unroll
    for (int q = 0; q < 2; ++q)
        boff[q] = (uint32_t)(min((int64_t)Side::column((wave * 2 + q) * 16 + (lane >> 2)), p.N - 1 - n0) * kb) + 16 * pos;
    // scales: the words of a row's bytes, 64 rows a copy (the waves past the
    // last row repeat the last 64)
    auto scale_base = [&](int r) { return r < TM ? p.a.scales : Side::scales(p, r - TM); };
    auto scale_row = [&](int r) -> const uint8_t * {
        const int64_t row = r < TM ? min(m0 + r, p.M - 1) : min(n0 + Side::column(r - TM), p.N - 1);
        return scale_base(r) + ((r < TM ? p.a.tile2d : p.b.tile2d) ? row / 16 : row) * ks;
    };
    int sgroup[SG];
    const uint8_t *ssrc[SG], *slast[SG];
#pragma unroll
    for (int k = 0; k < SG; ++k) {
        sgroup[k] = min(wave * SG + k, (TM + kRowsB) / 64 - 1) * 64;
        const int r = sgroup[k] + lane;
        const int64_t rows = r < TM ? p.a.rows : p.N;
        ssrc[k] = word_of(scale_row(r));
        slast[k] = word_of(scale_base(r) + ((r < TM ? p.a.tile2d : p.b.tile2d) ? rows / 16 : rows) * ks - 1);
    }
    // the last slab's copies are held inside the operands
    auto issue = [&](int64_t s, int stage) {
        Stage<TM> &d = st[stage];
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
        Stage<TM> &d = st[rd];
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
            const int64_t r = t == 0 ? p.a.rows - 1 - m0 : Side::row((int)min(col, (int64_t)Side::kCols)) + 32 * (t - 1);
            if (last && (t == 0 ? r < TM : t <= Side::kMats && col < Side::kCols)) {
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

    if constexpr (Side::kMats == 2) {
        join_groups<G>(smem, grp, wave, lane, reinterpret_cast<float(&)[RA * 32]>(acc));
        if (grp) return;
        finish(p, acc, m0 + wm * (TM / 2), n0, wn, lane);
    } else {
        f32x16 v[2][RA];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < RA; ++i) v[j][i] = acc[i][j];
        if constexpr (G == 1) {
#pragma unroll
            for (int j = 0; j < 2; ++j) finish(p, v[j], m0 + wm * (TM / 2), n0 + wn * 64 + j * 32, lane);
        } else {
            f32x16 o[RA];
            join_blocks<G>(smem, grp, wave, lane, reinterpret_cast<const float(&)[2][RA * 16]>(v),
                           reinterpret_cast<float(&)[RA * 16]>(o));
            if (grp < 2) finish(p, o, m0 + wm * (TM / 2), n0 + wn * 64 + grp * 32, lane);
        }
    }
}

// Launch with dynamic LDS; the kernel's limit is raised once per kernel.
template <auto Kernel, typename Params>
static hipError_t launch(int64_t tiles, int threads, size_t shm, const Params &p, hipStream_t s) {
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

static int64_t tiles_of(int64_t M, int64_t N, int tm, int tn) { return ((M + tm - 1) / tm) * ((N + tn - 1) / tn); }

}  // namespace small
}  // namespace bbs
