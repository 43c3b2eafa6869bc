// Gated feed-forward operators, kernels for any K the formats allow (gfx950).
//
//   forward   g = A Wg^T, u = A Wu^T (NVFP4 x NVFP4), h = act(g) * u, and
//             optionally MXFP8 checkpoints of the FP32 g and u
//   backward  dh = dY W (MXFP8 x MXFP8), dg = dh * u * act'(g),
//             du = dh * act(g), with g and u read back from the checkpoints
//
// Both products of the forward pass share one tile: its B side interleaves
// 32-column blocks of the gate and up weights, so the lane that holds g of an
// output also holds u, and h needs no exchange.  The activation works on the
// FP32 sums and each output is rounded once.
//
// These kernels take 128-row tiles and stage through registers; the large
// tile kernels beside the plain GEMMs serve K % 128 == 0.
#include "bbs_device.hpp"
#include "gated_epilogue.hpp"

namespace bbs {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

namespace {

constexpr int kBM = 128, kBF = 64, kBK = 64, kThreads = 256;
constexpr int kStride = kBK / 2 + 4;           // padded row of packed codes

struct FwdSmem {
    uint8_t a[kBM * kStride];
    uint8_t b[2 * kBF * kStride];
    uint8_t as[kBM * 4], bs[2 * kBF * 4];
};

// Eight E2M1 codes times one E4M3 scale in FP16 (exact: at most 6
// significant bits in [2^-10, 2688]).
__device__ __forceinline__ f16x8 expand8(uint32_t w, uint32_t scale_byte) {
    const f16x2 s2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scale_byte, 1.0f, false);
    const f16x2 s = {s2[0], s2[0]};
    const f16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s;
    const f16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s;
    const f16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s;
    const f16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s;
    return f16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// The tile's B row r holds weight row n0 + 32 (r / 64) + r % 32, of the gate
// matrix where r / 32 is even and of the up matrix where it is odd.
__device__ __forceinline__ int64_t b_column(int r) { return 32 * (r >> 6) + (r & 31); }

template <int ACT, bool BF16_OUT, bool CKPT>
__global__ __launch_bounds__(kThreads) void gated_gemm_kernel(GatedParams p) {
    __shared__ FwdSmem sm;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t tm = (p.M + kBM - 1) / kBM;
    const int64_t m0 = blockIdx.x % tm * kBM, n0 = blockIdx.x / tm * kBF;
    const int64_t kb = p.K / 2, ks = p.K / 16;
    // staging: thread t copies 32 codes (16 bytes) of row t / 2 of each side
    const int row = t >> 1, half = t & 1;
    const int64_t am = m0 + row, bn = n0 + b_column(row);
    const Fp4View &W = ((row >> 5) & 1) ? p.u : p.b;
    const bool a_ok = am < p.M, b_ok = bn < p.N;
    // scales: threads 0-127 the A side's rows, the others the B side's
    const int sr = t & 127;
    const bool sb = t >= 128;
    const Fp4View &S = sb ? (((sr >> 5) & 1) ? p.u : p.b) : p.a;
    const int64_t srow = sb ? n0 + b_column(sr) : m0 + sr;
    const bool s_ok = srow < (sb ? p.N : p.M);
    const uint8_t *sp = S.scales + (S.tile2d ? srow / 16 : srow) * ks;

    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{0};

    for (int64_t k0 = 0; k0 < p.K; k0 += kBK) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int64_t k = k0 + half * 32 + q * 16;
            uint2 va = make_uint2(0, 0), vb = make_uint2(0, 0);
            if (a_ok && k < p.K) va = *reinterpret_cast<const uint2 *>(p.a.codes + am * kb + k / 2);
            if (b_ok && k < p.K) vb = *reinterpret_cast<const uint2 *>(W.codes + bn * kb + k / 2);
            uint32_t *da = reinterpret_cast<uint32_t *>(sm.a + row * kStride + half * 16 + q * 8);
            uint32_t *db = reinterpret_cast<uint32_t *>(sm.b + row * kStride + half * 16 + q * 8);
            da[0] = va.x;
            da[1] = va.y;
            db[0] = vb.x;
            db[1] = vb.y;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t k = k0 / 16 + j;
            (sb ? sm.bs : sm.as)[sr * 4 + j] = (s_ok && k < ks) ? sp[k] : (uint8_t)0;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int h = lane >> 5, rl = lane & 31;
            f16x8 af[2], bf[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = wm * 64 + i * 32 + rl;
                af[i] = expand8(*reinterpret_cast<const uint32_t *>(sm.a + r * kStride + kk * 8 + h * 4),
                                sm.as[r * 4 + kk]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = wn * 64 + j * 32 + rl;
                bf[j] = expand8(*reinterpret_cast<const uint32_t *>(sm.b + r * kStride + kk * 8 + h * 4),
                                sm.bs[r * 4 + kk]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bf[j], af[i], acc[i][j], 0, 0, 0);
        }
        __syncthreads();
    }

    const float sg = p.b.s_dec[0], su = p.u.s_dec[0];
    const int64_t n = n0 + wn * 32 + 4 * (lane >> 5);      // the lane's first column
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t m = m0 + wm * 64 + i * 32 + (lane & 31);
        const int64_t ms = m < p.M ? m : p.M - 1;
        const float sa = p.a.s_dec[p.a.sdec_rows ? ms : 0];
        f32x16 g = acc[i][0], u = acc[i][1];
        scale16(g, sa * sg);
        scale16(u, sa * su);
        if (CKPT) {
            uint32_t w[4];
            const uint32_t bg = checkpoint16(g, w);
            if (m < p.M) store_checkpoint(w, bg, p.g_codes, p.g_scales, p.N, m, n, lane);
            const uint32_t bu = checkpoint16(u, w);
            if (m < p.M) store_checkpoint(w, bu, p.u_codes, p.u_scales, p.N, m, n, lane);
        }
        if (m >= p.M) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (n + 8 * q >= p.N) continue;
            store4<BF16_OUT>(p.h, m * p.ldh + n + 8 * q, gate_act<ACT, BF16_OUT>(g[4 * q]) * u[4 * q],
                             gate_act<ACT, BF16_OUT>(g[4 * q + 1]) * u[4 * q + 1],
                             gate_act<ACT, BF16_OUT>(g[4 * q + 2]) * u[4 * q + 2],
                             gate_act<ACT, BF16_OUT>(g[4 * q + 3]) * u[4 * q + 3]);
        }
    }
}

// Backward, 128 x 128 tiles with a K slab of 128 (one MFMA deep); operand
// layout of the scaled MFMA as in the plain MXFP8 GEMM: lane group g feeds
// bytes [16g, 16g + 16) and [64 + 16g, 64 + 16g + 16) of its row and the
// scale of the slab's 32-block g.
constexpr int kMxBK = 128, kMxStride = kMxBK + 16;

struct BwdSmem {
    uint8_t a[128 * kMxStride];
    uint8_t b[128 * kMxStride];
    uint8_t as[128 * 4], bs[128 * 4];
};

template <int ACT, bool BF16_OUT>
__global__ __launch_bounds__(kThreads) void gated_bwd_kernel(GatedBwdParams p) {
    __shared__ BwdSmem sm;
    const Mx8GemmParams &mm = p.mm;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t tm = (mm.M + 127) / 128;
    const int64_t m0 = blockIdx.x % tm * 128, n0 = blockIdx.x / tm * 128;
    const int64_t nkb = mm.K / 32;

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0};

    for (int64_t k0 = 0; k0 < mm.K; k0 += kMxBK) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int idx = q * kThreads + t;
            const int row = idx >> 3, seg = idx & 7;
            const int64_t k = k0 + seg * 16;
            uint4 va = make_uint4(0, 0, 0, 0), vb = make_uint4(0, 0, 0, 0);
            if (m0 + row < mm.M && k < mm.K)
                va = *reinterpret_cast<const uint4 *>(mm.a_codes + (m0 + row) * mm.K + k);
            if (n0 + row < mm.N && k < mm.K)
                vb = *reinterpret_cast<const uint4 *>(mm.b_codes + (n0 + row) * mm.K + k);
            *reinterpret_cast<uint4 *>(sm.a + row * kMxStride + seg * 16) = va;
            *reinterpret_cast<uint4 *>(sm.b + row * kMxStride + seg * 16) = vb;
        }
        {
            const int row = t & 127;
            const bool isb = t >= 128;
            const int64_t gr = (isb ? n0 : m0) + row;
            const uint8_t *sc = isb ? mm.b_scales : mm.a_scales;
            uint8_t *dst = isb ? sm.bs : sm.as;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t kb = k0 / 32 + j;
                dst[row * 4 + j] = (gr < (isb ? mm.N : mm.M) && kb < nkb) ? sc[gr * nkb + kb] : (uint8_t)0;
            }
        }
        __syncthreads();
        const int kg = lane >> 4;
        i32x8 af[4], bf[4];
        int as_[4], bs_[4];
        auto fragment = [&](const uint8_t *row) {
            const uint4 x0 = *reinterpret_cast<const uint4 *>(row + 16 * kg);
            const uint4 x1 = *reinterpret_cast<const uint4 *>(row + 64 + 16 * kg);
            return i32x8{(int)x0.x, (int)x0.y, (int)x0.z, (int)x0.w,
                         (int)x1.x, (int)x1.y, (int)x1.z, (int)x1.w};
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ra = wm * 64 + i * 16 + (lane & 15), rb = wn * 64 + i * 16 + (lane & 15);
            af[i] = fragment(sm.a + ra * kMxStride);
            bf[i] = fragment(sm.b + rb * kMxStride);
            as_[i] = sm.as[ra * 4 + kg];
            bs_[i] = sm.bs[rb * 4 + kg];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    bf[j], af[i], acc[i][j], 0, 0, 0, bs_[j], 0, as_[i]);
        __syncthreads();
    }

    // the B fragment goes first, so lane l holds row l % 16 and four
    // consecutive columns from 4 (l / 16) of every block
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + wm * 64 + i * 16 + (lane & 15);
        if (m >= mm.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + wn * 64 + j * 16 + 4 * (lane >> 4);
            if (n >= mm.N) continue;
            const int64_t at = m * mm.N + n, bl = m * (mm.N / 32) + n / 32;
            gated_bwd4<ACT, BF16_OUT>(p, m, n, acc[i][j], *reinterpret_cast<const uint32_t *>(p.g_codes + at),
                                      p.g_scales[bl], *reinterpret_cast<const uint32_t *>(p.u_codes + at),
                                      p.u_scales[bl]);
        }
    }
}

template <int ACT, bool BF16_OUT>
hipError_t fwd(const GatedParams &p, hipStream_t s) {
    const int64_t tiles = ((p.M + kBM - 1) / kBM) * ((p.N + kBF - 1) / kBF);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)tiles);
    if (p.g_codes)
        hipLaunchKernelGGL((gated_gemm_kernel<ACT, BF16_OUT, true>), grid, dim3(kThreads), 0, s, p);
    else
        hipLaunchKernelGGL((gated_gemm_kernel<ACT, BF16_OUT, false>), grid, dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

template <int ACT, bool BF16_OUT>
hipError_t bwd(const GatedBwdParams &p, hipStream_t s) {
    const int64_t tiles = ((p.mm.M + 127) / 128) * ((p.mm.N + 127) / 128);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)tiles);
    hipLaunchKernelGGL((gated_bwd_kernel<ACT, BF16_OUT>), grid, dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_gemm(const GatedParams &p, int act, bool bf16_out, hipStream_t s) {
    auto al8 = [](const void *q) { return reinterpret_cast<uintptr_t>(q) % 8 == 0; };
    if (p.K % 128 == 0 && al8(p.a.scales) && al8(p.b.scales) && al8(p.u.scales))
        return launch_gated_gemm_big(p, act, bf16_out, s);
    if (act == kActGelu) return bf16_out ? fwd<kActGelu, true>(p, s) : fwd<kActGelu, false>(p, s);
    return bf16_out ? fwd<kActSilu, true>(p, s) : fwd<kActSilu, false>(p, s);
}

hipError_t launch_gated_bwd(const GatedBwdParams &p, int act, bool bf16_out, hipStream_t s) {
    auto al4 = [](const void *q) { return reinterpret_cast<uintptr_t>(q) % 4 == 0; };
    // (the large tiles' row offsets are 32 bits wide)
    const int64_t lim = (int64_t)1 << 24;
    if (p.mm.K % 128 == 0 && p.mm.K < lim && p.mm.N < lim && al4(p.mm.a_scales) && al4(p.mm.b_scales))
        return launch_gated_bwd_big(p, act, bf16_out, s);
    if (act == kActGelu) return bf16_out ? bwd<kActGelu, true>(p, s) : bwd<kActGelu, false>(p, s);
    return bf16_out ? bwd<kActSilu, true>(p, s) : bwd<kActSilu, false>(p, s);
}

}  // namespace bbs
