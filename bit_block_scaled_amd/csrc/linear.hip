// A linear layer's NVFP4 product with bias, activation and residual, small-tile
// kernel for any K the format allows (gfx950), the choice between it and the
// large-tile kernel, and the backward pass of the bias and the activation.
//
//   forward   z = A W^T + b (NVFP4 x NVFP4), c = act(z) + r, optionally the MXFP8
//             checkpoint of z
//   backward  dz = dy * act'(z), db = sum over the rows of dz, with z read back
//             from the checkpoint
#include "gemm_nvfp4_small.hpp"
#include "linear.hpp"

namespace bbs {

namespace {

using small::kThreads;
using small::launch, small::run_tile, small::tiles_of;
using small::PlainSide;

// ---------------------------------------------------------------------------
// Forward: TM rows by 128 columns.  The epilogue of a 32 x 32 block loads all it
// needs before its first store: loads and stores share one counter, so a load behind a
// store would wait for it.  Where groups of waves split K, two of them finish a column
// block each.  Measured with GELU, bias and residual, replayed from a graph: 528 x 2736 x
// 1552, FP32, 16.6 us (loads between the stores, one group finishing: 19.4), 256 x 4096
// x 1536 14.8 (16.9), 2048 x 4096 x 1552, BF16, 41.5 (46.8).  64 x 512 x 512 takes 8.5: launch,
// first copies, join and epilogue; beyond that a slab costs 0.7 us on a CU, 45% of it
// the expansion.
// ---------------------------------------------------------------------------
// Sixteen consecutive values of a bias or a residual, as loaded.
struct Raw16 {
    uint4 v[4];
};

__device__ __forceinline__ void load16(Raw16 &o, const void *p, int bf16, int64_t at) {
    const uint4 *const from = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) + at * (bf16 ? 2 : 4));
    o.v[0] = from[0];
    o.v[1] = from[1];
    if (!bf16) {
        o.v[2] = from[2];
        o.v[3] = from[3];
    }
}

__device__ __forceinline__ void add16(f32x16 &v, const Raw16 &o, int bf16) {
    if (bf16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t w = big::word(o.v[e >> 2], e & 3);
            v[2 * e] += __uint_as_float(w << 16);
            v[2 * e + 1] += __uint_as_float(w & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] += __uint_as_float(big::word(o.v[e >> 2], e & 3));
    }
}

template <int TM, int NS, int G, bool BF16_OUT>
__global__ __launch_bounds__(kThreads * G, TM == 256 ? 2 : 1) void linear_kernel(LinearParams p) {
    constexpr int RA = TM / 64;                    // 32-row blocks of a wave
    extern __shared__ __align__(16) uint8_t smem[];
    auto finish = [](const LinearParams &p, const f32x16 (&acc)[RA], int64_t mw, int64_t nb, int lane)
                      __attribute__((always_inline)) {
        const int h = lane >> 5, rl = lane & 31;
        const float sb = p.b.s_dec[0];
        const int64_t n = nb + 16 * h, nc = n < p.N ? n : 0;        // the lane's first column
        Raw16 bias, res;
        if (p.bias) load16(bias, p.bias, p.bias_bf16, nc);
#pragma unroll
        for (int i = 0; i < RA; ++i) {
            const int64_t m = mw + i * 32 + rl, mc = min(m, p.M - 1);
            const bool in = m < p.M && n < p.N;
            const float scale = p.a.s_dec[p.a.sdec_rows ? mc : 0] * sb;
            if (p.r) load16(res, p.r, BF16_OUT, mc * p.ldr + nc);
            f32x16 v = acc[i];
            scale16(v, scale);
            if (p.bias) add16(v, bias, p.bias_bf16);
            if (p.z_codes) {
                uint32_t w[4];
                const uint32_t byte = checkpoint16(v, w);
                if (in) {
                    *reinterpret_cast<uint4 *>(p.z_codes + m * p.N + n) = make_uint4(w[0], w[1], w[2], w[3]);
                    if (h == 0) p.z_scales[m * (p.N / 32) + n / 32] = (uint8_t)byte;
                }
            }
            if (!in) continue;
            act_all<BF16_OUT, 16>(v, p.act);
            if (p.r) add16(v, res, BF16_OUT);
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
                const float y0[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                const float y1[4] = {v[4 * q + 4], v[4 * q + 5], v[4 * q + 6], v[4 * q + 7]};
                store8<BF16_OUT>(p.c, m * p.ldc + n + 4 * q, y0, y1);
            }
        }
    };
    run_tile<TM, NS, G, PlainSide>(smem, p, finish);
}

// ---------------------------------------------------------------------------
// Backward: a workgroup takes 128 columns of a range of rows, sixteen lanes to
// a row, eight columns a lane; column sums stay in registers over the rows and
// are joined in LDS.  The sums of the ranges go to memory and a second kernel
// adds them in order, so a call's bits do not depend on the order in which
// workgroups run.
// ---------------------------------------------------------------------------
constexpr int kBwdCols = 128, kBwdRows = 16;       // rows of one step of a workgroup
constexpr int kBwdDeep = 4;                        // steps whose loads are in flight together

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
}

template <bool BF16>
__device__ __forceinline__ void store_db(void *db, int64_t n, float v) {
    if (BF16) static_cast<uint16_t *>(db)[n] = (uint16_t)pk_bf16(v, v);
    else static_cast<float *>(db)[n] = v;
}

// DEEP steps from row m on; rows past `end` add nothing.
template <int ACT, int DEEP>
__device__ __forceinline__ void bwd_rows(const BiasActBwdParams &p, int64_t m, int64_t end, int64_t n,
                                         float (&sum)[8]) {
    uint4 dy[DEEP];
    uint2 z[DEEP];
    uint32_t zs[DEEP];
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
        const int64_t r = min(m + d * kBwdRows, end - 1);
        dy[d] = *reinterpret_cast<const uint4 *>(p.dy + r * p.ldy + n);
        if (ACT != kActNone) {
            z[d] = *reinterpret_cast<const uint2 *>(p.z_codes + r * p.N + n);
            zs[d] = p.z_scales[r * (p.N / 32) + n / 32];
        }
    }
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
        const int64_t r = m + d * kBwdRows;
        float v[8];
        unpack8(dy[d], v);
        if (ACT != kActNone) {
            float zv[8];
            decode4(z[d].x, zs[d], reinterpret_cast<float(&)[4]>(zv[0]));
            decode4(z[d].y, zs[d], reinterpret_cast<float(&)[4]>(zv[4]));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float slope;
                gate_act_grad<ACT == kActNone ? kActSilu : ACT, true>(zv[e], slope);
                v[e] = v[e] * slope;
            }
        }
        if (r >= end) break;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += v[e];
        if (p.dz)
            *reinterpret_cast<uint4 *>(p.dz + r * p.ldz + n) =
                make_uint4(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7]));
    }
}

template <int ACT>
__global__ __launch_bounds__(256) void bias_act_bwd_kernel(BiasActBwdParams p, int64_t rows, int parts) {
    __shared__ float part[kBwdRows][kBwdCols];
    const int t = threadIdx.x, rl = t >> 4, c = (t & 15) * 8;
    const int64_t n = (int64_t)blockIdx.x * kBwdCols + c;
    const int64_t m0 = (int64_t)blockIdx.y * rows, end = min(m0 + rows, p.M);
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n < p.N)
        for (int64_t m = m0 + rl; m < end; m += kBwdRows * kBwdDeep) bwd_rows<ACT, kBwdDeep>(p, m, end, n, sum);
    if (!p.db) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) part[rl][c + e] = sum[e];
    __syncthreads();
    const int64_t nc = (int64_t)blockIdx.x * kBwdCols + t;
    if (t < kBwdCols && nc < p.N) {
        float v = part[0][t];
#pragma unroll
        for (int r = 1; r < kBwdRows; ++r) v += part[r][t];
        if (parts > 1) p.part[(int64_t)blockIdx.y * p.N + nc] = v;
        else if (p.db_bf16) store_db<true>(p.db, nc, v);
        else store_db<false>(p.db, nc, v);
    }
}

// 64 columns a workgroup; wave w adds every fourth range from w on, with its loads in
// flight together.
template <bool BF16>
__global__ __launch_bounds__(256) void bias_sum_kernel(const float *part, int64_t N, int parts, void *db) {
    __shared__ float sums[4][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t n = (int64_t)blockIdx.x * 64 + lane;
    const float *const from = part + min(n, N - 1);
    float v = 0.0f;
    for (int i = w; i < parts; i += 32) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = from[min(i + 4 * j, parts - 1) * N];
#pragma unroll
        for (int j = 0; j < 8; ++j) v += i + 4 * j < parts ? x[j] : 0.0f;
    }
    sums[w][lane] = v;
    __syncthreads();
    if (w == 0 && n < N) store_db<BF16>(db, n, sums[0][lane] + sums[1][lane] + sums[2][lane] + sums[3][lane]);
}

template <int TM, int NS, int G>
hipError_t fwd(const LinearParams &p, bool bf16_out, hipStream_t s) {
    const int64_t tiles = tiles_of(p.M, p.N, TM, PlainSide::kCols);
    constexpr size_t shm = G * NS * sizeof(small::Stage<TM>);
    return bf16_out ? launch<linear_kernel<TM, NS, G, true>>(tiles, kThreads * G, shm, p, s)
                    : launch<linear_kernel<TM, NS, G, false>>(tiles, kThreads * G, shm, p, s);
}

}  // namespace

hipError_t launch_linear(const LinearParams &p, bool bf16_out, hipStream_t s) {
    auto al8 = [](const void *q) { return reinterpret_cast<uintptr_t>(q) % 8 == 0; };
    const bool large = p.K % 128 == 0 && al8(p.a.scales) && al8(p.b.scales);
    const int64_t cus = device_cus(s);
    if (tiles_of(p.M, p.N, 64, PlainSide::kCols) <= cus) return fwd<64, 2, 4>(p, bf16_out, s);
    if (tiles_of(p.M, p.N, 128, PlainSide::kCols) <= cus) return fwd<128, 3, 2>(p, bf16_out, s);
    if (large) return launch_linear_big(p, bf16_out, s);
    return fwd<256, 2, 1>(p, bf16_out, s);
}

hipError_t launch_bias_act_bwd(const BiasActBwdParams &p, hipStream_t s) {
    const int64_t cols = (p.N + kBwdCols - 1) / kBwdCols;
    const int64_t most = (p.M + kBwdRows - 1) / kBwdRows;
    int64_t parts = (8 * device_cus(s) + cols - 1) / cols;
    parts = parts > kBiasParts ? kBiasParts : parts;
    parts = parts > most ? most : parts;
    const int64_t rows = ((p.M + parts - 1) / parts + kBwdRows - 1) / kBwdRows * kBwdRows;
    parts = (p.M + rows - 1) / rows;
    const dim3 grid((unsigned)cols, (unsigned)parts);
    if (p.act == kActSilu) hipLaunchKernelGGL((bias_act_bwd_kernel<kActSilu>), grid, dim3(256), 0, s, p, rows, (int)parts);
    else if (p.act == kActGelu) hipLaunchKernelGGL((bias_act_bwd_kernel<kActGelu>), grid, dim3(256), 0, s, p, rows, (int)parts);
    else hipLaunchKernelGGL((bias_act_bwd_kernel<kActNone>), grid, dim3(256), 0, s, p, rows, (int)parts);
    if (p.db && parts > 1) {
        const dim3 g2((unsigned)((p.N + 63) / 64));
        if (p.db_bf16) hipLaunchKernelGGL(bias_sum_kernel<true>, g2, dim3(256), 0, s, p.part, p.N, (int)parts, p.db);
        else hipLaunchKernelGGL(bias_sum_kernel<false>, g2, dim3(256), 0, s, p.part, p.N, (int)parts, p.db);
    }
    return hipGetLastError();
}

}  // namespace bbs
