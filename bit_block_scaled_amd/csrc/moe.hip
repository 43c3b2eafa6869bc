// A whole mixture-of-experts layer for a few tokens with 4-bit weights (gfx950):
//   y[t] = r[t] + sum_j w[t, j] (act(x[t] Wg_e^T) * (x[t] Wu_e^T)) Wd_e^T,   e = ids[t, j]
// or, for plain experts, act(x[t] Wu_e^T) Wd_e^T, in two kernels.
//
// The chosen experts' weights bound the layer: each is read once, against 2 flops
// a weight and token.  The first kernel's workgroups take one expert and a few of
// its hidden rows; they find the expert's tokens themselves by looking through
// the ids (T k of them), so nothing has to be sorted first.  The second kernel's
// workgroups take a few output columns of all the chosen experts: an output's
// sum over the experts then stays in one workgroup, in a fixed order, without
// atomics.  Its waves share the steps of all experts evenly, whatever the routing.
//
// The hidden values go between the kernels as two BF16 parts (three for FP32
// outputs): h = hi + lo to 2^-16, below the output's rounding.  A part is one
// more token to the matrix instructions, which have rows to spare.
#include <algorithm>

#include "gemv_steps.hpp"
#include "moe.hpp"

namespace bbs {

namespace {

using namespace gemv;

// ---------------------------------------------------------------------------
// Routing.  A slot is a routed pair where there are fewer of these than experts
// (the first pair of an expert stands for all its pairs), else an expert.
// ---------------------------------------------------------------------------
struct MoePlan {
    int32_t *expert, *count;           // of each slot (count 0: nothing to do)
    MoeEntry *entry;                   // T a slot
    uint16_t *h;                       // parts x T k x F
};

__device__ __forceinline__ MoePlan plan_of(const MoeParams &p) {
    const int64_t pairs = p.T * p.k, slots = pairs < p.E ? pairs : p.E;
    MoePlan m;
    m.expert = reinterpret_cast<int32_t *>(p.ws);
    m.count = m.expert + slots;
    m.entry = reinterpret_cast<MoeEntry *>(m.count + slots);
    m.h = reinterpret_cast<uint16_t *>(p.ws + (slots * (8 + p.T * (int64_t)sizeof(MoeEntry)) + 15) / 16 * 16);
    return m;
}

// A slot's tokens in LDS, in ascending order.
struct Routed {
    int32_t tok[64], pair[64];
    int32_t expert, count;
};

// Every wave gets here; `keep` (the same for the workgroup): the slot's plan is
// written for the second kernel.
__device__ __forceinline__ void route(Routed &rt, const MoeParams &p, int slot, bool keep) {
    if (threadIdx.x < 64) {
        const int t = threadIdx.x;
        const bool by_pair = p.T * p.k < p.E;
        const int e = by_pair ? p.ids[slot] : slot;
        int first = -1;
        float w = 0.0f;
        if (t < p.T && e >= 0 && e < p.E) {
            for (int j = 0; j < p.k; ++j) {
                const int at = t * p.k + j;
                if (p.ids[at] != e) continue;
                if (first < 0) first = at;
                if (keep) w += p.weights ? p.weights[at] : 1.0f;      // an expert chosen twice counts twice
            }
        }
        uint64_t mask = __ballot(first >= 0);
        if (by_pair && mask && __shfl(first, __builtin_ctzll(mask), 64) != slot) mask = 0;
        const int count = __builtin_popcountll(mask);
        const int rank = __builtin_popcountll(mask & ((1ull << t) - 1));
        if (mask >> t & 1) {
            rt.tok[rank] = t;
            rt.pair[rank] = first;
        }
        if (t == 0) {
            rt.expert = e;
            rt.count = count;
        }
        if (keep) {
            const MoePlan m = plan_of(p);
            if (mask >> t & 1) m.entry[slot * p.T + rank] = {first, w};
            if (t == 0) {
                m.expert[slot] = e;
                m.count[slot] = count;
            }
        }
    }
    __syncthreads();
}

__device__ __forceinline__ GemvParams::Weight expert_of(const GemvParams::Weight &w, int e, int64_t rows, int64_t cols,
                                                        int sc) {
    return {w.codes + e * rows * (cols / 2),
            w.scales + e * (sc == kRows16   ? rows * (cols / 16)
                            : sc == kRows32 ? rows * (cols / 32)
                                            : rows / 16 * (cols / 16)),
            sc == kRows32 ? nullptr : w.s_dec + e};
}

template <int SC, int NM>
__device__ __forceinline__ GemvParams up_product(const MoeParams &p, int e) {
    GemvParams q{};
    q.K = p.K;
    q.N = p.F;
    q.w = expert_of(NM == 2 ? p.g : p.u, e, p.F, p.K, SC);
    if (NM == 2) q.u = expert_of(p.u, e, p.F, p.K, SC);
    return q;
}

// Hidden value n of a pair from its sums, as its parts.
template <int SC, int NM>
__device__ __forceinline__ void finish_hidden(const MoeParams &p, const GemvParams &q, const MoePlan &m, int pair,
                                              int64_t n, const float (&v)[2]) {
    float h = SC == kRows32 ? v[0] : v[0] * q.w.s_dec[0];
    if (p.act == kActSilu) h = gate_act<kActSilu, false>(h);
    else if (p.act == kActGelu) h = gate_act<kActGelu, false>(h);
    if (NM == 2) h *= SC == kRows32 ? v[1] : v[1] * q.u.s_dec[0];
    uint16_t *at = m.h + pair * p.F + n;
    const int64_t part = p.T * p.k * p.F;
    const int parts = p.bf16_out ? 2 : 3;
    for (int i = 0; i < parts; ++i) {
        const uint32_t b = pk_bf16(h, h) & 0xFFFFu;
        at[i * part] = (uint16_t)b;
        // an infinite part leaves nothing over (not infinity less infinity)
        h = (b & 0x7FFFu) == 0x7F80u ? 0.0f : h - bf16_to_f32(b);
    }
}

constexpr int kMoeSplit = 8;     // waves of a workgroup

// ---------------------------------------------------------------------------
// Up projections, up to four tokens at a time (4 x 4 x 4 products).
// ---------------------------------------------------------------------------
template <int SC, int NM, int TT, int R>
__global__ __launch_bounds__(64 * kMoeSplit) void moe_up_few_kernel(MoeParams p) {
    constexpr int NO = TT * R * 4;                       // outputs, of NM sums each
    __shared__ float part[kMoeSplit][NM * NO];
    __shared__ Routed rt;
    route(rt, p, blockIdx.y, blockIdx.x == 0);
    const int count = rt.count;
    if (count == 0) return;
    const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * (4 * R);
    const int64_t full = p.K / kStepK;
    const MoePlan m = plan_of(p);
    GemvParams q = up_product<SC, NM>(p, rt.expert);
    q.x = p.x;
    q.T = 1;
    Place<R> pl = place_of<SC, R>(q, n0);
    const uint16_t *const x0 = pl.x;
    for (int c = 0; c < count; c += TT) {
        pl.x = x0 + rt.tok[min(c + min(lane & 3, TT - 1), count - 1)] * p.ldx;
        float acc[NM][R][TT] = {};
        int64_t s = wave;
        if (s < full) {
            Step<NM, R> cur, nxt;
            load_step<SC, NM, R, false>(cur, q, pl, n0, s);
            for (; s + nw < full; s += nw) {
                load_step<SC, NM, R, false>(nxt, q, pl, n0, s + nw);
                add_step<SC, NM, TT, R>(acc, cur);
                cur = nxt;
            }
            add_step<SC, NM, TT, R>(acc, cur);
            s += nw;
        }
        if (s == full && p.K % kStepK) {
            Step<NM, R> last;
            load_step<SC, NM, R, true>(last, q, pl, n0, s);
            add_step<SC, NM, TT, R>(acc, last);
        }
#pragma unroll
        for (int w = 0; w < NM; ++w)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const float v = sum_blocks(acc[w][r][t]);
                    if (lane < 4) part[wave][w * NO + (t * R + r) * 4 + lane] = v;
                }
        __syncthreads();
        for (int o = threadIdx.x; o < NO; o += blockDim.x) {
            float v[2] = {0.0f, 0.0f};
            for (int k = 0; k < nw; ++k)
#pragma unroll
                for (int w = 0; w < NM; ++w) v[w] += part[k][w * NO + o];
            const int i = c + o / (R * 4);
            const int64_t n = n0 + o % (R * 4);
            if (i < count && n < p.F) finish_hidden<SC, NM>(p, q, m, rt.pair[i], n, v);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Up projections, sixteen tokens at a time (16 x 16 x 32 products, activations
// through LDS as in the matrix-vector products).
// ---------------------------------------------------------------------------
template <int SC, int NM, int NR>
__global__ __launch_bounds__(64 * kMoeSplit) void moe_up_tile_kernel(MoeParams p) {
    constexpr int NO = NR * 256;                          // sums of one matrix
    constexpr int kWave = NM * NO * 4 > 4096 ? NM * NO * 4 : 4096;
    __shared__ __align__(16) uint8_t lds[kMoeSplit * kWave];
    __shared__ Routed rt;
    route(rt, p, blockIdx.y, blockIdx.x == 0);
    const int count = rt.count;
    if (count == 0) return;
    const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NR);
    const MoePlan m = plan_of(p);
    const GemvParams q = up_product<SC, NM>(p, rt.expert);
    TilePlace<NR> pl;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const uint32_t row = (uint32_t)min((int64_t)(16 * r + i), p.F - 1 - n0);
        pl.code[r] = row * (uint32_t)(p.K / 2) + 16 * g;
        pl.scale[r] = SC == kRows16   ? row * (uint32_t)(p.K / 16) + 2 * g
                      : SC == kRows32 ? row * (uint32_t)(p.K / 32) + g
                                      : row / 16 * (uint32_t)(p.K / 16) + 2 * g;
    }
    uint8_t *const xl = lds + wave * kWave;
    const int64_t full = p.K / kTileK;
    for (int c = 0; c < count; c += 16) {
        const uint16_t *src[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = 4 * k + g;
            src[k] = p.x + rt.tok[min(c + t, count - 1)] * p.ldx + 8 * (i ^ t);
        }
        f32x4 acc[NM][NR][1];
#pragma unroll
        for (int w = 0; w < NM; ++w)
#pragma unroll
            for (int r = 0; r < NR; ++r) acc[w][r][0] = f32x4{0, 0, 0, 0};
        TileWeights<NM, NR> tw;
        for (int64_t s = wave; s < full; s += nw) {
            load_weights<SC, NM, NR, false>(tw, q, pl, n0, s * kTileK);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");    // the reads of the step before are done
#pragma unroll
            for (int k = 0; k < 4; ++k) copy_lds16(src[k] + s * kTileK, xl + k * 1024);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            tile_products<SC, NM, 1, NR>(acc, tw, [&](int, int j) {
                return *reinterpret_cast<const bf16x8 *>(xl + i * 256 + 16 * ((4 * g + j) ^ i));
            });
        }
        if (full % nw == wave && p.K % kTileK) {
            const int64_t k0 = full * kTileK;
            load_weights<SC, NM, NR, true>(tw, q, pl, n0, k0);
            const int left = (int)(p.K - k0) / 8;         // chunks of a token inside K
            const uint16_t *row = p.x + rt.tok[min(c + i, count - 1)] * p.ldx + k0;
            tile_products<SC, NM, 1, NR>(acc, tw, [&](int, int j) {
                const uint4 v = *reinterpret_cast<const uint4 *>(row + 8 * min(4 * g + j, left - 1));
                const bool in = 4 * g + j < left;
                return __builtin_bit_cast(bf16x8, make_uint4(in ? v.x : 0, in ? v.y : 0, in ? v.z : 0, in ? v.w : 0));
            });
        }
        __syncthreads();                                  // the activations' place is reused
        float *const part = reinterpret_cast<float *>(lds);
        // lane 16 g + i holds token i and rows 4 g .. 4 g + 3
#pragma unroll
        for (int w = 0; w < NM; ++w)
#pragma unroll
            for (int r = 0; r < NR; ++r)
                *reinterpret_cast<f32x4 *>(part + (wave * NM + w) * NO + r * 256 + lane * 4) = acc[w][r][0];
        __syncthreads();
        for (int o = threadIdx.x; o < NO; o += blockDim.x) {
            float v[2] = {0.0f, 0.0f};
            for (int s = 0; s < nw; ++s)
#pragma unroll
                for (int w = 0; w < NM; ++w) v[w] += part[(s * NM + w) * NO + o];
            // consecutive o: rows 4 g + v of one token
            const int l = (o >> 2) & 63, t = c + (l & 15);
            const int64_t n = n0 + (o >> 8) * 16 + (l >> 4) * 4 + (o & 3);
            if (t < count && n < p.F) finish_hidden<SC, NM>(p, q, m, rt.pair[t], n, v);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Down projection and the sum over the experts.  A unit is an expert and up to
// TOK of its tokens; the steps of all units lie in a row, and each wave takes an
// even share of them.  Whenever a wave leaves a unit it adds what it has, times
// the tokens' weights, to its own sums in LDS; the waves' sums are joined in
// order at the end.
// ---------------------------------------------------------------------------
struct DownUnits {
    int32_t *unit;                     // slot << 8 | chunk
    float *sums;                       // waves x T x rows
    int32_t *units;
};

__device__ __forceinline__ DownUnits down_lds(uint8_t *lds, const MoeParams &p) {
    DownUnits d;
    d.units = reinterpret_cast<int32_t *>(lds);
    d.unit = d.units + 4;
    d.sums = reinterpret_cast<float *>(d.unit + (p.T * p.k + 3) / 4 * 4);
    return d;
}

// The units in LDS, and the sums cleared.
template <int TOK, int ROWS>
__device__ __forceinline__ void list_units(const DownUnits &d, const MoeParams &p, const MoePlan &m) {
    const int slots = (int)(p.T * p.k < p.E ? p.T * p.k : p.E);
    for (int o = threadIdx.x; o < (int)(blockDim.x >> 6) * p.T * ROWS; o += blockDim.x) d.sums[o] = 0.0f;
    if (threadIdx.x < 64) {
        int at = 0;
        for (int s0 = 0; s0 < slots; s0 += 64) {
            const int s = s0 + threadIdx.x;
            const int n = s < slots ? (m.count[s] + TOK - 1) / TOK : 0;
            int sum = n;                                  // inclusive sum over the lanes
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int v = __shfl_up(sum, o, 64);
                if ((int)threadIdx.x >= o) sum += v;
            }
            for (int c = 0; c < n; ++c) d.unit[at + sum - n + c] = s << 8 | c;
            at += __shfl(sum, 63, 64);
        }
        if (threadIdx.x == 0) *d.units = at;
    }
    __syncthreads();
}

template <int ROWS>
__device__ __forceinline__ void join_waves(const DownUnits &d, const MoeParams &p, int64_t n0) {
    __syncthreads();
    const int nw = blockDim.x >> 6;
    for (int o = threadIdx.x; o < (int)p.T * ROWS; o += blockDim.x) {
        const int64_t t = o / ROWS, n = n0 + o % ROWS;
        if (n >= p.N) continue;
        float v = 0.0f;
        for (int w = 0; w < nw; ++w) v += d.sums[w * (int)p.T * ROWS + o];
        if (p.r) v += value_at(p.r, t * p.ldr + n, p.bf16_out);
        if (p.bf16_out) static_cast<uint16_t *>(p.y)[t * p.ldy + n] = (uint16_t)pk_bf16(v, v);
        else static_cast<float *>(p.y)[t * p.ldy + n] = v;
    }
}

// NP parts a value, TOK tokens of a unit: TOK NP <= 4 rows of the 4 x 4 x 4 products.
template <int SC, int NP, int TOK, int R>
__global__ __launch_bounds__(64 * kMoeSplit) void moe_down_few_kernel(MoeParams p) {
    constexpr int ROWS = 4 * R, TT = TOK * NP;
    extern __shared__ __align__(16) uint8_t lds[];
    const DownUnits d = down_lds(lds, p);
    const MoePlan m = plan_of(p);
    list_units<TOK, ROWS>(d, p, m);
    const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * ROWS;
    const int64_t full = p.F / kStepK, steps = (p.F + kStepK - 1) / kStepK, total = *d.units * steps;
    int64_t at = total * wave / nw;
    const int64_t end = total * (wave + 1) / nw;
    GemvParams q{};
    q.K = p.F;
    q.N = p.N;
    q.T = 1;
    Place<R> pl = place_of<SC, R>(q, n0);
    const int i = lane & 3, b = lane >> 2;
    float *const sums = d.sums + wave * (int)p.T * ROWS;
    while (at < end) {
        const int64_t u = at / steps;
        const int unit = __builtin_amdgcn_readfirstlane(d.unit[u]), slot = unit >> 8, c = (unit & 255) * TOK;
        const int e = m.expert[slot], count = m.count[slot];
        q.w = expert_of(p.d, e, p.N, p.F, SC);
        const MoeEntry *const entry = m.entry + slot * p.T;
        // row i of the products: part i % NP of the unit's token i / NP
        const MoeEntry own = entry[min(c + min(i / NP, TOK - 1), count - 1)];
        pl.x = m.h + ((int64_t)(i % NP) * p.T * p.k + own.pair) * p.F + b * 32;
        int64_t s = at - u * steps;
        const int64_t last = min(steps, s + end - at);
        at += last - s;
        float acc[1][R][TT] = {};
        const int64_t whole = min(last, full);
        if (s < whole) {
            Step<1, R> cur, nxt;
            load_step<SC, 1, R, false>(cur, q, pl, n0, s);
            for (; s + 1 < whole; ++s) {
                load_step<SC, 1, R, false>(nxt, q, pl, n0, s + 1);
                add_step<SC, 1, TT, R>(acc, cur);
                cur = nxt;
            }
            add_step<SC, 1, TT, R>(acc, cur);
            ++s;
        }
        if (s < last) {
            Step<1, R> tail;
            load_step<SC, 1, R, true>(tail, q, pl, n0, s);
            add_step<SC, 1, TT, R>(acc, tail);
        }
        const float sd = SC == kRows32 ? 1.0f : q.w.s_dec[0];
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            const MoeEntry en = entry[min(c + t, count - 1)];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float v = acc[0][r][t * NP];
#pragma unroll
                for (int k = 1; k < NP; ++k) v += acc[0][r][t * NP + k];
                v = sum_blocks(v);
                if (lane < 4 && c + t < count) sums[en.pair / p.k * ROWS + 4 * r + lane] += en.weight * (v * sd);
            }
        }
    }
    join_waves<ROWS>(d, p, n0);
}

// The same with 16 x 16 x 32 products: 16 / NP tokens a unit.
template <int SC, int NP>
__global__ __launch_bounds__(64 * kMoeSplit) void moe_down_tile_kernel(MoeParams p) {
    constexpr int ROWS = 16, TOK = 16 / NP;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint8_t *const xl = lds + wave * 4096;                // the waves' hidden values come first
    const DownUnits d = down_lds(lds + nw * 4096, p);
    const MoePlan m = plan_of(p);
    list_units<TOK, ROWS>(d, p, m);
    const int i = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * ROWS;
    const int64_t full = p.F / kTileK, steps = (p.F + kTileK - 1) / kTileK, total = *d.units * steps;
    int64_t at = total * wave / nw;
    const int64_t end = total * (wave + 1) / nw;
    GemvParams q{};
    q.K = p.F;
    q.N = p.N;
    TilePlace<1> pl;
    const uint32_t row = (uint32_t)min((int64_t)i, p.N - 1 - n0);
    pl.code[0] = row * (uint32_t)(p.F / 2) + 16 * g;
    pl.scale[0] = SC == kRows16   ? row * (uint32_t)(p.F / 16) + 2 * g
                  : SC == kRows32 ? row * (uint32_t)(p.F / 32) + g
                                  : 2 * g;
    float *const sums = d.sums + wave * (int)p.T * ROWS;
    while (at < end) {
        const int64_t u = at / steps;
        const int unit = __builtin_amdgcn_readfirstlane(d.unit[u]), slot = unit >> 8, c = (unit & 255) * TOK;
        const int e = m.expert[slot], count = m.count[slot];
        q.w = expert_of(p.d, e, p.N, p.F, SC);
        const MoeEntry *const entry = m.entry + slot * p.T;
        // row r of the products: part r % NP of the unit's token r / NP
        auto hidden = [&](int r) {
            const MoeEntry en = entry[min(c + min(r / NP, TOK - 1), count - 1)];
            return m.h + ((int64_t)(r % NP) * p.T * p.k + en.pair) * p.F;
        };
        const uint16_t *src[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) src[k] = hidden(4 * k + g) + 8 * (i ^ (4 * k + g));
        int64_t s = at - u * steps;
        const int64_t last = min(steps, s + end - at);
        at += last - s;
        f32x4 acc[1][1][1] = {{{f32x4{0, 0, 0, 0}}}};
        TileWeights<1, 1> tw;
        for (; s < min(last, full); ++s) {
            load_weights<SC, 1, 1, false>(tw, q, pl, n0, s * kTileK);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");    // the reads of the step before are done
#pragma unroll
            for (int k = 0; k < 4; ++k) copy_lds16(src[k] + s * kTileK, xl + k * 1024);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            tile_products<SC, 1, 1, 1>(acc, tw, [&](int, int j) {
                return *reinterpret_cast<const bf16x8 *>(xl + i * 256 + 16 * ((4 * g + j) ^ i));
            });
        }
        if (s < last) {
            const int64_t k0 = full * kTileK;
            load_weights<SC, 1, 1, true>(tw, q, pl, n0, k0);
            const int left = (int)(p.F - k0) / 8;         // chunks of a row inside F
            const uint16_t *hr = hidden(i) + k0;
            tile_products<SC, 1, 1, 1>(acc, tw, [&](int, int j) {
                const uint4 v = *reinterpret_cast<const uint4 *>(hr + 8 * min(4 * g + j, left - 1));
                const bool in = 4 * g + j < left;
                return __builtin_bit_cast(bf16x8, make_uint4(in ? v.x : 0, in ? v.y : 0, in ? v.z : 0, in ? v.w : 0));
            });
        }
        const float sd = SC == kRows32 ? 1.0f : q.w.s_dec[0];
        // lane 16 g + i holds row i of the products for outputs 4 g .. 4 g + 3
        f32x4 v = acc[0][0][0], sum = v;
#pragma unroll
        for (int k = 1; k < NP; ++k)
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) sum[e4] += __shfl_down(v[e4], k, 16);
        if (i % NP == 0 && i / NP < TOK && c + i / NP < count) {
            const MoeEntry en = entry[c + i / NP];
            float *const to = sums + en.pair / p.k * ROWS + 4 * g;
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) to[e4] += en.weight * (sum[e4] * sd);
        }
    }
    join_waves<ROWS>(d, p, n0);
}

// ---------------------------------------------------------------------------
// Launch rules
// ---------------------------------------------------------------------------
template <auto Kernel>
hipError_t launch_down(const MoeParams &p, int rows, size_t wave_bytes, hipStream_t s) {
    const int64_t pairs = p.T * p.k;
    const size_t shm = 16 + (pairs + 3) / 4 * 16 + kMoeSplit * (p.T * rows * 4 + wave_bytes);
    static const bool attr_set = [rows, wave_bytes] {
        const int most = 16 + 64 * kMoeSlots * 4 + kMoeSplit * (64 * rows * 4 + (int)wave_bytes);
        (void)hipFuncSetAttribute(reinterpret_cast<const void *>(Kernel), hipFuncAttributeMaxDynamicSharedMemorySize, most);
        return true;
    }();
    (void)attr_set;
    hipLaunchKernelGGL(Kernel, dim3((unsigned)((p.N + rows - 1) / rows)), dim3(64 * kMoeSplit), shm, s, p);
    return hipGetLastError();
}

template <int SC, int NM, int TT>
hipError_t up_few(const MoeParams &p, hipStream_t s) {
    constexpr int R = 4 / NM;
    const dim3 grid((unsigned)((p.F + 4 * R - 1) / (4 * R)), (unsigned)moe_slots(p.T, p.k, p.E));
    hipLaunchKernelGGL((moe_up_few_kernel<SC, NM, TT, R>), grid, dim3(64 * kMoeSplit), 0, s, p);
    return hipGetLastError();
}

template <int SC, int NM>
hipError_t up(const MoeParams &p, hipStream_t s) {
    if (p.T == 1) return up_few<SC, NM, 1>(p, s);
    if (p.T == 2) return up_few<SC, NM, 2>(p, s);
    if (p.T <= 4) return up_few<SC, NM, 4>(p, s);
    const dim3 grid((unsigned)((p.F + 15) / 16), (unsigned)moe_slots(p.T, p.k, p.E));
    hipLaunchKernelGGL((moe_up_tile_kernel<SC, NM, 1>), grid, dim3(64 * kMoeSplit), 0, s, p);
    return hipGetLastError();
}

template <int SC>
hipError_t down(const MoeParams &p, hipStream_t s) {
    if (p.T <= 4) {
        if (!p.bf16_out) return launch_down<moe_down_few_kernel<SC, 3, 1, 4>>(p, 16, 0, s);
        if (p.T == 1) return launch_down<moe_down_few_kernel<SC, 2, 1, 4>>(p, 16, 0, s);
        return launch_down<moe_down_few_kernel<SC, 2, 2, 4>>(p, 16, 0, s);
    }
    if (p.bf16_out) return launch_down<moe_down_tile_kernel<SC, 2>>(p, 16, 4096, s);
    return launch_down<moe_down_tile_kernel<SC, 3>>(p, 16, 4096, s);
}

template <int SC>
hipError_t run(const MoeParams &p, hipStream_t s) {
    const hipError_t e = p.gated ? up<SC, 2>(p, s) : up<SC, 1>(p, s);
    return e != hipSuccess ? e : down<SC>(p, s);
}

}  // namespace

hipError_t launch_moe(const MoeParams &p, bool mxfp4, hipStream_t s) {
    return mxfp4 ? run<kRows32>(p, s) : p.tile2d ? run<kTiles16>(p, s) : run<kRows16>(p, s);
}

}  // namespace bbs
