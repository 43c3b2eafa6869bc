// A whole mixture-of-experts layer for a few tokens with 4-bit weights (gfx950):
//   y[t] = r[t] + sum_j w[t, j] (act(x[t] Wg_e^T) * (x[t] Wu_e^T)) Wd_e^T,   e = ids[t, j]
// or, for plain experts, act(x[t] Wu_e^T) Wd_e^T.
//
// The chosen experts' weights bound the layer: each is read once, against 2 flops
// a weight and token.  Three forms, by the launch rules at the end:
//   - a few tokens, two kernels with 4 x 4 x 4 products.  The first kernel's
//     workgroups take one expert and a few of its hidden rows; they find the expert's
//     tokens themselves by looking through the ids (T k of them), so nothing has to be
//     sorted first.  The second kernel's workgroups take a few output columns of all
//     the chosen experts: an output's sum over the experts then stays in one
//     workgroup, in a fixed order, without atomics.  Its waves share the steps of all
//     experts evenly, whatever the routing.
//   - more tokens: the same two with 16 x 16 x 32 products.
//   - more tokens and large weights: one workgroup a CU streams its even share of all
//     the experts' weights through registers, a kernel for each projection, and a
//     third kernel adds up the experts' outputs.
// Measured, replayed from a graph (codes and scales at TB/s in brackets): 1 token,
// 8 of 64 plain experts, 50 MB: 17.7 us (2.9); 1 token, 2 of 8 gated, 177 MB: 41.0 us
// (4.3); 16 tokens, MXFP4, 430 MB: 112 us (3.8); 64 tokens, 8 of 64, NVFP4, 61 experts
// chosen, 582 MB: 184 us (3.2).
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
    m.h = reinterpret_cast<uint16_t *>(p.ws);
    m.entry = reinterpret_cast<MoeEntry *>(m.h + 3 * pairs * p.F);
    m.expert = reinterpret_cast<int32_t *>(m.entry + slots * p.T);
    m.count = m.expert + slots;
    return m;
}

// A slot's tokens in LDS, in ascending order.
struct Routed {
    int32_t tok[64], pair[64];
    int32_t expert, count;
};

// Every wave gets here; `keep` (the same for the workgroup): the slot's plan is
// written for the second kernel.  The ids are loaded eight at a time, all before
// the first is looked at (one after the other they took longer than the weights
// of a small expert).
__device__ __forceinline__ void route(Routed &rt, const MoeParams &p, int slot, bool keep) {
    if (threadIdx.x < 64) {
        const int t = threadIdx.x;
        const bool by_pair = p.T * p.k < p.E;
        const int e = by_pair ? p.ids[slot] : slot;
        const int row = min(t, (int)p.T - 1) * p.k;
        int first = -1;
        float w = 0.0f;
        for (int j0 = 0; j0 < p.k; j0 += 8) {
            int id[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) id[j] = p.ids[row + min(j0 + j, p.k - 1)];
#pragma unroll
            for (int j = 7; j >= 0; --j)
                if (id[j] == e && j0 + j < p.k && (first < 0 || first >= row + j0)) first = row + j0 + j;
            if (keep) {                                               // an expert chosen twice counts twice
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (id[j] == e && j0 + j < p.k) w += p.weights ? p.weights[row + j0 + j] : 1.0f;
            }
        }
        uint64_t mask = __ballot(first >= 0 && t < p.T && e >= 0 && e < p.E);
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
__device__ __forceinline__ void finish_hidden(const MoeParams &p, const GemvParams &q, uint16_t *hidden, int pair,
                                              int64_t n, const float (&v)[2]) {
    float h = SC == kRows32 ? v[0] : v[0] * q.w.s_dec[0];
    if (p.act == kActSilu) h = gate_act<kActSilu, false>(h);
    else if (p.act == kActGelu) h = gate_act<kActGelu, false>(h);
    if (NM == 2) h *= SC == kRows32 ? v[1] : v[1] * q.u.s_dec[0];
    uint16_t *at = hidden + pair * p.F + n;
    const int64_t part = p.T * p.k * p.F;
    const int parts = p.bf16_out ? 2 : 3;
    for (int i = 0; i < parts; ++i) {
        const uint32_t b = pk_bf16(h, h) & 0xFFFFu;
        at[i * part] = (uint16_t)b;
        // an infinite part leaves nothing over (not infinity less infinity)
        h = (b & 0x7FFFu) == 0x7F80u ? 0.0f : h - bf16_to_f32(b);
    }
}

constexpr int kSplit = 8;              // waves of a workgroup
// Of moe_up_few_kernel with 16 / NM rows a workgroup: 2 of 8 experts, 1 token, 30.1 us
// against 32.5 with four waves and 35 with eight; 8 of 64, 9.0 against 11.0 with one (where
// one wave is better, see up_few).
constexpr int kUpFewSplit = 2;

// ---------------------------------------------------------------------------
// Up projections, four tokens at a time (4 x 4 x 4 products).
// ---------------------------------------------------------------------------
template <int SC, int NM, int TT, int R>
__global__ __launch_bounds__(64 * kUpFewSplit) void moe_up_few_kernel(MoeParams p) {
    constexpr int NO = TT * R * 4;                       // outputs, of NM sums each
    __shared__ float part[kUpFewSplit][NM * NO];
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
            if (i < count && n < p.F) finish_hidden<SC, NM>(p, q, m.h, rt.pair[i], n, v);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Up projections, sixteen tokens at a time (16 x 16 x 32 products, activations
// through LDS as in the matrix-vector products).
// ---------------------------------------------------------------------------
template <int SC, int NM, int NR>
__global__ __launch_bounds__(64 * kSplit) void moe_up_tile_kernel(MoeParams p) {
    constexpr int NO = NR * 256;                          // sums of one matrix
    constexpr int kWave = NM * NO * 4 > 4096 ? NM * NO * 4 : 4096;
    __shared__ __align__(16) uint8_t lds[kSplit * kWave];
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
            if (t < count && n < p.F) finish_hidden<SC, NM>(p, q, m.h, rt.pair[t], n, v);
        }
        __syncthreads();
    }
}

// Four consecutive hidden values of a pair; sv, su: the decode scales.
template <int NM>
__device__ __forceinline__ void finish_hidden4(const MoeParams &p, uint16_t *hidden, int pair, int64_t n, const f32x4 &v,
                                               const f32x4 &u, float sv, float su) {
    float h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        h[q] = v[q] * sv;
        if (p.act == kActSilu) h[q] = gate_act<kActSilu, false>(h[q]);
        else if (p.act == kActGelu) h[q] = gate_act<kActGelu, false>(h[q]);
        if (NM == 2) h[q] *= u[q] * su;
    }
    uint16_t *at = hidden + pair * p.F + n;
    const int parts = p.bf16_out ? 2 : 3;
    for (int i = 0; i < parts; ++i, at += p.T * p.k * p.F) {
        const uint2 b = make_uint2(pk_bf16(h[0], h[1]), pk_bf16(h[2], h[3]));
        *reinterpret_cast<uint2 *>(at) = b;
        const uint32_t w[4] = {b.x << 16, b.x & 0xFFFF0000u, b.y << 16, b.y & 0xFFFF0000u};
        // an infinite part leaves nothing over (not infinity less infinity)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            h[q] = (w[q] & 0x7FFFFFFFu) == 0x7F800000u ? 0.0f : h[q] - __uint_as_float(w[q]);
    }
}

__device__ __forceinline__ void finish_output(const MoeParams &p, int64_t t, int64_t n, float v) {
    if (p.r) v += value_at(p.r, t * p.ldr + n, p.bf16_out);
    if (p.bf16_out) static_cast<uint16_t *>(p.y)[t * p.ldy + n] = (uint16_t)pk_bf16(v, v);
    else static_cast<float *>(p.y)[t * p.ldy + n] = v;
}

// ---------------------------------------------------------------------------
// Streaming kernels: 16 x 16 x 32 products, sixteen tokens (or rows of parts of hidden
// values) by sixteen weight rows, 512 K values a step.
//
// One workgroup of eight waves a CU.  Each lists the units first: an expert and up to
// a tile's rows of its tokens, in ascending order.
//
// Bound by the loads together with the expansion of the codes (NVFP4: two vector
// instructions a code and half of one for the exchange of lanes, vector units 65%
// busy; MXFP4: half an instruction and the exchange).  Up projections of 4096 to 1536,
// with the weights that a second unit of an expert reads again: 64 tokens, NVFP4, 464 MB
// in 113 us (4.1 TB/s); 16 tokens, MXFP4, 307 MB in 66 us (4.7); a plain read of such
// sizes reaches 5.7 to 6.3 TB/s.  About 10 us of each are the lists, the first loads
// and the last units.
// ---------------------------------------------------------------------------
struct Units {
    int32_t *entry;                    // pair | token << 16
    float *weight;                     // of each entry
    int32_t *unit;                     // expert | first entry << 10 | entries << 21
    int32_t *count;                    // the units
    // while they are listed, where the rows come afterwards
    uint64_t *mask;                    // the tokens of each expert
    int32_t *first;                    // its first entry
    int32_t *ids;                      // of each pair
};

__device__ __forceinline__ Units units_at(uint8_t *lds, uint8_t *scratch, const MoeParams &p) {
    const int pairs = (int)p.T * p.k;
    Units u;
    u.entry = reinterpret_cast<int32_t *>(lds);
    u.weight = reinterpret_cast<float *>(u.entry + pairs);
    u.unit = reinterpret_cast<int32_t *>(u.weight + pairs);
    u.count = u.unit + pairs;
    u.mask = reinterpret_cast<uint64_t *>(scratch);
    u.first = reinterpret_cast<int32_t *>(u.mask + p.E);
    u.ids = u.first + p.E;
    return u;
}

__device__ __forceinline__ void list_units(const Units &u, const MoeParams &p, int tok) {
    const int pairs = (int)p.T * p.k, n = blockDim.x;
    for (int e = threadIdx.x; e < p.E; e += n) u.mask[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += n) {
        const int e = p.ids[i];
        u.ids[i] = e;
        if (e >= 0 && e < p.E) atomicOr(reinterpret_cast<unsigned long long *>(u.mask + e), 1ull << (i / p.k));
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        int entries = 0, units = 0;
        for (int e0 = 0; e0 < p.E; e0 += 64) {
            const int e = e0 + threadIdx.x;
            const int c = e < p.E ? __builtin_popcountll(u.mask[e]) : 0;
            // inclusive sums over the lanes: entries low, units high
            const int n_units = (c + tok - 1) / tok;
            int sum = c | n_units << 16;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int v = __shfl_up(sum, o, 64);
                if ((int)threadIdx.x >= o) sum += v;
            }
            const int first = entries + (sum & 0xFFFF) - c;
            int at = units + (sum >> 16) - n_units;
            if (e < p.E) u.first[e] = first;
            for (int i = 0; i < c; i += tok) u.unit[at++] = e | (first + i) << 10 | min(tok, c - i) << 21;
            const int all = __shfl(sum, 63, 64);
            entries += all & 0xFFFF;
            units += all >> 16;
        }
        if (threadIdx.x == 0) *u.count = units;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += n) {
        const int e = u.ids[i], t = i / p.k, end = t * p.k + p.k;
        bool again = e < 0 || e >= p.E;
        for (int j = t * p.k; j < i; ++j) again |= u.ids[j] == e;
        if (again) continue;
        float w = p.weights ? p.weights[i] : 1.0f;
        for (int j = i + 1; j < end; ++j)                 // an expert chosen twice counts twice
            if (u.ids[j] == e) w += p.weights ? p.weights[j] : 1.0f;
        const int at = u.first[e] + __builtin_popcountll(u.mask[e] & ((1ull << t) - 1));
        u.entry[at] = i | t << 16;
        u.weight[at] = w;
    }
    __syncthreads();
}

// The weights of a step, 512 K values of NM NR tiles of 16 rows, in registers.  Lane
// 16 g + i multiplies row i at K values 128 g .. + 128 of the step: 64 bytes of
// codes.  They are loaded so that four lanes in a row (a quad) take 64 bytes in a
// row, each of its four rows with one load, and change lanes in registers: with each
// lane loading its own row, every 16 bytes were an access of their own in L1, one a
// cycle, and bound the kernel.
template <int NM, int NR>
struct TileStep {
    uint4 c[NM][NR][4];                // 16 bytes m: of the quad's row m
    uint2 s[NM][NR];                   // the lane's eight E4M3 bytes, or four E8M0 ones in x
};

template <int CTRL>
__device__ __forceinline__ uint32_t quad_perm(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}

// Lanes q and q ^ 1 (CTRL 0xB1, bit: q & 1) or q ^ 2 (0x4E, q & 2) swap b of the lower
// one with a of the upper one.
template <int CTRL>
__device__ __forceinline__ void quad_swap(uint32_t &a, uint32_t &b, bool upper) {
    const uint32_t t = quad_perm<CTRL>(upper ? a : b);
    a = upper ? t : a;
    b = upper ? b : t;
}

// From 16 bytes q of rows 0 .. 3 to 16 bytes 0 .. 3 of row q, q being the lane's place
// in its quad.
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4]) {
    const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll
    for (int m = 0; m < 4; m += 2) {
        quad_swap<0xB1>(v[m].x, v[m + 1].x, odd);
        quad_swap<0xB1>(v[m].y, v[m + 1].y, odd);
        quad_swap<0xB1>(v[m].z, v[m + 1].z, odd);
        quad_swap<0xB1>(v[m].w, v[m + 1].w, odd);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        quad_swap<0x4E>(v[m].x, v[m + 2].x, high);
        quad_swap<0x4E>(v[m].y, v[m + 2].y, high);
        quad_swap<0x4E>(v[m].z, v[m + 2].z, high);
        quad_swap<0x4E>(v[m].w, v[m + 2].w, high);
    }
}

// Where a wave loads weights from: the matrices at the tile's first row, and from
// there the lane's place in the quad's first row and its own row's scales.
template <int NM, int NR>
struct TileSource {
    const uint8_t *codes[NM], *scales[NM];
    uint32_t code, pitch, scale[NR];
};

// k0: K value of the step.
template <int SC, int NM, int NR>
__device__ __forceinline__ void load_tile(TileStep<NM, NR> &st, const TileSource<NM, NR> &t, int64_t k0) {
#pragma unroll
    for (int w = 0; w < NM; ++w)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
                st.c[w][r][m] = *reinterpret_cast<const uint4 *>(t.codes[w] + k0 / 2 + (t.code + (16 * r + m) * t.pitch));
            if (SC == kRows32) __builtin_memcpy(&st.s[w][r].x, t.scales[w] + k0 / 32 + t.scale[r], 4);
            else __builtin_memcpy(&st.s[w][r], t.scales[w] + k0 / 16 + t.scale[r], 8);
        }
}

// x: the step's rows in LDS, 1024 bytes each, NT tiles of 16; row: the lane's in a tile.
template <int SC, int NM, int NR, int NT>
__device__ __forceinline__ void add_tile(f32x4 (&acc)[NM][NR][NT], TileStep<NM, NR> &st, const uint8_t *x, int row) {
    const int g = (threadIdx.x & 63) >> 4;
    uint4 xv[2][4][NT];
    // the rows' 64 bytes m are read while those before them are multiplied
    auto read = [&](int m) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                xv[m & 1][j][t] = *reinterpret_cast<const uint4 *>(x + (16 * t + row) * 1024 + 256 * g +
                                                                   16 * ((4 * m + j) ^ row));
    };
    read(0);
#pragma unroll
    for (int w = 0; w < NM; ++w)
#pragma unroll
        for (int r = 0; r < NR; ++r) quad_transpose(st.c[w][r]);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if (m < 3) read(m + 1);
        __builtin_amdgcn_sched_barrier(0);
        f32x2 sc[NM][NR];                                 // of blocks 2 m and 2 m + 1 (MXFP4: m)
#pragma unroll
        for (int w = 0; w < NM; ++w)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const uint2 b = st.s[w][r];
                if (SC == kRows32) sc[w][r][0] = sc[w][r][1] = e8m0_value(b.x >> (8 * m) & 0xFFu);
                else if (m & 1) sc[w][r] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)(m < 2 ? b.x : b.y), 1.0f, true);
                else sc[w][r] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)(m < 2 ? b.x : b.y), 1.0f, false);
            }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int w = 0; w < NM; ++w)
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const bf16x8 c = expand8<SC>(word(st.c[w][r][m], j), sc[w][r][j >> 1]);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        acc[w][r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            c, __builtin_bit_cast(bf16x8, xv[m & 1][j][t]), acc[w][r][t], 0, 0, 0);
                }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// n steps through a ring of D in registers: issue(step) loads the next one (past
// the last it loads what is there again), use(step) multiplies the oldest; begun()
// comes between the first loads and the first use.  No load depends on a branch:
// the compiler then waits for a step's own loads and not for those behind them.
template <int D, typename Step, typename Issue, typename Begun, typename Use>
__device__ __forceinline__ void run_ring(int64_t n, Issue issue, Begun begun, Use use) {
    Step ring[D];
#pragma unroll
    for (int d = 0; d < D; ++d) issue(ring[d]);
    begun();
    for (int64_t i = D; i <= n; i += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            use(ring[d]);
            issue(ring[d]);
        }
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (d < n % D) use(ring[d]);
}

__device__ __forceinline__ float scalar(float v) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

// NP = 0: up projection, x rows to hidden values.  Else: down projection, NP parts of
// hidden values to a pair's outputs (weighted), of each range of K.
//
// A workgroup takes an even share of the tiles (16 NR weight rows of a range of a
// unit), unit by unit.  The unit's rows lie in LDS, and its tiles' steps, one tile's
// after another's, are cut into even parts for the waves.  A wave that comes into a
// tile behind its first step leaves its sums in LDS for the one that began it.
template <int SC, int NM, int NR, int NP, int NT, int D>
__global__ __launch_bounds__(64 * kMoeTileWaves, kMoeTileWaves / 4) void moe_stream_kernel(MoeParams p, MoeShape sh) {
    static_assert(NM * NR == 2, "a tile's sums fill a wave's buffer");
    constexpr int NW = kMoeTileWaves;
    extern __shared__ __align__(16) uint8_t lds[];
    const int64_t K = NP ? p.F : p.K, rows = NP ? p.N : p.F;
    const int64_t most = moe_rows_bytes(sh);
    uint8_t *const xs = lds;                                                   // [step][row][1024 bytes]
    float *const part = reinterpret_cast<float *>(lds + most);
    const Units un = units_at(lds + most + moe_sums_bytes(NT), lds, p);
    const int tok = NP ? sh.rows / 16 * (16 / (NP ? NP : 1)) : sh.rows;
    list_units(un, p, tok);
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = i & (sh.rows - 1);        // (rows: 4, 8, or 16 a tile)
    const int64_t blocks = (rows + 16 * NR - 1) / (16 * NR), tiles = *un.count * sh.ranges * blocks;
    int64_t at = tiles * blockIdx.x / gridDim.x;
    const int64_t last = tiles * (blockIdx.x + 1) / gridDim.x;
    uint16_t *const h = reinterpret_cast<uint16_t *>(p.ws);
    const int64_t pairs = p.T * p.k;

    while (at < last) {
        // blocks b0 .. b1 of one range of one unit
        const int64_t ur = at / blocks, b0 = at - ur * blocks, b1 = min(blocks, b0 + last - at);
        at += b1 - b0;
        const int u = (int)(ur / sh.ranges), range = (int)(ur - (int64_t)u * sh.ranges);
        const int unit = __builtin_amdgcn_readfirstlane(un.unit[u]), e = unit & 1023, n = unit >> 21;
        const int *const entry = un.entry + (unit >> 10 & 2047);
        const int64_t klo = range * sh.range, khi = min(K, klo + sh.range);
        const int steps = (int)((khi - klo + kMoeStep - 1) / kMoeStep);
        const int64_t all = (b1 - b0) * steps, s0 = all * wave / NW, s1 = all * (wave + 1) / NW;
        // the decode scales, loaded here: a load's wait among the steps would be one for
        // all the weights before it
        float sv = 1.0f, su = 1.0f;
        if (SC != kRows32) {
            sv = scalar((NP ? p.d : NM == 2 ? p.g : p.u).s_dec[e]);
            if (NM == 2) su = scalar(p.u.s_dec[e]);
        }
        // a last step that K ends in starts earlier, at K - 512; in LDS its rows are zero
        // where the step before has had them
        auto step_k = [&](int s) { return min(klo + s * kMoeStep, K - kMoeStep); };
        // a block at the end of the rows starts earlier, and leaves out the rows that the
        // block before it has: their sums are cut elsewhere there
        auto first_row = [&](int64_t blk) { return min(blk * (16 * NR), rows - 16 * NR); };
        GemvParams::Weight mat[NM];
        mat[0] = expert_of(NP ? p.d : NM == 2 ? p.g : p.u, e, rows, K, SC);
        if (NM == 2) mat[NM - 1] = expert_of(p.u, e, rows, K, SC);
        TileSource<NM, NR> src;
        src.pitch = (uint32_t)(K / 2);
        src.code = (lane >> 2 & 3) * 4 * src.pitch + 64 * g + 16 * (lane & 3);
#pragma unroll
        for (int r = 0; r < NR; ++r)
            src.scale[r] = (SC == kTiles16 ? r : 16 * r + i) * (uint32_t)(SC == kRows32 ? K / 32 : K / 16) +
                           (SC == kRows32 ? 4 : 8) * g;
        int64_t lb = b0 + s0 / steps;
        int ls = (int)(s0 % steps);
        auto issue = [&](TileStep<NM, NR> &st) __attribute__((always_inline)) {
            const int64_t n0 = first_row(lb);
#pragma unroll
            for (int w = 0; w < NM; ++w) {
                src.codes[w] = mat[w].codes + n0 * (K / 2);
                src.scales[w] = mat[w].scales + (SC == kRows16   ? n0 * (K / 16)
                                                 : SC == kRows32 ? n0 * (K / 32)
                                                                 : n0 / 16 * (K / 16));
            }
            load_tile<SC, NM, NR>(st, src, step_k(ls));
            const bool over = ls + 1 == steps;
            lb += over && lb + 1 < b1 ? 1 : 0;
            ls = over ? 0 : ls + 1;
        };
        // the unit's rows into LDS: a copy for each row of a step, chunk c (16 bytes) of
        // row r at place c ^ r of its sixteen
        auto begun = [&]() {
            __syncthreads();                              // the rows before are done with
            constexpr int P = NP ? NP : 1, TOK = 16 / P;
            const int used = n * P;
            for (int c = wave; c < steps * used; c += NW) {
                const int s = c / used, q = c - s * used, tk = q / P, r = tk / TOK * 16 + tk % TOK * P + q % P;
                const int en = entry[tk];
                const uint16_t *const from = NP ? h + ((q % P) * pairs + (en & 0xFFFF)) * p.F : p.x + (en >> 16) * p.ldx;
                copy_lds16(from + step_k(s) + 8 * (lane ^ (r & 15)), xs + (s * sh.rows + r) * 1024);
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            const int had = (int)(klo + (steps - 1) * kMoeStep - step_k(steps - 1)) / 8;   // chunks of eight values
            if (had > 0) {
                for (int r = wave; r < sh.rows; r += NW)
                    if (lane < had)
                        *reinterpret_cast<uint4 *>(xs + ((steps - 1) * sh.rows + r) * 1024 + 16 * (lane ^ (r & 15))) =
                            make_uint4(0, 0, 0, 0);
                __syncthreads();
            }
        };
        f32x4 acc[NM][NR][NT];
        int64_t cb = lb;
        int cs = ls;
        bool began = cs == 0;
        auto clear = [&]() {
#pragma unroll
            for (int w = 0; w < NM; ++w)
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[w][r][t] = f32x4{0, 0, 0, 0};
        };
        auto place = [&](int o, int w, int r, int t) {
            return reinterpret_cast<f32x4 *>(part + ((o * 2 + w * NR + r) * NT + t) * 256 + lane * 4);
        };
        auto leave = [&]() {
#pragma unroll
            for (int w = 0; w < NM; ++w)
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t) *place(wave, w, r, t) = acc[w][r][t];
        };
        // lane 16 g + i holds row i's sums for weight rows 4 g .. 4 g + 3 of each 16
        auto finish = [&]() __attribute__((always_inline)) {
            constexpr int P = NP ? NP : 1, TOK = 16 / P;   // tokens of a tile of rows
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int own = t * TOK + i / P, en = min(own, n - 1), pr = entry[en] & 0xFFFF;
                const bool in = i % P == 0 && i / P < TOK && own < n;
                const float w = NP ? un.weight[(unit >> 10 & 2047) + en] * sv : 0.0f;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const int64_t at4 = first_row(cb) + 16 * r + 4 * g;
                    if (NP == 0) {
                        if (in && at4 >= cb * (16 * NR))  // (all four: F is a multiple of 16)
                            finish_hidden4<NM>(p, h, pr, at4, acc[0][r][t], acc[NM - 1][r][t], sv, su);
                    } else {
                        f32x4 sum = acc[0][r][t];
#pragma unroll
                        for (int k = 1; k < NP; ++k)
#pragma unroll
                            for (int q = 0; q < 4; ++q) sum[q] += __shfl_down(acc[0][r][t][q], k, 16);
                        float *const y = p.part + (range * pairs + pr) * p.N + at4;
                        if (in) {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                if (at4 + q >= cb * (16 * NR)) y[q] = w * sum[q];
                        }
                    }
                }
            }
        };
        auto use = [&](TileStep<NM, NR> &st) __attribute__((always_inline)) {
            add_tile<SC, NM, NR, NT>(acc, st, xs + cs * sh.rows * 1024, row);
            if (++cs == steps) {
                if (began) finish();
                else leave();
                clear();
                cs = 0;
                ++cb;
                began = true;
            }
        };
        clear();
        if (s0 < s1) run_ring<D, TileStep<NM, NR>>(s1 - s0, issue, begun, use);
        else begun();
        // a tile that goes on in the next waves
        const bool open = s0 < s1 && cs != 0;
        if (open && !began) leave();
        __syncthreads();
        if (open && began) {
            const int64_t over = (cb - b0 + 1) * steps;
            for (int o = wave + 1; o < NW && all * o / NW < over; ++o) {
                if (all * o / NW == all * (o + 1) / NW) continue;
#pragma unroll
                for (int w = 0; w < NM; ++w)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const f32x4 v = *place(o, w, r, t);
                            acc[w][r][t] += v;
                        }
            }
            finish();
        }
    }
}

// An output from its pairs' and ranges' sums, in the order of the token's choice.
__global__ __launch_bounds__(64) void moe_sum_kernel(MoeParams p, int ranges) {
    __shared__ int64_t from[kMoeSlots];
    const int64_t n = (int64_t)blockIdx.x * 64 + threadIdx.x, t = blockIdx.y;
    const int j = threadIdx.x & (kMoeSlots - 1);
    const int e = j < p.k ? p.ids[t * p.k + j] : -1;
    bool first = e >= 0 && e < p.E;                       // an expert chosen again is with its first pair
    for (int q = 1; q < p.k; ++q) {
        const int o = __shfl(e, j - q, kMoeSlots);
        if (j >= q && o == e) first = false;
    }
    const uint64_t mask = __ballot(first && threadIdx.x < kMoeSlots);
    if (first && threadIdx.x < kMoeSlots) from[__builtin_popcountll(mask & ((1ull << j) - 1))] = (t * p.k + j) * p.N;
    const int count = __builtin_popcountll(mask);
    __syncthreads();
    if (n >= p.N) return;
    float v = 0.0f;
    for (int r = 0; r < ranges; ++r) {
        const float *const part = p.part + r * p.T * p.k * p.N + n;
#pragma unroll 4
        for (int q = 0; q < count; ++q) v += part[from[q]];
    }
    finish_output(p, t, n, v);
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
__device__ __forceinline__ void list_slots(const DownUnits &d, const MoeParams &p, const MoePlan &m) {
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
__device__ __forceinline__ void join_waves(const float *sums, const MoeParams &p, int64_t n0) {
    __syncthreads();
    const int nw = blockDim.x >> 6;
    for (int o = threadIdx.x; o < (int)p.T * ROWS; o += blockDim.x) {
        const int64_t t = o / ROWS, n = n0 + o % ROWS;
        if (n >= p.N) continue;
        float v = 0.0f;
        for (int w = 0; w < nw; ++w) v += sums[w * (int)p.T * ROWS + o];
        finish_output(p, t, n, v);
    }
}

// NP parts a value, TOK tokens of a unit: TOK NP <= 4 rows of the 4 x 4 x 4 products.
template <int SC, int NP, int TOK, int R>
__global__ __launch_bounds__(64 * kSplit) void moe_down_few_kernel(MoeParams p) {
    constexpr int ROWS = 4 * R, TT = TOK * NP;
    extern __shared__ __align__(16) uint8_t lds[];
    const DownUnits d = down_lds(lds, p);
    const MoePlan m = plan_of(p);
    list_slots<TOK, ROWS>(d, p, m);
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
    join_waves<ROWS>(d.sums, p, n0);
}

// The same with 16 x 16 x 32 products: 16 / NP tokens a unit.
template <int SC, int NP>
__global__ __launch_bounds__(64 * kSplit) void moe_down_tile_kernel(MoeParams p) {
    constexpr int ROWS = 16, TOK = 16 / NP;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint8_t *const xl = lds + wave * 4096;                // the waves' hidden values come first
    const DownUnits d = down_lds(lds + nw * 4096, p);
    const MoePlan m = plan_of(p);
    list_slots<TOK, ROWS>(d, p, m);
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
    join_waves<ROWS>(d.sums, p, n0);
}

// ---------------------------------------------------------------------------
// Launch rules
// ---------------------------------------------------------------------------
template <auto Kernel>
hipError_t launch_down(const MoeParams &p, int rows, size_t wave_bytes, hipStream_t s) {
    const int64_t pairs = p.T * p.k;
    const size_t shm = 16 + (pairs + 3) / 4 * 16 + kSplit * (p.T * rows * 4 + wave_bytes);
    static const bool attr_set = [rows, wave_bytes] {
        const int most = 16 + 64 * kMoeSlots * 4 + kSplit * (64 * rows * 4 + (int)wave_bytes);
        (void)hipFuncSetAttribute(reinterpret_cast<const void *>(Kernel), hipFuncAttributeMaxDynamicSharedMemorySize, most);
        return true;
    }();
    (void)attr_set;
    hipLaunchKernelGGL(Kernel, dim3((unsigned)((p.N + rows - 1) / rows)), dim3(64 * kSplit), shm, s, p);
    return hipGetLastError();
}

// Streaming pays from about 50 MB of codes of the experts that can be chosen: below it
// the lists and the third launch cost more than the earlier forms' uneven loads.
// Measured (streaming against not): 20 MB, 5 tokens, 25.7 and 17.4 us; 50 MB, 8
// tokens, 33.2 and 29.9, 16 tokens (MXFP4) 33.6 and 33.3, 64 tokens 52.5 and 60.9;
// 100 MB, 8 tokens, 37.4 and 45.0, 64 tokens 62.5 and 103; 604 MB, 5 tokens, 85.5 and 129.
// It needs a whole step of each K, a tile's rows, and room in LDS for four rows of x.
bool streams(const MoeParams &p) {
    const int64_t codes = moe_slots(p.T, p.k, p.E) * ((p.gated ? 2 : 1) * p.F * p.K + p.N * p.F) / 2;
    return codes > (48 << 20) && p.K >= kMoeStep && p.F >= kMoeStep && p.N >= 32 &&
           moe_up_shape(p.T, p.k, p.K).rows > 0;
}

// The 4 x 4 x 4 products leave no rows empty at a few tokens, but expand a code again for
// every four of an expert.  NVFP4, up to eight tokens, against the other two forms: 8 of
// 64 experts, 5 tokens 71.5 us and 85.9, 8 tokens 94.7 and 102; 2 of 8, 6 tokens 130 and
// 142, 8 tokens 154 and 152; 2 of 16 small ones, 8 tokens 15.3 and 17.2 (16 tokens and 8 of 64:
// 198 and 135).  That is with BF16 outputs; for FP32 ones the down projection takes one
// token at a time and expands its codes again for each: 8 of 64, 3 tokens 49.9 and 72.3, 5
// tokens 74.9 and 86.5, 8 tokens 102 and 104; 2 of 8, 3 tokens 90.6 and 93.8, but 6 tokens
// 151 and 143, 8 tokens 185 and 155: from about two tokens an expert on the bound of eight
// tokens is too high there.  MXFP4 streams sooner, as its codes are cheap to expand: 2 of 8,
// 3 tokens 103 and 85.8, 4 tokens 138 and 119; but below the streaming kernels' size 4 tokens
// 25.0 and 30.3, 5 tokens 20.7 and 17.5.
template <int SC>
bool few_tokens(const MoeParams &p) {
    if (SC != kRows32) return p.T <= 8;
    return p.T <= 2 || (p.T <= 4 && !streams(p));
}

// Steps in flight beside the one in use: two for NVFP4 (64 tokens, 118 us against 123
// with one), one for MXFP4, whose steps are short (16 tokens, 65 us against 68 with two).
template <int SC>
constexpr int kRing = SC == kRows32 ? 1 : 2;

template <auto Kernel>
hipError_t launch_stream(const MoeParams &p, const MoeShape &sh, hipStream_t s) {
    const int64_t shm = moe_tile_lds(p.T, p.k, sh);
    static const bool attr_set = [] {
        (void)hipFuncSetAttribute(reinterpret_cast<const void *>(Kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                  kMoeLds);
        return true;
    }();
    (void)attr_set;
    hipLaunchKernelGGL(Kernel, dim3((unsigned)device_cus(s)), dim3(64 * kMoeTileWaves), (size_t)shm, s, p, sh);
    return hipGetLastError();
}

// With gated NVFP4 experts one wave takes all of K, and 16 rows, where that leaves every
// CU six waves: a wave then loads twice as much a step, and joins nothing in LDS.
// Measured (against two waves of half the rows): 2 of 8 experts, 1 token, 1792 waves, 41.0
// us and 45.8, 4 tokens 121 and 147; 8 of 64, 2 tokens, 1536 waves, 36.8 and 40.0, 4
// tokens 58.7 and 67.6, but 1 token, 768 waves, 26.9 and 23.6.  MXFP4, 16 of 64 experts
// with 1536 waves, 48.3 and 44.7.
template <int SC, int NM, int TT>
hipError_t up_few(const MoeParams &p, hipStream_t s) {
    const int64_t slots = moe_slots(p.T, p.k, p.E);
    constexpr int R = 4 / NM, RW = 4;
    auto blocks = [&](int r) { return (unsigned)((p.F + 4 * r - 1) / (4 * r)); };
    if constexpr (SC != kRows32 && NM == 2) {
        if (blocks(RW) * slots >= 6 * device_cus(s)) {
            hipLaunchKernelGGL((moe_up_few_kernel<SC, NM, TT, RW>), dim3(blocks(RW), (unsigned)slots), dim3(64), 0, s, p);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((moe_up_few_kernel<SC, NM, TT, R>), dim3(blocks(R), (unsigned)slots), dim3(64 * kUpFewSplit), 0, s,
                       p);
    return hipGetLastError();
}

template <int SC, int NM>
hipError_t up(const MoeParams &p, hipStream_t s) {
    if (p.T == 1) return up_few<SC, NM, 1>(p, s);
    if (p.T == 2) return up_few<SC, NM, 2>(p, s);
    if (few_tokens<SC>(p)) return up_few<SC, NM, 4>(p, s);
    if (streams(p))
        return launch_stream<moe_stream_kernel<SC, NM, 2 / NM, 0, 1, kRing<SC>>>(p, moe_up_shape(p.T, p.k, p.K), s);
    const dim3 grid((unsigned)((p.F + 15) / 16), (unsigned)moe_slots(p.T, p.k, p.E));
    hipLaunchKernelGGL((moe_up_tile_kernel<SC, NM, 1>), grid, dim3(64 * kSplit), 0, s, p);
    return hipGetLastError();
}

template <int SC, int NP>
hipError_t down_stream(const MoeParams &p, hipStream_t s) {
    const MoeShape sh = moe_down_shape(p.T, p.k, p.F);
    hipError_t e;
    if (SC == kRows32 && sh.rows == 16) e = launch_stream<moe_stream_kernel<kRows32, 1, 2, NP, 1, kRing<kRows32>>>(p, sh, s);
    else e = launch_stream<moe_stream_kernel<SC, 1, 2, NP, 2, kRing<SC>>>(p, sh, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(moe_sum_kernel, dim3((unsigned)((p.N + 63) / 64), (unsigned)p.T), dim3(64), 0, s, p, sh.ranges);
    return hipGetLastError();
}

template <int SC>
hipError_t down(const MoeParams &p, hipStream_t s) {
    if (few_tokens<SC>(p)) {
        if (!p.bf16_out) return launch_down<moe_down_few_kernel<SC, 3, 1, 4>>(p, 16, 0, s);
        if (p.T == 1) return launch_down<moe_down_few_kernel<SC, 2, 1, 4>>(p, 16, 0, s);
        return launch_down<moe_down_few_kernel<SC, 2, 2, 4>>(p, 16, 0, s);
    }
    if (streams(p)) return p.bf16_out ? down_stream<SC, 2>(p, s) : down_stream<SC, 3>(p, s);
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
