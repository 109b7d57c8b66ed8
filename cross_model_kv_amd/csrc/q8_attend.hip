// Attention over the 8-bit paged cache.
//
// For query row i of sequence b at position pos = len - n_q + i, with y_t = scale * q . k_t, t <= pos:
//   lse = log sum exp y_t,   out = sum exp(y_t - lse) v_t.
// One pass over the tokens with a running maximum m and sum l; the query heads that share a KV head
// (G = H_q / H_kv of them) and the n_q queries of a sequence are the rows of one problem, row
// r = i * G + g, so the cache is read once for all of them.
//
// Matrix products on 16x16x32 tiles, a wave of 64 lanes on 64 tokens x 16 rows, transposed so that
// a row of the softmax is a column of the tiles (lane & 15) everywhere:
//   S^T = K Q^T   A = 16 tokens x 32 dims,  B = 32 dims x 16 rows   -> lane holds 4 tokens of one row
//   O^T = V^T P^T A = 16 dims x 32 tokens,  B = 32 tokens x 16 rows -> lane holds 4 dims of one row
// The order of a contraction is free as long as both operands share it, and so is the order of the
// tokens in S^T's tiles.  Both are chosen so that nothing crosses lanes and every load is 16 bytes:
// with g = lane >> 4, row 4 g' + j of S^T's tile m is token 16 g' + 4 m + j, so after the four tiles of 64
// tokens lane group g holds the tokens 16 g .. 16 g + 15 of its row, in order; and those are the 16 bytes of
// a dim that the lane's load of the (dim-major) values brings.  Keys are read as 16 adjacent dims of a
// token.  No shared memory and no barrier in the loop.
//
// 8 bits to 16: a code is exact in bf16 and in fp16, so scales stay out of the operands: the key's goes into
// the score, the value's into the weight.  bf16 calls: bf16 queries; weights in fp16 (11 bits; bf16's 8 would
// cost the output as much as its own rounding does).  Weights are held as pv = exp2(y2 + log2 v_scale - m) with m
// the running maximum of that exponent, so pv stays in fp16's range whatever the scales are, and
// l = sum pv / v_scale.  fp32 calls: queries and weights as three bf16 parts each (24 bits).

#include <algorithm>

#include "common.h"
#include "internal.h"
#include "q8_span.h"

namespace kvmap {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -1e30f;   // the running maximum of a row that has seen no token
constexpr float kSlack = 6.f;     // m is moved when a score passes it by this much (weights up to 2^6)
constexpr int kTile = 64;         // tokens of a wave's step
constexpr int kWaves = 4;
constexpr int kPerCu = 4;         // workgroups a CU that splits are made for

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float inf32() { return __uint_as_float(0x7F800000u); }
__device__ __forceinline__ float nan32() { return __uint_as_float(0x7FC00000u); }

template <bool BF16>
struct Weights;  // what PV's operands are made of

// 1 in every byte of w that is a NaN code
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7; }

// 8 codes (two dwords) as a matrix operand
__device__ __forceinline__ bf16x8_t bf16_codes(uint32_t a, uint32_t b) {
    const bf16x2_t x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false);
    const bf16x2_t x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true);
    const bf16x2_t x2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false);
    const bf16x2_t x3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true);
    return bf16x8_t{x0[0], x0[1], x1[0], x1[1], x2[0], x2[1], x3[0], x3[1]};
}
__device__ __forceinline__ f16x8_t f16_codes(uint32_t a, uint32_t b) {
    const f16x2_t x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, false);
    const f16x2_t x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, true);
    const f16x2_t x2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, false);
    const f16x2_t x3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, true);
    return f16x8_t{x0[0], x0[1], x1[0], x1[1], x2[0], x2[1], x3[0], x3[1]};
}

// x as a sum of three bf16 parts (8 bits each), exact to 2^-24
struct Parts3 {
    bf16x8_t p[3];
    __device__ __forceinline__ void set(const float* x) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float rest = x[i];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const __bf16 y = (__bf16)rest;
                p[k][i] = y;
                rest -= (float)y;
            }
        }
    }
};

template <>
struct Weights<true> {
    using Codes = f16x8_t;
    Codes p;
    __device__ __forceinline__ void set(const float* x) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const f16x2_t y = __builtin_convertvector((f32x2_t{x[i], x[i + 1]}), f16x2_t);
            p[i] = y[0];
            p[i + 1] = y[1];
        }
    }
    __device__ static __forceinline__ Codes codes(uint32_t a, uint32_t b) { return f16_codes(a, b); }
    __device__ __forceinline__ f32x4_t times(Codes v, f32x4_t o) const { return __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p, o, 0, 0, 0); }
};
template <>
struct Weights<false> : Parts3 {
    using Codes = bf16x8_t;
    __device__ static __forceinline__ Codes codes(uint32_t a, uint32_t b) { return bf16_codes(a, b); }
    __device__ __forceinline__ f32x4_t times(Codes v, f32x4_t o) const {
        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[2], o, 0, 0, 0);
        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[1], o, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[0], o, 0, 0, 0);
    }
};

template <bool BF16>
struct Query;  // 8 dims of a query row as a matrix operand
template <>
struct Query<true> {
    bf16x8_t p;
    __device__ __forceinline__ void load(const void* base, int64_t at) { p = *(const bf16x8_t*)((const __bf16*)base + at); }
    __device__ __forceinline__ void zero() { p = bf16x8_t{}; }
    __device__ __forceinline__ f32x4_t times(bf16x8_t k, f32x4_t s) const { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, p, s, 0, 0, 0); }
};
template <>
struct Query<false> : Parts3 {
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        const float4 a = ((const float4*)((const float*)base + at))[0], b = ((const float4*)((const float*)base + at))[1];
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        set(x);
    }
    __device__ __forceinline__ void zero() { p[0] = p[1] = p[2] = bf16x8_t{}; }
    __device__ __forceinline__ f32x4_t times(bf16x8_t k, f32x4_t s) const {
        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, p[2], s, 0, 0, 0);
        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, p[1], s, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, p[0], s, 0, 0, 0);
    }
};

// How a sequence's tokens are split over workgroups: split s takes the tiles [s * tps, (s + 1) * tps).
struct Q8Split {
    int n_splits, tps;   // tps: tiles of a split
    int row_blocks;
    float* part_o;       // [B * H][row_blocks][n_splits][ROWS][d]: sums of pv times codes
    float* part_ml;      // [B * H][row_blocks][n_splits][ROWS][2]: m, l
};

__host__ __device__ __forceinline__ int live_splits(int len, int tps) {
    const int t = (len + kTile - 1) / kTile;
    return t > tps ? (t + tps - 1) / tps : 1;
}

// One tile's codes as loaded: keys of 4 x 16 tokens, values of D dims, and the lane's scales (the
// tokens 16 g .. 16 g + 15 lie in one page, pages being whole 16 tokens).
template <int D>
struct TileData {
    u32x4_t k[4][D / 64];
    u32x4_t v[D / 16];
    float ks, vs;
};

// Waves a SIMD that the registers are held to.  An instance that spills is not built: the compiler's
// spills of parts of matrix operands have given wrong sums (an fp32 instance of four row tiles), so fp32
// stops at two row tiles and a test reads every instance's scratch size.
template <bool BF16, int D, int NT>
constexpr int kOccupancy = !BF16 ? (NT == 1 ? 2 : 1) : NT == 1 ? 3 : NT == 2 ? 2 : 1;

template <bool BF16, int D, int NT>
__global__ __launch_bounds__(256, (kOccupancy<BF16, D, NT>)) void q8_decode_kernel(Q8Attend a, Q8Split sp) {
    constexpr int ROWS = 16 * NT;
    constexpr int LDO = D + 4;
    __shared__ float s_o[kWaves][ROWS][LDO];
    __shared__ float s_ml[kWaves][ROWS][2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int split = blockIdx.x % sp.n_splits, rb = blockIdx.x / sp.n_splits, b = blockIdx.y / a.c.H, h = blockIdx.y % a.c.H;
    const int G = a.Hq / a.c.H, R = a.n_q * G;
    const int P = a.c.page, logP = 31 - __clz(P);
    const int len = a.len[b];
    const bool bad = len < 0 || len > a.max_len;
    const int tiles = bad ? 0 : (len + kTile - 1) / kTile;
    const int live = bad ? 1 : live_splits(len, sp.tps);
    if (split >= live) return;
    const int t_end = min(tiles, (split + 1) * sp.tps);

    // this lane's rows: their queries, and the tokens that they see
    Query<BF16> q[NT][D / 32];
    int end[NT];
    const int first_end = len - a.n_q + rb * ROWS / G + 1;  // the fewest tokens that a row of the block sees
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = rb * ROWS + n * 16 + c;
        const int i = r / G, hq = h * G + r % G;
        end[n] = len - a.n_q + i + 1;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            // step s contracts dims 64 (s / 2) + 16 g + 8 (s & 1) .. + 8, as the key loads hold them
            if (r < R)
                q[n][s].load(a.q.base, (int64_t)b * a.q.seq + (int64_t)hq * a.q.head + (int64_t)i * a.q.token + 64 * (s / 2) + 16 * g + 8 * (s & 1));
            else
                q[n][s].zero();
        }
    }
    const float y2 = a.scale * kLog2e;
    const int32_t* pages = a.pages + (int64_t)b * a.max_pages;
    f32x4_t o[NT][D / 16];
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = kNone;
        l[n] = 0.f;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) o[n][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    // the pages of the 16 tokens that this lane's key rows and its values come from
    auto pages_of = [&](int tile, int& pk, int& pv) {
        pk = q8_page_at(pages, (tile * kTile + 16 * (c >> 2)) >> logP, a.max_pages, a.c.n_pages);
        pv = q8_page_at(pages, (tile * kTile + 16 * g) >> logP, a.max_pages, a.c.n_pages);
    };
    auto load = [&](int tile, int pk, int pv, TileData<D>& x) {
        const int tk = tile * kTile + 16 * (c >> 2) + (c & 3), tv = tile * kTile + 16 * g;
        const int64_t pgk = (int64_t)max(pk, 0) * a.c.H + h, pgv = (int64_t)max(pv, 0) * a.c.H + h;
        const uint8_t* k = a.c.k + (pgk * P + (tk & (P - 1))) * D + 16 * g;
        const uint8_t* v = a.c.v + (pgv * D + c) * P + (tv & (P - 1));
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int kb = 0; kb < D / 64; ++kb) x.k[mt][kb] = *(const u32x4_t*)(k + 4 * mt * D + 64 * kb);
#pragma unroll
        for (int t = 0; t < D / 16; ++t) x.v[t] = *(const u32x4_t*)(v + 16 * t * P);
        // a page out of range makes the scores that need it NaN; past the sequence's end there is no page
        const bool held = pv >= 0 && tv < len;
        x.ks = held ? a.c.ks[pgv] : nan32();
        x.vs = held ? a.c.vs[pgv] : 1.f;
    };
    uint32_t hidden_nan = 0;
    auto step = [&](int tile, TileData<D>& x) {
        const int tok = tile * kTile + 16 * g;  // the lane's 16 tokens
        const bool edge = tile * kTile + kTile > first_end;
        // scores of the lane's tokens, token tok + 4 mt + i in s[n][mt][i]
        f32x4_t s[NT][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < D / 32; ++st) {
                const u32x4_t w = x.k[mt][st / 2];
                const bf16x8_t k = (st & 1) ? bf16_codes(w[2], w[3]) : bf16_codes(w[0], w[1]);
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][mt] = q[n][st].times(k, s[n][mt]);
            }
        }
        const int ev = (int)(__float_as_uint(x.vs) >> 23) - 127;
        const float bias = (float)max(ev, -90);  // (values under 2^-82: l would overflow on their 1 / v_scale)
        const float small = ev < -90 ? x.vs * 0x1p90f : 1.f;
        const float back = __uint_as_float((uint32_t)(127 - max(ev, -90)) << 23);  // 1 / v_scale
        const float cs = x.ks * y2;
        float top[NT];
        bool move = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            top[n] = -inf32();
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[n][mt][i] = fmaf(s[n][mt][i], cs, bias);
                    top[n] = fmaxf(top[n], s[n][mt][i]);
                }
        }
        if (edge) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                top[n] = -inf32();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (e >= end[n] - tok) s[n][e / 4][e % 4] = -inf32();
                    top[n] = fmaxf(top[n], s[n][e / 4][e % 4]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) move |= top[n] > m[n] + kSlack;
        if (__any(move)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float t = fmaxf(top[n], __shfl_xor(top[n], 16));
                t = fmaxf(t, __shfl_xor(t, 32));
                t = fmaxf(t, m[n]);
                const float keep = __builtin_amdgcn_exp2f(m[n] - t);
                m[n] = t;
                l[n] *= keep;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) o[n][d] *= keep;
            }
        }
        Weights<BF16> w[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float pv[16];
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                pv[e] = __builtin_amdgcn_exp2f(s[n][e / 4][e % 4] - m[n]);
                sum += pv[e];
            }
            l[n] = fmaf(sum, back, l[n]);
            if (__any(ev < -90))
#pragma unroll
                for (int e = 0; e < 16; ++e) pv[e] *= small;
            w[n][0].set(pv);
            w[n][1].set(pv + 8);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (edge) {
            // codes past the sequence's end may be anything: they become zeros, since 0 times NaN is NaN
            const int nv = min(max(len - tok, 0), 16);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int nb = nv - 4 * z;
                const uint32_t keep = nb >= 4 ? 0xFFFFFFFFu : nb <= 0 ? 0u : (1u << (8 * nb)) - 1u;
#pragma unroll
                for (int t = 0; t < D / 16; ++t) {
                    x.v[t][z] &= keep;
                    // and so do NaN codes that some of the rows do not see; put right after the loop
                    if (a.n_q > 1) {
                        const uint32_t bits = nan_codes(x.v[t][z]);
                        hidden_nan |= bits;
                        x.v[t][z] &= ~(bits * 0xFFu);
                    }
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
            const auto v0 = Weights<BF16>::codes(x.v[t][0], x.v[t][1]);
            const auto v1 = Weights<BF16>::codes(x.v[t][2], x.v[t][3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                o[n][t] = w[n][0].times(v0, o[n][t]);
                o[n][t] = w[n][1].times(v1, o[n][t]);
            }
        }
    };

    int tile = split * sp.tps + wave;
    if (tile < t_end) {
        int pk, pv;
        pages_of(tile, pk, pv);
        for (; tile < t_end; tile += kWaves) {
            TileData<D> x;
            load(tile, pk, pv, x);
            pages_of(tile + kWaves, pk, pv);
            step(tile, x);
        }
    }

    // Rows that see a NaN value taken out above: which dims of which rows is the product of where the NaNs are
    // with what the rows see.
    if (__any(hidden_nan != 0)) {
        for (int t1 = split * sp.tps + wave; t1 < t_end; t1 += kWaves) {
            if (t1 * kTile + kTile <= first_end) continue;
            const int tok = t1 * kTile + 16 * g;
            const int pv = tok < len ? q8_page_at(pages, tok >> logP, a.max_pages, a.c.n_pages) : -1;
            const uint8_t* v = a.c.v + (((int64_t)max(pv, 0) * a.c.H + h) * D + c) * P + (tok & (P - 1));
            for (int t = 0; t < D / 16; ++t) {
                u32x4_t is = *(const u32x4_t*)(v + 16 * t * P);
#pragma unroll
                for (int z = 0; z < 4; ++z) is[z] = nan_codes(is[z]) * 0x38u;  // the code of 1
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    f32x4_t hits = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = tok + 8 * half + e < min(end[n], len) ? 1.f : 0.f;
                        Weights<BF16> sees;
                        sees.set(f);
                        hits = sees.times(Weights<BF16>::codes(is[2 * half], is[2 * half + 1]), hits);
                    }
#pragma unroll
                    for (int tt = 0; tt < D / 16; ++tt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (tt == t && hits[i] > 0.f) o[n][tt][i] = nan32();
                }
            }
        }
    }

    // join the waves: a fixed order, so the result does not depend on who is first
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float t = l[n];
        t += __shfl_xor(t, 16);
        t += __shfl_xor(t, 32);
        if (g == 0) {
            s_ml[wave][n * 16 + c][0] = m[n];
            s_ml[wave][n * 16 + c][1] = t;
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) *(f32x4_t*)&s_o[wave][n * 16 + c][16 * d + 4 * g] = o[n][d];
    }
    __syncthreads();
    const int64_t slot = (((int64_t)blockIdx.y * sp.row_blocks + rb) * sp.n_splits + split) * ROWS;
    for (int x = tid; x < ROWS * (D / 4); x += 256) {
        const int row = x / (D / 4), d4 = x % (D / 4) * 4;
        const int r = rb * ROWS + row;
        if (r >= R) continue;
        float top = s_ml[0][row][0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, s_ml[w][row][0]);
        f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
        float lsum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(s_ml[w][row][0] - top);
            sum += f * *(const f32x4_t*)&s_o[w][row][d4];
            lsum = fmaf(f, s_ml[w][row][1], lsum);
        }
        if (bad) lsum = nan32();
        if (live > 1) {
            *(f32x4_t*)(sp.part_o + (slot + row) * D + d4) = sum;
            if (d4 == 0) *(float2*)(sp.part_ml + (slot + row) * 2) = make_float2(top, lsum);
            continue;
        }
        const int i = r / G, hq = h * G + r % G;
        const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
        sum *= inv;
        const int64_t at = (int64_t)b * a.out.seq + (int64_t)hq * a.out.head + (int64_t)i * a.out.token + d4;
        if (BF16)
            *(uint2*)((uint16_t*)a.out.base + at) = make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
        else
            *(f32x4_t*)((float*)a.out.base + at) = sum;
        if (d4 == 0 && a.lse)
            a.lse[((int64_t)b * a.n_q + i) * a.Hq + hq] = lsum == 0.f ? -inf32() : (top + __builtin_amdgcn_logf(lsum)) * kLn2;
    }
}

// The splits of one row joined, in order.  Sequences of one live split have their answer already.
template <bool BF16, int D>
__global__ __launch_bounds__(64) void q8_join_kernel(Q8Attend a, Q8Split sp, int rows) {
    constexpr int PER = D / 64;
    const int G = a.Hq / a.c.H, R = a.n_q * G;
    const int r = blockIdx.x, b = blockIdx.y / a.c.H, h = blockIdx.y % a.c.H, lane = threadIdx.x;
    const int len = a.len[b];
    if (len < 0 || len > a.max_len) return;
    const int live = live_splits(len, sp.tps);
    if (live == 1 || r >= R) return;
    const int64_t slot = (((int64_t)blockIdx.y * sp.row_blocks + r / rows) * sp.n_splits) * rows + r % rows;
    float top = -inf32();
    for (int s = 0; s < live; ++s) top = fmaxf(top, sp.part_ml[(slot + (int64_t)s * rows) * 2]);
    float o[PER], l = 0.f;
#pragma unroll
    for (int p = 0; p < PER; ++p) o[p] = 0.f;
    for (int s = 0; s < live; ++s) {
        const int64_t at = slot + (int64_t)s * rows;
        const float f = __builtin_amdgcn_exp2f(sp.part_ml[at * 2] - top);
        l = fmaf(f, sp.part_ml[at * 2 + 1], l);
#pragma unroll
        for (int p = 0; p < PER; ++p) o[p] = fmaf(f, sp.part_o[at * D + lane * PER + p], o[p]);
    }
    const int i = r / G, hq = h * G + r % G;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = (int64_t)b * a.out.seq + (int64_t)hq * a.out.head + (int64_t)i * a.out.token + lane * PER;
#pragma unroll
    for (int p = 0; p < PER; ++p) o[p] *= inv;
    if (BF16) {
        if (PER == 2) *(uint32_t*)((uint16_t*)a.out.base + at) = pack_bf16(o[0], o[PER - 1]);
        else ((uint16_t*)a.out.base)[at] = (uint16_t)pack_bf16(o[0], 0.f);
    } else {
#pragma unroll
        for (int p = 0; p < PER; ++p) ((float*)a.out.base)[at + p] = o[p];
    }
    if (lane == 0 && a.lse)
        a.lse[((int64_t)b * a.n_q + i) * a.Hq + hq] = l == 0.f ? -inf32() : (top + __builtin_amdgcn_logf(l)) * kLn2;
}

// Row tiles of a workgroup: as many as the rows fill and the registers hold.
int row_tiles(int64_t R, bool bf16, int d) { return R <= 16 ? 1 : R <= 32 || !bf16 || d > 64 ? 2 : 4; }

}  // namespace

Q8Plan q8_attend_plan(Elem e, int B, int n_q, int Hq, int H, int d, int max_len, int cus) {
    Q8Plan p;
    const int64_t R = (int64_t)n_q * (Hq / H);
    p.nt = row_tiles(R, e == Elem::BF16, d);
    p.row_blocks = (int)((R + 16 * p.nt - 1) / (16 * p.nt));
    const int tiles = std::max(1, (max_len + kTile - 1) / kTile);
    const int64_t blocks = (int64_t)B * H * p.row_blocks;
    // a split is worth its join from one step of each wave on; enough of them for a few workgroups a CU
    const int64_t want = std::max<int64_t>(1, kPerCu * (int64_t)cus / blocks);
    p.tps = (int)std::max<int64_t>(kWaves, (tiles + want - 1) / want);
    p.n_splits = (tiles + p.tps - 1) / p.tps;
    return p;
}

// Splits are only made while all workgroups stay within kPerCu * cus: so many blocks of at most 64 rows.
size_t q8_scratch_bytes(int cus) { return (size_t)kPerCu * cus * 64 * (128 + 2) * sizeof(float); }

template <bool BF16, int D>
static hipError_t launch_attend(const Q8Attend& a, const Q8Plan& p, void* scratch, hipStream_t s) {
    const size_t rows = p.n_splits > 1 ? (size_t)a.B * a.c.H * p.row_blocks * p.n_splits * 16 * p.nt : 0;
    const Q8Split sp{p.n_splits, p.tps, p.row_blocks, (float*)scratch, (float*)scratch + rows * D};
    const dim3 grid((unsigned)(p.n_splits * p.row_blocks), (unsigned)(a.B * a.c.H));
    if (p.nt == 1) hipLaunchKernelGGL((q8_decode_kernel<BF16, D, 1>), grid, dim3(256), 0, s, a, sp);
    else if (p.nt == 2) hipLaunchKernelGGL((q8_decode_kernel<BF16, D, 2>), grid, dim3(256), 0, s, a, sp);
    else if constexpr (BF16 && D == 64) hipLaunchKernelGGL((q8_decode_kernel<BF16, D, 4>), grid, dim3(256), 0, s, a, sp);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.n_splits == 1) return e;
    hipLaunchKernelGGL((q8_join_kernel<BF16, D>), dim3((unsigned)(a.n_q * (a.Hq / a.c.H)), (unsigned)(a.B * a.c.H)), dim3(64), 0, s, a,
                       sp, 16 * p.nt);
    return hipGetLastError();
}

hipError_t launch_q8_attend(Elem e, const Q8Attend& a, const Q8Plan& p, void* scratch, hipStream_t s) {
    if (e == Elem::BF16) return a.c.d == 128 ? launch_attend<true, 128>(a, p, scratch, s) : launch_attend<true, 64>(a, p, scratch, s);
    return a.c.d == 128 ? launch_attend<false, 128>(a, p, scratch, s) : launch_attend<false, 64>(a, p, scratch, s);
}

}  // namespace kvmap
