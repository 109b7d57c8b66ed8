// Attention of the last tokens of every sequence over the paged cache in the model's own type.
//
// For query row i of sequence b at position pos = len - n_q + i, with y_t = scale * q' . k_t, t <= pos:
//   lse = log sum exp y_t,   out = sum exp(y_t - lse) v_t,
// q' being q, or q turned at its position where the call has a table.  One pass over the tokens with a running
// maximum m and sum l; the query heads that share a KV head (G of them) and the n_q queries of a sequence are the
// rows of one problem, row r = i * G + g, so up to 32 rows read the cache once.
//
// A wave of 64 lanes takes 32 tokens x 16 rows a tile, transposed so that a row of the softmax is a column of the
// tiles (lane & 15) everywhere:
//   S^T = K Q^T   16 tokens x 16 rows, twice   -> lane holds 4 tokens of one row
//   O^T = V^T P^T 16 dims x 16 rows            -> lane holds 4 dims of one row
// The order of a contraction is free as long as both operands share it, and so are the orders of S^T's tokens and of
// O^T's dims.  They are chosen so that no score crosses lanes: with g = lane >> 4, row 4 g' + j of S^T's tile m is token
// 8 g' + 4 m + j, so that lane group g ends up with the tokens 8 g .. 8 g + 7 of its row; and row c of O^T's tile
// (half, j) is dim 64 half + 4 c + j, so that a lane reads 4 adjacent dims of each of those 8 tokens.  For bf16 products
// (16x16x32) the 8 tokens of a dim are brought side by side by byte permutes; fp32 products (16x16x4) take a token at
// a time and need none.  No shared memory and no barrier in the loop but for the low parts of turned queries.
//
// bf16 calls: weights as three bf16 parts (24 bits and the exponents of fp32, which they come in), queries that were turned as
// three too (what their turn in fp32 has).  fp32 calls: products of fp32 operands.  Sums and statistics in fp32, a row's sum of
// weights in fp64.
//
// What bounds it: bytes, where there are enough of them.  Keys and values are read once, past the caches and by whole lines of
// 128 bytes (but fp32 keys), a tile's 16 KB at a time by each of 8 waves a CU: 64 sequences of 8,192 tokens, 8 KV heads, 2.15 GB in
// 338 to 347 us by card, 6.2 to 6.35 TB/s (loads alone in the same pattern 6.8), one of 32,768 134 MB in 27 and 4 to join.  Asking
// for a tile's keys and values while the one before is multiplied was slower, 61 us for 56 on 8 sequences of 8,192.  Below some
// thousand tokens a sequence it is the way through one step: lengths, pages, keys, the tile's products and the joining of the waves
// one after the other, 7.4 us for 130 tokens.  Pieces are joined by a second kernel: by the last piece to come, through memory past
// the caches, it took 58 us for 38 on one sequence of 32,768 tokens and 63 for 61 on 8 of 8,192.

#include <algorithm>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "q8_mfma.h"
#include "q8_span.h"

namespace kvmap {
namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;  // tokens of a wave's step

// The upper 16 bits of two fp32 numbers side by side: the first bf16 parts that their remainders follow.
__device__ __forceinline__ uint32_t upper_halves(float x0, float x1) {
    return __builtin_amdgcn_perm(__float_as_uint(x1), __float_as_uint(x0), 0x07060302u);
}
// What x has beyond its upper 16 bits, of x's sign.
__device__ __forceinline__ float beyond_half(float x) { return x - __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }

// A turned query's 8 elements as three parts of 8 bits, each cut off, so that all have the element's sign, and raised by 2^-30 and 2^-40
// of it, so that none is zero where the element is not (from 2^-86 on): then a key's infinity times the element is the same one
// in every part's product, and the score has it.
struct SplitQuery {
    u32x4_t p[3];
    __device__ __forceinline__ void set(const float* x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x0 = x[2 * i], x1 = x[2 * i + 1];
            const float y0 = fmaf(x0, 0x1p-30f, beyond_half(x0)), y1 = fmaf(x1, 0x1p-30f, beyond_half(x1));
            const float z0 = fmaf(x0, 0x1p-40f, beyond_half(y0)), z1 = fmaf(x1, 0x1p-40f, beyond_half(y1));
            p[0][i] = upper_halves(x0, x1);
            p[1][i] = upper_halves(y0, y1);
            p[2][i] = upper_halves(z0, z1);
        }
    }
};

// A row's queries as operands of S^T.  load() asks for what ready() makes them of; low: the lane's place in shared memory for
// the second and third parts of turned bf16 queries (N row tiles side by side), which all waves share; OWN: they are in registers.
template <bool BF16, int D, bool TURN, bool OWN>
struct Queries;

template <int D, bool TURN, bool OWN>
struct Queries<true, D, TURN, OWN> {
    static constexpr int STEPS = D / 32;  // step s contracts dims 32 s + 8 g .. + 8
    bf16x8_t p[STEPS];
    u32x4_t own[TURN && OWN ? 2 * STEPS : 1];
    f32x4_t t[TURN ? STEPS * 2 : 1];
    // row: the query's first element; tab: its position's cosines and sines
    __device__ __forceinline__ void load(const void* row, int g, const float2* tab) {
        const __bf16* at = (const __bf16*)row + 8 * g;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) p[s] = *(const bf16x8_t*)(at + 32 * s);
        if (TURN)
#pragma unroll
            for (int s = 0; s < STEPS / 2; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) t[4 * s + e] = *(const f32x4_t*)(tab + 32 * s + 8 * g + 2 * e);
    }
    template <int N>
    __device__ __forceinline__ void ready(u32x4_t* low, bool write) {
        if (!TURN) return;
#pragma unroll
        for (int s = 0; s < STEPS / 2; ++s) {
            float a[8], b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = (float)p[s][e], y = (float)p[s + STEPS / 2][e];
                const float cs = t[4 * s + e / 2][2 * (e & 1)], sn = t[4 * s + e / 2][2 * (e & 1) + 1];
                a[e] = fmaf(-y, sn, x * cs);
                b[e] = fmaf(x, sn, y * cs);
            }
            SplitQuery lo, hi;
            lo.set(a);
            hi.set(b);
            p[s] = __builtin_bit_cast(bf16x8_t, lo.p[0]);
            p[s + STEPS / 2] = __builtin_bit_cast(bf16x8_t, hi.p[0]);
            if (OWN)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    own[k * STEPS + s] = lo.p[1 + k];
                    own[k * STEPS + s + STEPS / 2] = hi.p[1 + k];
                }
            else if (write)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    low[(k * STEPS + s) * N * 64] = lo.p[1 + k];
                    low[(k * STEPS + s + STEPS / 2) * N * 64] = hi.p[1 + k];
                }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // s0, s1 += step st of two tiles of keys
    template <int N>
    __device__ __forceinline__ void times(const u32x4_t (&k)[2], int st, const u32x4_t* low, f32x4_t& s0, f32x4_t& s1) const {
        const bf16x8_t x0 = __builtin_bit_cast(bf16x8_t, k[0]), x1 = __builtin_bit_cast(bf16x8_t, k[1]);
        if (TURN)
#pragma unroll
            for (int part = 1; part >= 0; --part) {
                const bf16x8_t y = __builtin_bit_cast(bf16x8_t, OWN ? own[part * STEPS + st] : low[(part * STEPS + st) * N * 64]);
                s0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x0, y, s0, 0, 0, 0);
                s1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x1, y, s1, 0, 0, 0);
            }
        s0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x0, p[st], s0, 0, 0, 0);
        s1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x1, p[st], s1, 0, 0, 0);
    }
};

template <int D, bool TURN, bool OWN>
struct Queries<false, D, TURN, OWN> {
    static constexpr int STEPS = D / 16;  // step s contracts dims 16 s + 4 g .. + 4
    f32x4_t p[STEPS];
    f32x4_t t[TURN ? STEPS : 1];
    __device__ __forceinline__ void load(const void* row, int g, const float2* tab) {
        const float* at = (const float*)row + 4 * g;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) p[s] = *(const f32x4_t*)(at + 16 * s);
        if (TURN)
#pragma unroll
            for (int s = 0; s < STEPS / 2; ++s)
#pragma unroll
                for (int e = 0; e < 2; ++e) t[2 * s + e] = *(const f32x4_t*)(tab + 16 * s + 4 * g + 2 * e);
    }
    template <int N>
    __device__ __forceinline__ void ready(u32x4_t*, bool) {
        if (!TURN) return;
#pragma unroll
        for (int s = 0; s < STEPS / 2; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = p[s][e], y = p[s + STEPS / 2][e];
                const float cs = t[2 * s + e / 2][2 * (e & 1)], sn = t[2 * s + e / 2][2 * (e & 1) + 1];
                p[s][e] = fmaf(-y, sn, x * cs);
                p[s + STEPS / 2][e] = fmaf(x, sn, y * cs);
            }
    }
    template <int N>
    __device__ __forceinline__ void times(const u32x4_t (&k)[2], int st, const u32x4_t*, f32x4_t& s0, f32x4_t& s1) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s0 = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[0][e]), p[st][e], s0, 0, 0, 0);
            s1 = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[1][e]), p[st][e], s1, 0, 0, 0);
        }
    }
};

template <bool STREAM, class T>
__device__ __forceinline__ T fetch(const T* p) { return STREAM ? __builtin_nontemporal_load(p) : *p; }

// A tile's keys, as operands of S^T: step st of tile mt is bytes 64 st + 16 g of row c.  at0, at1: where the lane's rows of
// the tile's first and last 16 tokens are.
template <bool BF16, int D>
struct Keys;

// bf16: a load brings whole lines of 128 bytes, of 8 tokens: lane (c, g) gets bytes 64 (c >> 3) + 16 g of the lines of row
// (c & 7) + 8 j, and lanes 8 apart change halves.
template <int D>
struct Keys<true, D> {
    static constexpr int LINES = D / 64, STEPS = 2 * LINES;
    u32x4_t k[2][2][LINES];  // [mt][j][line]
    __device__ static __forceinline__ int token(int c) { return 8 * ((c >> 2) & 1) + (c & 3); }
    __device__ static __forceinline__ int byte(int c, int g) { return 64 * (c >> 3) + 16 * g; }
    template <bool STREAM>
    __device__ __forceinline__ void load(const char* at0, const char* at1) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int l = 0; l < LINES; ++l) k[mt][j][l] = fetch<STREAM>((const u32x4_t*)((j ? at1 : at0) + 4 * mt * D * 2 + 128 * l));
    }
    __device__ __forceinline__ u32x4_t step(int mt, int st) const {
        const u32x4_t a = k[mt][0][st >> 1], b = k[mt][1][st >> 1];
        u32x4_t x;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = st & 1 ? (uint32_t)__builtin_amdgcn_update_dpp((int)b[i], (int)a[i], 0x128, 0xF, 0x3, false)
                          : (uint32_t)__builtin_amdgcn_update_dpp((int)a[i], (int)b[i], 0x128, 0xF, 0xC, false);
        return x;
    }
};

// fp32: half a line of 16 tokens a load, as the product wants them, and through the caches, where the next load finds the other half (past
// them 64 sequences of 8,192 tokens take 730 us for 676, 8 of 8,192 104 for 108, 4 of up to 7,091 19.1 for 19.9).
template <int D>
struct Keys<false, D> {
    static constexpr int STEPS = D / 16;
    u32x4_t k[2][STEPS];
    __device__ static __forceinline__ int token(int c) { return 8 * ((c >> 2) & 1) + (c & 3); }
    __device__ static __forceinline__ int byte(int, int g) { return 16 * g; }
    template <bool STREAM>
    __device__ __forceinline__ void load(const char* at0, const char* at1) {
        const char* at = threadIdx.x & 8 ? at1 : at0;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int s = 0; s < STEPS; ++s) k[mt][s] = *(const u32x4_t*)(at + 4 * mt * D * 4 + 64 * s);
    }
    __device__ __forceinline__ u32x4_t step(int mt, int st) const { return k[mt][st]; }
};

// The weights of a lane's 8 tokens.  In bf16 as three parts of 8 bits, each cut off, so that they hold all that fp32 does, none is
// negative, and none is zero where the weight is not: then an infinity that a row sees is one in its sum, and no 0 times it.
// (Where the weight is not zero itself, nor a factor that it meets later, as m grows and in the joins: each is a power of 2 by m's
// difference to a larger m.  A score is never more than kSlack over its m, and the largest m at most 1 over lse, in base 2: weights of
// 2^-110 of the row's sum and more stay.)
// (Two parts, 16 bits: where a row's values nearly cancel, outputs were up to 490 steps of bf16 off, for 21 now and 102 of the
// formula in 32-bit torch calls, on 64 sequences of up to 16,384 tokens.  The third is 1 to 3 % of the time of 1 to 4 tokens, 4 drafted ones of
// 64 sequences of up to 900 in 37.2 us for 36.0, and 6 to 9 % of 16, of 16 sequences of up to 8,192 in 173 for 161.)
struct SplitWeights {
    bf16x8_t p[3];
    __device__ __forceinline__ void set(const float* x) {
        u32x4_t w[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float r0 = x[2 * i], r1 = x[2 * i + 1];
            const float least0 = fminf(r0, 0x1p-126f), least1 = fminf(r1, 0x1p-126f);
            w[0][i] = upper_halves(r0, r1);
#pragma unroll
            for (int k = 1; k < 3; ++k) {
                r0 = fmaxf(beyond_half(r0), least0);
                r1 = fmaxf(beyond_half(r1), least1);
                w[k][i] = upper_halves(r0, r1);
            }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) p[k] = __builtin_bit_cast(bf16x8_t, w[k]);
    }
    __device__ __forceinline__ f32x4_t times(bf16x8_t v, f32x4_t o) const {
#pragma unroll
        for (int k = 3; k--;) o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[k], o, 0, 0, 0);
        return o;
    }
};
struct WholeWeights {
    float p[8];
    __device__ __forceinline__ void set(const float* x) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = x[e];
    }
};
template <bool BF16>
using RowWeights = std::conditional_t<BF16, SplitWeights, WholeWeights>;

// The values of a lane's 8 tokens, dims 64 half + 4 c .. + 4 of each, as operands of O^T; `row` bytes from token to token.
template <bool BF16, int D>
struct Values;

template <int D>
struct Values<true, D> {
    typedef RowWeights<true> Weights;
    u32x2_t v[8][D / 64];
    template <bool STREAM>
    __device__ __forceinline__ void load(const char* at, int row) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) v[e][h] = fetch<STREAM>((const u32x2_t*)(at + e * row + 128 * h));
    }
    __device__ __forceinline__ void keep(int e, bool yes) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) v[e][h][i] = yes ? v[e][h][i] : 0u;
    }
    __device__ __forceinline__ bool finite(int e) const {
        bool ok = true;
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) ok &= (v[e][h][i] & 0x7F80u) != 0x7F80u && (v[e][h][i] & 0x7F800000u) != 0x7F800000u;
        return ok;
    }
    // dim 64 half + 4 c + j of the 8 tokens
    __device__ __forceinline__ bf16x8_t dim(int half, int j) const {
        u32x4_t w;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = __builtin_amdgcn_perm(v[2 * e + 1][half][j >> 1], v[2 * e][half][j >> 1], j & 1 ? 0x07060302u : 0x05040100u);
        return __builtin_bit_cast(bf16x8_t, w);
    }
    __device__ __forceinline__ f32x4_t times(int half, int j, const Weights& w, f32x4_t o) const { return w.times(dim(half, j), o); }
    // with the first `count` tokens alone, whatever the others hold
    __device__ __forceinline__ f32x4_t times_first(int half, int j, int count, const Weights& w, f32x4_t o) const {
        u32x4_t x = __builtin_bit_cast(u32x4_t, dim(half, j));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] &= count >= 2 * e + 2 ? 0xFFFFFFFFu : count == 2 * e + 1 ? 0xFFFFu : 0u;
        return w.times(__builtin_bit_cast(bf16x8_t, x), o);
    }
};

template <int D>
struct Values<false, D> {
    typedef RowWeights<false> Weights;
    f32x4_t v[8][D / 64];
    template <bool STREAM>
    __device__ __forceinline__ void load(const char* at, int row) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) v[e][h] = fetch<STREAM>((const f32x4_t*)(at + e * row + 256 * h));
    }
    __device__ __forceinline__ void keep(int e, bool yes) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[e][h][j] = yes ? v[e][h][j] : 0.f;
    }
    __device__ __forceinline__ bool finite(int e) const {
        bool ok = true;
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) ok &= (__float_as_uint(v[e][h][j]) & 0x7F800000u) != 0x7F800000u;
        return ok;
    }
    __device__ __forceinline__ f32x4_t times(int half, int j, const Weights& w, f32x4_t o) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) o = __builtin_amdgcn_mfma_f32_16x16x4f32(v[e][half][j], w.p[e], o, 0, 0, 0);
        return o;
    }
    __device__ __forceinline__ f32x4_t times_first(int half, int j, int count, const Weights& w, f32x4_t o) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) o = __builtin_amdgcn_mfma_f32_16x16x4f32(e < count ? v[e][half][j] : 0.f, w.p[e], o, 0, 0, 0);
        return o;
    }
};

// Whether one of the tokens from .. to of a lane's 8 has values that are not finite.
template <class V>
__device__ __forceinline__ bool odd(const V& v, int from, int to) {
    bool any = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) any |= e >= from && e < to && !v.finite(e);
    return any;
}

// One value at an address that all lanes share and no workgroup writes, through the scalar cache.
template <class T>
__device__ __forceinline__ T uniform(const T* p) {
    typedef const T __attribute__((address_space(4))) * constant_ptr;
    return *(constant_ptr)(uintptr_t)p;
}

// Waves that a SIMD holds at once, as the registers allow.  bf16 rows of 128 dims in one 16-row tile, and of 64 dims in two, would fit three
// times, but steps divide better by two, and two have enough in flight.  The first: 64 sequences of 8,192 tokens 347 us, three 367, one of
// 32,768 30.6 and 34.5.  The second, 4 drafted tokens, 8 heads, G 8: 8 sequences of 8,192 36 us, three 42, one of 32,768 22 and 28, 16 of
// up to 16,384 67 and 72 (but 16 of up to 5,003 with 4 heads 25.0 and 24.1, 32 of up to 3,000 27.9 and 25.7).  fp32 spills three times.
__host__ __device__ constexpr int per_simd(bool bf16, int d, int nt) {
    if (d == 64) return nt == 2 ? 2 : 4;
    return nt == 2 && !bf16 ? 1 : 2;
}
// Waves of a workgroup.  (8 in one workgroup a CU: 24.1 us for 25.0 on 4 drafted tokens of 16 sequences of up to 5,003, 4 heads of 64 dims, but
// 29 for 22 on 9 of 20 of up to 900, 207 for 173 on 16 of 16 of up to 8,192, 8 heads of 128 dims, G 8, and 12.5 for 11.4 on one of 4,096.)
constexpr int kGroup = 4;

// Steps of one item of each of 64 sequences, summed up to and including the lane's.
__device__ __forceinline__ uint32_t steps_upto(const Q8Attend& a, int b0, int step, int lane) {
    return wave_scan(b0 + lane < a.B ? (uint32_t)steps_of(a.len[b0 + lane], a.max_len, step) : 0u);
}

template <bool BF16, int D, int NT, bool TURN, bool STREAM>
__global__ __launch_bounds__(64 * kGroup, (per_simd(BF16, D, NT))) void paged_decode_kernel(Q8Attend a, Rotation rot, Q8Pieces sp) {
    constexpr int W = kGroup, ROWS = 16 * NT, ES = BF16 ? 2 : 4, LDO = D + 4, THREADS = 64 * W, STEP = kTile * W;
    constexpr bool SHARES = BF16 && TURN && NT > 1;
    constexpr int LOW = SHARES ? 2 * (D / 32) * NT * 64 : 1;
    typedef Queries<BF16, D, TURN, !SHARES> Q;
    typedef Values<BF16, D> V;
    typedef RowWeights<BF16> Weights;
    static_assert(LOW * sizeof(u32x4_t) <= W * ROWS * LDO * sizeof(float), "the queries' parts lie where the sums come later");
    __shared__ __attribute__((aligned(16))) float s_o[W][ROWS][LDO];
    __shared__ float s_ml[W][ROWS][2];
    u32x4_t* const s_low = (u32x4_t*)&s_o[0][0][0];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int H = a.c.H, G = a.Hq / H, R = a.n_q * G;
    const int P = a.c.page, logP = 31 - __clz(P);
    const int rbs = sp.row_blocks;
    const float y2 = a.scale * kLog2e;
    const bool cuts = sp.cut != nullptr;
    const int lane0 = threadIdx.x & 63;
    // Where items may be cut: this workgroup's piece [at, stop) of the line of steps of all (sequence, KV head), the sequence that
    // it begins in, and its block of rows: the blocks of a piece are neighbours, and find what they share in the caches.
    // Else one whole item.
    const int pieces = gridDim.x / rbs;
    uint64_t stop = 0, share = 1, base = 0;
    uint32_t upto = 0, used = gridDim.x;
    int b = 0;
    if (cuts) {
        upto = steps_upto(a, 0, STEP, lane0);
        uint64_t total = lane_value(upto, 63);
        for (int b0 = 64; b0 < a.B; b0 += 64) total += lane_value(steps_upto(a, b0, STEP, lane0), 63);
        stop = total *= H;
        share = div64(total + pieces - 1, pieces);
        used = (uint32_t)div64(total + share - 1, share) * rbs;
        if (blockIdx.x >= used) {  // a piece of nothing
            const int j = blockIdx.x - used;
            if (threadIdx.x == 0 && !sp.few) sp.cut[j % rbs * pieces + used / rbs + j / rbs] = make_int2(0, 1);
            return;
        }
    }
    // neighbours on one XCD (workgroups go round the 8 XCDs), so that the heads of a page meet in its caches
    const uint32_t xcd = blockIdx.x % 8, place = xcd * (used / 8) + min(xcd, used % 8) + blockIdx.x / 8;
    const int rb = place % rbs, piece = rb * pieces + place / rbs;  // (pieces of one block of rows are numbered in order)
    uint64_t at = share * (place / rbs);
    if (cuts) {
        stop = min(stop, at + share);
        if (threadIdx.x == THREADS - 1 && !sp.few) sp.cut[piece] = make_int2(0, 1);  // (by the thread that may write it again)
        for (int b0 = 0;;) {
            const uint64_t past = __ballot(base + (uint64_t)upto * H > at);
            if (past) {
                const int n = __ffsll((unsigned long long)past) - 1;
                b = b0 + n;
                if (n) base += (uint64_t)lane_value(upto, n - 1) * H;
                break;
            }
            base += (uint64_t)lane_value(upto, 63) * H;
            b0 += 64;
            if (b0 >= a.B) return;  // (not reached while the lengths stay as they were summed)
            upto = steps_upto(a, b0, STEP, lane0);
        }
    } else {
        b = (int)at / H;
        stop = at + 1;
    }

    while (at < stop) {
        int h, steps, s_begin = 0, s_end;  // the head of sequence b, and its steps that are this workgroup's
        uint64_t item_at = at;
        b = __builtin_amdgcn_readfirstlane(b);
        const int len = uniform(a.len + b);
        steps = steps_of(len, a.max_len, STEP);
        if (cuts) {
            const uint64_t next = base + (uint64_t)steps * H;
            if (at >= next) {
                base = next;
                if (++b >= a.B) return;  // (as above)
                continue;
            }
            h = (int)div64(at - base, steps);
            item_at = base + (uint64_t)h * steps;
            s_begin = (int)(at - item_at);
            s_end = (int)min((uint64_t)steps, stop - item_at);
        } else {
            h = (int)at - b * H;
            s_end = steps;
        }
        h = __builtin_amdgcn_readfirstlane(h);
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));  // keeps products of it with strides from being held across items: registers are full
        const int lane = tid & 63, c = lane & 15, g = lane >> 4;
        const bool bad = len < 0 || len > a.max_len;
        const int tiles = bad ? 0 : (len + kTile - 1) / kTile;
        const int t_begin = s_begin * W, t_end = min(tiles, s_end * W);

        const int32_t* pages = a.pages + (int64_t)b * a.max_pages;
        // the pages of a tile's first and last 16 tokens
        auto page_of = [&](int tile, int half) {
            const int slot = (int)((int64_t)(tile * kTile + 16 * half) >> logP);
            if (slot >= a.max_pages) return -1;
            const int page = uniform(pages + slot);
            return page >= 0 && page < a.c.n_pages ? page : -1;
        };
        int tile = t_begin + wave;
        int p0 = page_of(tile, 0), p1 = page_of(tile, 1), n0 = -1, n1 = -1;  // of the tile in hand, and of the next one

        // this lane's rows: their queries, and the tokens that they see
        Q q[NT];
        int end[NT];
        const int first_end = len - a.n_q + 1;  // the fewest tokens that a row sees
        auto load_query = [&](auto& to, int n) {
            const int r = min(rb * ROWS + n * 16 + c, R - 1);  // (rows past the last are not stored)
            const int i = q8_query(a, r), hq = h * G + r - i * G;
            end[n] = first_end + i;
            const int pos = bad ? 0 : max(end[n] - 1, 0);
            to.load((const char*)a.q.base + ((int64_t)b * a.q.seq + (int64_t)hq * a.q.head + (int64_t)i * a.q.token) * ES, g,
                    TURN ? rot.tab + (int64_t)pos * (D / 2) : nullptr);
        };
#pragma unroll
        for (int n = 0; n < NT; ++n) load_query(q[n], n);
        // A tile's keys and values.  A lane's 8 tokens of values lie in one page, which has whole 16 tokens, and so do the rows of
        // keys of one load.  What one workgroup alone reads is read past the caches (STREAM).
        Keys<BF16, D> k;
        V v;
        const char* kbase = (const char*)a.c.k + Keys<BF16, D>::byte(c, g);
        auto load_keys = [&](int t0, int p0, int p1) {
            const int tk = t0 + Keys<BF16, D>::token(c);
            k.template load<STREAM>(kbase + ((((int64_t)max(p0, 0) * H + h) * P + (tk & (P - 1))) * D) * ES,
                                    kbase + ((((int64_t)max(p1, 0) * H + h) * P + ((tk + 16) & (P - 1))) * D) * ES);
        };
        auto values_at = [&](int t0, int p0, int p1) {
            const int tv = t0 + 8 * g, pv = g & 2 ? p1 : p0;
            return (const char*)a.c.v + ((((int64_t)max(pv, 0) * H + h) * P + (tv & (P - 1))) * D + 4 * c) * ES;
        };
        if (tile + W < t_end) n0 = page_of(tile + W, 0), n1 = page_of(tile + W, 1);
#pragma unroll
        for (int n = 0; n < NT; ++n) q[n].template ready<NT>(s_low + n * 64 + lane, wave == 0);
        if (SHARES) __syncthreads();
        int low = lane;

        f32x4_t o[NT][D / 16];
        float m[NT];
        double l[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = kNone;
            l[n] = 0.0;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[n][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        // A tile's scores y of the lane's tokens tok .. tok + 8.
        auto scores = [&](const auto& q, int t0, int p0, int p1, float (&y)[NT][8]) {
            const int tok = t0 + 8 * g;
            if (SHARES) asm volatile("" : "+v"(low));  // keeps the low parts where they are: registers are full
            f32x4_t s[2][NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) s[0][n] = s[1][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < Keys<BF16, D>::STEPS; ++st) {
                const u32x4_t x[2] = {k.step(0, st), k.step(1, st)};
#pragma unroll
                for (int n = 0; n < NT; ++n) q[n].template times<NT>(x, st, s_low + low + n * 64, s[0][n], s[1][n]);
                if (SHARES) __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[n][4 * mt + i] = s[mt][n][i] * y2;
            if ((p0 | p1) < 0) {  // a page out of range
                const bool lost = (g & 2 ? p1 : p0) < 0;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[n][e] = lost ? nan32() : y[n][e];
            }
            if (t0 + kTile > first_end) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[n][e] = tok + e < min(end[n], len) ? y[n][e] : -inf32();
            }
        };
        bool apart = false;
        for (; tile < t_end; tile += W) {
            const int t0 = tile * kTile, tok = t0 + 8 * g;
            float y[NT][8], top[NT];
            load_keys(t0, p0, p1);
            v.template load<STREAM>(values_at(t0, p0, p1), D * ES);
            scores(q, t0, p0, p1, y);
            bool move = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                top[n] = y[n][0];
#pragma unroll
                for (int e = 1; e < 8; ++e) top[n] = fmaxf(top[n], y[n][e]);
                move |= top[n] > m[n] + kSlack;
            }
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
            Weights w[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[n][e] = __builtin_amdgcn_exp2f(y[n][e] - m[n]);
                    sum += y[n][e];
                }
                l[n] += (double)sum;
                w[n].set(y[n]);
            }
            if (t0 + kTile > first_end) {
                // Values past the sequence's end may be anything: they become zeros, since 0 times NaN is NaN.  Where one
                // that only some of the rows see is not finite, the tile is multiplied after the loop, query by query.
                const bool later = __any(odd(v, first_end - tok, len - tok));
                apart |= later;
#pragma unroll
                for (int e = 0; e < 8; ++e) v.keep(e, tok + e < len && !later);
            }
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n) o[n][t] = v.times(t >> 2, t & 3, w[n], o[n][t]);
            p0 = n0, p1 = n1;
            if (tile + 2 * W < t_end) n0 = page_of(tile + 2 * W, 0), n1 = page_of(tile + 2 * W, 1);
        }
        if (SHARES) __syncthreads();  // the parts of the queries have been read
        // join the waves: a fixed order, so the result does not depend on who is first
        asm volatile("" : "+v"(tid));  // (nor across the loop above)
        const int row0 = tid & 15, dim0 = (tid & 63) >> 4 << 4;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            double t = l[n];
            t += __shfl_xor(t, 16);
            t += __shfl_xor(t, 32);
            float lf;
            const int down = settle_sum(t, m[n], lf);
            if (dim0 == 0) {
                s_ml[wave][n * 16 + row0][0] = m[n];
                s_ml[wave][n * 16 + row0][1] = lf;
            }
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4_t x;
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = __builtin_amdgcn_ldexpf(o[n][4 * hf + j][i], down);
                    *(f32x4_t*)&s_o[wave][n * 16 + row0][64 * hf + dim0 + 4 * i] = x;
                }
        }
        if (apart) {
            // The tiles left out above, query by query, each with what it sees, onto the wave's sums where they are now.  (The
            // queries once more: registers are free, and their parts are overwritten.)
            Queries<BF16, D, TURN, true> again[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                load_query(again[n], n);
                again[n].template ready<NT>(nullptr, false);
            }
            for (int t1 = t_begin + wave; t1 < t_end; t1 += W) {
                const int t0 = t1 * kTile, tok = t0 + 8 * g;
                if (t0 + kTile <= first_end) continue;
                p0 = page_of(t1, 0), p1 = page_of(t1, 1);
                const char* va = values_at(t0, p0, p1);
                v.template load<false>(va, D * ES);
                if (!__any(odd(v, first_end - tok, len - tok))) continue;
                load_keys(t0, p0, p1);
                float y[NT][8];
                scores(again, t0, p0, p1, y);
                Weights w[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[n][e] = __builtin_amdgcn_exp2f(y[n][e] - m[n]);
                    w[n].set(y[n]);
                }
                for (int upto = first_end; upto <= len; ++upto)
#pragma unroll
                    for (int t = 0; t < D / 16; ++t)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const f32x4_t by = v.times_first(t >> 2, t & 3, upto - tok, w[n], f32x4_t{0.f, 0.f, 0.f, 0.f});
                            float* to = &s_o[wave][n * 16 + row0][64 * (t >> 2) + dim0 + (t & 3)];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (end[n] == upto) to[4 * i] += by[i];
                        }
            }
        }
        if (tid == THREADS - 1 && cuts && s_begin == 0) {  // (of several items that begin here only the last may be cut)
            const int n = (int)div64(item_at + steps - 1, share) - place / rbs + 1, id = (b * H + h) * rbs + rb;
            sp.cut[sp.few ? id : piece] = make_int2(sp.few ? piece : id, n);
        }
        __syncthreads();
        const int rows = min(ROWS, R - rb * ROWS);
        const bool part = s_begin > 0 || s_end < steps;
        const int64_t slot = q8_slot(piece, s_begin == 0) * ROWS;
        for (int x = tid; x < rows * (D / 4); x += THREADS) {
            const int row = x / (D / 4), d4 = x % (D / 4) * 4;
            float top, lsum;
            f32x4_t sum;
            join_waves<W, ROWS, LDO>(s_o, s_ml, row, d4, top, lsum, sum);
            if (part) {
                *(f32x4_t*)(sp.part_o + (slot + row) * D + d4) = sum;
                if (d4 == 0) *(float2*)(sp.part_ml + (slot + row) * 2) = make_float2(top, lsum);
            } else {
                if (bad) lsum = nan32();
                const int r = rb * ROWS + row, i = q8_query(a, r);
                q8_store_row<BF16>(a, b, i, h * G + r - i * G, d4, top, lsum, sum);
            }
        }
        at = item_at + s_end;
        __syncthreads();  // the next item's sums come into the same memory
    }
}

}  // namespace

// Items of sequences of at most this many tokens are not cut, each a workgroup's that the chip takes up as others end: where there
// are few of them a workgroup's second step costs less than the joining kernel (130 tokens of one sequence 7.2 us, cut 9.1; 512:
// 14.7, cut 10.0); with one for every CU (32 sequences of 1,000, 8 heads: 28 us, cut 33); with one for every workgroup
// that the chip holds (128 of 1,500: 133, cut 144; 64 of up to 1,400: 42 and 48; with 256 items for 512 places, fp32: 37 and 28).
constexpr int kWhole = 256, kFull = 1024, kMany = 2048;

// Workgroups that the chip holds at once.
static int held_at_once(bool bf16, int d, int nt, int cus) { return 4 * per_simd(bf16, d, nt) / kGroup * cus; }

// The most that a plan below leaves for the join: a piece of every workgroup that the chip holds.
size_t paged_scratch_bytes(int cus) {
    size_t most = 0;
    for (bool bf16 : {false, true})
        for (int d : {64, 128})
            for (int nt : {1, 2}) most = std::max(most, q8_piece_bytes(held_at_once(bf16, d, nt, cus), 16 * nt, d));
    return most;
}

Q8Plan paged_attend_plan(Elem e, int B, int n_q, int Hq, int H, int d, int max_len, int cus) {
    Q8Plan p{};
    const bool bf16 = e == Elem::BF16;
    const int64_t R = (int64_t)n_q * (Hq / H);
    const int nt = R <= 16 ? 1 : 2;  // 16-row tiles of a workgroup
    p.rows = 16 * nt;
    p.row_blocks = (int)((R + p.rows - 1) / p.rows);
    const double items = (double)B * H * p.row_blocks;
    const int steps = steps_of(max_len, max_len, kTile * kGroup), held = held_at_once(bf16, d, nt, cus);
    p.splits = max_len > (items < cus ? kWhole : items < held ? kFull : kMany) && held / p.row_blocks > 1;
    // cut: a workgroup for every step that the lengths can bring, up to what the chip holds at once; else one for every item
    p.grid = p.splits ? (int)std::min<double>(held / p.row_blocks, (double)B * H * steps) * p.row_blocks : (int)items;
    return p;
}

template <bool BF16, int D, int NT, bool TURN>
static hipError_t launch_decode(const Q8Attend& a, const Rotation& rot, const Q8Pieces& sp, const Q8Plan& p, hipStream_t s) {
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)p.grid), dim3(64 * kGroup), 0, s, a, rot, sp); };
    if constexpr (NT == 2)
        if (p.row_blocks > 1) {
            go(paged_decode_kernel<BF16, D, NT, TURN, false>);
            return hipGetLastError();
        }
    go(paged_decode_kernel<BF16, D, NT, TURN, true>);
    return hipGetLastError();
}

template <bool BF16, int D>
static hipError_t launch_of(const Q8Attend& a, const Rotation& rot, const Q8Pieces& sp, const Q8Plan& p, hipStream_t s) {
    if (rot.tab) return p.rows == 16 ? launch_decode<BF16, D, 1, true>(a, rot, sp, p, s) : launch_decode<BF16, D, 2, true>(a, rot, sp, p, s);
    return p.rows == 16 ? launch_decode<BF16, D, 1, false>(a, rot, sp, p, s) : launch_decode<BF16, D, 2, false>(a, rot, sp, p, s);
}

hipError_t launch_paged_attend(Elem e, const Q8Attend& a, const Rotation& rot, const Q8Plan& p, void* scratch, hipStream_t s) {
    const Q8Pieces sp = q8_pieces(a, p, scratch);
    hipError_t r;
    if (e == Elem::BF16) r = a.c.d == 128 ? launch_of<true, 128>(a, rot, sp, p, s) : launch_of<true, 64>(a, rot, sp, p, s);
    else r = a.c.d == 128 ? launch_of<false, 128>(a, rot, sp, p, s) : launch_of<false, 64>(a, rot, sp, p, s);
    return r == hipSuccess && p.splits ? launch_q8_join(e, a, sp, s) : r;
}

}  // namespace kvmap
