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
// O^T's dims.  They are chosen so that nothing crosses lanes: with g = lane >> 4, row 4 g' + j of S^T's tile m is token
// 8 g' + 4 m + j, so that lane group g ends up with the tokens 8 g .. 8 g + 7 of its row; and row c of O^T's tile
// (half, j) is dim 64 half + 4 c + j, so that a lane reads 4 adjacent dims of each of those 8 tokens.  For bf16 products
// (16x16x32) the 8 tokens of a dim are brought side by side by byte permutes; fp32 products (16x16x4) take a token at
// a time and need none.  No shared memory and no barrier in the loop.
//
// bf16 calls: weights as two bf16 parts (16 bits, fp32's exponents: a weight counts however far below the row's largest
// it lies), queries that were turned as three (24 bits, what their turn in fp32 has).  fp32 calls:
// products of fp32 operands.  Sums and statistics in fp32, a row's sum of weights in fp64.

#include <algorithm>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "q8_mfma.h"
#include "q8_span.h"

namespace kvmap {
namespace {

constexpr int kTile = kPagedStep / kWaves;  // tokens of a wave's step
static_assert(kTile == 32, "the tiles' token order");

// A row's queries as operands of S^T, and a tile's keys: 16 bytes of a token's dims a step.
template <bool BF16, int D, bool TURN>
struct Queries;

template <int D, bool TURN>
struct Queries<true, D, TURN> {
    static constexpr int STEPS = D / 32;  // step s contracts dims 32 s + 8 g .. + 8
    static constexpr int N = TURN ? 3 : 1;
    Parts<N> p[STEPS];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int k = 0; k < N; ++k) p[s].p[k] = bf16x8_t{};
    }
    // row: the query's first element; tab: its position's cosines and sines
    __device__ __forceinline__ void load(const void* row, int g, const float2* tab) {
        const __bf16* at = (const __bf16*)row + 8 * g;
        if (!TURN) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) p[s].p[0] = *(const bf16x8_t*)(at + 32 * s);
            return;
        }
#pragma unroll
        for (int s = 0; s < STEPS / 2; ++s) {
            const bf16x8_t lo = *(const bf16x8_t*)(at + 32 * s), hi = *(const bf16x8_t*)(at + 32 * s + D / 2);
            float a[8], b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 t = tab[32 * s + 8 * g + e];
                const float x = (float)lo[e], y = (float)hi[e];
                a[e] = fmaf(-y, t.y, x * t.x);
                b[e] = fmaf(x, t.y, y * t.x);
            }
            p[s].set(a);
            p[s + STEPS / 2].set(b);
        }
    }
    __device__ __forceinline__ f32x4_t times(const u32x4_t (&k)[STEPS]) const {
        f32x4_t s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int st = 0; st < STEPS; ++st)
#pragma unroll
            for (int n = N; n--;) s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, k[st]), p[st].p[n], s, 0, 0, 0);
        return s;
    }
};

template <int D, bool TURN>
struct Queries<false, D, TURN> {
    static constexpr int STEPS = D / 16;  // step s contracts dims 16 s + 4 g .. + 4
    f32x4_t p[STEPS];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) p[s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    __device__ __forceinline__ void load(const void* row, int g, const float2* tab) {
        const float* at = (const float*)row + 4 * g;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) p[s] = *(const f32x4_t*)(at + 16 * s);
        if (!TURN) return;
#pragma unroll
        for (int s = 0; s < STEPS / 2; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 t = tab[16 * s + 4 * g + e];
                const float x = p[s][e], y = p[s + STEPS / 2][e];
                p[s][e] = fmaf(-y, t.y, x * t.x);
                p[s + STEPS / 2][e] = fmaf(x, t.y, y * t.x);
            }
    }
    __device__ __forceinline__ f32x4_t times(const u32x4_t (&k)[STEPS]) const {
        f32x4_t s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int st = 0; st < STEPS; ++st)
#pragma unroll
            for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[st][e]), p[st][e], s, 0, 0, 0);
        return s;
    }
};

// The weights of a lane's 8 tokens.  In bf16 as two parts, the first cut off, so that the second is not negative, and not
// zero where the weight is not: then an infinity that a row sees is one in its sum, and no 0 times it.
struct SplitWeights {
    bf16x8_t hi, lo;
    __device__ __forceinline__ void set(const float* x) {
        u32x4_t h, l;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float r[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float w = x[2 * i + k];
                r[k] = fmaxf(w - __uint_as_float(__float_as_uint(w) & 0xFFFF0000u), fminf(w, 0x1p-126f));
            }
            h[i] = __builtin_amdgcn_perm(__float_as_uint(x[2 * i + 1]), __float_as_uint(x[2 * i]), 0x07060302u);
            l[i] = pack_bf16(r[0], r[1]);
        }
        hi = __builtin_bit_cast(bf16x8_t, h);
        lo = __builtin_bit_cast(bf16x8_t, l);
    }
    __device__ __forceinline__ f32x4_t times(bf16x8_t v, f32x4_t o) const {
        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, lo, o, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, hi, o, 0, 0, 0);
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
    uint2 v[8][D / 64];
    __device__ __forceinline__ void load(const char* at, int row) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) v[e][h] = *(const uint2*)(at + e * row + 128 * h);
    }
    __device__ __forceinline__ void keep(int e, bool yes) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            v[e][h].x = yes ? v[e][h].x : 0u;
            v[e][h].y = yes ? v[e][h].y : 0u;
        }
    }
    __device__ __forceinline__ bool finite(int e) const {
        bool ok = true;
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
            for (uint32_t w : {v[e][h].x, v[e][h].y}) ok &= (w & 0x7F80u) != 0x7F80u && (w & 0x7F800000u) != 0x7F800000u;
        return ok;
    }
    // dim 64 half + 4 c + j of the 8 tokens
    __device__ __forceinline__ bf16x8_t dim(int half, int j) const {
        u32x4_t w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t a = j & 2 ? v[2 * e][half].y : v[2 * e][half].x, b = j & 2 ? v[2 * e + 1][half].y : v[2 * e + 1][half].x;
            w[e] = __builtin_amdgcn_perm(b, a, j & 1 ? 0x07060302u : 0x05040100u);
        }
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
    __device__ __forceinline__ void load(const char* at, int row) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) v[e][h] = *(const f32x4_t*)(at + e * row + 256 * h);
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

// Workgroups that a CU holds at once, as the registers and the shared memory allow.
__host__ __device__ constexpr int per_cu(bool bf16, int nt, bool turn) { return bf16 ? (nt == 1 ? (turn ? 2 : 3) : (turn ? 1 : 2)) : (nt == 1 ? 2 : 1); }

// Steps of one item of each of 64 sequences, summed up to and including the lane's.
__device__ __forceinline__ uint32_t steps_upto(const Q8Attend& a, int b0, int lane) {
    return wave_scan(b0 + lane < a.B ? (uint32_t)paged_steps(a.len[b0 + lane], a.max_len) : 0u);
}

template <bool BF16, int D, int NT, bool TURN>
__global__ __launch_bounds__(256, (per_cu(BF16, NT, TURN))) void paged_decode_kernel(Q8Attend a, Rotation rot, Q8Pieces sp) {
    constexpr int ROWS = 16 * NT, ES = BF16 ? 2 : 4, LDO = D + 4;
    typedef Queries<BF16, D, TURN> Q;
    typedef Values<BF16, D> V;
    typedef RowWeights<BF16> Weights;
    __shared__ float s_o[kWaves][ROWS][LDO];
    __shared__ float s_ml[kWaves][ROWS][2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int H = a.c.H, G = a.Hq / H, R = a.n_q * G;
    const int P = a.c.page, logP = 31 - __clz(P);
    const int items = H * sp.row_blocks;  // of one sequence
    const float y2 = a.scale * kLog2e;
    const bool cuts = sp.cut != nullptr;

    // Where items may be cut: this workgroup's piece [at, stop) of the line of steps, and the sequence that it begins in.
    // Else whole items, one after the other.
    uint64_t at = blockIdx.x, stop = (uint64_t)a.B * items, share = 1, base = 0;
    int b = 0;
    if (cuts) {
        uint32_t upto = steps_upto(a, 0, lane);
        uint64_t total = lane_value(upto, 63);
        for (int b0 = 64; b0 < a.B; b0 += 64) total += lane_value(steps_upto(a, b0, lane), 63);
        total *= items;
        share = div64(total + gridDim.x - 1, gridDim.x);
        at = share * blockIdx.x;
        stop = at + share < total ? at + share : total;
        if (tid == 255 && !sp.few) sp.cut[blockIdx.x] = make_int2(0, 1);  // (by the thread that may write it again)
        if (at >= stop) return;
        for (int b0 = 0;;) {
            const uint64_t past = __ballot(base + (uint64_t)upto * items > at);
            if (past) {
                const int n = __ffsll((unsigned long long)past) - 1;
                b = b0 + n;
                if (n) base += (uint64_t)lane_value(upto, n - 1) * items;
                break;
            }
            base += (uint64_t)lane_value(upto, 63) * items;
            b0 += 64;
            if (b0 >= a.B) return;  // (not reached while the lengths stay as they were summed)
            upto = steps_upto(a, b0, lane);
        }
    }

    while (at < stop) {
        int item, steps, s_begin = 0, s_end;  // the item of sequence b, and its steps that are this workgroup's
        uint64_t item_at = 0;
        if (cuts) {
            b = __builtin_amdgcn_readfirstlane(b);
            steps = paged_steps(a.len[b], a.max_len);
            const uint64_t next = base + (uint64_t)steps * items;
            if (at >= next) {
                base = next;
                if (++b >= a.B) return;  // (as above)
                continue;
            }
            item = (int)div64(at - base, steps);
            item_at = base + (uint64_t)item * steps;
            s_begin = (int)(at - item_at);
            s_end = (int)min((uint64_t)steps, stop - item_at);
        } else {
            b = __builtin_amdgcn_readfirstlane((int)((uint32_t)at / (uint32_t)items));
            item = (int)((uint32_t)at - (uint32_t)b * (uint32_t)items);
            s_end = steps = paged_steps(a.len[b], a.max_len);
        }
        item = __builtin_amdgcn_readfirstlane(item);
        const int len = a.len[b];
        const bool bad = len < 0 || len > a.max_len;
        const int tiles = bad ? 0 : (len + kTile - 1) / kTile;
        const int h = item / sp.row_blocks, rb = item - h * sp.row_blocks;
        const int t_begin = s_begin * kWaves, t_end = min(tiles, s_end * kWaves);

        const int32_t* pages = a.pages + (int64_t)b * a.max_pages;
        // the pages of a tile's first and last 16 tokens
        auto page_of = [&](int tile, int half) { return q8_page_at(pages, (int64_t)(tile * kTile + 16 * half) >> logP, a.max_pages, a.c.n_pages); };
        int tile = t_begin + wave;
        int p0 = -1, p1 = -1;
        if (tile < t_end) p0 = page_of(tile, 0), p1 = page_of(tile, 1);

        // this lane's rows: their queries, and the tokens that they see
        Q q[NT];
        int end[NT];
        const int first_end = len - a.n_q + 1;  // the fewest tokens that a row sees
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = rb * ROWS + n * 16 + c;
            const int i = q8_query(a, r);
            end[n] = first_end + i;
            const int pos = first_end + i - 1;
            if (r < R && pos >= 0 && !bad) {
                const int hq = h * G + r - i * G;
                q[n].load((const char*)a.q.base + ((int64_t)b * a.q.seq + (int64_t)hq * a.q.head + (int64_t)i * a.q.token) * ES, g,
                          TURN ? rot.tab + (int64_t)pos * (D / 2) : nullptr);
            } else {
                q[n].zero();
            }
        }
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

        // A tile's scores y of the lane's tokens tok .. tok + 8, and where their values are.
        auto scores = [&](int t0, int p0, int p1, float (&y)[NT][8], V& v, const char*& va) {
            u32x4_t k[2][Q::STEPS];
            const int tk = t0 + 8 * (c >> 2) + (c & 3), tok = t0 + 8 * g;
            const int pk = (c >> 2) & 2 ? p1 : p0, pv = g & 2 ? p1 : p0;
            const char* ka = (const char*)a.c.k + ((((int64_t)max(pk, 0) * H + h) * P + (tk & (P - 1))) * D) * ES + 16 * g;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int s = 0; s < Q::STEPS; ++s) k[mt][s] = *(const u32x4_t*)(ka + 4 * mt * D * ES + 64 * s);
            va = (const char*)a.c.v + ((((int64_t)max(pv, 0) * H + h) * P + (tok & (P - 1))) * D + 4 * c) * ES;
            v.load(va, D * ES);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    const f32x4_t s = q[n].times(k[mt]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[n][4 * mt + i] = s[i] * y2;
                }
            if ((p0 | p1) < 0) {  // a page out of range
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[n][e] = pv < 0 ? nan32() : y[n][e];
            }
            if (t0 + kTile > first_end) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[n][e] = tok + e < min(end[n], len) ? y[n][e] : -inf32();
            }
        };
        bool apart = false;
        for (; tile < t_end; tile += kWaves) {
            const int t0 = tile * kTile, tok = t0 + 8 * g;
            float y[NT][8], top[NT];
            V v;
            const char* va;
            const int at0 = p0, at1 = p1;
            if (tile + kWaves < t_end) p0 = page_of(tile + kWaves, 0), p1 = page_of(tile + kWaves, 1);
            scores(t0, at0, at1, y, v, va);
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
                bool odd = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) odd |= tok + e >= first_end && tok + e < len && !v.finite(e);
                const bool later = __any(odd);
                apart |= later;
#pragma unroll
                for (int e = 0; e < 8; ++e) v.keep(e, tok + e < len && !later);
            }
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n) o[n][t] = v.times(t >> 2, t & 3, w[n], o[n][t]);
        }
        if (apart) {
            for (int t1 = t_begin + wave; t1 < t_end; t1 += kWaves) {
                const int t0 = t1 * kTile, tok = t0 + 8 * g;
                if (t0 + kTile <= first_end) continue;
                float y[NT][8];
                V v;
                const char* va;
                scores(t0, page_of(t1, 0), page_of(t1, 1), y, v, va);
                bool odd = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) odd |= tok + e >= first_end && tok + e < len && !v.finite(e);
                if (!__any(odd)) continue;
                Weights w[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[n][e] = __builtin_amdgcn_exp2f(y[n][e] - m[n]);
                    w[n].set(y[n]);
                }
                for (int hf = 0; hf < D / 64; ++hf) {
                    Values<BF16, 64> x;
                    x.load(va + 64 * ES * hf, D * ES);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            f32x4_t before = o[n][j], sum;
#pragma unroll
                            for (int i = 0; i < 4; ++i) sum[i] = before[i] = hf ? o[n][D / 16 - 4 + j][i] : before[i];
#pragma unroll 1
                            for (int upto = first_end; upto <= len; ++upto) {
                                const f32x4_t by = x.times_first(0, j, upto - tok, w[n], before);
#pragma unroll
                                for (int i = 0; i < 4; ++i) sum[i] = end[n] == upto ? by[i] : sum[i];
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                o[n][j][i] = hf ? o[n][j][i] : sum[i];
                                o[n][D / 16 - 4 + j][i] = hf == D / 64 - 1 ? sum[i] : o[n][D / 16 - 4 + j][i];
                            }
                        }
                }
            }
        }

        // join the waves: a fixed order, so the result does not depend on who is first
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            double t = l[n];
            t += __shfl_xor(t, 16);
            t += __shfl_xor(t, 32);
            float lf;
            const int down = settle_sum(t, m[n], lf);
            if (g == 0) {
                s_ml[wave][n * 16 + c][0] = m[n];
                s_ml[wave][n * 16 + c][1] = lf;
            }
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4_t x;
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = __builtin_amdgcn_ldexpf(o[n][4 * hf + j][i], down);
                    *(f32x4_t*)&s_o[wave][n * 16 + c][64 * hf + 16 * g + 4 * i] = x;
                }
        }
        if (tid == 255 && cuts && s_begin == 0) {  // (of several items that begin here only the last may be cut)
            const int pieces = (int)div64(item_at + steps - 1, share) - (int)blockIdx.x + 1, id = b * items + item;
            sp.cut[sp.few ? id : (int)blockIdx.x] = make_int2(sp.few ? (int)blockIdx.x : id, pieces);
        }
        __syncthreads();
        const int rows = min(ROWS, R - rb * ROWS);
        const bool part = s_begin > 0 || s_end < steps;
        const int64_t slot = q8_slot(blockIdx.x, s_begin == 0) * ROWS;
        for (int x = tid; x < rows * (D / 4); x += 256) {
            const int row = x / (D / 4), d4 = x % (D / 4) * 4;
            float top, lsum;
            f32x4_t sum;
            join_waves<ROWS, LDO>(s_o, s_ml, row, d4, top, lsum, sum);
            if (part) {
                *(f32x4_t*)(sp.part_o + (slot + row) * D + d4) = sum;
                if (d4 == 0) *(float2*)(sp.part_ml + (slot + row) * 2) = make_float2(top, lsum);
            } else {
                if (bad) lsum = nan32();
                const int r = rb * ROWS + row, i = q8_query(a, r);
                q8_store_row<BF16>(a, b, i, h * G + r - i * G, d4, top, lsum, sum);
            }
        }
        at = cuts ? item_at + s_end : at + gridDim.x;
        __syncthreads();  // the next item's sums come into the same memory
    }
}

}  // namespace

// Sequences of at most this many steps are never cut: a workgroup's further steps cost less than the joining kernel.
constexpr int kWhole = 4;

Q8Plan paged_attend_plan(Elem e, int B, int n_q, int Hq, int H, int max_len, bool turn, int cus) {
    Q8Plan p{};
    const int64_t R = (int64_t)n_q * (Hq / H);
    const int nt = R <= 16 ? 1 : 2;  // 16-row tiles of a workgroup
    p.rows = 16 * nt;
    p.row_blocks = (int)((R + p.rows - 1) / p.rows);
    const double items = (double)B * H * p.row_blocks;
    const int steps = paged_steps(max_len, max_len);
    p.splits = steps > kWhole;
    // a workgroup for every step that the lengths can bring, up to what the chip holds at once
    p.grid = (int)std::min<double>((double)per_cu(e == Elem::BF16, nt, turn) * cus, p.splits ? items * steps : items);
    return p;
}

template <bool BF16, int D, bool TURN>
static hipError_t launch_decode(const Q8Attend& a, const Rotation& rot, const Q8Pieces& sp, hipStream_t s) {
    const dim3 grid((unsigned)sp.grid);
    if (sp.rows == 16) hipLaunchKernelGGL((paged_decode_kernel<BF16, D, 1, TURN>), grid, dim3(256), 0, s, a, rot, sp);
    else hipLaunchKernelGGL((paged_decode_kernel<BF16, D, 2, TURN>), grid, dim3(256), 0, s, a, rot, sp);
    return hipGetLastError();
}

hipError_t launch_paged_attend(Elem e, const Q8Attend& a, const Rotation& rot, const Q8Plan& p, void* scratch, hipStream_t s) {
    const Q8Pieces sp = q8_pieces(a, p, scratch);
    const bool bf16 = e == Elem::BF16, wide = a.c.d == 128;
    hipError_t r;
    if (rot.tab) {
        if (bf16) r = wide ? launch_decode<true, 128, true>(a, rot, sp, s) : launch_decode<true, 64, true>(a, rot, sp, s);
        else r = wide ? launch_decode<false, 128, true>(a, rot, sp, s) : launch_decode<false, 64, true>(a, rot, sp, s);
    } else {
        if (bf16) r = wide ? launch_decode<true, 128, false>(a, rot, sp, s) : launch_decode<true, 64, false>(a, rot, sp, s);
        else r = wide ? launch_decode<false, 128, false>(a, rot, sp, s) : launch_decode<false, 64, false>(a, rot, sp, s);
    }
    return r == hipSuccess && p.splits ? launch_q8_join(e, a, sp, s) : r;
}

}  // namespace kvmap
