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
// 8 bits to 16: a code is exact in bf16, so scales stay out of the operands: the key's goes into the score, the value's into the
// weight, pv = exp2(y2 + log2 v_scale - m) with m the running maximum of that exponent, and l = sum pv / v_scale, in 64 bits.  bf16
// calls: bf16 queries, weights as two bf16 parts (16 bits).  fp32 calls: queries and weights as three (24 bits).  Parts have fp32's
// exponents, so a weight counts however far below the row's largest it lies; in fp16, 11 bits in one part, weights under 2^-24 are
// gone, and they are the whole answer of a row whose weight lies on tokens with values of zero.  (The second part costs a step of 32,768
// tokens of one sequence 2 %, 21.0 -> 21.5 us, 64 sequences of up to 16,384 1 %, 202.6 -> 204, 4 drafted tokens of 16 sequences of up to
// 5,003 5 %, 19.5 -> 20.6.)
//
// What bounds it: bytes, where there are enough of them.  64 sequences of up to 16,384 tokens, 64 query and 8 KV heads: 1.08 GB
// in 197 us and 5 to join, 5.46 TB/s (a copy of 4 GiB reaches 4.75); 32,768 tokens of one: 67 MB in 18 us and 4 to join.  Below some
// thousand tokens a sequence it is the way through one step: 2,500 cycles until a workgroup knows its piece, 6,000 to 8,500 for
// its item, queries and a tile (900 instructions at 4.5 cycles, and the CU's 64 bytes a cycle), 2,500 to join the
// waves and store: 7.2 us for 130 tokens.

#include <algorithm>

#include "common.h"
#include "internal.h"
#include "q8_mfma.h"
#include "q8_span.h"

namespace kvmap {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = kQ8Step / kWaves;  // tokens of a wave's step

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
constexpr int kOccupancy = BF16 ? (NT == 1 ? 3 : 2) : (NT == 1 ? 2 : 1);

template <bool BF16>
using RowWeights = PartWeights<BF16 ? 2 : 3>;

// Workgroups that a CU holds at once, as the registers (kOccupancy) and the shared memory allow.
__host__ __device__ constexpr int per_cu(bool bf16, int nt) { return bf16 ? (nt == 1 ? 3 : 2) : (nt == 1 ? 2 : 1); }
template <bool BF16, int NT>
constexpr bool kThird = per_cu(BF16, NT) == 3;

// One row and 4 dims of the waves' sums, joined.
template <int ROWS, int LDO>
__device__ __forceinline__ void join_waves(const float (&s_o)[kWaves][ROWS][LDO], const float (&s_ml)[kWaves][ROWS][2], int row, int d4,
                                           float& top, float& lsum, f32x4_t& sum) {
    top = s_ml[0][row][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, s_ml[w][row][0]);
    sum = f32x4_t{0.f, 0.f, 0.f, 0.f};
    lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(s_ml[w][row][0] - top);
        sum += f * *(const f32x4_t*)&s_o[w][row][d4];
        lsum = fmaf(f, s_ml[w][row][1], lsum);
    }
}

// Steps of one item of each of 64 sequences, summed up to and including the lane's (at most 64 * 2^22).
__device__ __forceinline__ uint32_t steps_upto(const Q8Attend& a, int b0, int end, int lane) {
    return wave_scan(b0 + lane < end ? (uint32_t)q8_steps(a.len[b0 + lane], a.max_len) : 0u);
}

template <bool BF16, int D, int NT>
__global__ __launch_bounds__(256, (kOccupancy<BF16, D, NT>)) void q8_decode_kernel(Q8Attend a, Q8Pieces sp) {
    constexpr int ROWS = 16 * NT;
    constexpr int LDO = D + 4;
    __shared__ float s_o[kWaves][ROWS][LDO];
    __shared__ float s_ml[kWaves][ROWS][2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = a.Hq / a.c.H, R = a.n_q * G;
    const int P = a.c.page, logP = 31 - __clz(P);
    const int items = a.c.H;  // of one sequence
    const float y2 = a.scale * kLog2e;

    // this workgroup's piece [at, stop) of the line of steps, and the sequence that it begins in
    uint32_t upto = a.B == 1 ? (uint32_t)q8_steps(a.len[0], a.max_len) : steps_upto(a, 0, a.B, lane);
    uint64_t total = lane_value(upto, 63);
    for (int b0 = 64; b0 < a.B; b0 += 64) total += lane_value(steps_upto(a, b0, a.B, lane), 63);
    total *= items;
    uint64_t share = 1;
    if (total > gridDim.x) {
        share = div64(total + gridDim.x - 1, gridDim.x);
        if (kThird<BF16, NT>) {
            // Of three workgroups a CU the third may go at once: two move 3 % more bytes a second (64 sequences of up to 16,384
            // tokens 204 us, by three 209.5), and the pieces' whole steps may fit better (64 of 1,000: 34 and 40 us; 48 of
            // 1,000: 32 and 29).
            const uint64_t two = gridDim.x - gridDim.x / 3, share2 = div64(total + two - 1, two);
            if (2 * share2 < 3 * share + share / 8) share = share2;
        }
    }
    uint64_t at = share * blockIdx.x;
    const uint64_t stop = at + share < total ? at + share : total;
    if (tid == 255 && sp.cut && !sp.few) sp.cut[blockIdx.x] = make_int2(0, 1);  // (by the thread that may write it again)
    if (at >= stop) return;
    int b = 0;
    uint64_t base = 0;  // the sequence's first step
    if (a.B > 1)
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
            upto = steps_upto(a, b0, a.B, lane);
        }

    while (at < stop) {
        b = __builtin_amdgcn_readfirstlane(b);
        const int len = a.len[b], steps = q8_steps(len, a.max_len);
        const uint64_t next = base + (uint64_t)steps * items;
        if (at >= next) {
            base = next;
            if (++b >= a.B) return;  // (as above)
            continue;
        }
        const bool bad = len < 0 || len > a.max_len;
        const int tiles = bad ? 0 : (len + kTile - 1) / kTile;
        const int h = __builtin_amdgcn_readfirstlane((int)div64(at - base, steps));
        const uint64_t item_at = base + (uint64_t)h * steps;
        const int s_begin = (int)(at - item_at), s_end = (int)min((uint64_t)steps, stop - item_at);
        int x0 = tid;
        asm volatile("" : "+v"(x0));  // keeps products of it with strides from being held across items: registers are full
        const int c = x0 & 15, g = (x0 & 63) >> 4;
        const int t_begin = s_begin * kWaves, t_end = min(tiles, s_end * kWaves);

        const int32_t* pages = a.pages + (int64_t)b * a.max_pages;
        // the pages of the 16 tokens that this lane's key rows and its values come from
        auto pages_of = [&](int tile, int& pk, int& pv) {
            pk = q8_page_at(pages, (tile * kTile + 16 * (c >> 2)) >> logP, a.max_pages, a.c.n_pages);
            pv = q8_page_at(pages, (tile * kTile + 16 * g) >> logP, a.max_pages, a.c.n_pages);
        };
        int tile = t_begin + wave, pk = -1, pv = -1;
        if (tile < t_end) pages_of(tile, pk, pv);  // (on their way while the queries are found)
        __builtin_amdgcn_sched_barrier(0);

        // this lane's rows: their queries, and the tokens that they see
        Query<BF16> q[NT][D / 32];
        int end[NT];
        const int first_end = len - a.n_q + 1;  // the fewest tokens that a row sees
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = n * 16 + c;
            const int i = q8_query(a, r), hq = h * G + r - i * G;
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
            const int ev = scale_exponent(x.vs);
            const float bias = (float)ev;
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
            RowWeights<BF16> w[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float pv[16];
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    pv[e] = __builtin_amdgcn_exp2f(s[n][e / 4][e % 4] - m[n]);
                    sum += pv[e];
                }
                l[n] = fma((double)sum, inverse_scale(ev), l[n]);
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
                const auto v0 = RowWeights<BF16>::codes(x.v[t][0], x.v[t][1]);
                const auto v1 = RowWeights<BF16>::codes(x.v[t][2], x.v[t][3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][t] = w[n][0].times(v0, o[n][t]);
                    o[n][t] = w[n][1].times(v1, o[n][t]);
                }
            }
        };

        for (; tile < t_end; tile += kWaves) {
            TileData<D> x;
            load(tile, pk, pv, x);
            pages_of(tile + kWaves, pk, pv);
            step(tile, x);
        }

        // Rows that see a NaN value taken out above: which dims of which rows is the product of where the NaNs are
        // with what the rows see.
        if (__any(hidden_nan != 0)) {
            for (int t1 = t_begin + wave; t1 < t_end; t1 += kWaves) {
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
                            RowWeights<BF16> sees;
                            sees.set(f);
                            hits = sees.times(RowWeights<BF16>::codes(is[2 * half], is[2 * half + 1]), hits);
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
            for (int d = 0; d < D / 16; ++d) {
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][d][i] = __builtin_amdgcn_ldexpf(o[n][d][i], down);
                *(f32x4_t*)&s_o[wave][n * 16 + c][16 * d + 4 * g] = o[n][d];
            }
        }
        asm volatile("" : "+v"(x0));  // (nor across the loop above)
        if (x0 == 255 && sp.cut && s_begin == 0) {  // (of several items that begin here only the last may be cut)
            const int pieces = (int)div64(item_at + steps - 1, share) - (int)blockIdx.x + 1, id = b * items + h;
            sp.cut[sp.few ? id : (int)blockIdx.x] = make_int2(sp.few ? (int)blockIdx.x : id, pieces);
        }
        __syncthreads();
        const int rows = min(ROWS, R);
        if (s_begin > 0 || s_end < steps) {
            const int64_t slot = q8_slot(blockIdx.x, s_begin == 0) * ROWS;
            for (int x = x0; x < rows * (D / 4); x += 256) {
                const int row = x / (D / 4), d4 = x % (D / 4) * 4;
                float top, lsum;
                f32x4_t sum;
                join_waves<ROWS, LDO>(s_o, s_ml, row, d4, top, lsum, sum);
                *(f32x4_t*)(sp.part_o + (slot + row) * D + d4) = sum;
                if (d4 == 0) *(float2*)(sp.part_ml + (slot + row) * 2) = make_float2(top, lsum);
            }
        } else {
            for (int x = x0; x < rows * (D / 4); x += 256) {
                const int row = x / (D / 4), d4 = x % (D / 4) * 4;
                float top, lsum;
                f32x4_t sum;
                join_waves<ROWS, LDO>(s_o, s_ml, row, d4, top, lsum, sum);
                if (bad) lsum = nan32();
                const int i = q8_query(a, row);
                q8_store_row<BF16>(a, b, i, h * G + row - i * G, d4, top, lsum, sum);
            }
        }
        at = item_at + s_end;
        __syncthreads();  // the next item's sums come into the same memory
    }
}

}  // namespace

Q8Plan q8_attend_plan(Elem e, int B, int n_q, int Hq, int H, int d, int max_len, int cus) {
    Q8Plan p = q8_prompt_plan(e, B, n_q, Hq, H, d, max_len, cus);
    if (p.rows) return p;
    const int64_t R = (int64_t)n_q * (Hq / H);
    const int nt = R <= 16 ? 1 : 2;  // 16-row tiles of a workgroup (q8_prompt.hip takes more than 32 rows)
    p.rows = 16 * nt;
    p.row_blocks = 1;
    // a workgroup for every step that the lengths can bring, up to what the chip holds at once
    const double steps = (double)B * H * q8_steps(max_len, max_len);
    p.grid = (int)std::min<double>((double)per_cu(e == Elem::BF16, nt) * cus, steps);
    p.splits = p.grid > 1 && q8_steps(max_len, max_len) > 1;  // (items of one step are never cut)
    return p;
}

size_t q8_scratch_bytes(int cus) {
    // the most rows of all workgroups together: 256 a CU (q8_prompt.hip); the most workgroups: 3 a CU
    return q8_piece_bytes(3 * cus, 0, 128) + q8_piece_bytes(cus, 256, 128);
}

template <bool BF16, int D>
static hipError_t launch_decode(const Q8Attend& a, const Q8Pieces& sp, hipStream_t s) {
    const dim3 grid((unsigned)sp.grid);
    if (sp.rows == 16) hipLaunchKernelGGL((q8_decode_kernel<BF16, D, 1>), grid, dim3(256), 0, s, a, sp);
    else hipLaunchKernelGGL((q8_decode_kernel<BF16, D, 2>), grid, dim3(256), 0, s, a, sp);
    return hipGetLastError();
}

hipError_t launch_q8_attend(Elem e, const Q8Attend& a, const Q8Plan& p, void* scratch, hipStream_t s) {
    const Q8Pieces sp = q8_pieces(a, p, scratch);
    hipError_t r;
    if (p.prompt) r = launch_q8_prompt(e, a, sp, s);
    else if (e == Elem::BF16) r = a.c.d == 128 ? launch_decode<true, 128>(a, sp, s) : launch_decode<true, 64>(a, sp, s);
    else r = a.c.d == 128 ? launch_decode<false, 128>(a, sp, s) : launch_decode<false, 64>(a, sp, s);
    return r == hipSuccess && p.splits ? launch_q8_join(e, a, sp, s) : r;
}

}  // namespace kvmap
