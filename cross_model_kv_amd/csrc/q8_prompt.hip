// Attention over the 8-bit paged cache for many rows: prompts (the mathematics is q8_attend.hip's).
//
// A workgroup of 8 waves holds 256 rows of one sequence and KV head (row r = i * G + g, query i, head g), a wave 32 of them, and
// walks the tokens in tiles of 64.  A tile's codes are turned to 16 bits once for the workgroup, on their way into
// shared memory, and every wave reads all of it as the left operand:
//   S^T = K Q^T   A = 32 tokens x 16 dims,  B = 16 dims x 32 rows   (32x32x16 tiles; queries stay in registers)
//   O^T = V^T P^T A = 32 dims x 16 tokens,  B = 16 tokens x 32 rows
// Row m of S^T's 32 tokens is token (m & 3) + 4 (m >> 3) + 16 (m >> 2 & 1), so that a lane's 16 scores of a row
// are 16 adjacent tokens, which is what P^T's operand wants of it: nothing crosses lanes, and the 16
// tokens lie in one page, with one scale.
//
// What bounds it: a tile costs a SIMD (64 rows) 2050 cycles of matrix products, 2350 of issuing vector instructions
// (these among them) and takes 4140; the clock meanwhile falls to 1.6 - 1.8 GHz: 1.10 - 1.20 ms by card for 8,192 rows a head,
// 8 heads and 33,792 tokens (930 - 1015 TFLOP/s, against 1430 - 1550 of large library products here).  Waves of 64 rows, one a SIMD,
// read half as much shared memory but cannot issue fast enough (an instruction every 5 cycles, 580 of them a tile): the same
// time within 3 %.  Products next to the vector work in the order in which they are written, not the compiler's, took waves
// of 64 rows from 1470 us to 1220 - 1300.

#include <algorithm>
#include <utility>

#include "common.h"
#include "internal.h"
#include "q8_mfma.h"
#include "q8_span.h"

namespace kvmap {
namespace {

// f(integral_constant<0>), .., f(integral_constant<N - 1>): unrolled whatever f's body looks like.
template <int... I, class F>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F&& f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
    each(std::make_integer_sequence<int, N>{}, f);
}

constexpr int kTile = 64;

// The weights of bf16 calls are fp16, 2^(y - m): 11 bits from 2^-14 to 2^kTop, fewer below, one at 2^-24.  A row may have nearly all
// of its weight on a few tokens whose values are zero, and is made of the others then, however far below those they lie.  So m
// follows the scores up and down, and what fp16 does not hold is not lost: where the largest weight of 16 adjacent tokens is not
// inside 2^kDrop .. 2^kTop, or that of 4 is below 2^kThin, rows that do not fit move their m, and where it is not enough, what the
// rounding takes of the half tile's weights below 2^-14 is multiplied on its own, 2^38 times as large (11 bits down to 2^-52).  So
// a weight is off by 2^-11 of the largest of 16 adjacent ones at most, and by 2^-8 of itself next to the row's own token.  (With m
// at the largest score and no more than that, a row that had 0.9999 of its weight on one token lost all of its answer.)  Looking for
// it costs 1 to 2 % of a call (1,024 queries on 33,792 tokens 1,107 -> 1,118 us).  Where scores have a deviation of 2 or 3 nats, as there,
// it is needed in hardly any half; by 4 the call takes a sixth longer, by 6 more than twice as long: a row then reaches further
// than fp16 does.
constexpr float kTop = 15.f, kDrop = -14.f, kThin = -24.f;
// m is put so far below the largest score of a half: by the item's first half and where it moves down; where it moves up (no more than it
// has to, for the tokens before); and where it moves down and the half's scores reach further than from there to 2^kThin.
constexpr float kFirst = 5.f, kUp = 13.f, kWide = 11.f;
constexpr float kEdge = -17.f;  // 8 bits: where a row does not see all of a half, which may be few tokens, of every weight that it sees
constexpr float kCalm = -8.f;  // rows whose largest weight is below this move along when others move: each on its own costs more
constexpr float kDeep = 60.f;  // m at most this far below where it has been: 2^60 times 2^15 times 2^30 tokens' codes stays finite
#define STEP() __builtin_amdgcn_sched_barrier(0)

// Tokens that the last row of a row block sees, and its tiles: one at least, so that its rows are answered.
__device__ __forceinline__ int block_end(const Q8Attend& a, int G, int len, int rb, int bm) {
    const int last = min((rb + 1) * bm, a.n_q * G) - 1;
    return len - a.n_q + q8_query(a, last) + 1;
}
__device__ __forceinline__ int block_tiles(const Q8Attend& a, int G, int len, int rb, int bm) {
    if (len < 1 || len > a.max_len) return 1;
    const int end = block_end(a, G, len, rb, bm);
    return end < 1 ? 1 : (end - 1) / kTile + 1;
}
// An item costs as much as its tiles and kItemCost more: page table, queries, first tiles, answers.  (Counted as its tiles
// alone, 333 queries of 3 heads in 4 sequences, one of them empty, took 209 us instead of 73.)
template <bool BF16>
constexpr int kItemCost = BF16 ? 5 : 2;

// Cost of all row blocks of one head: of sequence b0 + lane (0 past the last), lanes going over the sequences or over the row
// blocks, whichever is fewer rounds.
__device__ __forceinline__ uint64_t head_cost(const Q8Attend& a, int G, int b0, int row_blocks, int bm, int extra, int lane) {
    uint64_t sum = 0;
    const int n = min(a.B - b0, 64);
    if (n * ((row_blocks + 63) / 64) < row_blocks) {
        for (int i = 0; i < n; ++i) {
            const int len = a.len[b0 + i];
            uint64_t s = 0;
            for (int r0 = 0; r0 < row_blocks; r0 += 64)
                s += lane_value(wave_scan<uint32_t>(r0 + lane < row_blocks ? block_tiles(a, G, len, r0 + lane, bm) + extra : 0), 63);
            if (i == lane) sum = s;
        }
    } else if (lane < n) {
        const int len = a.len[b0 + lane];
        for (int rb = 0; rb < row_blocks; ++rb) sum += block_tiles(a, G, len, rb, bm) + extra;
    }
    return sum;
}

// An item, and where it lies in the line.
struct Item {
    int b, h, rb, cost;
    uint64_t at;
};
// The line's length; `first` is what head_cost gives for the first 64 sequences.  Every lane of the wave alike.
__device__ __forceinline__ uint64_t line_length(const Q8Attend& a, int G, int row_blocks, int bm, int extra, int lane, uint64_t first) {
    uint64_t total = lane_value(wave_scan(first), 63);
    for (int b0 = 64; b0 < a.B; b0 += 64) total += lane_value(wave_scan(head_cost(a, G, b0, row_blocks, bm, extra, lane)), 63);
    return total * a.c.H;
}
// The item that holds the line's unit u (less than its length).
__device__ __forceinline__ Item find_item(const Q8Attend& a, int G, int row_blocks, int bm, int extra, int lane, uint64_t first, uint64_t u) {
    Item it;
    uint64_t base = 0, mine = first;
    int b0 = 0;
    while (true) {
        const uint64_t upto = wave_scan(mine) * a.c.H;
        const uint64_t past = __ballot(base + upto > u);
        const int n = past ? __ffsll((unsigned long long)past) - 1 : 63;
        it.b = min(b0 + n, a.B - 1);  // (past is not 0 in the end, while the lengths stay as they were summed)
        if (past || b0 + 64 >= a.B) {
            mine = lane_value(mine, n);
            base += lane_value(upto, n) - mine * a.c.H;
            break;
        }
        base += lane_value(upto, 63);
        b0 += 64;
        mine = head_cost(a, G, b0, row_blocks, bm, extra, lane);
    }
    it.h = min((int)div64(u - base, max(mine, (uint64_t)1)), a.c.H - 1);
    base += (uint64_t)it.h * mine;
    const int len = a.len[it.b];
    for (int r0 = 0;; r0 += 64) {
        const uint32_t cost = r0 + lane < row_blocks ? block_tiles(a, G, len, r0 + lane, bm) + extra : 0;
        const uint32_t upto = wave_scan(cost);
        const uint64_t past = __ballot(base + upto > u);
        if (past || r0 + 64 >= row_blocks) {
            const int n = past ? __ffsll((unsigned long long)past) - 1 : row_blocks - 1 - r0;
            it.rb = r0 + n;
            it.cost = (int)lane_value(cost, n);
            it.at = base + lane_value(upto, n) - it.cost;
            return it;
        }
        base += lane_value(upto, 63);
    }
}

// The lane, computed where it is wanted: registers are full, and the compiler would hold it, and its products with strides,
// across loops.
__device__ __forceinline__ int fresh_lane() {
    int lane;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(lane));
    return lane;
}

// The larger, and the smaller, of two or three.  Written out they stay where they are written, and the compiler does not put an
// instruction in front of each that makes its operands quiet.
__device__ __forceinline__ float max2(float a, float b) {
    float r;
    asm volatile("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm volatile("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float min2(float a, float b) {
    float r;
    asm volatile("v_min_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm volatile("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// What the wave's lanes have written to shared memory is there for its other lanes.
__device__ __forceinline__ void wave_memory() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Workgroups that a CU holds at once.  bf16 with 128 dims: one of 8 waves, or two of 4, which have shared memory for two tiles of
// keys each, not three, and so a barrier more a tile.  (One of 4 waves and three tiles: 64 rows of 8 sequences of 8,192 tokens 66 us
// for 61.5, of one of 32,768 38 for 37.)
template <bool BF16, int D, int WAVES>
constexpr int kPerCu = D == 64 || (BF16 && WAVES == 4) ? 2 : 1;

template <bool BF16, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, (kPerCu<BF16, D, WAVES> * WAVES / 4)) void q8_prompt_kernel(Q8Attend a, Q8Pieces sp) {
    constexpr int BM = 32 * WAVES;             // rows of a workgroup
    constexpr int KROW = 2 * D + 16;           // bytes of a token's keys in shared memory: the 16 spread the banks
    constexpr int KBYTES = kTile * KROW;
    constexpr int VROW = 2 * kTile + 16;       // bytes of a dim's tokens
    constexpr int THREADS = 64 * WAVES;
    constexpr int NC = D * kTile / 16 / THREADS;  // 16-byte loads of a thread for a tile's keys, and for its values
    constexpr int NQ = D / 8, NV = D / 8;      // operands of a tile: keys, values
    constexpr int AHEAD = 3;
    constexpr int CPT = D / 16;                // such loads of a token's keys
    constexpr int RING = D == 128 && kPerCu<BF16, D, WAVES> == 2 ? 2 : 3;  // tiles of keys
    __shared__ __align__(16) uint8_t s_k[RING * KBYTES + 2 * D * VROW];
    uint8_t* const s_v = s_k + RING * KBYTES;
    __shared__ int s_nan;                      // some value was taken out
    __shared__ float2 s_scale[4][4];           // k_scale, v_scale of 16 tokens each; a tile's are written with its keys
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int G = a.Hq / a.c.H, R = a.n_q * G;
    const int P = a.c.page, logP = 31 - __clz(P);
    const float y2 = a.scale * kLog2e;

    // this workgroup's piece; those of one XCD (workgroups 8 apart) are neighbours, which share a head's keys and values
    const int piece = gridDim.x % 8 ? blockIdx.x : blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
    constexpr int COST = kItemCost<BF16>;
    const uint64_t first = head_cost(a, G, 0, sp.row_blocks, BM, COST, fresh_lane());
    const uint64_t total = line_length(a, G, sp.row_blocks, BM, COST, fresh_lane(), first);
    const uint64_t share = div64(total + sp.grid - 1, sp.grid), at = share * piece, stop = at + share < total ? at + share : total;
    if (threadIdx.x == 0 && sp.cut && !sp.few) sp.cut[piece] = make_int2(0, 1);

    if (at >= stop) return;
    Item it = find_item(a, G, sp.row_blocks, BM, COST, fresh_lane(), first, at);
    bool again = false;
    for (; it.at < stop; it.at += it.cost, ++it.rb) {
        if (it.rb == sp.row_blocks) {
            it.rb = 0;
            if (++it.h == a.c.H) {
                it.h = 0;
                if (++it.b == a.B) return;  // (not reached while the lengths stay as they were summed)
            }
        }
        const int b = __builtin_amdgcn_readfirstlane(it.b), h = __builtin_amdgcn_readfirstlane(it.h);
        const int rb = __builtin_amdgcn_readfirstlane(it.rb);
        const int len = a.len[b], tiles = block_tiles(a, G, len, rb, BM);
        it.cost = tiles + COST;
        const Q8Cut cut = q8_cut(it.at + COST, tiles, share, piece);
        const int t0 = __builtin_amdgcn_readfirstlane(cut.t0), t1 = __builtin_amdgcn_readfirstlane(cut.t1);
        if (t0 >= t1) continue;
        if (again) __syncthreads();  // this item's tiles come into the memory of the one before
        again = true;
        const bool bad = len < 0 || len > a.max_len;
        const int first_end = bad ? 0 : len - a.n_q + q8_query(a, rb * BM) + 1;               // the fewest tokens that a row sees
        const int wave_end = bad ? 0 : len - a.n_q + q8_query(a, rb * BM + wave * 32) + 1;  // the same of the wave's rows
        const int32_t* pages = a.pages + (int64_t)b * a.max_pages;

        const int tid = 64 * wave + fresh_lane(), c = tid & 31, hi = tid >> 5 & 1;
        const int row = rb * BM + wave * 32 + c;  // of the sequence and head
        const int query = q8_query(a, row);  // (rows past the last are fewer than 2^28 too)
        const int end = bad ? 0 : min(len - a.n_q + query + 1, len);

        // A thread's part of a tile: keys as 16 dims of the tokens ktok(j), values as 16 tokens (group tid & 3) of the dims
        // vdim(j), and the group's scales.
        auto ktok = [&](int j) { return (tid + THREADS * j) / CPT; };
        auto wave_tok = [&](int j) { return (64 * wave + THREADS * j) / CPT; };  // the wave's first: all of them lie in one page
        auto vdim = [&](int j) { return (tid + THREADS * j) / 4; };
        // The table's entry of a token, and that entry checked: apart, because a check waits for the load.  Without a branch,
        // because the main loop's body has to stay one block.
        auto entry_of = [&](int tok) { return pages[min(tok >> logP, a.max_pages - 1)]; };
        auto page_of = [&](int tok, int p) { return (tok >> logP) < a.max_pages && p >= 0 && p < a.c.n_pages ? p : -1; };
        const uint8_t *kh = a.c.k + (int64_t)h * P * D, *vh = a.c.v + (int64_t)h * P * D;
        const float *ksh = a.c.ks + h, *vsh = a.c.vs + h;
        const uint32_t page_bytes = a.c.H * P * D;  // of all heads (H < 2^16)
        u32x4_t kx[NC], vx[NC];
        int pk[NC], pg, pv;
        float2 sc;
        auto find_pages = [&](int tile) {
#pragma unroll
            for (int j = 0; j < NC; ++j) pk[j] = entry_of(tile * kTile + wave_tok(j));
            pg = entry_of(tile * kTile + 16 * (tid & 3));
        };
        uint32_t koff[NC], voff;
#pragma unroll
        for (int j = 0; j < NC; ++j) koff[j] = (ktok(j) & (P - 1)) * D + 16 * (tid % CPT);
        voff = (16 * (tid & 3) & (P - 1)) + vdim(0) * P;
        auto load_k = [&](int tile) {
            const uint8_t* at = kh + ((tile * kTile) & (P - 1)) * D;  // (64 tokens begin a page, or the second half of one)
#pragma unroll
            for (int j = 0; j < NC; ++j)
                kx[j] = *(const u32x4_t*)(at + (uint64_t)(uint32_t)max(page_of(tile * kTile + wave_tok(j), __builtin_amdgcn_readfirstlane(pk[j])), 0) * page_bytes + koff[j]);
            pv = page_of(tile * kTile + 16 * (tid & 3), pg);
            const uint64_t g = (uint64_t)(uint32_t)max(pv, 0) * (uint32_t)a.c.H;
            sc = make_float2(ksh[g], vsh[g]);
        };
        auto load_v = [&](int tile) {
            const uint8_t* v = vh + ((tile * kTile) & (P - 1)) + ((uint64_t)(uint32_t)max(pv, 0) * page_bytes + voff);
#pragma unroll
            for (int j = 0; j < NC; ++j) vx[j] = *(const u32x4_t*)(v + THREADS / 4 * j * P);
        };
        auto store_k = [&](int at, const u32x4_t (&kx)[NC]) {
            uint8_t* to = s_k + at;
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const int t = ktok(j), row = (t & 32) + (t & 3) + 4 * (t >> 4 & 1) + 8 * (t >> 2 & 3);
                bf16x8_t* w = (bf16x8_t*)(to + row * KROW + 32 * (tid % CPT));
                w[0] = bf16_codes(kx[j][0], kx[j][1]);
                w[1] = bf16_codes(kx[j][2], kx[j][3]);
            }
        };
        // A page out of range makes the scores that need it NaN; past the sequence's end there is no page.
        auto store_scale = [&](int tile, float2 sc, int pv) {
            if (tid < 4) s_scale[tile & 3][tid] = pv < 0 || tile * kTile + 16 * tid >= len ? make_float2(nan32(), 1.f) : sc;
        };
        uint32_t hidden_nan = 0;
        if (tid == 0) s_nan = 0;
        auto clean_v = [&](int tile) {
            if (tile * kTile + kTile <= first_end) return;
            // codes past the sequence's end may be anything: they become zeros, since 0 times NaN is NaN; and so do
            // NaN codes that some of the rows do not see, which is put right after the loop
            const int nv = min(max(len - tile * kTile - 16 * (tid & 3), 0), 16);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int nb = nv - 4 * z;
                const uint32_t keep = nb >= 4 ? 0xFFFFFFFFu : nb <= 0 ? 0u : (1u << (8 * nb)) - 1u;
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    vx[j][z] &= keep;
                    const uint32_t bits = nan_codes(vx[j][z]);
                    hidden_nan |= bits;
                    vx[j][z] &= ~(bits * 0xFFu);
                }
            }
        };
        auto store_v = [&](int tile) {
            uint8_t* to = s_v + (tile & 1) * (D * VROW);
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                auto* w = (typename Weights<BF16>::Codes*)(to + vdim(j) * VROW + 32 * (tid & 3));
                w[0] = Weights<BF16>::codes(vx[j][0], vx[j][1]);
                w[1] = Weights<BF16>::codes(vx[j][2], vx[j][3]);
            }
        };

        // The walk goes by halves of a tile, 32 tokens: half 2 t + mt is tokens 32 mt .. of tile t.  Scores of a half: token
        // 16 hi + i in x[n][i].
        f32x16_t even, odd;    // of the halves 2 t and 2 t + 1
        float top, bottom;     // the largest and the smallest of the half that comes next
        float cs, bias;        // its scales, made of
        float2 scl;
        int ev;                // the value scale's exponent
        int k_at = 0, k_next = KBYTES, k_last = RING == 3 ? 2 * KBYTES : 0;  // where tiles t, t + 1, t + 2 keep their keys
        auto read_scale = [&](int tile, int mt) { scl = s_scale[tile & 3][2 * mt + hi]; };
        auto use_scale = [&]() {
            ev = scale_exponent(scl.y);
            cs = scl.x * y2;
            bias = (float)ev;
        };
        // Two tiles of keys and one of values into shared memory.  All loads first: they wait for one another only through the
        // page table.
        Query<BF16> q[D / 16];
        f32x16_t o[D / 32];
        float m = kNone, highest = kNone;
        double l = 0.0;
        {
            int pk1[NC];
#pragma unroll
            for (int j = 0; j < NC; ++j) pk1[j] = entry_of((t0 + 1) * kTile + wave_tok(j));
            const int pg1 = entry_of((t0 + 1) * kTile + 16 * (tid & 3));
            find_pages(t0);
            load_k(t0);
            load_v(t0);
            u32x4_t k0[NC];
            const float2 sc0 = sc;
            const int pv0 = pv;
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                k0[j] = kx[j];
                pk[j] = pk1[j];
            }
            pg = pg1;
            load_k(t0 + 1);
            find_pages(t0 + 2);
            const int64_t q_at = (int64_t)b * a.q.seq + (int64_t)(h * G + row - query * G) * a.q.head + (int64_t)query * a.q.token + 8 * hi;
#pragma unroll
            for (int st = 0; st < D / 16; ++st) {
                if (row < R) q[st].load(a.q.base, q_at + 16 * st);
                else q[st].zero();
            }
            store_scale(t0, sc0, pv0);
            store_scale(t0 + 1, sc, pv);
            store_k(k_at, k0);
            clean_v(t0);
            store_v(t0);
            store_k(k_next, kx);
#pragma unroll
            for (int st = 0; st < D / 16; ++st) q[st].keep();
#pragma unroll
            for (int d = 0; d < D / 32; ++d) {
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
                keep_accumulated(o[d]);
            }
        }
        __syncthreads();

        // Operands read ahead, keys of a tile at `at`.
        u32x4_t op[AHEAD + 1];
        const uint8_t* lane_k = s_k + c * KROW + 16 * hi;
        const uint8_t* lane_v = s_v + c * VROW + 32 * hi;
        auto fetch_k = [&](auto U, int at, int mt) { op[U % (AHEAD + 1)] = *(const u32x4_t*)(lane_k + at + 32 * mt * KROW + 32 * U); };

        // The mask, where some row of the wave does not see all of the half; m moved; and what fp16 does not hold of weights added.
        auto settle = [&](auto FIRST, int tile, int mt, f32x16_t& x) {
            const int from = tile * kTile + 32 * mt;
            if (from + 32 > wave_end) {
                const int see = end - from - 16 * hi;
                top = -inf32();
                bottom = inf32();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float y = fmaf(x[i], cs, bias);
                    x[i] = i < see ? y : -inf32();
                    top = fmaxf(top, x[i]);
                    if (BF16) bottom = fminf(bottom, i < see ? y : inf32());
                }
                if (BF16) bottom += kThin - kEdge;
                // 16 hidden tokens move nothing, and a part of 16, often one token or two, only where it keeps fewer than 8 bits (a
                // repair in one workgroup of a short call is a tenth of it: 16 prompts of 64 tokens 15.6 us, so 14).
                if (BF16 && (top == -inf32() || top >= m + kEdge)) top = fmaxf(top, m + kCalm);
                cs = 1.f;
                bias = 0.f;
            }
            const float off = bias - m;
            float t = fmaf(top, cs, off);  // relative to m, as the weights are
            if (!BF16) {
                if (__any(t > kSlack)) {
                    t = fmaxf(fmaxf(t, __shfl_xor(t, 32)), 0.f) + m;
                    const float keep = __builtin_amdgcn_exp2f(m - t);
                    m = t;
                    if constexpr (!FIRST) {  // (nothing is summed yet)
                        l *= keep;
#pragma unroll
                        for (int d = 0; d < D / 32; ++d) scale_product(o[d], keep);
                    }
                }
            } else if (__any(fabsf(t - (kTop + kDrop) / 2) > (kTop - kDrop) / 2 || fmaf(bottom, cs, off) < kThin)) {
                const float own_top = fmaf(top, cs, bias), own_low = fmaf(bottom, cs, bias);  // (of the lane's 16 tokens)
                t = fmaxf(own_top, __shfl_xor(own_top, 32));
                const float low = fminf(own_low, __shfl_xor(own_low, 32));
                float to = m;
                if (t > m + kTop) to = t - (FIRST ? kFirst : kUp);
                else if (t < m + kCalm || low < m + kThin) to = fminf(m, fmaxf(t - (low - t < kThin - kFirst ? kWide : kFirst), highest - kDeep));
                highest = fmaxf(highest, to);
                const float keep = __builtin_amdgcn_exp2f(m - to);
                m = to;
                if constexpr (!FIRST) l *= keep;  // (else nothing is summed yet)
                const bool thin = __any(own_low < m + kThin || (own_top < m + kDrop && own_low < inf32()));  // (16 hidden tokens are not)
                if (!FIRST || thin) {
                    f16x8_t rest[2];
                    if (thin) {
                        float shift = bias - m;
                        asm volatile("" : "+v"(shift));  // (or the compiler makes the step's weights here, ahead of its products)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float p = __builtin_amdgcn_exp2f(fmaf(x[i], cs, shift));
                            rest[i / 8][i % 8] = (_Float16)(p < 0x1p-14f ? (p - (float)(_Float16)p) * 0x1p38f : 0.f);
                        }
                    }
                    const uint8_t* from_v = s_v + (32 * hi + (tile & 1) * (D * VROW) + 64 * mt);
                    each<D / 32>([&](auto I) {
                        f32x16_t sum;
                        if (thin) {
                            const f16x8_t* v = (const f16x8_t*)(from_v + (c + 32 * I) * VROW);
                            first_product(v[0], rest[0], sum);
                            STEP();
                            next_product(v[1], rest[1], sum);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) sum[i] = 0.f;
                        }
                        add_product(o[I], FIRST ? 1.f : keep, sum, 0x1p-38f);
                        STEP();
                    });
                }
            }
        };

        // the first half's scores
        each<D / 16>([&](auto S) {
            const bf16x8_t k = *(const bf16x8_t*)(s_k + k_at + c * KROW + 16 * hi + 32 * S);
            q[S].template to_vector<S == 0>(k, even);
        });
        product_done(even);
        top = -inf32();
        bottom = inf32();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float four = fmaxf(fmaxf(even[i], even[i + 1]), fmaxf(even[i + 2], even[i + 3]));
            top = fmaxf(top, four);
            bottom = fminf(bottom, four);
        }
        read_scale(t0, 0);
        use_scale();

        // A step: one half's weights and sums, and the next one's scores, instruction by instruction.  Operand u of its products is
        // read from shared memory AHEAD operands before its use, and behind every product comes the vector work that fits
        // into its time (left to itself the compiler puts the products in one heap and the exponentials in another).
        auto step = [&](auto MT, int tile, const f32x16_t& s, f32x16_t& next) {
            constexpr int mt = MT, NP = (NQ + NV) / 2, E = 16;  // products, and weights of a lane
            const uint8_t* from_v = lane_v + (tile & 1) * (D * VROW) + 64 * mt;
            Weights<BF16> w[2];
            float sum[2], p[2];
            const float shift = bias - m;
            // Weight x of the lane's 16 tokens; what is made of x - 2 and x - 1 comes with x, when they are there.
            auto weight = [&](auto X) {
                constexpr int x = X;
                if constexpr (x % 2 == 0 && x > 0) {
                    sum[0] = x == 2 ? p[0] : sum[0] + p[0];
                    sum[1] = x == 2 ? p[1] : sum[1] + p[1];
                    asm volatile("" : "+v"(sum[0]), "+v"(sum[1]));  // here and not later, with all of p's registers held for it
                    w[(x - 2) / 8].put((x - 2) % 8, p[0], p[1]);
                    if constexpr (x == E) l = fma((double)(sum[0] + sum[1]), inverse_scale(ev), l);
                }
                if constexpr (x < E) p[x & 1] = __builtin_amdgcn_exp2f(fmaf(s[x], cs, shift));
            };
            float four[2];
            auto largest = [&](auto X) {
                constexpr int x = X;
                float& f = four[x / 2 % 2];
                f = x % 2 == 0 ? max2(next[2 * x], next[2 * x + 1]) : max3(next[2 * x], next[2 * x + 1], f);
                if constexpr (x % 4 == 3) {
                    top = x == 3 ? max2(four[0], four[1]) : max3(four[0], four[1], top);
                    if constexpr (BF16) bottom = x == 3 ? min2(four[0], four[1]) : min3(four[0], four[1], bottom);
                }
            };
            each<NP>([&](auto F) {
                constexpr int f = F, ahead = f + AHEAD;
                if constexpr (ahead < NQ / 2) fetch_k(std::integral_constant<int, ahead>{}, mt ? k_next : k_at, 1 - mt);
                else if constexpr (ahead < NP) {
                    constexpr int d = (ahead - NQ / 2) % (D / 32), j = (ahead - NQ / 2) / (D / 32);
                    op[ahead % (AHEAD + 1)] = *(const u32x4_t*)(from_v + 32 * d * VROW + 16 * j);
                } else fetch_k(std::integral_constant<int, ahead - NP>{}, k_next, mt);  // the next step's
                const u32x4_t x = op[f % (AHEAD + 1)];
                if constexpr (f < NQ / 2) q[f].template to_vector<f == 0>(__builtin_bit_cast(bf16x8_t, x), next);
                else {
                    constexpr int d = (f - NQ / 2) % (D / 32), j = (f - NQ / 2) / (D / 32);
                    o[d] = w[j].times(__builtin_bit_cast(typename Weights<BF16>::Codes, x), o[d]);
                }
                // the weights, all of them by the last quarter of the products, which is what the second half of them is for
                constexpr int e0 = std::min(f * 4 * (E + 1) / (3 * NP), E + 1), e1 = std::min((f + 1) * 4 * (E + 1) / (3 * NP), E + 1);
                each<e1 - e0>([&](auto I) { weight(std::integral_constant<int, e0 + I>{}); });
                // the next half's largest and smallest scores, from a little after its last product on
                constexpr int first = NP / 2 + (NP >= 16 ? 3 : 2), span = NP - first;
                if constexpr (f == first && NP < 16) product_done(next);  // (with 128 dims three products are issued between)
                if constexpr (f >= first) {
                    constexpr int g0 = (f - first) * (E / 2) / span, g1 = (f - first + 1) * (E / 2) / span;
                    each<g1 - g0>([&](auto I) { largest(std::integral_constant<int, g0 + I>{}); });
                }
                // the tiles to come: loaded in a tile's first step, stored at the end of its second (no step reads there before
                // the barrier behind it)
                if constexpr (mt == 0) {
                    if constexpr (f == NP / 4) load_v(tile + 1);
                    if constexpr (f == NP / 4 + 1) load_k(tile + 2);
                    if constexpr (f == NP / 4 + 2) find_pages(tile + 3);
                } else {
                    if constexpr (f == NP - 4) clean_v(tile + 1);
                    if constexpr (f == NP - 3) store_v(tile + 1);
                    if constexpr (f == NP - 2) store_k(k_last, kx);
                }
                if constexpr (f == NP / 2) read_scale(tile + mt, 1 - mt);
                if constexpr (f == NP - 1) use_scale();
                STEP();
            });
        };
        settle(std::true_type{}, t0, 0, even);
        each<AHEAD>([&](auto U) { fetch_k(U, k_at, 1); });
        for (int tile = t0; tile < t1; ++tile) {
            step(std::integral_constant<int, 0>{}, tile, even, odd);
            settle(std::false_type{}, tile, 1, odd);
            if constexpr (RING == 2) __syncthreads();  // no wave reads this tile's keys any more: tile + 2's come there
            step(std::integral_constant<int, 1>{}, tile, odd, even);
            store_scale(tile + 2, sc, pv);
            const int k = k_at;
            k_at = k_next;
            k_next = RING == 3 ? k_last : k;
            k_last = RING == 3 ? k : k_at;
            __syncthreads();
            if (tile + 1 < t1) settle(std::false_type{}, tile + 1, 0, even);
        }

        // the rows' answers, or what this piece of the item adds to them
        const int own = fresh_lane(), col = own & 31, half = own >> 5;
        const bool whole = t0 == 0 && t1 == tiles;
        const int64_t slot = q8_slot(piece, t0 == 0) * BM + wave * 32 + col;
        if (wave == 0 && own == 0 && sp.cut && t0 == 0) {  // (of several items that begin here only the last may be cut)
            const int id = (b * a.c.H + h) * sp.row_blocks + rb;
            sp.cut[sp.few ? id : piece] = make_int2(sp.few ? piece : id, cut.pieces);
        }
        float sum;
        const int down = settle_sum(l + __shfl_xor(l, 32), m, sum);
        if (bad) sum = nan32();
        const int r = rb * BM + wave * 32 + col, i = q8_query(a, r), hq = h * G + r - i * G;
        if (r < R && half == 0) {
            if (!whole) *(float2*)(sp.part_ml + slot * 2) = make_float2(m, sum);
            else if (a.lse) a.lse[((int64_t)b * a.n_q + i) * a.Hq + hq] = q8_lse(m, sum);
        }
        // A lane holds 4 dims here and 4 there of one row; turned in the wave's part of shared memory, 64 dims at a time, rows leave
        // in whole pieces (as the lanes hold them, 16 bytes a row and store, they took 9,000 cycles).
        {
            constexpr int LD = 64 + 4, DIMS = BF16 ? 8 : 4;  // floats of a row; dims of a lane's store
            static_assert(WAVES * 32 * LD * 4 <= sizeof(s_k), "the waves' parts");
            float* mine = (float*)s_k + wave * (32 * LD);
            const float scale = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int p = 0; p < D / 64; ++p) {
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const f32x16_t& x = o[2 * p + d];
                        *(f32x4_t*)(mine + col * LD + 32 * d + 8 * z + 4 * half) =
                            f32x4_t{__builtin_amdgcn_ldexpf(x[4 * z], down) * scale, __builtin_amdgcn_ldexpf(x[4 * z + 1], down) * scale,
                                    __builtin_amdgcn_ldexpf(x[4 * z + 2], down) * scale, __builtin_amdgcn_ldexpf(x[4 * z + 3], down) * scale};
                    }
                wave_memory();
                if (whole) {
#pragma unroll
                    for (int k = 0; k < 32 * 64 / (64 * DIMS); ++k) {
                        const int y = (k * 64 + own) / (64 / DIMS), at = own % (64 / DIMS) * DIMS, ry = rb * BM + wave * 32 + y;
                        if (ry >= R) continue;
                        const int iy = q8_query(a, ry);
                        const int64_t to = (int64_t)b * a.out.seq + (int64_t)(h * G + ry - iy * G) * a.out.head + (int64_t)iy * a.out.token + 64 * p + at;
                        const f32x4_t x0 = *(const f32x4_t*)(mine + y * LD + at);
                        if (BF16) {
                            const f32x4_t x1 = *(const f32x4_t*)(mine + y * LD + at + 4);
                            *(uint4*)((uint16_t*)a.out.base + to) = make_uint4(pack_bf16(x0[0], x0[1]), pack_bf16(x0[2], x0[3]), pack_bf16(x1[0], x1[1]), pack_bf16(x1[2], x1[3]));
                        } else
                            *(f32x4_t*)((float*)a.out.base + to) = x0;
                    }
                } else {
                    float* to = sp.part_o + (slot - col) * D + 64 * p;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int y = k * 4 + own / 16, at = own % 16 * 4;
                        if (rb * BM + wave * 32 + y < R) *(f32x4_t*)(to + y * D + at) = *(const f32x4_t*)(mine + y * LD + at);
                    }
                }
                wave_memory();
            }
        }

        // Rows that see a NaN value taken out above: which dims of which rows is the product of where the NaNs are
        // with what the rows see.  Other lanes of the wave have stored those elements (the rows were turned); the NaN goes over
        // them, and the barrier in front of it keeps that order.
        if (__any(hidden_nan != 0)) s_nan = 1;
        __syncthreads();
        if (s_nan) {
            const int sees_to = bad || r >= R ? 0 : min(len - a.n_q + i + 1, len);
#pragma unroll 1
            for (int t = max(t0, max(first_end, 0) / kTile); t < t1; ++t)
#pragma unroll 1
                for (int d = 0; d < D / 32; ++d) {
                    f32x16_t hits;
#pragma unroll
                    for (int z = 0; z < 16; ++z) hits[z] = 0.f;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const int tok = t * kTile + 32 * mt + 16 * half;
                        const int slot_of = min(tok >> logP, a.max_pages - 1), p = pages[slot_of];
                        const int page = tok < len && p >= 0 && p < a.c.n_pages ? p : 0;
                        u32x4_t is = *(const u32x4_t*)(a.c.v + (((int64_t)page * a.c.H + h) * D + 32 * d + col) * P + (tok & (P - 1)));
#pragma unroll
                        for (int z = 0; z < 4; ++z) is[z] = nan_codes(is[z]) * 0x38u;  // the code of 1
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float f[8];
#pragma unroll
                            for (int z = 0; z < 8; ++z) f[z] = tok + 8 * j + z < sees_to ? 1.f : 0.f;
                            Weights<BF16> sees;
                            sees.set(f);
                            hits = sees.times(Weights<BF16>::codes(is[2 * j], is[2 * j + 1]), hits);
                        }
                    }
#pragma unroll
                    for (int z = 0; z < 16; ++z) {
                        if (!(hits[z] > 0.f)) continue;  // (rows past the last see nothing)
                        const int dim = 32 * d + (z & 3) + 8 * (z >> 2) + 4 * half;
                        if (!whole) sp.part_o[slot * D + dim] = nan32();
                        else {
                            const int64_t to = (int64_t)b * a.out.seq + (int64_t)hq * a.out.head + (int64_t)i * a.out.token + dim;
                            if (BF16) ((uint16_t*)a.out.base)[to] = 0x7FC0;
                            else ((float*)a.out.base)[to] = nan32();
                        }
                    }
                }
        }
    }
}

}  // namespace

// More rows of a sequence and KV head than this take this kernel.  (48 rows in fp32 and 64 in bf16 of 16 sequences of up to 3,000
// tokens with 8 heads: 61 and 35 us here, 79 and 42 in a kernel like q8_attend.hip's with three and four row tiles; 24 and 32 rows:
// 35 here, 27 and 29 there.)
constexpr int64_t kPromptRows = 32;

Q8Plan q8_prompt_plan(Elem e, int B, int n_q, int Hq, int H, int d, int max_len, int cus) {
    Q8Plan p{};
    const int64_t R = (int64_t)n_q * (Hq / H);
    if (R <= kPromptRows) return p;
    const bool bf16 = e == Elem::BF16;
    p.prompt = true;
    p.rows = bf16 && d == 128 && R > 128 ? 256 : 128;
    p.row_blocks = (int)((R + p.rows - 1) / p.rows);
    const int tiles = std::max(1, (max_len + kTile - 1) / kTile);
    // Two workgroups of 4 waves from 16 tiles a CU on (below, the pieces are so short that joining more of them costs more): 64 rows
    // of 4 sequences of 4,000 tokens with 8 heads are 8 a CU, and take 27 us by one workgroup a CU, 30 by two.
    const double work = (double)B * H * p.row_blocks * (tiles + kItemCost<true>);
    const int per_cu = d == 64 || (bf16 && p.rows == 128 && work >= 16.0 * cus) ? 2 : 1;
    p.grid = (int)std::min<double>((double)per_cu * cus, (double)B * H * p.row_blocks * tiles);
    p.splits = p.grid > 1 && tiles > 1;
    return p;
}

template <bool BF16, int D>
static hipError_t launch(const Q8Attend& a, const Q8Pieces& sp, hipStream_t s) {
    const dim3 grid((unsigned)sp.grid);
    if (sp.rows == 128) hipLaunchKernelGGL((q8_prompt_kernel<BF16, D, 4>), grid, dim3(256), 0, s, a, sp);
    else if constexpr (BF16 && D == 128) hipLaunchKernelGGL((q8_prompt_kernel<BF16, D, 8>), grid, dim3(512), 0, s, a, sp);
    return hipGetLastError();
}

hipError_t launch_q8_prompt(Elem e, const Q8Attend& a, const Q8Pieces& sp, hipStream_t s) {
    if (e == Elem::BF16) return a.c.d == 128 ? launch<true, 128>(a, sp, s) : launch<true, 64>(a, sp, s);
    return a.c.d == 128 ? launch<false, 128>(a, sp, s) : launch<false, 64>(a, sp, s);
}

}  // namespace kvmap
