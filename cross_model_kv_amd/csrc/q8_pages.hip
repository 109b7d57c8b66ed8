// Writing rows into the 8-bit paged cache and reading them back.
//
// One workgroup owns one page of one (layer, sequence, head), keys or values, so the page's scale
// needs no agreement between workgroups and every element moves once.  For n new rows x of a page
//   a = max |x| (finite),  e = min { e : a <= 448 * 2^e },  code = rne_e4m3(x * 2^-e),
// all exact but for that one rounding.  Bytes bound it: es bytes read and one written an element.
//
// Thread layout: d / VEC threads side by side on a token's row (16-byte loads), each holding PASSES
// consecutive tokens, so that a thread has PASSES tokens of VEC dims in registers: a row's codes
// leave as they are for keys; for values, whose page is dim-major, a thread's PASSES tokens of one dim
// are adjacent bytes and the page is turned in LDS.  A page that a wave can hold so is a wave's, not a
// workgroup's (bf16 pages of 16 tokens with 64 dims: 1.9 -> 4.0 to 5.2 TB/s written, 2.2 -> 5.3 read).
//
// Writing 8,192 mapped bf16 tokens of 64 layers with 8 heads takes 585 us, 5.5 TB/s, reading 4,096 of 40 layers 178 us,
// 5.65 TB/s; a copy of 4 GiB reaches 4.75 TB/s.  A decode step's write (4.7 us for 64 sequences, 3.6 for one) is the launch
// and one page's way through memory.

#include "common.h"
#include "internal.h"
#include "q8_span.h"

namespace kvmap {
namespace {

constexpr float kTop = 448.f;  // largest e4m3 value
constexpr int kMinExp = -110, kMaxExp = 119;

// The smallest power of two 2^e with amax <= 448 * 2^e, e clamped to the scales' range.  With
// amax = (1 + f) * 2^(x - 1): 448 = 0.875 * 2^9, so e is x - 9, or x - 8 where (1 + f) / 2 > 0.875.
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 126 - 9 + ((u & 0x7FFFFFu) > 0x600000u);
    e = min(max(e, kMinExp), kMaxExp);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Four values to four codes: nearest even, saturating; NaN for what is not finite.
__device__ __forceinline__ uint32_t codes4(const float* x, float inv) {
    float y[4];
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = fminf(fmaxf(x[i] * inv, -kTop), kTop);
        odd |= (__float_as_uint(x[i]) & 0x7F800000u) == 0x7F800000u ? 0xFFu << (8 * i) : 0u;
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
    return ((uint32_t)w & ~odd) | (0x7F7F7F7Fu & odd);
}

__device__ __forceinline__ void values4(uint32_t w, float* x) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[0] = a[0];
    x[1] = a[1];
    x[2] = b[0];
    x[3] = b[1];
}

// Codes of one scale rounded to a larger one (NaN stays NaN).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    float x[4];
    values4(w, x);
    return codes4(x, ratio);
}

template <bool BF16>
struct Row16 {  // 16 bytes of a row as fp32
    static constexpr int N = BF16 ? 8 : 4;
    uint4 raw;
    __device__ __forceinline__ void get(float* x) const {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        if (BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16lo(w[i]);
                x[2 * i + 1] = bf16hi(w[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
        }
    }
    __device__ __forceinline__ void set(const float* x) {
        if (BF16)
            raw = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        else
            raw = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

// In a scalar register, so that a page's item, its lookups and its addresses stay scalar.
__device__ __forceinline__ uint32_t wave_of_thread() { return (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / 64)); }

// What one group of threads works on.
struct Item {
    int j, b, h, layer, kv;
};
__device__ __forceinline__ Item item_of(uint32_t i, int n_slots, int B, int H) {
    Item t;
    t.j = (int)(i % n_slots);
    i /= n_slots;
    t.h = (int)(i % H);
    i /= H;
    t.b = (int)(i % B);
    i /= B;
    t.kv = (int)(i & 1);
    t.layer = (int)(i >> 1);
    return t;
}

// What a wave's lanes have written, to LDS or the page, is there for the rest of it.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// WAVE: the most 16-byte parts of rows that one wave takes a page of.  Measured on pages of 512 parts, by waves and by
// workgroups: writes 5.7 and 5.2 TB/s (bf16, 32 tokens of 128 dims), fp32 reads 5.5 and 4.8 (32 tokens of 64), bf16 reads 5.2
// and 5.6.
template <bool BF16, int D, int P, int WAVE>
struct Tile {
    static constexpr int ES = BF16 ? 2 : 4;
    static constexpr int VEC = 16 / ES;
    static constexpr int TPR = D / VEC;                          // threads on a row
    static constexpr int GROUP = P * TPR <= WAVE ? 64 : 256;     // threads on a page
    static constexpr int PASSES = P * TPR / GROUP;               // consecutive tokens of a thread
    static constexpr int LDW = P / 4 + 1;                        // LDS dwords of a dim's tokens (odd: spreads the banks)
    static constexpr int TURN = D * LDW * (256 / GROUP);         // of all groups of a workgroup
    __device__ static __forceinline__ void sync() {
        if (GROUP == 256) __syncthreads();
        else wave_sync();
    }
};

template <bool BF16, int D, int P>
using WriteTile = Tile<BF16, D, P, 512>;
template <bool BF16, int D, int P>
using ReadTile = Tile<BF16, D, P, BF16 ? 256 : 512>;

// The codes of a page's first `lo` tokens rounded to a scale 1 / ratio times as large, by `threads` threads.
template <int D, int P>
__device__ __forceinline__ void rescale_page(uint8_t* dst, int kv, int lo, float ratio, int tid, int threads) {
    if (kv == 0) {
        for (int i = tid; i < lo * (D / 4); i += threads) {
            uint32_t* w = (uint32_t*)dst + i;
            *w = rescale4(*w, ratio);
        }
        return;
    }
    const int wpd = (lo + 3) / 4;  // dwords of a dim that hold such tokens
    for (int i = tid; i < D * wpd; i += threads) {
        const int dim = i / wpd, k = i - dim * wpd;
        uint32_t* w = (uint32_t*)(dst + dim * P) + k;
        const uint32_t keep = lo - 4 * k >= 4 ? 0u : 0xFFFFFFFFu << (8 * (lo - 4 * k));
        *w = (*w & keep) | (rescale4(*w, ratio) & ~keep);
    }
}

// The bytes [from, to) of 4 tokens' codes of one dim; the others stay as they are.
__device__ __forceinline__ void store_tokens(uint32_t* at, uint32_t w, int from, int to) {
    if (from <= 0 && to >= 4) {
        *at = w;
    } else if (from < 4 && to > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i >= from && i < to) ((uint8_t*)at)[i] = (uint8_t)(w >> (8 * i));
    }
}

template <bool BF16, int D, int P>
__global__ __launch_bounds__(256) void q8_write_kernel(Q8Pools c, Q8Seqs q, int n_slots, uint32_t items, int n, Q8Rows kr, Q8Rows vr,
                                                       unsigned int* __restrict__ dropped) {
    using T = WriteTile<BF16, D, P>;
    __shared__ uint32_t s_max[4];
    __shared__ uint32_t s_turn[T::TURN];
    const uint32_t group = T::GROUP == 256 ? 0 : wave_of_thread(), index = blockIdx.x * (256 / T::GROUP) + group;
    if (index >= items) return;
    const Item it = item_of(index, n_slots, q.B, c.H);
    const int tid = threadIdx.x % T::GROUP;
    uint32_t* turn = s_turn + group * (D * T::LDW);
    const Q8Span sp = q8_span(q.start[it.b], q.count ? q.count[it.b] : n, n, it.j, q.pages + (int64_t)it.b * q.max_pages,
                              q.max_pages, c.n_pages, P);
    if (sp.lo >= sp.live) return;
    if (sp.page < 0) {
        if (tid == 0 && (!sp.bad_seq || it.j == 0)) atomicAdd(dropped, 1u);
        return;
    }
    const int lo = sp.lo, hi = sp.live;

    const Q8Rows& r = it.kv ? vr : kr;
    const char* src = (const char*)r.base +
                      (it.layer * r.layer + it.b * r.seq + it.h * r.head + sp.p0 * r.token) * T::ES;
    const int row0 = tid / T::TPR * T::PASSES, col = tid % T::TPR * T::VEC;
    Row16<BF16> x[T::PASSES];
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < T::PASSES; ++p) {
        const int row = row0 + p;
        x[p].raw = make_uint4(0, 0, 0, 0);
        if (row >= lo && row < hi) x[p].raw = *(const uint4*)(src + (row * r.token + col) * T::ES);
        float f[T::VEC];
        x[p].get(f);
#pragma unroll
        for (int i = 0; i < T::VEC; ++i) {
            const uint32_t u = __float_as_uint(f[i]) & 0x7FFFFFFFu;
            top = max(top, u < 0x7F800000u ? u : 0u);
        }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if (T::GROUP == 256) {
        if ((tid & 63) == 0) s_max[tid >> 6] = top;
        __syncthreads();
        top = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
    }

    const int64_t page = it.layer * c.layer_scales + (int64_t)sp.page * c.H + it.h;
    float* scale_at = (it.kv ? c.vs : c.ks) + page;
    uint8_t* dst = (it.kv ? c.v : c.k) + page * (P * D);
    float scale = scale_for(__uint_as_float(top));
    if (lo) {
        const float before = *scale_at;
        if (before >= scale) {
            scale = before;
        } else {  // the tokens before start are rounded to the new scale
            rescale_page<D, P>(dst, it.kv, lo, before / scale, tid, T::GROUP);
        }
        T::sync();  // `before` is read, and shared dwords of values are written, before the stores below
    }
    if (tid == 0) *scale_at = scale;
    const float inv = 1.f / scale;  // exact: a power of two

    if (it.kv == 0) {
#pragma unroll
        for (int p = 0; p < T::PASSES; ++p) {
            const int row = row0 + p;
            if (row < lo || row >= hi) continue;
            float f[T::VEC];
            x[p].get(f);
            uint32_t* w = (uint32_t*)(dst + row * D + col);
            if (BF16)
                *(uint2*)w = make_uint2(codes4(f, inv), codes4(f + T::VEC - 4, inv));
            else
                *w = codes4(f, inv);
        }
        return;
    }
    // values: PASSES tokens of each of VEC dims
    uint32_t w[T::PASSES][T::VEC / 4];
#pragma unroll
    for (int p = 0; p < T::PASSES; ++p) {
        float f[T::VEC];
        x[p].get(f);
#pragma unroll
        for (int i = 0; i < T::VEC / 4; ++i) w[p][i] = codes4(f + 4 * i, inv);
    }
    uint8_t* lds = (uint8_t*)turn;
#pragma unroll
    for (int i = 0; i < T::VEC; ++i)
#pragma unroll
        for (int p = 0; p < T::PASSES; ++p)
            lds[(col + i) * (T::LDW * 4) + row0 + p] = (uint8_t)(w[p][i / 4] >> (8 * (i & 3)));
    T::sync();
    for (int i = tid; i < D * (P / 16); i += T::GROUP) {
        const int dim = i / (P / 16), k = i % (P / 16);
        const uint32_t* a = turn + dim * T::LDW + 4 * k;
        uint32_t* to = (uint32_t*)(dst + dim * P + 16 * k);
        if (lo <= 16 * k && 16 * k + 16 <= hi) {
            *(uint4*)to = make_uint4(a[0], a[1], a[2], a[3]);
        } else {  // (byte by byte, pages of 128 tokens of which 81 enter took five times as long)
#pragma unroll
            for (int z = 0; z < 4; ++z) store_tokens(to + z, a[z], lo - 16 * k - 4 * z, hi - 16 * k - 4 * z);
        }
    }
}

template <bool BF16, int D, int P>
__global__ __launch_bounds__(256) void q8_read_kernel(Q8Pools c, Q8Seqs q, int n_slots, uint32_t items, int n, Q8Rows kr, Q8Rows vr) {
    using T = ReadTile<BF16, D, P>;
    __shared__ uint32_t s_turn[T::TURN];
    const uint32_t group = T::GROUP == 256 ? 0 : wave_of_thread(), index = blockIdx.x * (256 / T::GROUP) + group;
    if (index >= items) return;
    const Item it = item_of(index, n_slots, q.B, c.H);
    const int tid = threadIdx.x % T::GROUP;
    uint32_t* turn = s_turn + group * (D * T::LDW);
    const Q8Span sp = q8_span(q.start[it.b], q.count ? q.count[it.b] : n, n, it.j, q.pages + (int64_t)it.b * q.max_pages,
                              q.max_pages, c.n_pages, P);
    if (sp.lo >= sp.hi) return;
    const bool held = sp.page >= 0;
    const int lo = sp.lo, hi = sp.hi, live = sp.live;  // rows [live, hi) are zeros

    const Q8Rows& r = it.kv ? vr : kr;
    char* out = (char*)r.base + (it.layer * r.layer + it.b * r.seq + it.h * r.head + sp.p0 * r.token) * T::ES;
    const int64_t page = it.layer * c.layer_scales + (int64_t)(held ? sp.page : 0) * c.H + it.h;
    const uint8_t* src = (it.kv ? c.v : c.k) + page * (P * D);
    const float scale = held ? (it.kv ? c.vs : c.ks)[page] : __uint_as_float(0x7FC00000u);
    const int row0 = tid / T::TPR * T::PASSES, col = tid % T::TPR * T::VEC;
    uint32_t w[T::PASSES][T::VEC / 4];  // keys: all of a thread's loads before its first store
    if (it.kv == 0 && held && live > lo) {
#pragma unroll
        for (int p = 0; p < T::PASSES; ++p)
#pragma unroll
            for (int g = 0; g < T::VEC / 4; ++g) w[p][g] = *(const uint32_t*)(src + (row0 + p) * D + col + 4 * g);
    }
    if (it.kv && held && live > lo) {
        for (int i = tid; i < D * (P / 16); i += T::GROUP) {
            const int dim = i / (P / 16), k = i % (P / 16);
            if (16 * k + 16 <= lo || 16 * k >= live) continue;
            const uint4 a = *(const uint4*)(src + dim * P + 16 * k);
            uint32_t* w = turn + dim * T::LDW + 4 * k;
            w[0] = a.x;
            w[1] = a.y;
            w[2] = a.z;
            w[3] = a.w;
        }
    }
    T::sync();
    const uint8_t* lds = (const uint8_t*)turn;
#pragma unroll
    for (int p = 0; p < T::PASSES; ++p) {
        const int row = row0 + p;
        if (row < lo || row >= hi) continue;
        float f[T::VEC];
        if (row >= live) {
#pragma unroll
            for (int i = 0; i < T::VEC; ++i) f[i] = 0.f;
        } else if (!held) {
#pragma unroll
            for (int i = 0; i < T::VEC; ++i) f[i] = scale;  // NaN
        } else {
#pragma unroll
            for (int g = 0; g < T::VEC / 4; ++g) {
                if (it.kv) {
                    const uint8_t* a = lds + (col + 4 * g) * (T::LDW * 4) + row;
                    w[p][g] = a[0] | (uint32_t)a[T::LDW * 4] << 8 | (uint32_t)a[2 * T::LDW * 4] << 16 | (uint32_t)a[3 * T::LDW * 4] << 24;
                }
                values4(w[p][g], f + 4 * g);
            }
#pragma unroll
            for (int i = 0; i < T::VEC; ++i) f[i] *= scale;
        }
        Row16<BF16> y;
        y.set(f);
        *(uint4*)(out + (row * r.token + col) * T::ES) = y.raw;
    }
}

// Writes of at most FEW tokens a sequence: a wave takes a page, its lanes D / 64 dims of every row that enters, so that a
// page's other rows cost nothing.
template <bool BF16, int D, int P, int FEW>
__global__ __launch_bounds__(256) void q8_write_few_kernel(Q8Pools c, Q8Seqs q, int n_slots, uint32_t items, int n, Q8Rows kr, Q8Rows vr,
                                                           unsigned int* __restrict__ dropped) {
    constexpr int V = D / 64, ES = BF16 ? 2 : 4;
    const uint32_t index = blockIdx.x * 4 + wave_of_thread();
    if (index >= items) return;
    const Item it = item_of(index, n_slots, q.B, c.H);
    const int lane = threadIdx.x & 63;
    const Q8Span sp = q8_span(q.start[it.b], q.count ? q.count[it.b] : n, n, it.j, q.pages + (int64_t)it.b * q.max_pages,
                              q.max_pages, c.n_pages, P);
    if (sp.lo >= sp.live) return;
    if (sp.page < 0) {
        if (lane == 0 && (!sp.bad_seq || it.j == 0)) atomicAdd(dropped, 1u);
        return;
    }
    const int lo = sp.lo, rows = sp.live - lo;
    const int64_t page = it.layer * c.layer_scales + (int64_t)sp.page * c.H + it.h;
    float* scale_at = (it.kv ? c.vs : c.ks) + page;
    uint8_t* dst = (it.kv ? c.v : c.k) + page * (P * D);
    const float before = lo ? *scale_at : 0.f;
    const Q8Rows& r = it.kv ? vr : kr;
    const char* src = (const char*)r.base +
                      (it.layer * r.layer + it.b * r.seq + it.h * r.head + (sp.p0 + lo) * r.token + lane * V) * ES;
    float x[FEW][V];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < FEW; ++i) {
        if (i >= rows) break;
        const char* at = src + i * r.token * ES;
        if (BF16 && V == 2) {
            const uint32_t w = *(const uint32_t*)at;
            x[i][0] = bf16lo(w);
            x[i][V - 1] = bf16hi(w);
        } else if (BF16) {
            x[i][0] = __uint_as_float((uint32_t)*(const uint16_t*)at << 16);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) x[i][k] = ((const float*)at)[k];
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const uint32_t u = __float_as_uint(x[i][k]) & 0x7FFFFFFFu;
            top = max(top, u < 0x7F800000u ? u : 0u);
        }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    float scale = scale_for(__uint_as_float(top));
    if (lo) {
        if (before >= scale) scale = before;
        else rescale_page<D, P>(dst, it.kv, lo, before / scale, lane, 64);
        wave_sync();  // dwords of values that also hold new tokens are written before the bytes below
    }
    if (lane == 0) *scale_at = scale;
    const float inv = 1.f / scale;  // exact: a power of two
    uint64_t w[FEW / 8][V] = {};  // a dim's tokens side by side
#pragma unroll
    for (int i = 0; i < FEW; ++i) {
        if (i >= rows) break;
        const float y[4] = {x[i][0], x[i][V - 1], 0.f, 0.f};
        const uint32_t codes = codes4(y, inv);
        if (it.kv) {
#pragma unroll
            for (int k = 0; k < V; ++k) w[i / 8][k] |= (uint64_t)(codes >> (8 * k) & 0xFF) << (8 * (i & 7));
        } else if (V == 2) {
            *(uint16_t*)(dst + (lo + i) * D + 2 * lane) = (uint16_t)codes;
        } else {
            dst[(lo + i) * D + lane] = (uint8_t)codes;
        }
    }
    if (it.kv == 0) return;
    const int skip = lo & 3;  // they begin in a dword's middle
#pragma unroll
    for (int e = 0; e < FEW / 8; ++e) {
        const int live = rows - 8 * e + skip;
        if (live <= skip) break;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            uint32_t* to = (uint32_t*)(dst + (lane * V + k) * P) + lo / 4 + 2 * e;
            const uint64_t low = w[e][k] << (8 * skip);
            store_tokens(to, (uint32_t)low, skip, live);
            store_tokens(to + 1, (uint32_t)(low >> 32), skip - 4, live - 4);
            if (skip && live > 8) store_tokens(to + 2, (uint32_t)(w[e][k] >> (64 - 8 * skip)), 0, min(live, 8 + skip) - 8);
        }
    }
}

// Reads of at most FEW tokens a sequence, in the same way.
template <bool BF16, int D, int P, int FEW>
__global__ __launch_bounds__(256) void q8_read_few_kernel(Q8Pools c, Q8Seqs q, int n_slots, uint32_t items, int n, Q8Rows kr, Q8Rows vr) {
    constexpr int V = D / 64, ES = BF16 ? 2 : 4;
    const uint32_t index = blockIdx.x * 4 + wave_of_thread();
    if (index >= items) return;
    const Item it = item_of(index, n_slots, q.B, c.H);
    const int lane = threadIdx.x & 63;
    const Q8Span sp = q8_span(q.start[it.b], q.count ? q.count[it.b] : n, n, it.j, q.pages + (int64_t)it.b * q.max_pages,
                              q.max_pages, c.n_pages, P);
    if (sp.lo >= sp.hi) return;
    const bool held = sp.page >= 0;
    const int lo = sp.lo, rows = sp.hi - lo, live = sp.live - lo;  // rows [live, rows) are zeros
    const int64_t page = it.layer * c.layer_scales + (int64_t)(held ? sp.page : 0) * c.H + it.h;
    const uint8_t* src = (it.kv ? c.v : c.k) + page * (P * D);
    const float scale = held ? (it.kv ? c.vs : c.ks)[page] : __uint_as_float(0x7FC00000u);
    uint32_t codes[FEW] = {};  // of a row's V dims
    if (held && it.kv == 0) {
#pragma unroll
        for (int i = 0; i < FEW; ++i)
            if (i < live) codes[i] = V == 2 ? *(const uint16_t*)(src + (lo + i) * D + 2 * lane) : src[(lo + i) * D + lane];
    } else if (held) {
        const int skip = lo & 3;  // they begin in a dword's middle
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const uint32_t* from = (const uint32_t*)(src + (lane * V + k) * P) + lo / 4;
            uint32_t w[FEW / 4 + 1] = {};
#pragma unroll
            for (int j = 0; j <= FEW / 4; ++j)
                if (4 * j < skip + live) w[j] = from[j];
#pragma unroll
            for (int j = 0; j < FEW / 4; ++j) {
                const uint32_t four = (uint32_t)(((uint64_t)w[j + 1] << 32 | w[j]) >> (8 * skip));
#pragma unroll
                for (int i = 0; i < 4; ++i) codes[4 * j + i] |= (four >> (8 * i) & 0xFF) << (8 * k);
            }
        }
    }
    const Q8Rows& r = it.kv ? vr : kr;
    char* out = (char*)r.base + (it.layer * r.layer + it.b * r.seq + it.h * r.head + (sp.p0 + lo) * r.token + lane * V) * ES;
#pragma unroll
    for (int i = 0; i < FEW; ++i) {
        if (i >= rows) break;
        float f[4];
        values4(codes[i], f);
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = i >= live ? 0.f : held ? f[k] * scale : scale;
        char* at = out + i * r.token * ES;
        if (BF16 && V == 2) *(uint32_t*)at = pack_bf16(f[0], f[1]);
        else if (BF16) *(uint16_t*)at = (uint16_t)pack_bf16(f[0], 0.f);
        else
#pragma unroll
            for (int k = 0; k < V; ++k) ((float*)at)[k] = f[k];
    }
}

// A row range of n tokens touches at most this many pages.
int slots(int n, int page) { return (int)(((int64_t)n + 2 * page - 2) / page); }

// f(Shape<bf16, d, page>()) for what a call has.
template <bool B, int DIMS, int TOKENS>
struct Shape {
    static constexpr bool BF16 = B;
    static constexpr int D = DIMS, P = TOKENS;
};
template <bool BF16, int D, class F>
void with_page(int page, F&& f) {
    if (page == 16) f(Shape<BF16, D, 16>());
    else if (page == 32) f(Shape<BF16, D, 32>());
    else if (page == 64) f(Shape<BF16, D, 64>());
    else f(Shape<BF16, D, 128>());
}
template <class F>
void with_shape(Elem e, const Q8Pools& c, F&& f) {
    if (e == Elem::BF16) c.d == 128 ? with_page<true, 128>(c.page, f) : with_page<true, 64>(c.page, f);
    else c.d == 128 ? with_page<false, 128>(c.page, f) : with_page<false, 64>(c.page, f);
}

// Workgroups for items that 256 / GROUP of them take.
template <int GROUP>
dim3 grid_of(uint32_t items) { return dim3((items + 256 / GROUP - 1) / (256 / GROUP)); }

}  // namespace

// Which tokens are few.  One token of 16 sequences in 40 layers: 13 us by the wave (bf16 pages of 64, fp32 ones of 128), 33 and
// 49 by the workgroup; 8 tokens of 4 sequences in 8 layers 7.2 and 7.7.  Up to 16 tokens only where there are many pages, each a
// workgroup's, since the wave's rows come 4 bytes a lane: 16 tokens of 16 sequences in 40 layers (20,480 pages) 52 and 75 us, of
// 8 in 16 (4,096) 16.8 and 20.0, of 8 in 8 (2,048) 12.7 and 12.2.  Reads: 8 tokens of those 16 sequences 15 and 39 us, 16 of 8 in
// 16 layers 10.1 and 12.4.
constexpr int kFew = 8, kSome = 16;
constexpr uint32_t kManyPages = 4096;

hipError_t launch_q8_write(Elem e, const Q8Pools& c, const Q8Seqs& q, int n_layers, int n, const Q8Rows& k,
                           const Q8Rows& v, unsigned int* dropped, hipStream_t s) {
    const int ns = slots(n, c.page);
    const uint32_t items = (uint32_t)((int64_t)ns * q.B * c.H * n_layers * 2);
    with_shape(e, c, [&](auto shape) {
        using S = decltype(shape);
        constexpr int GROUP = WriteTile<S::BF16, S::D, S::P>::GROUP;
        if (n <= kFew) {
            hipLaunchKernelGGL((q8_write_few_kernel<S::BF16, S::D, S::P, kFew>), grid_of<64>(items), dim3(256), 0, s, c, q, ns, items, n, k, v, dropped);
            return;
        }
        if constexpr (GROUP == 256)
            if (n <= kSome && items >= kManyPages) {
                hipLaunchKernelGGL((q8_write_few_kernel<S::BF16, S::D, S::P, kSome>), grid_of<64>(items), dim3(256), 0, s, c, q, ns, items, n, k, v, dropped);
                return;
            }
        hipLaunchKernelGGL((q8_write_kernel<S::BF16, S::D, S::P>), grid_of<GROUP>(items), dim3(256), 0, s, c, q, ns, items, n, k, v, dropped);
    });
    return hipGetLastError();
}

hipError_t launch_q8_read(Elem e, const Q8Pools& c, const Q8Seqs& q, int n_layers, int n, const Q8Rows& k,
                          const Q8Rows& v, hipStream_t s) {
    const int ns = slots(n, c.page);
    const uint32_t items = (uint32_t)((int64_t)ns * q.B * c.H * n_layers * 2);
    with_shape(e, c, [&](auto shape) {
        using S = decltype(shape);
        constexpr int GROUP = ReadTile<S::BF16, S::D, S::P>::GROUP;
        if (n <= kFew) {
            hipLaunchKernelGGL((q8_read_few_kernel<S::BF16, S::D, S::P, kFew>), grid_of<64>(items), dim3(256), 0, s, c, q, ns, items, n, k, v);
            return;
        }
        if constexpr (GROUP == 256)
            if (n <= kSome && items >= kManyPages) {
                hipLaunchKernelGGL((q8_read_few_kernel<S::BF16, S::D, S::P, kSome>), grid_of<64>(items), dim3(256), 0, s, c, q, ns, items, n, k, v);
                return;
            }
        hipLaunchKernelGGL((q8_read_kernel<S::BF16, S::D, S::P>), grid_of<GROUP>(items), dim3(256), 0, s, c, q, ns, items, n, k, v);
    });
    return hipGetLastError();
}

}  // namespace kvmap
