// Rows into the paged cache of the model's own type, with the keys' rotation on the way, and back.
//
// Pair (i, i + d/2) of a key at position p turns by a = p f_i: (lo, hi) -> (lo cos a - hi sin a, hi cos a + lo sin a),
// and by -a when it is read back.  Products and sums in fp32 from fp32 cosines and sines (formed in float64),
// rounded once; values, and keys without a table, are moved as they are.
//
// A thread owns 16 bytes of a token's low half and the 16 bytes of the high half that pair with them, in one layer and head, of
// keys or of values: nothing crosses lanes.  Every element moves once, past the caches.  Bytes bound it: 8,192 bf16 tokens
// of 64 layers and 8 heads enter in 721 us, 6.0 TB/s (a copy of 4 GiB: 4.7; through the caches and with keys and values in
// one thread, four slabs at a time, 883), 4,096 of 40 layers are read back stripped in 223, 6.0 TB/s (265).  One decode step's
// tokens (2.3 us for one sequence, 2.6 for 64) are the launch and a row's way through memory.

#include <algorithm>

#include "common.h"
#include "internal.h"
#include "q8_span.h"

namespace kvmap {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

template <bool BF16>
struct Piece {  // 16 bytes of a row
    static constexpr int N = BF16 ? 8 : 4;
    u32x4_t w;
    __device__ __forceinline__ void load(const char* at) { w = __builtin_nontemporal_load((const u32x4_t*)at); }
    __device__ __forceinline__ void store(char* at) const { __builtin_nontemporal_store(w, (u32x4_t*)at); }
    __device__ __forceinline__ float get(int i) const {
        if (!BF16) return __uint_as_float(w[i]);
        return (i & 1) ? bf16hi(w[i >> 1]) : bf16lo(w[i >> 1]);
    }
    __device__ __forceinline__ void set(const float* x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = BF16 ? pack_bf16(x[2 * i], x[2 * i + 1]) : __float_as_uint(x[i]);
    }
};

// One token's cosines and sines of a thread's pairs; sign -1 turns back.
template <bool BF16>
struct Turn {
    static constexpr int N = Piece<BF16>::N;
    float c[N], s[N];
    __device__ __forceinline__ void load(const float2* at, float sign) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float4 x = ((const float4*)at)[i];
            c[2 * i] = x.x;
            s[2 * i] = sign * x.y;
            c[2 * i + 1] = x.z;
            s[2 * i + 1] = sign * x.w;
        }
    }
    __device__ __forceinline__ void apply(Piece<BF16>& lo, Piece<BF16>& hi) const {
        float a[N], b[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float x = lo.get(i), y = hi.get(i);
            a[i] = fmaf(-y, s[i], x * c[i]);
            b[i] = fmaf(x, s[i], y * c[i]);
        }
        lo.set(a);
        hi.set(b);
    }
};

// What a token's threads need to know of it.
struct Token {
    int64_t pos;
    int i, b, page, row;
    bool live;     // belongs to the sequence's count
    bool bad_seq;  // start or count out of range
};
__device__ __forceinline__ Token token_of(const Q8Seqs& q, uint32_t n, uint32_t t, int n_pages, int P, const Rotation& rot) {
    Token x;
    x.b = (int)(t / n);
    x.i = (int)(t - (uint32_t)x.b * n);
    const int start = q.start[x.b], count = q.count ? q.count[x.b] : (int)n;
    x.bad_seq = start < 0 || count < 0 || count > (int)n;
    x.pos = (int64_t)start + x.i;
    x.live = x.bad_seq || x.i < count;
    const bool there = x.live && !x.bad_seq && (!rot.tab || x.pos < rot.n_pos);
    x.page = there ? q8_page_at(q.pages + (int64_t)x.b * q.max_pages, x.pos >> (31 - __clz(P)), q.max_pages, n_pages) : -1;
    x.row = (int)(x.pos & (P - 1));
    return x;
}

template <bool BF16, int D, bool TURN, bool READ>
__global__ __launch_bounds__(256) void paged_rows_kernel(PagedPools c, Q8Seqs q, int n_layers, int n, uint32_t tokens, Q8Rows kr, Q8Rows vr,
                                                         Rotation rot, unsigned int* __restrict__ dropped) {
    using X = Piece<BF16>;
    constexpr int ES = BF16 ? 2 : 4;
    constexpr int TPT = D / 2 / X::N;  // threads on a token
    const uint32_t t = blockIdx.x * (256 / TPT) + threadIdx.x / TPT;
    if (t >= tokens) return;
    const int p = threadIdx.x % TPT * X::N;  // the first of this thread's pairs
    const Token x = token_of(q, n, t, c.n_pages, c.page, rot);
    if (!READ) {
        if (!x.live) return;
        if (x.page < 0) {
            if (p == 0 && blockIdx.y == 0) atomicAdd(dropped, 1u);
            return;
        }
    }
    const bool values = blockIdx.y & 1;
    const bool turns = TURN && !values && x.page >= 0;
    Turn<BF16> turn;
    if (turns) turn.load(rot.tab + x.pos * (D / 2) + p, READ ? -1.f : 1.f);

    const Q8Rows& r = values ? vr : kr;
    char* pool = values ? c.v : c.k;
    const int64_t in_page = ((int64_t)max(x.page, 0) * c.H * c.page + x.row) * D + p;
    constexpr int HIGH = D / 2 * ES;
    for (int slab = blockIdx.y >> 1; slab < n_layers * c.H; slab += gridDim.y >> 1) {
        const int layer = slab / c.H, h = slab - layer * c.H;
        char* held = pool + (int64_t)layer * c.layer + (in_page + (int64_t)h * c.page * D) * ES;
        char* row = (char*)r.base + (layer * r.layer + x.b * r.seq + h * r.head + x.i * r.token + p) * ES;
        X lo, hi;
        if (READ && x.page < 0) {  // rows past a sequence's count are zeros, what is out of range is NaN
            const uint32_t w = !x.live ? 0u : BF16 ? 0x7FC07FC0u : 0x7FC00000u;
            lo.w = hi.w = u32x4_t{w, w, w, w};
        } else {
            const char* from = READ ? held : row;
            lo.load(from);
            hi.load(from + HIGH);
            if (turns) turn.apply(lo, hi);
        }
        char* to = READ ? row : held;
        lo.store(to);
        hi.store(to + HIGH);
    }
}

template <bool READ>
hipError_t launch_rows_of(Elem e, const PagedPools& c, const Q8Seqs& q, int n_layers, int n, const Q8Rows& k, const Q8Rows& v,
                          const Rotation& rot, unsigned int* dropped, hipStream_t s) {
    const uint32_t tokens = (uint32_t)q.B * (uint32_t)n;  // at most 2^27
    const uint32_t per_block = 256 / (c.d / 2 / (e == Elem::BF16 ? 8 : 4));
    const uint32_t bx = (tokens + per_block - 1) / per_block;
    const int64_t by = std::min<int64_t>(2 * (int64_t)n_layers * c.H, 65534);  // keys and values of a slab side by side
    const dim3 grid(bx, (unsigned)by);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, c, q, n_layers, n, tokens, k, v, rot, dropped); };
    const bool turn = rot.tab != nullptr;
    if (e == Elem::BF16) {
        if (c.d == 128) turn ? go(paged_rows_kernel<true, 128, true, READ>) : go(paged_rows_kernel<true, 128, false, READ>);
        else turn ? go(paged_rows_kernel<true, 64, true, READ>) : go(paged_rows_kernel<true, 64, false, READ>);
    } else {
        if (c.d == 128) turn ? go(paged_rows_kernel<false, 128, true, READ>) : go(paged_rows_kernel<false, 128, false, READ>);
        else turn ? go(paged_rows_kernel<false, 64, true, READ>) : go(paged_rows_kernel<false, 64, false, READ>);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_paged_append(Elem e, const PagedPools& c, const Q8Seqs& q, int n_layers, int n, const Q8Rows& k,
                               const Q8Rows& v, const Rotation& rot, unsigned int* dropped, hipStream_t s) {
    return launch_rows_of<false>(e, c, q, n_layers, n, k, v, rot, dropped, s);
}
hipError_t launch_paged_read(Elem e, const PagedPools& c, const Q8Seqs& q, int n_layers, int n, const Q8Rows& k,
                             const Q8Rows& v, const Rotation& rot, hipStream_t s) {
    return launch_rows_of<true>(e, c, q, n_layers, n, k, v, rot, nullptr, s);
}

}  // namespace kvmap
