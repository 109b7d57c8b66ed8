// What the kernels that attend over the 8-bit cache share: e4m3 codes, queries and softmax weights as matrix
// operands, and the constants of the running softmax.
#pragma once

#include "common.h"
#include "internal.h"
#include "q8_span.h"

namespace kvmap {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -3.4028235e38f;  // the running maximum of a row that has seen no token
constexpr float kSlack = 14.f;   // m is moved when a score passes it by more than this (not the prompt kernel's fp16 weights)

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

// x as a sum of N bf16 parts of 8 bits each: off by at most 2^(-8 N) of itself, over fp32's range of exponents
template <int N>
struct Parts {
    bf16x8_t p[N];
    __device__ __forceinline__ void put(int i, float x0, float x1) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const bf16x2_t y = __builtin_convertvector((f32x2_t{x0, x1}), bf16x2_t);
            p[k][i] = y[0];
            p[k][i + 1] = y[1];
            x0 -= (float)y[0];
            x1 -= (float)y[1];
        }
    }
    __device__ __forceinline__ void set(const float* x) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) put(i, x[i], x[i + 1]);
    }
};

// Weights in N bf16 parts.
template <int N>
struct PartWeights : Parts<N> {
    using Codes = bf16x8_t;
    __device__ static __forceinline__ Codes codes(uint32_t a, uint32_t b) { return bf16_codes(a, b); }
    __device__ __forceinline__ f32x4_t times(Codes v, f32x4_t o) const {
#pragma unroll
        for (int k = N; k--;) o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, this->p[k], o, 0, 0, 0);
        return o;
    }
    __device__ __forceinline__ f32x16_t times(Codes v, f32x16_t o) const {
#pragma unroll
        for (int k = N; k--;) o = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, this->p[k], o, 0, 0, 0);
        return o;
    }
};

template <>
struct Weights<true> {
    using Codes = f16x8_t;
    Codes p;
    __device__ __forceinline__ void put(int i, float x0, float x1) {
        const f16x2_t y = __builtin_convertvector((f32x2_t{x0, x1}), f16x2_t);
        p[i] = y[0];
        p[i + 1] = y[1];
    }
    __device__ __forceinline__ void set(const float* x) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) put(i, x[i], x[i + 1]);
    }
    __device__ static __forceinline__ Codes codes(uint32_t a, uint32_t b) { return f16_codes(a, b); }
    __device__ __forceinline__ f32x16_t times(Codes v, f32x16_t o) const { return __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p, o, 0, 0, 0); }
};
template <>
struct Weights<false> : PartWeights<3> {};

// s (+)= k q with s in vector registers and q in accumulation registers.  Where a kernel may use accumulation registers the
// compiler puts every product's result there, and moves what vector instructions need of it, one register an instruction:
// a quarter of the vector work of a tile.  Written out, the compiler does not know that it is a matrix product, whose result
// may not be touched by a vector instruction close behind it (8 passes): the caller keeps them apart, and
// tests/test_q8_listing.py reads the listing for 13 instructions between them.
template <bool FIRST>
__device__ __forceinline__ void mfma_to_vector(bf16x8_t k, bf16x8_t q, f32x16_t& s) {
    if (FIRST) asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(s) : "v"(k), "a"(q));
    else asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(s) : "v"(k), "a"(q));
}

// Puts q where mfma_to_vector takes it from, once and for all: copied there in front of a use, it would not be there in time.
template <class T>
__device__ __forceinline__ void keep_accumulated(T& q) { asm volatile("" : "+a"(q)); }

// From here on vector instructions may read s.
__device__ __forceinline__ void product_done(f32x16_t& s) { asm volatile("s_nop 15" : "+v"(s)); }

// o *= by, o in accumulation registers.  (As plain arithmetic in a branch, the compiler moves all of o to vector registers in
// front of the branch, taken or not.)
__device__ __forceinline__ void scale_product(f32x16_t& o, float by) {
    asm volatile("s_nop 15" : "+a"(o));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float x = o[i], t;
        asm volatile("v_accvgpr_read_b32 %1, %0\n\tv_mul_f32 %1, %2, %1\n\tv_accvgpr_write_b32 %0, %1" : "+a"(x), "=&v"(t) : "v"(by));
        o[i] = x;
    }
}

// x (+)= v w, and o = keep o + by x, in the same way.
__device__ __forceinline__ void first_product(f16x8_t v, f16x8_t w, f32x16_t& x) {
    asm volatile("s_nop 15\n\tv_mfma_f32_32x32x16_f16 %0, %1, %2, 0" : "=&v"(x) : "v"(v), "v"(w));
}
__device__ __forceinline__ void next_product(f16x8_t v, f16x8_t w, f32x16_t& x) {
    asm volatile("s_nop 15\n\tv_mfma_f32_32x32x16_f16 %0, %1, %2, %0\n\ts_nop 15" : "+v"(x) : "v"(v), "v"(w));
}
__device__ __forceinline__ void add_product(f32x16_t& o, float keep, f32x16_t x, float by) {
    asm volatile("s_nop 15" : "+a"(o));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float y = o[i], t;
        asm volatile("v_accvgpr_read_b32 %1, %0\n\tv_mul_f32 %1, %4, %1\n\tv_fmac_f32 %1, %3, %2\n\tv_accvgpr_write_b32 %0, %1"
                     : "+a"(y), "=&v"(t) : "v"(x[i]), "s"(by), "v"(keep));
        o[i] = y;
    }
}

template <bool BF16>
struct Query;  // 8 dims of a query row as a matrix operand
template <>
struct Query<true> {
    bf16x8_t p;
    __device__ __forceinline__ void load(const void* base, int64_t at) { p = *(const bf16x8_t*)((const __bf16*)base + at); }
    __device__ __forceinline__ void zero() { p = bf16x8_t{}; }
    __device__ __forceinline__ f32x4_t times(bf16x8_t k, f32x4_t s) const { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, p, s, 0, 0, 0); }
    __device__ __forceinline__ void keep() { keep_accumulated(p); }
    // s (+)= k times the queries, s in vector registers.
    template <bool FIRST>
    __device__ __forceinline__ void to_vector(bf16x8_t k, f32x16_t& s) const { mfma_to_vector<FIRST>(k, p, s); }
};
template <>
struct Query<false> : Parts<3> {
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
    __device__ __forceinline__ void keep() {
#pragma unroll
        for (int k = 0; k < 3; ++k) keep_accumulated(p[k]);
    }
    template <bool FIRST>
    __device__ __forceinline__ void to_vector(bf16x8_t k, f32x16_t& s) const {
        mfma_to_vector<FIRST>(k, p[2], s);
        mfma_to_vector<false>(k, p[1], s);
        mfma_to_vector<false>(k, p[0], s);
    }
};

// Lane n's value, n the same in all lanes.
__device__ __forceinline__ uint32_t lane_value(uint32_t x, int n) { return (uint32_t)__builtin_amdgcn_readlane((int)x, n); }
__device__ __forceinline__ uint64_t lane_value(uint64_t x, int n) {
    return (uint64_t)lane_value((uint32_t)(x >> 32), n) << 32 | lane_value((uint32_t)x, n);
}

// Sums of the lanes up to and including one's own; all 64 lanes take part.  Through registers: a step through shared memory's
// crossbar (a shuffle) is 100 cycles of waiting, and a workgroup finds its work with four such sums.
template <int FROM, int ROWS>
__device__ __forceinline__ uint32_t lanes_from(uint32_t x) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, FROM, ROWS, 0xF, false); }
template <int FROM, int ROWS>
__device__ __forceinline__ uint64_t lanes_from(uint64_t x) {
    return (uint64_t)lanes_from<FROM, ROWS>((uint32_t)(x >> 32)) << 32 | lanes_from<FROM, ROWS>((uint32_t)x);
}
template <class T>
__device__ __forceinline__ T wave_scan(T x) {
    x += lanes_from<0x111, 0xF>(x);  // 1, 2, 4, 8 lanes below, inside rows of 16 (0 where there is none)
    x += lanes_from<0x112, 0xF>(x);
    x += lanes_from<0x114, 0xF>(x);
    x += lanes_from<0x118, 0xF>(x);
    x += lanes_from<0x142, 0xA>(x);  // a row's last lane, for the odd rows
    x += lanes_from<0x143, 0xC>(x);  // lane 31, for the rows above it
    return x;
}

// Division with the usual case of small numbers in 32 bits.
__device__ __forceinline__ uint64_t div64(uint64_t a, uint64_t b) {
    return (a | b) >> 32 ? a / b : (uint64_t)((uint32_t)a / (uint32_t)b);
}

// A piece's slots: one for an item that it begins (its last), one for an item that began before (its first).
__host__ __device__ __forceinline__ int64_t q8_slot(int64_t piece, bool begins) { return 2 * piece + begins; }

// A value scale 2^e, and 2^-e.  The sum of a row's weights l = sum exp2(y - m) is held in 64 bits: m follows the largest
// y + e, and where scales are 2^-110 (a page of zeros) 32 bits would overflow.
__device__ __forceinline__ int scale_exponent(float s) { return (int)(__float_as_uint(s) >> 23) - 127; }
__device__ __forceinline__ double inverse_scale(int e) { return __hiloint2double((1023 - e) << 20, 0); }

// A row's sums as they are stored and joined: l in [0.5, 1) with its exponent in m, and the factor 2^-exponent for o.
__device__ __forceinline__ int settle_sum(double l, float& m, float& lf) {
    const int e = __builtin_amdgcn_frexp_exp(l);
    lf = (float)__builtin_amdgcn_frexp_mant(l);
    m += (float)e;
    return -e;
}

// The query of a row.
__device__ __forceinline__ int q8_query(const Q8Attend& a, int r) { return q8_divide(r, a.g_mul, a.g_shift); }

// A row's lse; one whose weights sum to 0 saw no token.
__device__ __forceinline__ float q8_lse(float top, float lsum) { return lsum == 0.f ? -inf32() : (top + __builtin_amdgcn_logf(lsum)) * kLn2; }

// 4 dims of one answered row, and at dim 0 its lse.
template <bool BF16>
__device__ __forceinline__ void q8_store_row(const Q8Attend& a, int b, int i, int hq, int d4, float top, float lsum, f32x4_t sum) {
    sum *= lsum == 0.f ? 0.f : 1.f / lsum;
    const int64_t at = (int64_t)b * a.out.seq + (int64_t)hq * a.out.head + (int64_t)i * a.out.token + d4;
    if (BF16)
        *(uint2*)((uint16_t*)a.out.base + at) = make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
    else
        *(f32x4_t*)((float*)a.out.base + at) = sum;
    if (d4 == 0 && a.lse)
        a.lse[((int64_t)b * a.n_q + i) * a.Hq + hq] = q8_lse(top, lsum);
}

}  // namespace
}  // namespace kvmap
