// Attention over the 8-bit paged cache.
//
// For query row i of sequence b at position pos = len - n_q + i, with y_t = scale * q . k_t, t <= pos:
//   m = max y_t,  l = sum exp(y_t - m),  out = sum exp(y_t - m) v_t / l,  lse = m + log l,
// in one pass over the tokens with a running m and l.

#include "common.h"
#include "internal.h"
#include "q8_span.h"

namespace kvmap {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float inf() { return __uint_as_float(0x7F800000u); }
__device__ __forceinline__ float nan32() { return __uint_as_float(0x7FC00000u); }

__device__ __forceinline__ void values4(uint32_t w, float* x) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[0] = a[0];
    x[1] = a[1];
    x[2] = b[0];
    x[3] = b[1];
}

// One workgroup a query row: 256 tokens a step, a thread a token for the scores and then a thread
// a dim for the values.
template <bool BF16, int D>
__global__ __launch_bounds__(256) void q8_attend_row_kernel(Q8Attend a) {
    __shared__ float sq[D];
    __shared__ float sp[256];
    __shared__ float red[4];
    __shared__ float part[256];
    const int tid = threadIdx.x;
    const int row = blockIdx.x % (a.n_q * a.Hq), b = blockIdx.x / (a.n_q * a.Hq);
    const int i = row / a.Hq, hq = row % a.Hq, h = hq / (a.Hq / a.c.H);
    const int P = a.c.page;
    const int len = a.len[b];
    const bool bad = len < 0 || len > a.max_len;
    const int end = bad ? 0 : len - a.n_q + i + 1;  // tokens that the row sees
    const int64_t qo = b * a.q.seq + hq * a.q.head + i * a.q.token;
    if (tid < D) {
        sq[tid] = (BF16 ? __uint_as_float((uint32_t)((const uint16_t*)a.q.base)[qo + tid] << 16) : ((const float*)a.q.base)[qo + tid]) *
                  (a.scale * kLog2e);
    }
    __syncthreads();
    const int32_t* pages = a.pages + (int64_t)b * a.max_pages;
    float m = -inf(), l = 0.f, o = 0.f;
    const int dim = tid % D, half = tid / D, parts = 256 / D;
    for (int t0 = 0; t0 < end; t0 += 256) {
        const int t = t0 + tid;
        float y = -inf();
        if (t < end) {
            const int pid = q8_page_at(pages, t / P, a.max_pages, a.c.n_pages);
            const bool held = pid >= 0;
            const int64_t page = (int64_t)(held ? pid : 0) * a.c.H + h;
            const uint4* k = (const uint4*)(a.c.k + (page * P + t % P) * D);
            float s = 0.f;
            for (int g = 0; g < D / 16; ++g) {
                const uint4 w = k[g];
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x[4];
                    values4(ww[e], x);
#pragma unroll
                    for (int z = 0; z < 4; ++z) s = fmaf(sq[16 * g + 4 * e + z], x[z], s);
                }
            }
            y = held ? s * a.c.ks[page] : nan32();
        }
        float top = y;
#pragma unroll
        for (int s = 32; s; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
        if ((tid & 63) == 0) red[tid >> 6] = top;
        __syncthreads();
        top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float m1 = fmaxf(m, top);
        const float ms = m1 == -inf() ? 0.f : m1;
        const float keep = exp2f(m - ms);
        const float p = t < end ? exp2f(y - ms) : 0.f;
        sp[tid] = p;
        float sum = p;
#pragma unroll
        for (int s = 32; s; s >>= 1) sum += __shfl_xor(sum, s);
        __syncthreads();
        if ((tid & 63) == 0) red[tid >> 6] = sum;
        __syncthreads();
        l = l * keep + (red[0] + red[1] + red[2] + red[3]);
        m = m1;
        o *= keep;
        for (int u = half * (256 / parts); u < (half + 1) * (256 / parts) && t0 + u < end; ++u) {
            const int tt = t0 + u;
            const int pid = q8_page_at(pages, tt / P, a.max_pages, a.c.n_pages);
            const bool held = pid >= 0;
            const int64_t page = (int64_t)(held ? pid : 0) * a.c.H + h;
            float x[4];
            values4(a.c.v[(page * D + dim) * P + tt % P], x);
            o = fmaf(sp[u], held ? x[0] * a.c.vs[page] : nan32(), o);
        }
        __syncthreads();
    }
    part[tid] = o;
    __syncthreads();
    if (tid < D) {
        for (int p = 1; p < parts; ++p) o += part[tid + p * D];
        o = bad ? nan32() : end > 0 ? o / l : 0.f;
        const int64_t oo = b * a.out.seq + hq * a.out.head + i * a.out.token;
        if (BF16)
            ((uint16_t*)a.out.base)[oo + tid] = (uint16_t)pack_bf16(o, 0.f);
        else
            ((float*)a.out.base)[oo + tid] = o;
    }
    if (tid == 0 && a.lse) a.lse[((int64_t)b * a.n_q + i) * a.Hq + hq] = bad ? nan32() : end > 0 ? (m + log2f(l)) * kLn2 : -inf();
}

}  // namespace

hipError_t launch_q8_attend(Elem e, const Q8Attend& a, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.B * a.n_q * a.Hq));
    if (e == Elem::BF16) {
        if (a.c.d == 128) hipLaunchKernelGGL((q8_attend_row_kernel<true, 128>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((q8_attend_row_kernel<true, 64>), grid, dim3(256), 0, s, a);
    } else {
        if (a.c.d == 128) hipLaunchKernelGGL((q8_attend_row_kernel<false, 128>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((q8_attend_row_kernel<false, 64>), grid, dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace kvmap
