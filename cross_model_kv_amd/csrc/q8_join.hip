// Joining the pieces of cut items (the last step of attention over the 8-bit cache).
//
// A piece's sums are relative to its own maximum m: out = sum_w 2^(m_w - M) o_w / sum_w 2^(m_w - M) l_w with M the
// largest m_w.  The pieces are added in their order, so the result does not depend on who was first.  Bytes bound it
// (a row of a piece is 4 d + 8), and latency where they are few: loads of 8 pieces are in flight a thread, and the
// pieces of a row are dealt out over the workgroup where they are many.

#include <algorithm>

#include "common.h"
#include "internal.h"
#include "q8_mfma.h"

namespace kvmap {
namespace {

// COOP: a workgroup takes one row, its groups of d / 4 threads the pieces in turn; else a group takes a row.
template <bool BF16, int D, bool COOP>
__global__ __launch_bounds__(256) void q8_join_kernel(Q8Attend a, Q8Pieces sp) {
    constexpr int LANES = D / 4, NG = 256 / LANES, STEP = COOP ? NG : 1;
    constexpr int U = 8;  // pieces in flight
    __shared__ f32x4_t s_o[COOP ? NG : 1][LANES];
    __shared__ float s_ml[COOP ? NG : 1][2];
    const int group = threadIdx.x / LANES, d4 = threadIdx.x % LANES * 4;
    const int2 cut = sp.cut[blockIdx.x];
    const int item = sp.few ? blockIdx.x : cut.x, w0 = sp.few ? cut.x : blockIdx.x, n = cut.y;
    const int G = a.Hq / a.c.H, R = a.n_q * G;
    const int rb = item % sp.row_blocks, h = item / sp.row_blocks % a.c.H, b = item / sp.row_blocks / a.c.H;
    const int row = COOP ? blockIdx.y : blockIdx.y * NG + group;
    const int r = rb * sp.rows + row;
    if (n < 2 || row >= sp.rows || r >= R) return;
    float top = kNone, lsum = 0.f;
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = COOP ? group : 0; j0 < n; j0 += U * STEP) {
        float2 ml[U];
        f32x4_t po[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int w = min(j0 + u * STEP, n - 1);
            const int64_t from = q8_slot(w0 + w, w == 0) * sp.rows + row;
            ml[u] = *(const float2*)(sp.part_ml + from * 2);
            po[u] = *(const f32x4_t*)(sp.part_o + from * D + d4);
        }
        float t = top;
#pragma unroll
        for (int u = 0; u < U; ++u) t = fmaxf(t, ml[u].x);
        const float keep = __builtin_amdgcn_exp2f(top - t);
        lsum *= keep;
        sum *= keep;
        top = t;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j0 + u * STEP < n) {
                const float f = __builtin_amdgcn_exp2f(ml[u].x - t);
                lsum = fmaf(f, ml[u].y, lsum);
                sum += f * po[u];
            }
    }
    if (COOP) {
        s_o[group][threadIdx.x % LANES] = sum;
        if (d4 == 0) {
            s_ml[group][0] = top;
            s_ml[group][1] = lsum;
        }
        __syncthreads();
        if (group) return;
        top = s_ml[0][0];
#pragma unroll
        for (int k = 1; k < NG; ++k) top = fmaxf(top, s_ml[k][0]);
        lsum = 0.f;
        sum = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            const float f = __builtin_amdgcn_exp2f(s_ml[k][0] - top);
            lsum = fmaf(f, s_ml[k][1], lsum);
            sum += f * s_o[k][threadIdx.x];
        }
    }
    const int i = q8_query(a, r);
    q8_store_row<BF16>(a, b, i, h * G + r - i * G, d4, top, lsum, sum);
}

}  // namespace

// Where a plan's pieces leave what has to be joined; nowhere, if nothing can be cut.
Q8Pieces q8_pieces(const Q8Attend& a, const Q8Plan& p, void* scratch) {
    Q8Pieces s;
    s.row_blocks = p.row_blocks;
    s.rows = p.rows;
    s.grid = p.grid;
    s.few = (int64_t)a.B * a.c.H * p.row_blocks <= p.grid;
    s.cut = nullptr;
    s.part_ml = s.part_o = nullptr;
    if (!p.splits) return s;
    s.cut = (int2*)scratch;
    s.part_ml = (float*)(s.cut + p.grid);
    s.part_o = s.part_ml + (size_t)2 * p.grid * p.rows * 2;
    s.part_o += -((uintptr_t)s.part_o / 4) & 3;  // 16-byte aligned
    return s;
}
size_t q8_piece_bytes(int grid, int rows, int d) { return (size_t)grid * sizeof(int2) + (size_t)2 * grid * rows * (d + 2) * sizeof(float) + 16; }

template <bool BF16, int D>
static hipError_t launch(const Q8Attend& a, const Q8Pieces& sp, hipStream_t s) {
    const int64_t items = (int64_t)a.B * a.c.H * sp.row_blocks;
    const int rows = (int)std::min<int64_t>(sp.rows, (int64_t)a.n_q * (a.Hq / a.c.H));
    const unsigned jobs = (unsigned)std::min<int64_t>(items, sp.grid);
    // a group for a row joins 8 pieces in about the time of one; a workgroup for a row is worth it from twice that on
    if (items * 16 <= sp.grid) hipLaunchKernelGGL((q8_join_kernel<BF16, D, true>), dim3(jobs, rows), dim3(256), 0, s, a, sp);
    else hipLaunchKernelGGL((q8_join_kernel<BF16, D, false>), dim3(jobs, (rows + 1024 / D - 1) / (1024 / D)), dim3(256), 0, s, a, sp);
    return hipGetLastError();
}

hipError_t launch_q8_join(Elem e, const Q8Attend& a, const Q8Pieces& sp, hipStream_t s) {
    if (e == Elem::BF16) return a.c.d == 128 ? launch<true, 128>(a, sp, s) : launch<true, 64>(a, sp, s);
    return a.c.d == 128 ? launch<false, 128>(a, sp, s) : launch<false, 64>(a, sp, s);
}

}  // namespace kvmap
