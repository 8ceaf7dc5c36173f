// Linear attention with a fixed decay for each head, recurrent form.
#include "mfma_common.h"
#include "pace_layers.h"

namespace pace {
namespace {

template <class T>
__device__ inline float in_elem(const void *p, size_t i) {
    if constexpr (sizeof(T) == 2) return bf2f(((const uint16_t *)p)[i]);
    return ((const float *)p)[i];
}

// Recurrent form.  One workgroup per (sequence, head, block of 4 CG columns):
// a thread holds 4 adjacent columns of DK / RG state rows in registers over
// all tokens, so the state is read and written once.  o_t = M_t^T q_t is
// summed over a thread's rows, then over the row groups in LDS.
template <class T, int DK, int CG>
__global__ void __launch_bounds__(256) linear_step_kernel(LinearArgs a, int col_blocks) {
    constexpr int RG = 256 / CG, NR = DK / RG;
    __shared__ f32x4 part[RG][CG];
    __shared__ float kq[2][DK];
    const int cb = blockIdx.x % col_blocks, bh = blockIdx.x / col_blocks;
    const int b = bh / a.H, h = bh - b * a.H;
    const int cg = threadIdx.x % CG, rg = threadIdx.x / CG, col = (cb * CG + cg) * 4;
    const int n = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const float g = a.decay[h];
    const size_t base = (size_t)bh * DK * a.dv + (size_t)(rg * NR) * a.dv + col;
    f32x4 M[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        M[i] = a.state_in ? *(const f32x4 *)(a.state_in + base + (size_t)i * a.dv) : f32x4{0.f, 0.f, 0.f, 0.f};
    for (int t = 0; t < n; ++t) {
        const size_t row = (size_t)t * a.B * a.H + bh;
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * DK; i += 256)
            kq[i / DK][i % DK] = in_elem<T>(i < DK ? a.k : a.q, row * DK + i % DK);
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = in_elem<T>(a.v, row * a.dv + col + e);
        __syncthreads();
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const float kk = kq[0][rg * NR + i], qq = kq[1][rg * NR + i];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                M[i][e] = fmaf(kk, v[e], M[i][e] * g);
                o[e] = fmaf(qq, M[i][e], o[e]);
            }
        }
        part[rg][cg] = o;
        __syncthreads();
        if (rg == 0) {
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
            for (int r = 0; r < RG; ++r) sum += part[r][cg];
            *(f32x4 *)(a.out + row * a.dv + col) = sum * a.scale;
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) *(f32x4 *)(a.state_out + base + (size_t)i * a.dv) = M[i];
}

template <class T, int DK>
hipError_t launch_step(const LinearArgs &a, hipStream_t s) {
    const int cg = a.dv % 128 == 0 ? 32 : a.dv % 64 == 0 ? 16 : a.dv % 32 == 0 ? 8 : 4;
    const int cb = a.dv / (4 * cg);
    const dim3 grid((unsigned)((long long)a.B * a.H * cb)), wg(256);
    switch (cg) {
        case 32: hipLaunchKernelGGL((linear_step_kernel<T, DK, 32>), grid, wg, 0, s, a, cb); break;
        case 16: hipLaunchKernelGGL((linear_step_kernel<T, DK, 16>), grid, wg, 0, s, a, cb); break;
        case 8: hipLaunchKernelGGL((linear_step_kernel<T, DK, 8>), grid, wg, 0, s, a, cb); break;
        default: hipLaunchKernelGGL((linear_step_kernel<T, DK, 4>), grid, wg, 0, s, a, cb); break;
    }
    return hipGetLastError();
}

}  // namespace

uint64_t linear_attn_workspace(int, int, int, int, int, int) { return 0; }

hipError_t launch_linear_attn(const LinearArgs &a, int bf16, hipStream_t s) {
    if (bf16) return a.dk == 128 ? launch_step<uint16_t, 128>(a, s) : launch_step<uint16_t, 64>(a, s);
    return a.dk == 128 ? launch_step<float, 128>(a, s) : launch_step<float, 64>(a, s);
}

}  // namespace pace
