// Head norms of queries and keys with the position rotation.
#include "../../include/pace.h"
#include "mfma_common.h"
#include "pace_layers.h"

namespace pace {
namespace {

template <class T>
struct Elem;
template <>
struct Elem<float> {
    static __device__ inline float get(const void *p, long long i) { return ((const float *)p)[i]; }
    static __device__ inline void put(void *p, long long i, float x) { ((float *)p)[i] = x; }
};
template <>
struct Elem<uint16_t> {
    static __device__ inline float get(const void *p, long long i) { return bf2f(((const uint16_t *)p)[i]); }
    static __device__ inline void put(void *p, long long i, float x) {
        ((uint16_t *)p)[i] = (uint16_t)(pk_bf16(x, 0.f) & 0xffff);
    }
};

__device__ inline float wave_sum(float x) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
    return x;
}

// one wave per (row, head), a lane takes channels lane, lane + 64, ...; a
// pair of rotated channels is read and written by one lane, so outputs may
// be the inputs
template <class T>
__global__ void __launch_bounds__(256) norm_any_kernel(NormArgs a, long long units) {
    const int lane = threadIdx.x & 63;
    const long long u = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (u >= units) return;
    const long long t = u / a.heads;
    const int hh = (int)(u - t * a.heads), key = hh >= a.heads_q;
    const int h = key ? hh - a.heads_q : hh, H = key ? a.heads - a.heads_q : a.heads_q;
    const void *x = a.x[key];
    const long long in = t * a.stride[key] + (long long)h * a.d, to = (t * H + h) * a.d;
    float ss = 0.f;
    for (int i = lane; i < a.d; i += 64) {
        const float e = Elem<T>::get(x, in + i);
        ss = fmaf(e, e, ss);
    }
    ss = wave_sum(ss);
    float r = 1.f;
    if (a.norm == PACE_NORM_L2) r = 1.f / sqrtf(ss + a.eps);
    if (a.norm == PACE_NORM_RMS) r = 1.f / sqrtf(ss / (float)a.d + a.eps);
    const float scale = key ? 1.f : a.q_scale;
    const float *w = a.weight[key];
    const int half = a.rot / 2;
    for (int i = lane; i < half; i += 64) {
        const int c0 = a.adjacent ? 2 * i : i, c1 = a.adjacent ? 2 * i + 1 : i + half;
        const float x0 = Elem<T>::get(x, in + c0) * r * (w ? w[c0] : 1.f);
        const float x1 = Elem<T>::get(x, in + c1) * r * (w ? w[c1] : 1.f);
        double turns = (double)a.pos[t] * (double)a.inv_freq[i] * 0.15915494309189535;
        turns -= rint(turns);
        float sn, cs;
        sincospif(2.f * (float)turns, &sn, &cs);
        Elem<T>::put(a.y[key], to + c0, (x0 * cs - x1 * sn) * scale);
        Elem<T>::put(a.y[key], to + c1, (x1 * cs + x0 * sn) * scale);
    }
    for (int i = a.rot + lane; i < a.d; i += 64)
        Elem<T>::put(a.y[key], to + i, Elem<T>::get(x, in + i) * r * (w ? w[i] : 1.f) * scale);
}

}  // namespace

hipError_t launch_qk_norm_rope(const NormArgs &a, int bf16, hipStream_t s) {
    const long long units = a.tokens * a.heads;
    const unsigned blocks = (unsigned)((units + 3) / 4);
    if (bf16)
        hipLaunchKernelGGL(norm_any_kernel<uint16_t>, dim3(blocks), dim3(256), 0, s, a, units);
    else
        hipLaunchKernelGGL(norm_any_kernel<float>, dim3(blocks), dim3(256), 0, s, a, units);
    return hipGetLastError();
}

}  // namespace pace
