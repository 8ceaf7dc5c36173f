// Head norms of queries and keys with the position rotation: one pass,
// y = R(pos) (x / norm(x) * weight) * scale, bound by reading x and writing y.
//
// A lane owns units of 2 V channels: V pairs that turn together, or 2 V
// channels that do not turn.  So the rotation needs no exchange between
// lanes, outputs may be the inputs, and the only cross-lane step is the sum of
// squares over the lanes of a row.  A workgroup takes a few tokens with all
// their heads and computes the tokens' sines and cosines once, into LDS: the
// angle pos * freq needs float64 to be reduced (a float32 product of a far
// position is off by whole radians), which is too slow to repeat for each head.
//
// 16384 rows of 32 + 8 heads of 128 channels, bf16, half of them rotated: 66 us,
// 5.1 TB/s (a large copy reaches 6.6).  32 rows of 16 + 16 heads: 3.2 us, the
// launch and one round of loads.
#include <algorithm>

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

// sine and cosine of pos * freq: the product and its reduction to a turn in
// float64 (within 2^-24 of a turn), the functions in float32
__device__ inline f32x2 turn(int pos, float freq) {
    double turns = (double)pos * (double)freq * 0.15915494309189535;
    turns -= rint(turns);
    float sn, cs;
    sincospif(2.f * (float)turns, &sn, &cs);
    return f32x2{cs, sn};
}

__device__ inline float norm_factor(const NormArgs &a, float ss) {
    if (a.norm == PACE_NORM_L2) return 1.f / sqrtf(ss + a.eps);
    if (a.norm == PACE_NORM_RMS) return 1.f / sqrtf(ss / (float)a.d + a.eps);
    return 1.f;
}

template <class T, int V>
struct Vec {
    typedef T type __attribute__((ext_vector_type(V)));
};

template <class T>
__device__ inline float widen(T x) {
    if constexpr (sizeof(T) == 2) return bf2f(x);
    return x;
}

// V elements, with the alignment of the vector
template <class T, int V>
__device__ inline void load_vec(float *x, const T *p) {
    const auto v = *(const typename Vec<T, V>::type *)p;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = widen<T>(v[i]);
}
template <class T, int V>
__device__ inline void store_vec(T *p, const float *x) {
    typename Vec<T, V>::type v;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const uint32_t w = pk_bf16(x[i], x[i + 1]);
            v[i] = (uint16_t)w, v[i + 1] = (uint16_t)(w >> 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = x[i];
    }
    *(typename Vec<T, V>::type *)p = v;
}

// L lanes a row (a power of two), U units a lane; `per` tokens a workgroup
template <class T, int V, int U>
__global__ void __launch_bounds__(256) norm_units_kernel(NormArgs a, int L, int per, int splits) {
    extern __shared__ __align__(16) f32x2 table[];   // [per][rot / 2] (cos, sin)
    const long long t0 = (long long)(blockIdx.x / splits) * per;
    const int part = blockIdx.x % splits, half = a.rot / 2;
    const int n_tok = (int)min((long long)per, a.tokens - t0);
    if (half) {
        for (int i = threadIdx.x; i < n_tok * half; i += 256)
            table[i] = turn(a.pos[t0 + i / half], a.inv_freq[i % half]);
    }
    float *weights = (float *)(table + ((per * half + 1) & ~1));   // [2][d]
    const bool weighted = a.weight[0] || a.weight[1];
    if (weighted) {
        for (int i = threadIdx.x; i < 2 * a.d; i += 256) {
            const float *w = a.weight[i >= a.d];
            weights[i] = w ? w[i >= a.d ? i - a.d : i] : 1.f;
        }
    }
    if (half || weighted) __syncthreads();
    const int sub = threadIdx.x % L, rows = 256 / L, units = a.d / (2 * V), turning = half / V;
    // channels of a lane's units and their place in the table
    int c0[U], c1[U], at[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int u = sub + j * L;
        at[j] = u < turning ? u * V : -1;
        if (u < turning && !a.adjacent)
            c0[j] = u * V, c1[j] = half + u * V;
        else
            c0[j] = 2 * V * u, c1[j] = 2 * V * u + V;
    }
    const int total = n_tok * a.heads, share = (total + splits - 1) / splits;
    const int first = part * share, last = min(first + share, total);
    for (int base = first; base < last; base += rows) {
        const int row = base + threadIdx.x / L;
        const bool live = row < last;   // every lane takes part in the sums
        const int tt = live ? row / a.heads : 0, hh = live ? row - tt * a.heads : 0, key = hh >= a.heads_q;
        const int h = key ? hh - a.heads_q : hh, H = key ? a.heads - a.heads_q : a.heads_q;
        const T *x = (const T *)a.x[key] + (t0 + tt) * a.stride[key] + (long long)h * a.d;
        T *y = (T *)a.y[key] + ((t0 + tt) * H + h) * a.d;
        float v[U][2 * V];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (!live || sub + j * L >= units) continue;
            load_vec<T, V>(v[j], x + c0[j]);
            load_vec<T, V>(v[j] + V, x + c1[j]);
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) ss = fmaf(v[j][i], v[j][i], ss);
        }
        for (int m = 1; m < L; m <<= 1) ss += __shfl_xor(ss, m);
        const float r = norm_factor(a, ss) * (key ? 1.f : a.q_scale);
        const float *w = weights + key * a.d;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (!live || sub + j * L >= units) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) v[j][i] *= r, v[j][V + i] *= r;
            if (weighted) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[j][i] *= w[c0[j] + i], v[j][V + i] *= w[c1[j] + i];
            }
            if (at[j] >= 0) {
                const f32x2 *cs = table + tt * half + at[j];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const f32x2 k = cs[i];
                    float *p = a.adjacent ? &v[j][2 * i] : &v[j][i], *q = a.adjacent ? &v[j][2 * i + 1] : &v[j][V + i];
                    const float x0 = *p, x1 = *q;
                    *p = x0 * k[0] - x1 * k[1];
                    *q = x1 * k[0] + x0 * k[1];
                }
            }
            store_vec<T, V>(y + c0[j], v[j]);
            store_vec<T, V>(y + c1[j], v[j] + V);
        }
    }
}

// Any size and alignment: one wave per (row, head), channel by channel
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
    const float r = norm_factor(a, ss);
    const float scale = key ? 1.f : a.q_scale;
    const float *w = a.weight[key];
    const int half = a.rot / 2;
    for (int i = lane; i < half; i += 64) {
        const int c0 = a.adjacent ? 2 * i : i, c1 = a.adjacent ? 2 * i + 1 : i + half;
        const float x0 = Elem<T>::get(x, in + c0) * r * (w ? w[c0] : 1.f);
        const float x1 = Elem<T>::get(x, in + c1) * r * (w ? w[c1] : 1.f);
        const f32x2 k = turn(a.pos[t], a.inv_freq[i]);
        Elem<T>::put(a.y[key], to + c0, (x0 * k[0] - x1 * k[1]) * scale);
        Elem<T>::put(a.y[key], to + c1, (x1 * k[0] + x0 * k[1]) * scale);
    }
    for (int i = a.rot + lane; i < a.d; i += 64)
        Elem<T>::put(a.y[key], to + i, Elem<T>::get(x, in + i) * r * (w ? w[i] : 1.f) * scale);
}

template <class T, int V, int U>
void launch_units(const NormArgs &a, int L, int per, int splits, hipStream_t s) {
    const unsigned blocks = (unsigned)((a.tokens + per - 1) / per * splits);
    const size_t lds = (((size_t)per * (a.rot / 2) + 1) & ~(size_t)1) * sizeof(f32x2) +
                       (a.weight[0] || a.weight[1] ? 2 * a.d * sizeof(float) : 0);
    hipLaunchKernelGGL((norm_units_kernel<T, V, U>), dim3(blocks), dim3(256), lds, s, a, L, per, splits);
}

template <class T, int V>
bool try_units(const NormArgs &a, hipStream_t s) {
    // whole vectors everywhere: the halves, the channels behind the rotation,
    // the rows' strides and the pointers
    const int half = a.rot / 2;
    if (a.d % (2 * V) || a.rot % (2 * V) || (!a.adjacent && half % V)) return false;
    for (int i = 0; i < 2; ++i) {
        if (i ? a.heads == a.heads_q : a.heads_q == 0) continue;
        if (a.stride[i] % V || (uintptr_t)a.x[i] % (V * sizeof(T)) || (uintptr_t)a.y[i] % (V * sizeof(T))) return false;
    }
    const int units = a.d / (2 * V);
    int L = 1;
    while (L < units && L < 64) L *= 2;
    const int U = (units + L - 1) / L;
    if (U > 2) return false;
    // tokens of a workgroup: two passes of its rows where there are many
    // tokens (the table of angles is shared by a token's heads), less where
    // that would leave units idle, down to parts of a token
    const int rows = 256 / L;
    long long per = std::max(1, 2 * rows / a.heads);
    if (half) per = std::min(per, (long long)std::max(1, 4096 / half));   // 32 KB of angles
    per = std::max(1ll, std::min(per, a.tokens / 1024));
    const long long groups = (a.tokens + per - 1) / per;
    const int splits = groups >= 256 ? 1 : (int)std::max(1ll, std::min(512 / groups, (long long)(a.heads + rows - 1) / rows));
    if (U == 1)
        launch_units<T, V, 1>(a, L, (int)per, splits, s);
    else
        launch_units<T, V, 2>(a, L, (int)per, splits, s);
    return true;
}

}  // namespace

hipError_t launch_qk_norm_rope(const NormArgs &a, int bf16, hipStream_t s) {
    // the widest vectors that the sizes allow (12986 rows of 48 heads of 96 channels, 24 rotated,
    // bf16: 55 us by four elements, 85 us by two)
    if (bf16 ? try_units<uint16_t, 8>(a, s) || try_units<uint16_t, 4>(a, s) || try_units<uint16_t, 2>(a, s)
             : try_units<float, 4>(a, s) || try_units<float, 2>(a, s) || try_units<float, 1>(a, s))
        return hipGetLastError();
    const long long units = a.tokens * a.heads;
    const unsigned blocks = (unsigned)((units + 3) / 4);
    if (bf16)
        hipLaunchKernelGGL(norm_any_kernel<uint16_t>, dim3(blocks), dim3(256), 0, s, a, units);
    else
        hipLaunchKernelGGL(norm_any_kernel<float>, dim3(blocks), dim3(256), 0, s, a, units);
    return hipGetLastError();
}

}  // namespace pace
