// The 4-bit paged cache: quantize and append tokens, read them back.
#include "kv4_layout.h"
#include "mfma_common.h"

namespace pace {
namespace {

template <class T>
__device__ inline float kv_elem(const void *p, size_t i) {
    if constexpr (sizeof(T) == 2) return bf2f(((const uint16_t *)p)[i]);
    return ((const float *)p)[i];
}

// Quantize and write.  One workgroup per (sequence, head, tile of 32 tokens)
// and keys and values in turn; it owns the tile's words, so words of
// values that hold older tokens too are read, changed and written without
// a race.  Codes are staged in LDS as bytes, then packed by word.
template <class T>
__global__ void __launch_bounds__(256) kv4_append_kernel(Kv4View c, const int32_t *start, const int32_t *count,
                                                         int n_tok, const void *k, const void *v, int tiles) {
    extern __shared__ uint8_t codes[];   // [32][d]
    const int j = blockIdx.x % tiles, bh = blockIdx.x / tiles, b = bh / c.Hk, h = bh - b * c.Hk;
    const long long first = start[b];
    const int n = count ? min(max(count[b], 0), n_tok) : n_tok;
    const long long base = first >= 0 ? first / KV4_TILE : -((-first + KV4_TILE - 1) / KV4_TILE);
    const long long tile = base + j, p0 = tile * KV4_TILE;   // first position of the tile
    if (tile < 0 || tile > 0x7fffffff || p0 >= first + n) return;
    uint8_t *to = kv4_tile(c, b, h, (int)tile);
    if (!to) return;
    const int lo = first > p0 ? (int)(first - p0) : 0;                                   // live tokens of the tile
    const int hi = first + n < p0 + KV4_TILE ? (int)(first + n - p0) : KV4_TILE;
    const int groups = c.d / KV4_GROUP;
    for (int what = 0; what < 2; ++what) {
        const void *src = what ? v : k;
        float *scales = (float *)(to + (what ? kv4_value_scales(c.d) : kv4_key_scales(c.d)));
        // a wave per token and group: 64 lanes, 64 channels
        for (int u = threadIdx.x >> 6; u < KV4_TILE * groups; u += 4) {
            const int t = u / groups, g = u - t * groups, lane = threadIdx.x & 63;
            if (t < lo || t >= hi) continue;
            const size_t row = ((size_t)(p0 + t - first) * c.B + b) * c.Hk + h;
            const float x = kv_elem<T>(src, row * c.d + g * KV4_GROUP + lane);
            float top = fabsf(x);
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) top = xor_max(top, m);
            const float y = top > 0.f ? rintf((x * 7.f) / top) : 0.f;
            codes[t * c.d + g * KV4_GROUP + lane] = (uint8_t)((int)y + 8);
            if (lane == 0) scales[g * KV4_TILE + t] = top / 7.f;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 4 * c.d; i += 256) {
            const int w = (i >> 8) * 4 + (i & 3), lane = (i >> 2) & 63;   // the word at byte 4 i
            uint32_t word = 0, mask = 0;
            for (int e = 0; e < 8; ++e) {
                int t, ch, nib;
                if (what) {
                    t = (e >> 2) * 16 + (lane >> 4) * 4 + (e & 3);
                    ch = w * 16 + (lane & 15);
                    nib = e;
                } else {
                    const int per = c.d >> 5;
                    t = (w / per) * 16 + (lane & 15);
                    ch = (w % per) * 32 + (lane >> 4) * 8 + e;
                    nib = (e & 1) * 4 + (e >> 1);
                }
                if (t < lo || t >= hi) continue;
                word |= (uint32_t)(codes[t * c.d + ch] & 15) << (4 * nib);
                mask |= 15u << (4 * nib);
            }
            if (!mask) continue;
            uint32_t *dst = (uint32_t *)(to + what * 16 * c.d) + i;
            *dst = mask == 0xffffffffu ? word : ((*dst & ~mask) | word);
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4View c, const int32_t *start, const int32_t *count,
                                                       int n_tok, float *k, float *v, long long total) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int ch = (int)(i % c.d);
    const long long row = i / c.d;
    const int h = (int)(row % c.Hk), b = (int)(row / c.Hk % c.B), t = (int)(row / c.Hk / c.B);
    const long long p = (long long)start[b] + t;
    const int n = count ? min(max(count[b], 0), n_tok) : n_tok;
    const uint8_t *tile = t < n && p >= 0 && p / KV4_TILE <= 0x7fffffff ? kv4_tile(c, b, h, (int)(p / KV4_TILE)) : nullptr;
    float kx = 0.f, vx = 0.f;
    if (tile) {
        const int tt = (int)(p % KV4_TILE), g = ch / KV4_GROUP;
        int nib;
        const uint32_t wk = *(const uint32_t *)(tile + kv4_key_word(c.d, tt, ch, &nib));
        kx = (float)((int)((wk >> (4 * nib)) & 15) - 8) * ((const float *)(tile + kv4_key_scales(c.d)))[g * KV4_TILE + tt];
        const uint32_t wv = *(const uint32_t *)(tile + kv4_value_word(c.d, tt, ch, &nib));
        vx = (float)((int)((wv >> (4 * nib)) & 15) - 8) * ((const float *)(tile + kv4_value_scales(c.d)))[g * KV4_TILE + tt];
    }
    if (k) k[i] = kx;
    if (v) v[i] = vx;
}

}  // namespace

hipError_t launch_kv4_append(const Kv4View &c, const int32_t *start, const int32_t *count, int T,
                             const void *k, const void *v, int bf16, hipStream_t s) {
    const int tiles = (T + KV4_TILE - 2) / KV4_TILE + 1;   // most tiles that T tokens touch
    const dim3 grid((unsigned)((long long)c.B * c.Hk * tiles));
    const size_t lds = (size_t)KV4_TILE * c.d;
    if (bf16)
        hipLaunchKernelGGL(kv4_append_kernel<uint16_t>, grid, dim3(256), lds, s, c, start, count, T, k, v, tiles);
    else
        hipLaunchKernelGGL(kv4_append_kernel<float>, grid, dim3(256), lds, s, c, start, count, T, k, v, tiles);
    return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4View &c, const int32_t *start, const int32_t *count, int T,
                           float *k, float *v, hipStream_t s) {
    const long long total = (long long)T * c.B * c.Hk * c.d;
    hipLaunchKernelGGL(kv4_read_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s, c, start, count, T,
                       k, v, total);
    return hipGetLastError();
}

}  // namespace pace
