// The 4-bit paged cache: quantize and append tokens, read them back.
#include "kv4_layout.h"
#include "mfma_common.h"

namespace pace {
namespace {

// eight elements
template <class T>
__device__ inline void load8(float *x, const void *p, size_t i) {
    if constexpr (sizeof(T) == 2) {
        const u32x4 w = *(const u32x4 *)((const uint16_t *)p + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[2 * e] = lo_f32(w[e]), x[2 * e + 1] = hi_f32(w[e]);
    } else {
        const f32x4 a = *(const f32x4 *)((const float *)p + i), b = *(const f32x4 *)((const float *)p + i + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = a[e], x[e + 4] = b[e];
    }
}

// Quantize and write.  One workgroup per (sequence, head, tile of 32 tokens),
// for keys and values in turn; it owns the tile's words, so value words that
// hold older tokens too are read, changed and written without a race.  Eight
// lanes take a token's group, eight channels each: the group's largest value
// is three lane swaps away, and the eight key codes are a word of the layout.
// Value words hold eight tokens of a channel and are collected through LDS.
// Codes are 7 x / max in float32: exact quotients where they can tie (bf16
// inputs have 8 bits, so a quotient that is not a tie is no nearer to one
// than 2^-9), rounded half to even.
template <class T, int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(Kv4View c, const int32_t *start, const int32_t *count,
                                                         int n_tok, const void *k, const void *v, int tiles) {
    constexpr int ROW = D + 4;   // bytes: rows of four-token steps in different banks
    __shared__ __align__(16) uint8_t codes[KV4_TILE * ROW];
    const int j = blockIdx.x % tiles, bh = blockIdx.x / tiles, b = bh / c.Hk, h = bh - b * c.Hk;
    const long long first = start[b];
    const int n = count ? min(max(count[b], 0), n_tok) : n_tok;
    const long long base = first >= 0 ? first / KV4_TILE : -((-first + KV4_TILE - 1) / KV4_TILE);
    const long long tile = base + j, p0 = tile * KV4_TILE;   // first position of the tile
    if (tile < 0 || tile >= (1 << 26) || p0 >= first + n) return;
    uint8_t *to = kv4_tile(c, b, h, (int)tile);
    if (!to) return;
    const int lo = first > p0 ? (int)(first - p0) : 0;                                   // live tokens of the tile
    const int hi = first + n < p0 + KV4_TILE ? (int)(first + n - p0) : KV4_TILE;
    constexpr int PER = D / 8;   // lanes of a token
#pragma unroll
    for (int what = 0; what < 2; ++what) {
        const void *src = what ? v : k;
        float *scales = (float *)(to + (what ? kv4_value_scales(D) : kv4_key_scales(D)));
        // the tokens from lo on, in whole steps of 256 / PER
        for (int t0 = lo; t0 < hi; t0 += 256 / PER) {
            const int t = t0 + threadIdx.x / PER, ch = threadIdx.x % PER * 8;
            const bool live = t < hi;
            float x[8] = {};
            if (live) load8<T>(x, src, (((size_t)(p0 + t - first) * c.B + b) * c.Hk + h) * D + ch);
            float top = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
            for (int m = 1; m < 8; m <<= 1) top = xor_max(top, m);
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = (uint32_t)((int)(top > 0.f ? rintf((x[e] * 7.f) / top) : 0.f) + 8);
            if (!live) continue;
            if ((threadIdx.x & 7) == 0) scales[ch / KV4_GROUP * KV4_TILE + t] = top / 7.f;
            if (what == 0) {
                uint32_t w = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) w |= y[e] << (4 * ((e & 1) * 4 + (e >> 1)));
                int nibble;
                *(uint32_t *)(to + kv4_key_word(D, t, ch, &nibble)) = w;
            } else {
                u32x2 w;
                w[0] = y[0] | y[1] << 8 | y[2] << 16 | y[3] << 24;
                w[1] = y[4] | y[5] << 8 | y[6] << 16 | y[7] << 24;
                *(uint32_t *)(codes + t * ROW + ch) = w[0];
                *(uint32_t *)(codes + t * ROW + ch + 4) = w[1];
            }
        }
    }
    __syncthreads();
    // value words: four channels of eight tokens at a time, 4 x 8 bytes to 4 words
    for (int i = threadIdx.x; i < D; i += 256) {
        const int quad = i / (D / 4), ch = i % (D / 4) * 4;   // tokens 4 quad .. and 16 + 4 quad ..
        uint32_t w[4] = {}, mask = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int t = (e >> 2) * 16 + quad * 4 + (e & 3);
            if (t < lo || t >= hi) continue;
            const uint32_t y = *(const uint32_t *)(codes + t * ROW + ch);
            mask |= 15u << (4 * e);
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x] |= ((y >> (8 * x)) & 15u) << (4 * e);
        }
        if (!mask) continue;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            int nibble;
            uint32_t *dst = (uint32_t *)(to + kv4_value_word(D, quad * 4, ch + x, &nibble));
            *dst = mask == 0xffffffffu ? w[x] : ((*dst & ~mask) | w[x]);
        }
    }
}

// Read back: a thread takes four adjacent channels of a token
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4View c, const int32_t *start, const int32_t *count,
                                                       int n_tok, float *k, float *v, long long total) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int per = c.d / 4, ch = (int)(i % per) * 4;
    const long long row = i / per, bt = row / c.Hk;
    const int h = (int)(row - bt * c.Hk), t = (int)(bt / c.B), b = (int)(bt - (long long)t * c.B);
    const long long p = (long long)start[b] + t;
    const int n = count ? min(max(count[b], 0), n_tok) : n_tok;
    const uint8_t *tile = t < n && p >= 0 && p < 0x7fffffff ? kv4_tile(c, b, h, (int)(p / KV4_TILE)) : nullptr;
    f32x4 kx = {0.f, 0.f, 0.f, 0.f}, vx = kx;
    if (tile) {
        const int tt = (int)(p % KV4_TILE), g = ch / KV4_GROUP;
        int nib;
        const uint32_t wk = *(const uint32_t *)(tile + kv4_key_word(c.d, tt, ch, &nib));
        const float sk = ((const float *)(tile + kv4_key_scales(c.d)))[g * KV4_TILE + tt];
        const float sv = ((const float *)(tile + kv4_value_scales(c.d)))[g * KV4_TILE + tt];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int kn = ((e & 1) * 4 + (((ch & 7) + e) >> 1));
            kx[e] = (float)((int)((wk >> (4 * kn)) & 15) - 8) * sk;
            const uint32_t wv = *(const uint32_t *)(tile + kv4_value_word(c.d, tt, ch + e, &nib));
            vx[e] = (float)((int)((wv >> (4 * nib)) & 15) - 8) * sv;
        }
    }
    if (k) *(f32x4 *)(k + 4 * i) = kx;
    if (v) *(f32x4 *)(v + 4 * i) = vx;
}

template <class T>
void launch_append(const Kv4View &c, const int32_t *start, const int32_t *count, int n_tok, const void *k,
                   const void *v, hipStream_t s) {
    const int tiles = (n_tok + KV4_TILE - 2) / KV4_TILE + 1;   // most tiles that n_tok tokens touch
    const dim3 grid((unsigned)((long long)c.B * c.Hk * tiles)), wg(256);
    if (c.d == 64)
        hipLaunchKernelGGL((kv4_append_kernel<T, 64>), grid, wg, 0, s, c, start, count, n_tok, k, v, tiles);
    else if (c.d == 128)
        hipLaunchKernelGGL((kv4_append_kernel<T, 128>), grid, wg, 0, s, c, start, count, n_tok, k, v, tiles);
    else
        hipLaunchKernelGGL((kv4_append_kernel<T, 256>), grid, wg, 0, s, c, start, count, n_tok, k, v, tiles);
}

}  // namespace

hipError_t launch_kv4_append(const Kv4View &c, const int32_t *start, const int32_t *count, int T,
                             const void *k, const void *v, int bf16, hipStream_t s) {
    bf16 ? launch_append<uint16_t>(c, start, count, T, k, v, s) : launch_append<float>(c, start, count, T, k, v, s);
    return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4View &c, const int32_t *start, const int32_t *count, int T,
                           float *k, float *v, hipStream_t s) {
    const long long total = (long long)T * c.B * c.Hk * (c.d / 4);
    hipLaunchKernelGGL(kv4_read_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s, c, start, count, T,
                       k, v, total);
    return hipGetLastError();
}

}  // namespace pace
