// The 4-bit paged cache: quantize and append tokens, read them back.
#include "kv4_layout.h"
#include "mfma_common.h"

namespace pace {
namespace {

// The part of a call that one workgroup works on: a tile of 32 positions of one
// (sequence, head).  Its arguments come by scalar loads.
struct TileWork {
    int b, h, lo, hi, upto;      // tokens lo .. hi - 1 of the tile are the call's, those below `upto` live
    long long tile, t0;          // t0: the call's token at the tile's first position
    __device__ inline TileWork(const Kv4View &c, const int32_t *start, const int32_t *count, int n_tok, int tiles) {
        typedef const __attribute__((address_space(4))) int32_t *scalar_ptr;
        const int j = blockIdx.x % tiles, bh = blockIdx.x / tiles;
        b = bh / c.Hk, h = bh - b * c.Hk;
        const long long first = ((scalar_ptr)(uintptr_t)start)[b];
        const int n = count ? min(max(((scalar_ptr)(uintptr_t)count)[b], 0), n_tok) : n_tok;
        tile = (first >> 5) + j;   // rounds down
        t0 = tile * KV4_TILE - first;
        lo = (int)max(-t0, 0ll);
        hi = (int)min((long long)n_tok - t0, (long long)KV4_TILE);
        upto = (int)min(max((long long)n - t0, 0ll), (long long)KV4_TILE);
    }
    __device__ inline uint8_t *address(const Kv4View &c) const {
        typedef const __attribute__((address_space(4))) int32_t *scalar_ptr;
        if (tile < 0 || tile >= (1 << 26)) return nullptr;
        const int per = c.page_tokens / KV4_TILE, col = kv4_column(c, (int)tile);
        if (col >= c.max_pages) return nullptr;
        const int page = ((scalar_ptr)(uintptr_t)c.table)[(size_t)b * c.max_pages + col];
        if (page < 0 || page >= c.n_pages) return nullptr;
        return c.pool + (((size_t)page * c.Hk + h) * per + ((int)tile - col * per)) * kv4_tile_bytes(c.d);
    }
};

// eight elements as they stand in memory, and as floats
template <class T>
struct Eight {
    u32x4 w[sizeof(T) / 2];
    __device__ inline void load(const void *p, size_t i) {
        const u32x4 *from = (const u32x4 *)((const T *)p + i);
        w[0] = from[0];
        if constexpr (sizeof(T) == 4) w[1] = from[1];
    }
    __device__ inline float get(int e) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e >> 2][e & 3]);
        return e & 1 ? hi_f32(w[0][e >> 1]) : lo_f32(w[0][e >> 1]);
    }
};

// Quantize and write.  One workgroup per (sequence, head, tile of 32 tokens); it
// owns the tile's words, so value words that hold older tokens too are read,
// changed and written without a race.  Eight lanes take a token's group, eight
// channels each: the group's largest value is three lane swaps away, and the
// eight key codes are a word of the layout.  Value words hold eight tokens of a
// channel and are collected through LDS.  A call's time is that of its chain of
// loads (arguments, table, data), so the data are asked for before the table
// entry is there, and the old value words before the new ones are known.
// Codes are 7 x / max in float32, rounded half to even.  bf16 inputs have 8
// bits, so a quotient above 1/2 that is no tie is at least 2^-14 from one, and a
// quotient within two roundings is enough where it is exact at the ties: the
// product with a reciprocal, once corrected by its remainder (the remainder of
// a tie is exact, so the correction ends on it).  float32 inputs take the
// correctly rounded division.  One token of 256 sequences, 8 heads of 128: 6.3 us;
// 4 x 4096 tokens, 15 to 22 us for 53 MB.
template <class T, int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(Kv4View c, const int32_t *start, const int32_t *count,
                                                         int n_tok, const void *k, const void *v, int tiles) {
    constexpr int ROW = D + 4, PER = D / 8, STEP = 256 / PER, STEPS = KV4_TILE / STEP;   // lanes of a token; tokens a step
    __shared__ __align__(16) uint8_t codes[KV4_TILE * ROW];
    const TileWork w(c, start, count, n_tok, tiles);
    if (w.lo >= w.upto) return;
    const int t_in = threadIdx.x / PER, ch = threadIdx.x % PER * 8;
    Eight<T> x[2][STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int t = s * STEP + t_in;
        if (t < w.lo || t >= w.upto) continue;
        const size_t at = (((size_t)(w.t0 + t) * c.B + w.b) * c.Hk + w.h) * D + ch;
        x[0][s].load(k, at);
        x[1][s].load(v, at);
    }
    uint8_t *to = w.address(c);
    if (!to) return;
    // thread i < D packs the four value words at byte 16 i: channels 64 (i / 64) +
    // 16 e + i % 16, e = 0..3, tokens of lane group (i / 16) % 4
    u32x4 *words = (u32x4 *)(to + 16 * D) + threadIdx.x;
    const bool packs = threadIdx.x < D;
    u32x4 old = {0, 0, 0, 0};
    if (packs && (w.lo > 0 || w.upto < KV4_TILE)) old = *words;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int t = s * STEP + t_in;
        const bool live = t >= w.lo && t < w.upto;   // the lanes of a group agree
        if (!live) continue;
#pragma unroll
        for (int what = 0; what < 2; ++what) {
            float top = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[what][s].get(e)));
#pragma unroll
            for (int m = 1; m < 8; m <<= 1) top = xor_max(top, m);
            // codes by the rounding of 1.5 * 2^23 + 8 + quotient: c + 8 in the low
            // bits of y, above them those of BASE
            constexpr float MAGIC = 12582912.f + 8.f;
            constexpr uint32_t BASE = 0x4b400000u;
            uint32_t y[8];
            if (sizeof(T) == 2 && top > 1e-30f && top < 1e30f) {   // the reciprocal is a normal number
                const float r = __builtin_amdgcn_rcpf(top);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x7 = x[what][s].get(e) * 7.f, q = x7 * r;
                    y[e] = __float_as_uint(fmaf(fmaf(-q, top, x7), r, q) + MAGIC);
                }
            } else {
                const float f = top > 1e30f ? 0.0625f : 1.f;   // 7 x of the largest values would overflow
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = __float_as_uint((top > 0.f ? (x[what][s].get(e) * f * 7.f) / (top * f) : 0.f) + MAGIC);
            }
            float *scales = (float *)(to + (what ? kv4_value_scales(D) : kv4_key_scales(D)));
            if ((threadIdx.x & 7) == 0) scales[ch / KV4_GROUP * KV4_TILE + t] = top / 7.f;
            if (what == 0) {
                uint32_t word = 0u - BASE * 0x11111111u;   // takes BASE from every place
#pragma unroll
                for (int e = 0; e < 8; ++e) word += y[e] << (4 * ((e & 1) * 4 + (e >> 1)));
                *(uint32_t *)(to + kv4_key_word(D, t, ch)) = word;
            } else {   // the four channels of a packing thread side by side
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    codes[t * ROW + (ch & ~63) + ((ch + e) & 15) * 4 + ((ch >> 4) & 3)] = (uint8_t)y[e];
            }
        }
    }
    __syncthreads();
    if (!packs) return;
    const int quad = (threadIdx.x >> 4) & 3, at = (threadIdx.x & ~63) + (threadIdx.x & 15) * 4;
    u32x4 word = {0, 0, 0, 0};
    uint32_t mask = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int t = (e >> 2) * 16 + quad * 4 + (e & 3);
        if (t < w.lo || t >= w.upto) continue;
        const uint32_t y = *(const uint32_t *)(codes + t * ROW + at);
        mask |= 15u << (4 * e);
#pragma unroll
        for (int i = 0; i < 4; ++i) word[i] |= ((y >> (8 * i)) & 15u) << (4 * e);
    }
    if (!mask) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) word[i] = ((word[i] ^ 0x88888888u) & mask) | (old[i] & ~mask);   // c + 8 to two's complement
    *words = word;
}

// Read back: one workgroup per tile, thread i < D takes the 16 bytes of key codes
// and of value codes at byte 16 i (4 x 4096 tokens, 8 heads of 128: 26 us, 5.8 TB/s,
// nearly all of it the float32 values written)
template <int D>
__global__ void __launch_bounds__(D) kv4_read_kernel(Kv4View c, const int32_t *start, const int32_t *count,
                                                     int n_tok, float *k, float *v, int tiles) {
    const TileWork w(c, start, count, n_tok, tiles);
    if (w.lo >= w.hi) return;
    const uint8_t *tile = w.upto > w.lo ? w.address(c) : nullptr;
    const int lane = threadIdx.x & 63, group = threadIdx.x >> 6, n16 = lane & 15, quad = lane >> 4;
    const size_t row = (size_t)c.B * c.Hk * D, base = ((size_t)w.b * c.Hk + w.h) * D;
    if (k) {
        u32x4 words = {0, 0, 0, 0};
        if (tile) words = ((const u32x4 *)tile)[threadIdx.x];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int x = 4 * group + e, t = x / (D / 32) * 16 + n16, ch = x % (D / 32) * 32 + 8 * quad;
            if (t < w.lo || t >= w.hi) continue;
            const bool live = tile && t < w.upto;
            const float s = live ? ((const float *)(tile + kv4_key_scales(D)))[ch / KV4_GROUP * KV4_TILE + t] : 0.f;
            f32x4 out[2];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int nibble = (i & 1) * 4 + (i >> 1);
                out[i >> 2][i & 3] = live ? (float)((int)((words[e] >> (4 * nibble)) & 15) - 8) * s : 0.f;
            }
            f32x4 *to = (f32x4 *)(k + (size_t)(w.t0 + t) * row + base + ch);
            to[0] = out[0], to[1] = out[1];
        }
    }
    if (v) {
        u32x4 words = {0, 0, 0, 0};
        f32x4 s[2] = {};
        if (tile) {
            words = ((const u32x4 *)(tile + 16 * D))[threadIdx.x];
            const float *scales = (const float *)(tile + kv4_value_scales(D)) + group * KV4_TILE + 4 * quad;
            s[0] = *(const f32x4 *)scales, s[1] = *(const f32x4 *)(scales + 16);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int t = (i >> 2) * 16 + 4 * quad + (i & 3);
            if (t < w.lo || t >= w.hi) continue;
            const bool live = tile && t < w.upto;
            float *to = v + (size_t)(w.t0 + t) * row + base + 64 * group + n16;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                to[16 * e] = live ? (float)(int)__builtin_amdgcn_sbfe(words[e], 4 * i, 4) * s[i >> 2][i & 3] : 0.f;
        }
    }
}

// most tiles that n tokens touch
int tiles_of(int n) { return (n + KV4_TILE - 2) / KV4_TILE + 1; }

template <class T>
void launch_append(const Kv4View &c, const int32_t *start, const int32_t *count, int n_tok, const void *k,
                   const void *v, hipStream_t s) {
    const int tiles = tiles_of(n_tok);
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
    const int tiles = tiles_of(T);
    const dim3 grid((unsigned)((long long)c.B * c.Hk * tiles)), wg((unsigned)c.d);
    if (c.d == 64)
        hipLaunchKernelGGL(kv4_read_kernel<64>, grid, wg, 0, s, c, start, count, T, k, v, tiles);
    else if (c.d == 128)
        hipLaunchKernelGGL(kv4_read_kernel<128>, grid, wg, 0, s, c, start, count, T, k, v, tiles);
    else
        hipLaunchKernelGGL(kv4_read_kernel<256>, grid, wg, 0, s, c, start, count, T, k, v, tiles);
    return hipGetLastError();
}

}  // namespace pace
