// Softmax attention over the 4-bit paged cache.
#include "kv4_layout.h"
#include "mfma_common.h"

namespace pace {
namespace {

__device__ inline float code_of(const uint8_t *tile, int off, int nib) {
    return (float)((int)((*(const uint32_t *)(tile + off) >> (4 * nib)) & 15) - 8);
}

// One wave per query row: 64 positions at a time, a lane scores one of them;
// then each lane sums its channels over the 64.
template <class T>
__global__ void __launch_bounds__(64) kv4_attention_row_kernel(Kv4AttnArgs a) {
    __shared__ float q[256], p[64];
    const Kv4View &c = a.c;
    const int lane = threadIdx.x, Hq = c.Hk * a.G;
    const int hq = blockIdx.x % Hq, b = blockIdx.x / Hq % c.B, t = blockIdx.x / Hq / c.B;
    const int h = hq / a.G, cap = (int)min((long long)c.max_pages * c.page_tokens, 0x7fffffffll);
    const int len = min(max(a.lens[b], 0), cap), n = a.count ? min(max(a.count[b], 0), a.T) : a.T;
    if (t >= n) return;
    const size_t row = (((size_t)t * c.B + b) * Hq + hq) * c.d;
    for (int i = lane; i < c.d; i += 64)
        q[i] = sizeof(T) == 2 ? bf2f(((const uint16_t *)a.q)[row + i]) : ((const float *)a.q)[row + i];
    __syncthreads();
    const int at = len - n + t;
    float top = -INFINITY, sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 <= at; j0 += 64) {
        const int j = j0 + lane;
        const bool see = j <= at && (a.window == 0 || j > at - a.window || j < a.sinks);
        const uint8_t *tile = see ? kv4_tile(c, b, h, j / KV4_TILE) : nullptr;
        float score = -INFINITY;
        if (tile) {
            score = 0.f;
            const float *sc = (const float *)(tile + kv4_key_scales(c.d));
            for (int g = 0; g < c.d / KV4_GROUP; ++g) {
                float dot = 0.f;
                for (int i = g * KV4_GROUP; i < (g + 1) * KV4_GROUP; ++i) {
                    int nib;
                    const int off = kv4_key_word(c.d, j % KV4_TILE, i, &nib);
                    dot = fmaf(q[i], code_of(tile, off, nib), dot);
                }
                score = fmaf(dot, sc[g * KV4_TILE + j % KV4_TILE], score);
            }
            score *= a.scale;
        }
        float m = score;
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) m = xor_max(m, x);
        m = fmaxf(m, top);
        if (m == -INFINITY) continue;
        const float e = expf(score - m), old = expf(top - m);
        float es = e;
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) es += __shfl_xor(es, x);
        sum = sum * old + es;
        top = m;
        __syncthreads();
        p[lane] = tile ? e : -1.f;
        __syncthreads();
        for (int r = 0; r < c.d / 64; ++r) {
            o[r] *= old;
            const int ch = r * 64 + lane;
            for (int x = 0; x < 64; ++x) {
                if (p[x] < 0.f) continue;
                const uint8_t *tv = kv4_tile(c, b, h, (j0 + x) / KV4_TILE);
                int nib;
                const int off = kv4_value_word(c.d, (j0 + x) % KV4_TILE, ch, &nib);
                o[r] = fmaf(p[x] * ((const float *)(tv + kv4_value_scales(c.d)))[r * KV4_TILE + (j0 + x) % KV4_TILE],
                            code_of(tv, off, nib), o[r]);
            }
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    for (int r = 0; r < c.d / 64; ++r) {
        if constexpr (sizeof(T) == 2)
            ((uint16_t *)a.out)[row + r * 64 + lane] = (uint16_t)(pk_bf16(o[r] * inv, 0.f) & 0xffff);
        else
            ((float *)a.out)[row + r * 64 + lane] = o[r] * inv;
    }
}

}  // namespace

uint64_t kv4_attention_workspace(const Kv4View &, int, int, int) { return 0; }

hipError_t launch_kv4_attention(const Kv4AttnArgs &a, int bf16, hipStream_t s) {
    const dim3 grid((unsigned)((long long)a.T * a.c.B * a.c.Hk * a.G));
    if (bf16)
        hipLaunchKernelGGL(kv4_attention_row_kernel<uint16_t>, grid, dim3(64), 0, s, a);
    else
        hipLaunchKernelGGL(kv4_attention_row_kernel<float>, grid, dim3(64), 0, s, a);
    return hipGetLastError();
}

}  // namespace pace
