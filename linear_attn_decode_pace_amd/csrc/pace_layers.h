// Arguments and launchers of the layers beside the gated delta rule: head
// norms with rotation, linear attention with a decay for each head, and the
// 4-bit paged cache with the attention that reads it.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace pace {

// ---- head norms with rotation (qk_norm_rope.hip) ---------------------------

struct NormArgs {
    const void *x[2];       // queries, keys
    void *y[2];
    const float *weight[2];
    long long stride[2];    // elements between rows
    const int32_t *pos;
    const float *inv_freq;
    long long tokens;
    int heads_q, heads;     // query heads; query + key heads
    int d, rot, adjacent, norm;
    float eps, q_scale;
};
hipError_t launch_qk_norm_rope(const NormArgs &a, int bf16, hipStream_t s);

// ---- linear attention with a decay for each head (linear_attn.hip) ---------

struct LinearArgs {
    const void *q, *k, *v;
    const float *decay;     // [H]
    const int32_t *lens;    // [B] or NULL
    const float *state_in;  // [B, H, dk, dv] or NULL
    float *state_out;
    float *out;             // [T, B, H, dv]
    float *workspace;
    float scale;
    int B, H, dk, dv, T;
};
uint64_t linear_attn_workspace(int B, int H, int dk, int dv, int T, int bf16);
hipError_t launch_linear_attn(const LinearArgs &a, int bf16, hipStream_t s);

// ---- 4-bit paged cache (kv4_cache.hip, kv4_attention.hip) ------------------

struct Kv4View {
    uint8_t *pool;
    const int32_t *table;   // [B, max_pages]
    int B, Hk, d, page_tokens, n_pages, max_pages;
    // ceil(2^32 / tiles of a page), or 0 for one tile: the high word of its
    // product with a tile number is the page's column, exactly for numbers
    // below 2^27 (cache positions have 31 bits and a page at most 32 tiles)
    uint32_t per_inv;
};
// append: src k / v [T, B, Hk, d]; read: dst float32 (either may be NULL)
hipError_t launch_kv4_append(const Kv4View &c, const int32_t *start, const int32_t *count, int T,
                             const void *k, const void *v, int bf16, hipStream_t s);
hipError_t launch_kv4_read(const Kv4View &c, const int32_t *start, const int32_t *count, int T,
                           float *k, float *v, hipStream_t s);

struct Kv4AttnArgs {
    Kv4View c;
    const int32_t *lens, *count;
    const void *q;
    void *out;
    float *workspace;
    float scale;
    int T, G, window, sinks;   // G: query heads that share a key / value head
};
uint64_t kv4_attention_workspace(const Kv4View &c, int G, int T, int bf16);
hipError_t launch_kv4_attention(const Kv4AttnArgs &a, int bf16, hipStream_t s);

}  // namespace pace
