// C ABI of the layers beside the gated delta rule (head norms with rotation,
// linear attention, the 4-bit paged cache): argument checks and dispatch.
// Every check runs before the first HIP call.
#include <math.h>

#include "pace_layers.h"
#include "pace_status.h"

using namespace pace;

namespace {

// Most workgroups one launch is given.  The kernels index their work by one
// grid dimension; calls that would need more are refused.
constexpr double MAX_GRID = 2147483647.0;

int check_buffer(const void *p, const char *name) {
    if (!p || !aligned(p, 16)) return fail(PACE_EINVAL, "%s must be a 16-byte aligned device pointer", name);
    return PACE_OK;
}

int check_i32(const void *p, const char *name, bool required) {
    if (!p && required) return fail(PACE_EINVAL, "%s must not be NULL", name);
    if (!aligned(p, 4)) return fail(PACE_EINVAL, "%s must be 4-byte aligned", name);
    return PACE_OK;
}

int check_linear(int32_t batch, int32_t heads, int32_t d_k, int32_t d_v, int32_t n_tok, int32_t in_dtype) {
    int rc = check_shape(batch, heads, d_k, d_v);
    if (rc) return rc;
    if ((rc = check_dtype(in_dtype))) return rc;
    if (n_tok < 1) return fail(PACE_EINVAL, "n_tok must be >= 1");
    if (n_tok > (1 << 30)) return fail(PACE_EUNSUPPORTED, "n_tok must be at most 2^30");
    if ((double)batch * heads * (d_v / 16) * ((double)n_tok / 64 + 1) > MAX_GRID)
        return fail(PACE_EUNSUPPORTED, "batch * heads * n_tok too large for one call");
    return PACE_OK;
}

// what every cache entry point shares; n_tok < 0: not used by the call
int check_kv4(const pace_kv4_config *cfg, int32_t n_tok) {
    if (!cfg) return fail(PACE_EINVAL, "cfg must not be NULL");
    if (cfg->heads_kv < 1) return fail(PACE_EINVAL, "heads_kv must be >= 1");
    if (cfg->n_pages < 1) return fail(PACE_EINVAL, "n_pages must be >= 1");
    if (cfg->d != 64 && cfg->d != 128 && cfg->d != 256) return fail(PACE_EUNSUPPORTED, "d must be 64, 128 or 256");
    if (cfg->page_tokens < 32 || cfg->page_tokens > 1024 || cfg->page_tokens % 32)
        return fail(PACE_EUNSUPPORTED, "page_tokens must be a multiple of 32 up to 1024");
    if (n_tok < 0) return PACE_OK;
    if (cfg->batch < 1 || cfg->max_pages < 1) return fail(PACE_EINVAL, "batch and max_pages must be >= 1");
    if ((int64_t)cfg->max_pages * cfg->page_tokens > 0x7fffffff - 2048)
        return fail(PACE_EUNSUPPORTED, "max_pages * page_tokens must fit 31 bits");
    int rc = check_dtype(cfg->in_dtype);
    if (rc) return rc;
    if (n_tok < 1) return fail(PACE_EINVAL, "n_tok must be >= 1");
    if ((double)n_tok * cfg->batch * cfg->heads_kv * cfg->d / 32 > MAX_GRID)
        return fail(PACE_EUNSUPPORTED, "n_tok * batch * heads_kv too large for one call");
    return PACE_OK;
}

int check_heads_q(const pace_kv4_config *cfg, int32_t n_tok) {
    if (cfg->heads_q < 1 || cfg->heads_q % cfg->heads_kv)
        return fail(PACE_EINVAL, "heads_q must be a multiple of heads_kv");
    if ((double)n_tok * cfg->batch * cfg->heads_q * cfg->d / 32 > MAX_GRID)
        return fail(PACE_EUNSUPPORTED, "n_tok * batch * heads_q too large for one call");
    return PACE_OK;
}

Kv4View kv4_view(const pace_kv4_config *cfg, const void *pool, const int32_t *table) {
    const uint64_t per = cfg->page_tokens / 32;
    return Kv4View{(uint8_t *)pool, table,           cfg->batch,   cfg->heads_kv,
                   cfg->d,          cfg->page_tokens, cfg->n_pages, cfg->max_pages,
                   per == 1 ? 0 : (uint32_t)(((1ull << 32) + per - 1) / per)};
}

}  // namespace

PACE_API int pace_qk_norm_rope(const pace_norm_config *cfg, const void *q, const void *k,
                               const float *q_weight, const float *k_weight, const int32_t *pos,
                               const float *inv_freq, void *q_out, void *k_out, void *stream) {
    if (!cfg) return fail(PACE_EINVAL, "cfg must not be NULL");
    const pace_norm_config &c = *cfg;
    if (c.tokens < 0 || c.heads_q < 0 || c.heads_k < 0) return fail(PACE_EINVAL, "tokens, heads_q, heads_k must be >= 0");
    if (c.d < 1) return fail(PACE_EINVAL, "d must be >= 1");
    if (c.d > PACE_NORM_MAX_D) return fail(PACE_EUNSUPPORTED, "d must be at most %d", PACE_NORM_MAX_D);
    int rc = check_dtype(c.in_dtype);
    if (rc) return rc;
    if (c.norm != PACE_NORM_NONE && c.norm != PACE_NORM_L2 && c.norm != PACE_NORM_RMS)
        return fail(PACE_EINVAL, "unknown norm %d", c.norm);
    if (!(c.eps >= 0.f) || !isfinite(c.eps)) return fail(PACE_EINVAL, "eps must be finite and >= 0");
    if (!isfinite(c.q_scale)) return fail(PACE_EINVAL, "q_scale must be finite");
    if (c.rot < 0 || c.rot > c.d || c.rot % 2) return fail(PACE_EINVAL, "rot must be even, 0..d");
    if (c.rot_pairs != PACE_ROT_HALVES && c.rot_pairs != PACE_ROT_ADJACENT)
        return fail(PACE_EINVAL, "unknown rot_pairs %d", c.rot_pairs);
    if ((q_weight || k_weight) && c.norm != PACE_NORM_RMS) return fail(PACE_EINVAL, "weights need PACE_NORM_RMS");
    if (c.rot && (!pos || !inv_freq)) return fail(PACE_EINVAL, "a rotation needs pos and inv_freq");
    const size_t e = c.in_dtype == PACE_DTYPE_BF16 ? 2 : 4;
    const struct {
        const char *name;
        const void *x, *y;
        int64_t heads, stride;
    } sides[2] = {{"q", q, q_out, c.heads_q, c.q_stride}, {"k", k, k_out, c.heads_k, c.k_stride}};
    for (const auto &s : sides) {
        if (s.heads == 0) continue;
        if (!s.x || !s.y) return fail(PACE_EINVAL, "%s and %s_out must not be NULL", s.name, s.name);
        if (!aligned(s.x, e) || !aligned(s.y, e)) return fail(PACE_EINVAL, "%s, %s_out: misaligned", s.name, s.name);
        if (s.stride < s.heads * c.d) return fail(PACE_EINVAL, "%s_stride must be at least heads * d", s.name);
        if (s.x == s.y && s.stride != s.heads * c.d) return fail(PACE_EINVAL, "%s_out = %s needs dense rows", s.name, s.name);
    }
    if (!aligned(pos, 4) || !aligned(inv_freq, 4) || !aligned(q_weight, 4) || !aligned(k_weight, 4))
        return fail(PACE_EINVAL, "pos, inv_freq and weights must be 4-byte aligned");
    if ((double)c.tokens * ((double)c.heads_q + c.heads_k) > MAX_GRID)
        return fail(PACE_EUNSUPPORTED, "tokens * heads too large for one call");
    if (c.tokens == 0 || (int64_t)c.heads_q + c.heads_k == 0) return ok();
    NormArgs a{{q, k},     {q_out, k_out}, {q_weight, k_weight}, {c.q_stride, c.k_stride}, pos,
               inv_freq,   c.tokens,       c.heads_q,            c.heads_q + c.heads_k,    c.d,
               c.rot,      c.rot_pairs == PACE_ROT_ADJACENT,     c.norm,                   c.eps, c.q_scale};
    hipError_t err = launch_qk_norm_rope(a, c.in_dtype == PACE_DTYPE_BF16, (hipStream_t)stream);
    if (err != hipSuccess) return hip_fail(err, "norm launch");
    return ok();
}

PACE_API int pace_linear_attn_workspace(int32_t batch, int32_t heads, int32_t d_k, int32_t d_v,
                                        int32_t n_tok, int32_t in_dtype, uint64_t *out) {
    if (!out) return fail(PACE_EINVAL, "out must not be NULL");
    int rc = check_linear(batch, heads, d_k, d_v, n_tok, in_dtype);
    if (rc) return rc;
    *out = linear_attn_workspace(batch, heads, d_k, d_v, n_tok, in_dtype == PACE_DTYPE_BF16);
    return ok();
}

PACE_API int pace_linear_attn(int32_t batch, int32_t heads, int32_t d_k, int32_t d_v, int32_t n_tok,
                              int32_t in_dtype, const void *q, const void *k, const void *v,
                              const float *decay, const int32_t *lens, float scale,
                              const float *state_in, float *state_out, float *out, void *workspace,
                              uint64_t workspace_bytes, void *stream) {
    int rc = check_linear(batch, heads, d_k, d_v, n_tok, in_dtype);
    if (rc) return rc;
    if ((rc = check_buffer(q, "q")) || (rc = check_buffer(k, "k")) || (rc = check_buffer(v, "v")) ||
        (rc = check_buffer(state_out, "state_out")) || (rc = check_buffer(out, "out")))
        return rc;
    if (!aligned(state_in, 16)) return fail(PACE_EINVAL, "state_in must be 16-byte aligned");
    if (!decay || !aligned(decay, 4)) return fail(PACE_EINVAL, "decay must be a 4-byte aligned device pointer");
    if ((rc = check_i32(lens, "lens", false))) return rc;
    if (!isfinite(scale)) return fail(PACE_EINVAL, "scale must be finite");
    const int bf16 = in_dtype == PACE_DTYPE_BF16;
    const uint64_t need = linear_attn_workspace(batch, heads, d_k, d_v, n_tok, bf16);
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
        return fail(PACE_EINVAL, "workspace must be 16-byte aligned and hold %llu bytes", (unsigned long long)need);
    LinearArgs a{q,   k,         v,   decay,                        lens,  state_in, state_out,
                 out, (float *)workspace, scale, batch, heads, d_k, d_v, n_tok};
    hipError_t e = launch_linear_attn(a, bf16, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "linear attention launch");
    return ok();
}

PACE_API int pace_kv4_pool_bytes(const pace_kv4_config *cfg, uint64_t *out) {
    if (!out) return fail(PACE_EINVAL, "out must not be NULL");
    int rc = check_kv4(cfg, -1);
    if (rc) return rc;
    *out = (uint64_t)cfg->n_pages * cfg->heads_kv * cfg->page_tokens * (36 * cfg->d / 32);
    return ok();
}

PACE_API int pace_kv4_append(const pace_kv4_config *cfg, void *pool, const int32_t *table,
                             const int32_t *start, const int32_t *count, int32_t n_tok, const void *k,
                             const void *v, void *stream) {
    int rc = check_kv4(cfg, n_tok < 0 ? 0 : n_tok);
    if (rc) return rc;
    if ((rc = check_buffer(pool, "pool")) || (rc = check_buffer(k, "k")) || (rc = check_buffer(v, "v")) ||
        (rc = check_i32(table, "table", true)) || (rc = check_i32(start, "start", true)) ||
        (rc = check_i32(count, "count", false)))
        return rc;
    hipError_t e = launch_kv4_append(kv4_view(cfg, pool, table), start, count, n_tok, k, v,
                                     cfg->in_dtype == PACE_DTYPE_BF16, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "cache append launch");
    return ok();
}

PACE_API int pace_kv4_read(const pace_kv4_config *cfg, const void *pool, const int32_t *table,
                           const int32_t *start, const int32_t *count, int32_t n_tok, float *k_out,
                           float *v_out, void *stream) {
    int rc = check_kv4(cfg, n_tok < 0 ? 0 : n_tok);
    if (rc) return rc;
    if ((rc = check_buffer(pool, "pool")) || (rc = check_i32(table, "table", true)) ||
        (rc = check_i32(start, "start", true)) || (rc = check_i32(count, "count", false)))
        return rc;
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return fail(PACE_EINVAL, "k_out and v_out must be 16-byte aligned");
    if (!k_out && !v_out) return ok();
    hipError_t e = launch_kv4_read(kv4_view(cfg, pool, table), start, count, n_tok, k_out, v_out, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "cache read launch");
    return ok();
}

PACE_API int pace_kv4_attention_workspace(const pace_kv4_config *cfg, int32_t n_tok, uint64_t *out) {
    if (!out) return fail(PACE_EINVAL, "out must not be NULL");
    int rc = check_kv4(cfg, n_tok < 0 ? 0 : n_tok);
    if (rc || (rc = check_heads_q(cfg, n_tok))) return rc;
    *out = kv4_attention_workspace(kv4_view(cfg, nullptr, nullptr), cfg->heads_q / cfg->heads_kv, n_tok,
                                   cfg->in_dtype == PACE_DTYPE_BF16);
    return ok();
}

PACE_API int pace_kv4_attention(const pace_kv4_config *cfg, const void *pool, const int32_t *table,
                                const int32_t *lens, const int32_t *count, int32_t n_tok, const void *q,
                                float scale, int32_t window, int32_t sinks, void *out, void *workspace,
                                uint64_t workspace_bytes, void *stream) {
    int rc = check_kv4(cfg, n_tok < 0 ? 0 : n_tok);
    if (rc || (rc = check_heads_q(cfg, n_tok))) return rc;
    if ((rc = check_buffer(pool, "pool")) || (rc = check_buffer(q, "q")) || (rc = check_buffer(out, "out")) ||
        (rc = check_i32(table, "table", true)) || (rc = check_i32(lens, "lens", true)) ||
        (rc = check_i32(count, "count", false)))
        return rc;
    if (!isfinite(scale)) return fail(PACE_EINVAL, "scale must be finite");
    if (window < 0 || sinks < 0) return fail(PACE_EINVAL, "window and sinks must be >= 0");
    const int G = cfg->heads_q / cfg->heads_kv, bf16 = cfg->in_dtype == PACE_DTYPE_BF16;
    const Kv4View c = kv4_view(cfg, pool, table);
    const uint64_t need = kv4_attention_workspace(c, G, n_tok, bf16);
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
        return fail(PACE_EINVAL, "workspace must be 16-byte aligned and hold %llu bytes", (unsigned long long)need);
    Kv4AttnArgs a{c, lens, count, q, out, (float *)workspace, scale, n_tok, G, window, window ? sinks : 0};
    hipError_t e = launch_kv4_attention(a, bf16, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "cache attention launch");
    return ok();
}
