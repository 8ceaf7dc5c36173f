// Softmax attention over the 4-bit paged cache, on bf16 matrix cores straight
// from the codes.
//
// For one key / value head, the query rows are the G heads that share it times
// the call's tokens (row r = token * G + head).  A wavefront takes 16 NT rows and
// tiles of 32 cached tokens, and works transposed, tokens by rows:
//   S^T = K Q^T   (16 x 16 x 32 products: A = keys, B = queries),
//   P   = exp2(S * scale * log2 e - m),
//   O^T = V^T P   (A = values, B = probabilities).
// S^T leaves a lane with four tokens of each 16 of one query, which are the
// operand elements of the second product if its k-slots are taken in that order
// (kv4_layout.h stores values so): nothing passes through LDS, and the row
// statistics are a lane's own values plus two lane swaps.
//
// Codes.  Values become bf16 c / 16, exactly.  Keys, where every wave unpacks
// for itself, take a cheaper form: a nibble n = c + 8 is the bf16 16 + n by one shift and
// one and-or for two codes (exponent 4, n in the upper mantissa bits), so operands
// hold c + 24, and the accumulators of S start at -24 sum(q) of their 64
// channels.  (Values in that form too, less 24 sum(p) at the end, take 1% less
// time on 64 caches of up to 32768 tokens, but leave the rounding of the
// 24 sum(p) in outputs that should be zero.)  Scales multiply S per token
// and group, and p per token and group before it is rounded.
//
// One token of 64 sequences of up to 32768 tokens, 8 heads of 128 channels, four
// query heads each: 276 us, 5.1 TB/s of codes and scales; a tile of 4.6 KB takes a wave
// about 300 VALU instructions (a third unpack codes) and 16 matrix
// products, so the VALU is busy for more than half of that time.  Four such
// sequences of 8192 tokens: 13 + 4 us, of which the loads' chain (lengths,
// table, codes) and the launches are most.
//
// Row maxima are lazy: a wave rescales its sums only where a score exceeds the
// row's reference by 2^8 or more, which is exact in float32 and keeps the
// cross-lane work out of nearly all tiles.
#include <algorithm>

#include "kv4_layout.h"
#include "mfma_common.h"

namespace pace {
namespace {

constexpr float CODE_BIAS = 24.f;

// The and-or's constants, one in a scalar and one in a vector register: the
// instruction takes one scalar operand and no literal.
struct CodeBits {
    uint32_t mask = 0x00780078u, one = 0x41804180u;
    __device__ inline CodeBits() { asm volatile("" : "+s"(mask), "+v"(one)); }
};

// eight codes of a word as bf16 c + 24
__device__ inline bf16x8 biased_codes(uint32_t w, const CodeBits &k) {
    return __builtin_bit_cast(bf16x8, u32x4{((w << 3) & k.mask) | k.one, ((w >> 1) & k.mask) | k.one,
                                            ((w >> 5) & k.mask) | k.one, ((w >> 9) & k.mask) | k.one});
}

// eight two's complement codes of a word as bf16 c / 16, exactly (see Loader::nibble_f32)
__device__ inline bf16x8 exact_codes(uint32_t lo) {
    using L = Loader<128, 4>;
    const uint32_t hi = lo >> 4;
    return __builtin_bit_cast(bf16x8, u32x4{pk_bf16(L::nibble_f32<0>(lo), L::nibble_f32<2>(lo)),
                                            pk_bf16(L::nibble_f32<0>(hi), L::nibble_f32<2>(hi)),
                                            pk_bf16(L::nibble_f32<1>(lo), L::nibble_f32<3>(lo)),
                                            pk_bf16(L::nibble_f32<1>(hi), L::nibble_f32<3>(hi))});
}

constexpr uint32_t KEY_SIGNS = 0x88888888u;   // keys' c + 8 to two's complement

// max / sum over the four lanes that share lane % 16
__device__ inline float quad_max(float x) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ inline float quad_sum(float x) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// a wavefront's share of one tile: the operand words of D of its CH D channels,
// and D / 64 of their 2 D scales, which the wave spreads through LDS when it comes
// to the tile
template <int D, int CH>
struct TileRegs {
    static_assert(CH == 1 || D == 128, "a half has whole groups of four words");
    typedef float scales_t __attribute__((ext_vector_type(D / 64)));
    u32x4 k[D / 64], v[D / 64];
    scales_t sc;
    // ONCE: codes that no other workgroup of the call reads, past the caches
    // (64 caches of up to 32768 tokens: 276 us against 288 us)
    template <bool ONCE>
    __device__ inline void load(const uint8_t *tile, int half, int lane) {
        auto get = [](const uint8_t *p) {
            return ONCE ? __builtin_nontemporal_load((const u32x4 *)p) : *(const u32x4 *)p;
        };
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            k[i] = get(tile + (i * CH + half) * 1024 + lane * 16);
            v[i] = get(tile + 16 * CH * D + (half * (D / 64) + i) * 1024 + lane * 16);
        }
        sc = *(const scales_t *)(tile + 32 * CH * D + half * 2 * D + lane * (D / 16) + (lane >> 5) * 2 * (CH - 1) * D);
    }
};

// operands of a tile from its words in registers, with D floats of LDS for its scales
template <int D, int CH, bool EXACT>
struct RegTile {
    const TileRegs<D, CH> &t;
    const float *scales;
    const CodeBits &bits;
    __device__ inline bf16x8 key(int sub, int m, int) const {
        const int w = sub * (D / 32) + m;
        return EXACT ? exact_codes(t.k[w >> 2][w & 3] ^ KEY_SIGNS) : biased_codes(t.k[w >> 2][w & 3], bits);
    }
    __device__ inline bf16x8 value(int c, int) const { return exact_codes(t.v[c >> 2][c & 3]); }
};

// operands of a tile that its workgroup has unpacked into LDS: [words][64 lanes]
template <int D>
struct SharedTile {
    const bf16x8 *ops;
    const float *scales;
    __device__ inline bf16x8 key(int sub, int m, int lane) const { return ops[(sub * (D / 32) + m) * 64 + lane]; }
    __device__ inline bf16x8 value(int c, int lane) const { return ops[(D / 16 + c) * 64 + lane]; }
};

// What a wave works on: 16 NT rows, D channels (from ch0 on) of a head
template <int D, int QP, int NT, bool EXACT>
struct Attn {
    static constexpr int NG = D / 64, NM = D / 32, NC = D / 16;
    bf16x8 q[NT][QP][NM];
    float qoff[NT][NG];
    f32x4 o[NT][NC];
    float m[NT], l[NT];
    int at[NT];   // last position that the lane's row sees, -1 for none
    float c;
    int window, sinks;

    // queries of rows r0 .. as operands, empty sums
    __device__ inline void init(const Kv4AttnArgs &a, int b, int h, int ch0, int r0, int len, int n, int lane) {
        const int n16 = lane & 15, quad = lane >> 4, R = a.T * a.G;
        window = a.window, sinks = a.sinks;
        const float sign = a.scale < 0.f ? -1.f : 1.f;
        this->c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f) * (EXACT ? 16.f : 1.f);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = r0 + nt * 16 + n16, t = r / a.G;
            const bool ok = r < R && t < n;
            at[nt] = ok ? len - n + t : -1;
            const size_t row = (((size_t)t * a.c.B + b) * a.c.Hk * a.G + (size_t)h * a.G + (r - t * a.G)) * a.c.d + ch0;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float sum = 0.f;
#pragma unroll
                for (int i = 2 * g; i < 2 * g + 2; ++i) {
                    const size_t from = row + 32 * i + 8 * quad;
                    float x[8];
                    if constexpr (QP == 1) {
                        u32x4 v = {0, 0, 0, 0};
                        if (ok) v = *(const u32x4 *)((const uint16_t *)a.q + from);
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[2 * e] = lo_f32(v[e]) * sign, x[2 * e + 1] = hi_f32(v[e]) * sign;
                    } else {
                        f32x4 v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
                        if (ok) v0 = *(const f32x4 *)((const float *)a.q + from), v1 = *(const f32x4 *)((const float *)a.q + from + 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] = v0[e] * sign, x[e + 4] = v1[e] * sign;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum += x[e];
#pragma unroll
                    for (int part = 0; part < QP; ++part) {
                        u32x4 v;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v[e] = pk_bf16(x[2 * e], x[2 * e + 1]);
                            x[2 * e] -= lo_f32(v[e]);
                            x[2 * e + 1] -= hi_f32(v[e]);
                        }
                        q[nt][part][i] = __builtin_bit_cast(bf16x8, v);
                    }
                }
                qoff[nt][g] = -CODE_BIAS * quad_sum(sum);
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) o[nt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
            m[nt] = -INFINITY, l[nt] = 0.f;
        }
    }

    // a row's sums, which its four lanes hold in parts, in the values' own units
    __device__ inline void close() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt] = quad_sum(l[nt]);
#pragma unroll
            for (int x = 0; x < NC; ++x) o[nt][x] *= 16.f;
        }
    }

    // one tile, positions p0 .. p0 + 31; full: every row sees all of them
    template <class Tile>
    __device__ inline void step(const Tile &t, int p0, bool full, int lane) {
        f32x4 sc[NT][2];
        scores(t, sc, lane);
        gather(t, sc, p0, full, lane);
    }

    // what the wave's channels give to the scores
    template <class Tile>
    __device__ inline void scores(const Tile &t, f32x4 (&sc)[NT][2], int lane) {
        const float *lds = t.scales;   // key scales [group][token], then value scales
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                // (operands of few products at a time: registers)
                if (D == 256) __builtin_amdgcn_sched_barrier(0);
                const bf16x8 ka[2] = {t.key(s, 2 * g, lane), t.key(s, 2 * g + 1, lane)};
                const f32x4 ks = *(const f32x4 *)(lds + g * 32 + s * 16 + (lane >> 4) * 4);   // tokens 4 quad ..
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float off = EXACT ? 0.f : qoff[nt][g];
                    f32x4 acc = {off, off, off, off};
#pragma unroll
                    for (int i = 2 * g; i < 2 * g + 2; ++i)
#pragma unroll
                        for (int part = QP - 1; part >= 0; --part) acc = mfma_bf16_k32(ka[i - 2 * g], q[nt][part][i], acc);
                    if (g == 0) {
                        sc[nt][s] = acc * ks;
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) sc[nt][s][r] = fmaf(acc[r], ks[r], sc[nt][s][r]);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // softmax and values
    template <class Tile>
    __device__ inline void gather(const Tile &t, f32x4 (&sc)[NT][2], int p0, bool full, int lane) {
        const float *lds = t.scales;
        f32x4 vs[NG][2];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int s = 0; s < 2; ++s) vs[g][s] = *(const f32x4 *)(lds + D / 2 + g * 32 + s * 16 + (lane >> 4) * 4);
        bf16x8 pb[NT][QP][NG];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            bool see[2][4];
            if (!full) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int p = p0 + 16 * s + 4 * (lane >> 4) + r;
                        see[s][r] = p <= at[nt] && (window == 0 || p > at[nt] - window || p < sinks);
                        sc[nt][s][r] = see[s][r] ? sc[nt][s][r] : -INFINITY;
                    }
            }
            float top = sc[nt][0][0];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, sc[nt][e >> 2][e & 3]);
            if (__any(top * c > m[nt] + 8.f)) {
                const float m2 = fmaxf(m[nt], quad_max(top) * c);
                const float f = m2 > m[nt] ? __builtin_amdgcn_exp2f(m[nt] - m2) : 1.f;
                m[nt] = m2;
                l[nt] *= f;
#pragma unroll
                for (int i = 0; i < NC; ++i) o[nt][i] *= f;
            }
            const float mm = m[nt] == -INFINITY ? 0.f : m[nt];
            float p[2][4];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    p[s][r] = __builtin_amdgcn_exp2f(fmaf(sc[nt][s][r], c, -mm));
                    l[nt] += p[s][r];
                }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float x[2][4];
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        x[s][r] = p[s][r] * vs[g][s][r];
                        if (!full) x[s][r] = see[s][r] ? x[s][r] : 0.f;   // scales of unseen tokens may be anything
                    }
#pragma unroll
                for (int part = 0; part < QP; ++part) {
                    u32x4 w;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        w[r] = pk_bf16(x[0][r], x[1][r]);
                        if (part + 1 < QP) {
                            x[0][r] -= lo_f32(w[r]);
                            x[1][r] -= hi_f32(w[r]);
                        }
                    }
                    pb[nt][part][g] = __builtin_bit_cast(bf16x8, w);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (D == 256 && i && i % 4 == 0) __builtin_amdgcn_sched_barrier(0);
            const bf16x8 va = t.value(i, lane);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int part = QP - 1; part >= 0; --part)
                    o[nt][i] = mfma_bf16_k32(va, pb[nt][part][i >> 2], o[nt][i]);
        }
    }
};

// Tiles that some of the rows r0 .. r0 + rows - 1 see: those of the sinks, then
// from the first row's window to the last row's position
struct TileList {
    int at_lo, at_hi, n_sink, lo, total;
    __device__ inline TileList(const Kv4AttnArgs &a, int r0, int rows, int len, int n) {
        const int t_lo = r0 / a.G, t_hi = min((r0 + rows - 1) / a.G, n - 1);
        at_lo = len - n + t_lo, at_hi = t_lo <= t_hi ? len - n + t_hi : -1;
        const int end = at_hi < 0 ? 0 : at_hi / KV4_TILE + 1;
        n_sink = a.window ? min((int)(((long long)a.sinks + KV4_TILE - 1) / KV4_TILE), end) : 0;
        lo = a.window ? min(max((int)max((long long)at_lo - a.window + 1, 0ll) / KV4_TILE, n_sink), end) : 0;
        total = n_sink + end - lo;
    }
    __device__ inline int tile(int i) const { return i < n_sink ? i : lo + i - n_sink; }
};

// Address of a tile of (sequence b, head h), and whether it has a page (the
// pool's first tile otherwise, which may be loaded).  Table entries come by
// scalar loads, which do not stand in the tiles' queue.
template <int D>
struct TileTable {
    typedef const __attribute__((address_space(4))) int32_t *scalar_ptr;
    const Kv4View &c;
    scalar_ptr table;
    int h, per_page;
    __device__ inline TileTable(const Kv4View &c, int b, int h)
        : c(c), table((scalar_ptr)(uintptr_t)(c.table + (size_t)b * c.max_pages)), h(h),
          per_page(c.page_tokens / KV4_TILE) {}
    __device__ inline int page(int tile) const { return table[kv4_column(c, tile)]; }
    __device__ inline bool live(int page) const { return page >= 0 && page < c.n_pages; }
    __device__ inline const uint8_t *tile(int page, int tile) const {
        const size_t at = ((size_t)(uint32_t)page * c.Hk + h) * per_page + (tile - kv4_column(c, tile) * per_page);
        return c.pool + (live(page) ? at * kv4_tile_bytes(D) : 0);
    }
};

// partial results of a split: [splits][B * Hk][R][D + 4] floats: sums, then (m, l)
__device__ inline float *partial_row(const Kv4AttnArgs &a, int D, int split, int bh, int r) {
    const size_t R = (size_t)a.T * a.G;
    return a.workspace + (((size_t)split * a.c.B * a.c.Hk + bh) * R + r) * (D + 4);
}

template <int QP>
__device__ inline void store4(void *out, size_t i, f32x4 x) {
    if constexpr (QP == 1)
        *(u32x2 *)((uint16_t *)out + i) = u32x2{pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3])};
    else
        *(f32x4 *)((float *)out + i) = x;
}

// a wave's rows and channels: the result, or its part of it
template <int D, int QP, int NT, class A>
__device__ inline void store_rows(const Kv4AttnArgs &a, const A &w, int b, int h, int ch0, int r0, int n, int split,
                                  int splits, int lane) {
    const int n16 = lane & 15, quad = lane >> 4, R = a.T * a.G, bh = b * a.c.Hk + h;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + nt * 16 + n16, t = r / a.G;
        if (r >= R || t >= n) continue;
        if (splits == 1) {
            const float inv = w.l[nt] > 0.f ? 1.f / w.l[nt] : 0.f;
            const size_t at = (((size_t)t * a.c.B * a.c.Hk + bh) * a.G + (r - t * a.G)) * D + ch0;
#pragma unroll
            for (int x = 0; x < A::NC; ++x) store4<QP>(a.out, at + 16 * x + 4 * quad, w.o[nt][x] * inv);
        } else {
            float *p = partial_row(a, D, split, bh, r);
#pragma unroll
            for (int x = 0; x < A::NC; ++x) *(f32x4 *)(p + ch0 + 16 * x + 4 * quad) = w.o[nt][x];
            if (quad == 0 && ch0 == 0) *(f32x2 *)(p + D) = f32x2{w.m[nt], w.l[nt]};
        }
    }
}

// Workgroup barrier that orders LDS only: loads of the tiles ahead stay in flight
__device__ inline void local_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Few rows.  The four waves of a workgroup are WR row waves of 16 NT rows, CH parts
// of the channels and WK waves that take tiles in turn.  CH = 2 for heads of 256
// channels: the registers of a whole head leave one wave a SIMD; halves of a head,
// which add their scores through LDS, leave two (64 caches of up to 4096 tokens, 8 such
// heads, four query heads each: 115 us against 190 us, float32 in proportion).
template <int D, int QP, int NT, int WR, int CH, int PF, int WAVES>
__global__ void __launch_bounds__(256, WAVES) kv4_attention_kernel(Kv4AttnArgs a, int row_blocks, int splits) {
    constexpr bool EXACT = QP == 3;
    constexpr int DW = D / CH, WK = 4 / (WR * CH);
    using A = Attn<DW, QP, NT, EXACT>;
    constexpr int ROWS = 16 * NT * WR, LDW = D + 4;
    __shared__ float scales[4][DW];
    __shared__ f32x4 parts[CH == 1 ? 1 : 2][4][NT * 2][64];   // of the scores, for two tiles in turn
    const Kv4View &c = a.c;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n16 = lane & 15, quad = lane >> 4;
    const int wr = wave / (4 / WR), wk = wave / CH % WK, half = wave % CH;
    const int BH = c.B * c.Hk, R = a.T * a.G;
    // (sequence, head) runs fastest: the row blocks that share a head's cache
    // then meet in one XCD's L2 where B * Hk is a multiple of 8; the last rows,
    // which see most, come first
    const int bh = blockIdx.x % BH, rest = blockIdx.x / BH;
    const int split = rest % splits, rb = row_blocks - 1 - rest / splits;
    const int b = bh / c.Hk, h = bh - b * c.Hk;
    const int cap = c.max_pages * c.page_tokens;
    const int len = min(max(a.lens[b], 0), cap), n = a.count ? min(max(a.count[b], 0), a.T) : a.T;
    if (rb * ROWS / a.G >= n) return;   // all rows behind the sequence's queries
    const int r0 = rb * ROWS + wr * 16 * NT;

    const CodeBits bits;

    // (waves that meet at barriers walk the same tiles)
    const TileList mine(a, r0, 16 * NT, len, n), list = CH == 1 ? mine : TileList(a, rb * ROWS, ROWS, len, n);
    const int at_lo = mine.at_lo, at_hi = mine.at_hi;
    const int per = (list.total + splits - 1) / splits;
    const int first = min(split * per, list.total), last = min(first + per, list.total);
    auto tile_of = [&](int i) { return list.tile(i); };
    const TileTable<D> table(c, b, h);
    // PF tiles in flight: while the wave works on one, the loads of the next
    // PF - 1 are under way and the table entry of the one behind them is read
    // (past the last tile, and where a tile has no page, the pool's first tile
    // is loaded and not used: loads without branches can be waited for one by one)
    TileRegs<DW, CH> buf[PF];
    bool live[PF];
    int i = first + wk, ahead = i;
    int page = ahead < last ? table.page(tile_of(ahead)) : -1;
    auto fetch = [&](int j) {   // tile `ahead` into slot j
        const int tile = tile_of(ahead);
        live[j] = table.live(page);
        buf[j].template load<true>(table.tile(page, tile), half, lane);
        ahead += WK;
        page = ahead < last ? table.page(tile_of(ahead)) : -1;
    };
#pragma unroll
    for (int j = 0; j < PF - 1; ++j) fetch(j);
    A w;   // the queries' loads follow those of the first tiles
    w.init(a, b, h, half * DW, r0, len, n, lane);
    const int stop = CH == 1 ? last : last + wk;   // CH = 2: as many steps for each wave
    while (i < stop) {
#pragma unroll
        for (int j = 0; j < PF; ++j) {
            if (i >= stop) break;
            fetch((j + PF - 1) % PF);
            const int tile = tile_of(i), p0 = tile * KV4_TILE;
            bool use = live[j];
            if (CH > 1) use = use && i < last && p0 <= at_hi && (tile < mine.n_sink || tile >= mine.lo);
            i += WK;
            if (CH == 1 && !use) continue;
            const bool full = p0 + KV4_TILE - 1 <= at_lo &&
                              (a.window == 0 || p0 > at_hi - a.window || p0 + KV4_TILE <= a.sinks);
            const RegTile<DW, CH, EXACT> t{buf[j], scales[wave], bits};
            if (use) {
                *(typename TileRegs<DW, CH>::scales_t *)(scales[wave] + lane * A::NG) = buf[j].sc;
                wave_sync();
            }
            if constexpr (CH == 2) {
                f32x4 sc[NT][2];
                if (use) {
                    w.scores(t, sc, lane);
#pragma unroll
                    for (int x = 0; x < NT * 2; ++x) parts[j][wave][x][lane] = sc[x / 2][x % 2];
                }
                local_barrier();
                if (!use) continue;
#pragma unroll
                for (int x = 0; x < NT * 2; ++x) sc[x / 2][x % 2] += parts[j][wave ^ 1][x][lane];
                if (full)
                    w.gather(t, sc, p0, true, lane);
                else
                    w.gather(t, sc, p0, false, lane);
            } else if (full)
                w.step(t, p0, true, lane);
            else
                w.step(t, p0, false, lane);
        }
    }

    w.close();
    const size_t out_row = ((size_t)b * c.Hk + h) * a.G;   // + t * B * Hk * G + head
    if constexpr (WK == 1) {
        store_rows<D, QP, NT>(a, w, b, h, half * DW, r0, n, split, splits, lane);
    } else {
        __shared__ float part[4 / CH][16][LDW];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt) __syncthreads();
            float *own = part[wave / CH][n16];
#pragma unroll
            for (int x = 0; x < A::NC; ++x) *(f32x4 *)(own + half * DW + 16 * x + 4 * quad) = w.o[nt][x];
            if (quad == 0 && half == 0) own[D] = w.m[nt], own[D + 1] = w.l[nt];
            __syncthreads();
            for (int u = threadIdx.x; u < WR * 16 * (D / 4); u += 256) {
                const int x = u % (D / 4), row = u / (D / 4), g = row / 16, rr = row % 16;
                const int r = rb * ROWS + g * 16 * NT + nt * 16 + rr, t = r / a.G;
                if (r >= R || t >= n) continue;
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < WK; ++k) top = fmaxf(top, part[g * WK + k][rr][D]);
                f32x4 sum = {0.f, 0.f, 0.f, 0.f};
                float l = 0.f;
#pragma unroll
                for (int k = 0; k < WK; ++k) {
                    const float *p = part[g * WK + k][rr];
                    const float f = p[D] > -INFINITY ? __builtin_amdgcn_exp2f(p[D] - top) : 0.f;
                    sum += f * *(const f32x4 *)(p + 4 * x);
                    l = fmaf(f, p[D + 1], l);
                }
                if (splits == 1) {
                    const float inv = l > 0.f ? 1.f / l : 0.f;
                    store4<QP>(a.out, ((size_t)t * BH * a.G + out_row + (r - t * a.G)) * D + 4 * x, sum * inv);
                } else {
                    float *p = partial_row(a, D, split, bh, r);
                    *(f32x4 *)(p + 4 * x) = sum;
                    if (x == 0) *(f32x2 *)(p + D) = f32x2{top, l};
                }
            }
        }
    }
}

// Many rows (blocks of a prompt): four waves of 16 NT rows unpack each TP tiles
// once, into LDS in operand order, and all read them; the loads and the unpacking of the
// next run beside these ones' products.  TP = 2 but for heads of 256 channels,
// where LDS has room for one tile twice.  512 tokens of two sequences, 32 heads of 128,
// behind a window of 4096: 140 + 11 us, 458 TFLOP/s, bound by the VALU work of the
// softmax (about 100 instructions for 16 rows and 32 tokens, against 16 matrix
// products) at two waves a SIMD; one row tile a wave and three or four waves took 180 us
// and more.  512 tokens of 16 sequences of 4096, 32 heads of 256: 2.11 ms, 488 TFLOP/s
// (3.47 ms with tiles unpacked by each wave), bound by reading operands from LDS.
template <int D, int QP, int NT, int TP>
__global__ void __launch_bounds__(256, 2) kv4_block_kernel(Kv4AttnArgs a, int row_blocks, int splits) {
    constexpr int ROWS = 64 * NT, NW = D / 8;   // operands of a tile
    constexpr int NL = TP * D / 128;                // 16-byte loads of a lane for TP tiles: TP D / 32 KiB in all
    using A = Attn<D, QP, NT, true>;
    __shared__ bf16x8 ops[2][TP][NW * 64];
    __shared__ float scales[2][TP][D];
    const Kv4View &c = a.c;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int BH = c.B * c.Hk, R = a.T * a.G;
    const int bh = blockIdx.x % BH, rest = blockIdx.x / BH;
    const int split = rest % splits, rb = row_blocks - 1 - rest / splits;
    const int b = bh / c.Hk, h = bh - b * c.Hk;
    const int cap = c.max_pages * c.page_tokens;
    const int len = min(max(a.lens[b], 0), cap), n = a.count ? min(max(a.count[b], 0), a.T) : a.T;
    if (rb * ROWS / a.G >= n) return;
    const int r0 = rb * ROWS + wave * 16 * NT;
    A w;
    w.init(a, b, h, 0, r0, len, n, lane);

    const TileList list(a, rb * ROWS, ROWS, len, n), mine(a, r0, 16 * NT, len, n);
    const int per = ((list.total + splits - 1) / splits + TP - 1) / TP * TP;
    const int first = min(split * per, list.total), last = min(first + per, list.total);
    const TileTable<D> table(c, b, h);
    u32x4 word[NL];
    float scale = 0.f;
    const int st = threadIdx.x / D, sx = threadIdx.x % D;   // a thread's scale: tile of the TP, place
    int live[2] = {}, next[2] = {};   // whether the tiles have a page
    auto fetch = [&](int i) {   // tiles i (and i + 1) of the list
        const int t0 = list.tile(i), t1 = list.tile(min(i + 1, last - 1));
        const int g0 = table.page(t0), g1 = table.page(t1);
        const uint8_t *p0 = table.tile(g0, t0), *p1 = table.tile(g1, t1);
        next[0] = table.live(g0), next[1] = i + 1 < last && table.live(g1);
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int x = wave + 4 * j;
            word[j] = *(const u32x4 *)((x < D / 32 ? p0 : p1) + x % (D / 32) * 1024 + lane * 16);
        }
        if (st < TP) scale = ((const float *)((st ? p1 : p0) + 32 * D))[sx];
    };
    auto unpack = [&](int buf) {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int x = wave + 4 * j;
            bf16x8 *to = ops[buf][x / (D / 32)] + x % (D / 32) * 256 + lane;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                to[e * 64] = exact_codes(x % (D / 32) < D / 64 ? word[j][e] ^ KEY_SIGNS : word[j][e]);
        }
        if (st < TP) scales[buf][st][sx] = scale;
        live[0] = next[0], live[1] = next[1];
    };
    if (first < last) {
        fetch(first);
        unpack(0);
    }
    local_barrier();
    int buf = 0;
    for (int i = first; i < last; i += TP, buf ^= 1) {
        const bool more = i + TP < last;
        if (more) fetch(i + TP);
#pragma unroll
        for (int j = 0; j < TP; ++j) {
            const int tile = list.tile(i + j), p0 = tile * KV4_TILE;
            // none, without a page, or not one of this wave's rows
            if (!live[j] || p0 > mine.at_hi || (tile >= mine.n_sink && tile < mine.lo)) continue;
            const SharedTile<D> t{ops[buf][j], scales[buf][j]};
            const bool full = p0 + KV4_TILE - 1 <= mine.at_lo &&
                              (a.window == 0 || p0 > mine.at_hi - a.window || p0 + KV4_TILE <= a.sinks);
            if (full)
                w.step(t, p0, true, lane);
            else
                w.step(t, p0, false, lane);
        }
        if (more) unpack(buf ^ 1);
        local_barrier();
    }
    w.close();
    store_rows<D, QP, NT>(a, w, b, h, 0, r0, n, split, splits, lane);
}

// Joins the splits of a row.  W waves take its splits in turn; W = 1: one wave a
// row, four rows a workgroup (few splits of many rows: 16384 rows in two parts
// take 11 us so and 25 us with W = 4, 2048 rows in eight parts 6.8 and 4.8 us).
template <int D, int QP, int W>
__global__ void __launch_bounds__(256) kv4_join_kernel(Kv4AttnArgs a, int splits) {
    constexpr int NL = D / 4;   // lanes that hold a row
    __shared__ float part[W == 1 ? 1 : 4][D + 4];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, R = a.T * a.G;
    const long long row = W == 1 ? (long long)blockIdx.x * 4 + wave : blockIdx.x;
    if (row >= (long long)a.c.B * a.c.Hk * R) return;
    const int bh = (int)(row / R), r = (int)(row - (long long)bh * R), t = r / a.G, b = bh / a.c.Hk;
    const int n = a.count ? min(max(a.count[b], 0), a.T) : a.T;
    if (t >= n) return;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    float top = -INFINITY, l = 0.f;
    for (int s = W == 1 ? 0 : wave; s < splits; s += W) {
        const float *p = partial_row(a, D, s, bh, r);
        const f32x2 ml = *(const f32x2 *)(p + D);
        const f32x4 x = lane < NL ? *(const f32x4 *)(p + 4 * lane) : sum;
        if (ml[0] == -INFINITY) continue;
        const float m2 = fmaxf(top, ml[0]);
        const float f0 = __builtin_amdgcn_exp2f(top - m2), f1 = __builtin_amdgcn_exp2f(ml[0] - m2);
        sum = sum * f0 + x * f1;
        l = l * f0 + ml[1] * f1;
        top = m2;
    }
    if constexpr (W > 1) {
        if (lane < NL) *(f32x4 *)&part[wave][4 * lane] = sum;
        if (lane == 0) part[wave][D] = top, part[wave][D + 1] = l;
        __syncthreads();
        if (wave > 0 || lane >= NL) return;
        top = fmaxf(fmaxf(part[0][D], part[1][D]), fmaxf(part[2][D], part[3][D]));
        sum = f32x4{0.f, 0.f, 0.f, 0.f}, l = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float f = part[k][D] > -INFINITY ? __builtin_amdgcn_exp2f(part[k][D] - top) : 0.f;
            sum += f * *(const f32x4 *)&part[k][4 * lane];
            l = fmaf(f, part[k][D + 1], l);
        }
    }
    if (lane >= NL) return;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    store4<QP>(a.out, (((size_t)t * a.c.B * a.c.Hk + bh) * a.G + (r - t * a.G)) * D + 4 * lane, sum * inv);
}

// rows of a workgroup, and the number of parts a row's tokens are split into
struct Plan {
    int nt, wr, row_blocks, splits;
};
// at most what a row block sees of a cache with a window: see TileList
long long window_tiles(int window, int sinks, int rows, int G) {
    return ((long long)window + (rows + G - 1) / G) / KV4_TILE + 2 + ((long long)sinks + KV4_TILE - 1) / KV4_TILE;
}
Plan plan_for(const Kv4View &c, int G, int T, int window, int sinks, int bf16) {
    Plan p;
    const long long R = (long long)T * G, heads = (long long)c.B * c.Hk;
    auto tiles_of = [&](int rows) {   // at most what a row block sees
        const long long all = ((long long)c.max_pages * c.page_tokens + KV4_TILE - 1) / KV4_TILE;
        const long long seen = ((long long)window + rows / G + 1) / KV4_TILE + 2 + ((long long)sinks + KV4_TILE - 1) / KV4_TILE;
        return window ? std::min(all, seen) : all;
    };
    // 16 or 32 rows a wave (registers: 32 for bf16 heads of up to 128 channels).  32
    // halve the unpacking for a row and double a workgroup's, so they pay where a
    // workgroup, two to a unit, has 24 tiles or more: 64 tokens of 32 heads in a cache of 8192,
    // 8 tiles, 37 us with 16 rows and 45 with 32; 256 tokens, 32 tiles, 98 and 91 us.  At 33
    // to 64 rows, halves of a tile list (WR = 2) with 32 rows a wave beat four waves
    // of 16 for 64 channels (37 and 39 us for 160 heads), not for 128 (34 and 25 us for 55).
    const bool wide = bf16 && c.d <= 128;
    p.nt = wide && (R <= 64 ? R > 32 && c.d == 64 : heads * ((R + 127) / 128) * tiles_of(128) >= 24 * 512) ? 2 : 1;
    p.wr = R <= 16 ? 1 : R <= (p.nt == 2 ? 64 : 32) ? 2 : 4;
    const int rows = 16 * p.nt * p.wr;
    p.row_blocks = (int)((R + rows - 1) / rows);
    const long long groups = heads * p.row_blocks, tiles = tiles_of(rows);
    if (p.wr == 4) {
        // many rows: their partial results cost more than idle units, so only until all
        // have a place on the card at once (two a unit, three of 64 channels); from eight
        // tiles a workgroup on also to the fewest parts that leave at most 15% of the places
        // empty in the last round (384 workgroups of 256 tiles: 469 us whole, 378 us in
        // four parts; 320 of 128 tiles: 243 and 188 us)
        const long long places = c.d == 64 ? 768 : 512;
        p.splits = (int)std::max(1ll, std::min(places / groups, tiles / 4));
        for (long long s = p.splits; s <= std::min(tiles / 8, 8ll); ++s)
            if (groups * s * 100 >= 85 * places * ((groups * s + places - 1) / places)) {
                p.splits = (int)s;
                break;
            }
    } else {
        // few rows: to two workgroups a unit at four tiles a wave, and beyond, as lengths
        // differ, to sixteen at 32 tiles (at four: 64 caches of up to 1024 tokens, 23 us against
        // 16; of 4096 tokens, 256 channels, 117 against 105)
        const int wk = std::max(1, 4 / (p.wr * (c.d == 256 ? 2 : 1)));   // waves that share a row's tiles
        p.splits = (int)std::max(std::min((511 + groups) / groups, tiles / (4 * wk)),
                                 std::min((4095 + groups) / groups, tiles / (32 * wk)));
    }
    p.splits = std::max(1, std::min(p.splits, 256));
    // the workspace is that of a call without a window
    if (window) p.splits = std::min(p.splits, plan_for(c, G, T, 0, 0, bf16).splits);
    return p;
}

template <int D, int QP, int NT, int WR>
void launch(const Kv4AttnArgs &a, const Plan &p, hipStream_t s) {
    const dim3 grid((unsigned)((long long)a.c.B * a.c.Hk * p.row_blocks * p.splits));
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, p.row_blocks, p.splits); };
    if constexpr (WR == 4)
        go(kv4_block_kernel<D, QP, NT, D == 256 ? 1 : 2>);
    else
        go(kv4_attention_kernel<D, QP, NT, WR, D == 256 ? 2 : 1, 2, NT == 1 ? 2 : 1>);
    const long long rows = (long long)a.c.B * a.c.Hk * a.T * a.G;
    if (p.splits > 8 || (p.splits > 1 && rows <= 8192))
        hipLaunchKernelGGL((kv4_join_kernel<D, QP, 4>), dim3((unsigned)rows), dim3(256), 0, s, a, p.splits);
    else if (p.splits > 1)
        hipLaunchKernelGGL((kv4_join_kernel<D, QP, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, s, a, p.splits);
}

template <int D, int QP>
void dispatch(const Kv4AttnArgs &a, const Plan &p, hipStream_t s) {
    if (p.wr == 1) return launch<D, QP, 1, 1>(a, p, s);
    if constexpr (QP == 1 && D <= 128) {
        if constexpr (D == 64)
            if (p.nt == 2 && p.wr == 2) return launch<D, QP, 2, 2>(a, p, s);
        if (p.nt == 2) return launch<D, QP, 2, 4>(a, p, s);
        return p.wr == 2 ? launch<D, QP, 1, 2>(a, p, s) : launch<D, QP, 1, 4>(a, p, s);
    } else {
        return p.wr == 2 ? launch<D, QP, 1, 2>(a, p, s) : launch<D, QP, 1, 4>(a, p, s);
    }
}

}  // namespace

uint64_t kv4_attention_workspace(const Kv4View &c, int G, int T, int bf16) {
    const Plan p = plan_for(c, G, T, 0, 0, bf16);
    return p.splits == 1 ? 0 : (uint64_t)p.splits * c.B * c.Hk * T * G * (c.d + 4) * 4;
}

hipError_t launch_kv4_attention(const Kv4AttnArgs &a, int bf16, hipStream_t s) {
    const Plan p = plan_for(a.c, a.G, a.T, a.window, a.sinks, bf16);
    if (a.c.d == 64)
        bf16 ? dispatch<64, 1>(a, p, s) : dispatch<64, 3>(a, p, s);
    else if (a.c.d == 128)
        bf16 ? dispatch<128, 1>(a, p, s) : dispatch<128, 3>(a, p, s);
    else
        bf16 ? dispatch<256, 1>(a, p, s) : dispatch<256, 3>(a, p, s);
    return hipGetLastError();
}

}  // namespace pace
