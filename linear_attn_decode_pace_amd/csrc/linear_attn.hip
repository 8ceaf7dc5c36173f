// Linear attention with a fixed decay g for each head:
//     M_t = g M_{t-1} + k_t v_t^T,   o_t = scale M_t^T q_t.
//
// Recurrent form (decode steps): the state goes through registers, one read and
// one write of it bound the step.
//
// Chunked form (bf16 prompts): for the tokens i = 0..C-1 of a chunk and the
// state M before it,
//     O = diag(g^{i+1}) Q M + (Q K^T o D) V,   D_ij = g^{i-j} for i >= j, else 0,
//     M <- g^C M + K^T diag(g^{C-1-i}) V,
// on bf16 matrix cores with float32 sums.  Q, K and V are exact operands; the
// three float32 factors (M, the weighted scores, the weighted V) are taken in
// three bf16 parts each, which keep their 24 bits, so outputs and state are as
// exact as float32 products.
//
// 1024 states of 128 x 128 over 4096 tokens take 1.26 ms: 273 TFLOP/s of the
// formulas above (without the parts' factor of three), 4.3 TB/s of q, k, v and o.
// Neither matrix cores (38% busy) nor VALU (35%) nor LDS (23%) fill that time:
// the shader clock falls to 1.9 GHz under it, and the phases of a chunk (scores,
// Q M, update) depend on each other within two waves a SIMD.  With neither
// loads nor stores it takes 1.02 ms, with a third of the products 1.16 ms.
// 16 states over 16384 tokens are cut into 32 segments each: 44 us for the
// segments' own states, 13 us to add them up, 88 us for the outputs.
#include <algorithm>
#include <type_traits>

#include "mfma_common.h"
#include "pace_layers.h"

namespace pace {
namespace {

// four elements as floats
template <class T>
__device__ inline f32x4 in_four(const void *p, size_t i) {
    if constexpr (sizeof(T) == 2) {
        const u32x2 w = *(const u32x2 *)((const uint16_t *)p + i);
        return f32x4{lo_f32(w[0]), hi_f32(w[0]), lo_f32(w[1]), hi_f32(w[1])};
    }
    return *(const f32x4 *)((const float *)p + i);
}

template <class T>
__device__ inline float in_elem(const void *p, size_t i) {
    if constexpr (sizeof(T) == 2) return bf2f(((const uint16_t *)p)[i]);
    return ((const float *)p)[i];
}

// Recurrent form.  One workgroup per (sequence, head, block of 4 CG columns): a
// thread holds 4 adjacent columns of DK / RG state rows in registers over all
// tokens, so the state is read and written once.
// STREAM: states larger than the last-level cache are read and written past
// it (16384 states of 128 x 128: 361 us, 6.0 TB/s, 25 us less).
// ONE: one column block; otherwise a state's blocks follow each other on one XCD, as
// they share lines of it (15756 states of 128 x 48: 147 us, blocks in the order
// of the grid 198 us).
template <int DK, int CG, bool STREAM, bool ONE>
struct StepState {
    static constexpr int RG = 256 / CG, NR = DK / RG;
    int bh, col0, cg, rg, n;
    float g;
    f32x4 M[NR];
    __device__ inline bool place(const LinearArgs &a, int col_blocks) {
        int cb = 0;
        bh = blockIdx.x;
        if constexpr (!ONE) {
            const int turn = blockIdx.x / 8;
            cb = turn % col_blocks, bh = turn / col_blocks * 8 + blockIdx.x % 8;
        }
        cg = threadIdx.x % CG, rg = threadIdx.x / CG, col0 = cb * CG * 4;
        return ONE || bh < a.B * a.H;
    }
    __device__ inline size_t base(const LinearArgs &a) const {
        return (size_t)bh * DK * a.dv + (size_t)(rg * NR) * a.dv + col0 + cg * 4;
    }
    __device__ inline void load(const LinearArgs &a) {
        const int b = bh / a.H;
        n = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
        g = a.decay[bh - b * a.H];
        const size_t at = base(a);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const f32x4 *from = (const f32x4 *)(a.state_in + at + (size_t)i * a.dv);
            M[i] = !a.state_in ? f32x4{0.f, 0.f, 0.f, 0.f} : STREAM ? __builtin_nontemporal_load(from) : *from;
        }
    }
    __device__ inline void store(const LinearArgs &a) const {
        const size_t at = base(a);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            f32x4 *to = (f32x4 *)(a.state_out + at + (size_t)i * a.dv);
            if (STREAM)
                __builtin_nontemporal_store(M[i], to);
            else
                *to = M[i];
        }
    }
    // one token; returns what the thread's rows give to its output
    __device__ inline f32x4 step(const float *k, const float *q, f32x4 v) {
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const float kk = k[rg * NR + i], qq = q[rg * NR + i];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                M[i][e] = fmaf(kk, v[e], M[i][e] * g);
                o[e] = fmaf(qq, M[i][e], o[e]);
            }
        }
        return o;
    }
};

// A single token: its output is summed over the row groups in LDS (in a wave's lanes first,
// as below, costs registers and with them a wave a SIMD: 378 us for those 16384 states)
template <class T, int DK, int CG, bool STREAM, bool ONE>
__global__ void __launch_bounds__(256) linear_token_kernel(LinearArgs a, int col_blocks) {
    using S = StepState<DK, CG, STREAM, ONE>;
    __shared__ f32x4 part[S::RG][CG];
    __shared__ float kq[2][DK];
    S s;
    if (!s.place(a, col_blocks)) return;
    s.load(a);
    if (s.n > 0) {
        for (int i = threadIdx.x; i < 2 * DK; i += 256)
            kq[i / DK][i % DK] = in_elem<T>(i < DK ? a.k : a.q, (size_t)s.bh * DK + i % DK);
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = in_elem<T>(a.v, (size_t)s.bh * a.dv + s.col0 + s.cg * 4 + e);
        __syncthreads();
        part[s.rg][s.cg] = s.step(kq[0], kq[1], v);
        __syncthreads();
        if (s.rg == 0) {
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
            for (int r = 0; r < S::RG; ++r) sum += part[r][s.cg];
            *(f32x4 *)(a.out + (size_t)s.bh * a.dv + s.col0 + s.cg * 4) = sum * a.scale;
        }
    }
    s.store(a);
}

// Several tokens: q, k and v of TB tokens are fetched at a time, into LDS, and o_t =
// M_t^T q_t is summed over a thread's rows, a wave's lanes, and for the TB tokens
// together the waves in LDS (15756 states of 128 x 48, 8 tokens: 203 us, with a
// token's loads and sums after each other 436 us)
template <class T, int DK, int CG, bool STREAM, bool ONE>
__global__ void __launch_bounds__(256) linear_step_kernel(LinearArgs a, int col_blocks) {
    constexpr int TB = 8;
    using S = StepState<DK, CG, STREAM, ONE>;
    __shared__ f32x4 part[TB][4][CG], vs[TB][CG];
    __shared__ __align__(16) float kq[TB][2][DK];
    S s;
    if (!s.place(a, col_blocks)) return;
    s.load(a);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, bh = s.bh, col0 = s.col0;
    const size_t BH = (size_t)a.B * a.H;
    for (int t0 = 0; t0 < s.n; t0 += TB) {
        const int m = min(TB, s.n - t0);
        if (t0) __syncthreads();
        for (int u = threadIdx.x; u < m * (DK / 2); u += 256) {
            const int t = u / (DK / 2), x = u % (DK / 2), what = x / (DK / 4), at = x % (DK / 4) * 4;
            *(f32x4 *)&kq[t][what][at] = in_four<T>(what ? a.q : a.k, ((t0 + t) * BH + bh) * DK + at);
        }
        for (int u = threadIdx.x; u < m * CG; u += 256)
            vs[u / CG][u % CG] = in_four<T>(a.v, ((t0 + u / CG) * BH + bh) * a.dv + col0 + u % CG * 4);
        __syncthreads();
        for (int t = 0; t < m; ++t) {
            const f32x4 o = s.step(kq[t][0], kq[t][1], vs[t][s.cg]);
            // over the wave's lanes of a column group, halving what a lane holds in each step
            const bool hi = lane & CG, hi2 = lane & (2 * CG);
            float x = hi ? o[2] : o[0], y = hi ? o[3] : o[1];
            x += __shfl_xor(hi ? o[0] : o[2], CG);
            y += __shfl_xor(hi ? o[1] : o[3], CG);
            float *to = (float *)&part[t][wave][s.cg] + 2 * hi;
            if constexpr (CG == 32) {
                *(f32x2 *)to = f32x2{x, y};
            } else {
                float z = hi2 ? y : x;
                z += __shfl_xor(hi2 ? x : y, 2 * CG);
#pragma unroll
                for (int d = 4 * CG; d < 64; d <<= 1) z += __shfl_xor(z, d);
                if (lane < 4 * CG) to[hi2] = z;
            }
        }
        __syncthreads();
        for (int u = threadIdx.x; u < m * CG; u += 256) {
            const int t = u / CG, x = u % CG;
            const f32x4 sum = (part[t][0][x] + part[t][1][x]) + (part[t][2][x] + part[t][3][x]);
            *(f32x4 *)(a.out + ((t0 + t) * BH + bh) * a.dv + col0 + x * 4) = sum * a.scale;
        }
    }
    s.store(a);
}

template <class T, int DK, int CG>
void launch_step_columns(const LinearArgs &a, hipStream_t s) {
    const int cb = a.dv / (4 * CG);
    const dim3 grid((unsigned)(cb == 1 ? (long long)a.B * a.H : ((long long)a.B * a.H + 7) / 8 * 8 * cb));
    // (rows of 64 bytes share lines: 1313 x 12 states of 128 x 112, 331 us, 388 us past the cache)
    const bool stream = (double)a.B * a.H * a.dk * a.dv * 4 > 256e6;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, cb); };
    auto form = [&](auto past, auto one) {
        constexpr bool STREAM = decltype(past)::value, ONE = decltype(one)::value;
        a.T == 1 ? go(linear_token_kernel<T, DK, CG, STREAM, ONE>) : go(linear_step_kernel<T, DK, CG, STREAM, ONE>);
    };
    auto columns = [&](auto past) { cb == 1 ? form(past, std::true_type()) : form(past, std::false_type()); };
    if constexpr (CG > 4)
        if (stream) return columns(std::true_type());
    columns(std::false_type());
}

template <class T, int DK>
hipError_t launch_step(const LinearArgs &a, hipStream_t s) {
    if (a.dv % 128 == 0)
        launch_step_columns<T, DK, 32>(a, s);
    else if (a.dv % 64 == 0)
        launch_step_columns<T, DK, 16>(a, s);
    else if (a.dv % 32 == 0)
        launch_step_columns<T, DK, 8>(a, s);
    else
        launch_step_columns<T, DK, 4>(a, s);
    return hipGetLastError();
}

// ---- chunked form -----------------------------------------------------------

constexpr int LC = 64;   // tokens of a chunk

// Workgroup barrier that orders LDS only: the next chunk's global loads and
// this one's stores stay in flight across it
__device__ inline void local_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// g^n from repeated squares in float64
__device__ inline float power(float g, int n) {
    double p = 1.0, b = g;
    for (; n > 0; n >>= 1) {
        if (n & 1) p *= b;
        b *= b;
    }
    return (float)p;
}

// The pairs (-1, 0) and (0, -1) in bf16, kept in registers: as a literal the
// second would be taken for the inline constant -1.0 of a float32 operand
struct Minus {
    uint32_t lo = 0x0000bf80u, hi = 0xbf800000u;
    __device__ inline Minus() { asm volatile("" : "+s"(lo), "+s"(hi)); }
    // x minus the first / second element of the pair w, in one dot product
    __device__ inline float first(uint32_t w, float x) const {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, lo), x, false);
    }
    __device__ inline float second(uint32_t w, float x) const {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, hi), x, false);
    }
};

// 2 N float32 values as three lists of bf16 pairs whose sum has 24 bits (the
// remainders x - bf16(x) are exact)
template <int N>
__device__ inline void split3(float *x, uint32_t (*part)[N], const Minus &minus) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const uint32_t w = part[i][e] = pk_bf16(x[2 * e], x[2 * e + 1]);
            if (i < 2) x[2 * e] = minus.first(w, x[2 * e]), x[2 * e + 1] = minus.second(w, x[2 * e + 1]);
        }
}
__device__ inline bf16x8 operand(const uint32_t *w) { return __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]}); }

// 16 x 16 tile of the scores S: place of its probabilities' k-slice (query
// tile i, slice ks of 32 keys) among the six that are not zero
__device__ inline int score_slice(int i, int ks) { return i < 2 ? i : 2 * i - 2 + ks; }

enum { LIN_WHOLE, LIN_LOCAL, LIN_OUTPUTS };

// One workgroup: a block of 64 CT columns of one (sequence, head), 16 CT
// columns for each wave, whose part of M stays in its registers.  All products
// run over k-slots in the order in which a 16 x 16 accumulator tile leaves
// its rows in the lanes (slot j of lane group x: row 16 (j / 4) + 4 x + j % 4), so M and
// the scores are operands as they stand; K^T and V are read from LDS
// transposed.  Outputs are formed transposed, four adjacent columns of
// a token in a lane.
//   LIN_WHOLE: the state from state_in through all tokens to state_out.
//   LIN_LOCAL: segment `seg` alone, from zero, its state to the workspace.
//   LIN_OUTPUTS: a segment's outputs from the state before it in the workspace.
template <int DK, int CT, int MODE>
__global__ void __launch_bounds__(256, 2) linear_chunk_kernel(LinearArgs a, int col_blocks, int segs, int seg_len) {
    constexpr int RT = DK / 16, KS = DK / 32, CB = 64 * CT;
    constexpr int KP = 64 * (DK / 8) / 256, VP = 2 * CT;   // 16-byte pieces a thread moves
    constexpr int ROW = DK + 8, VROW = CB + 8;   // rows 4 banks apart, offsets that fit an instruction
    __shared__ __align__(16) uint16_t kx[LC][ROW], qx[MODE == LIN_LOCAL ? 1 : LC][ROW], vx[LC][VROW];
    __shared__ u32x4 px[3][6][MODE == LIN_LOCAL ? 1 : 64];
    __shared__ __align__(16) float rw[LC], ps[LC + 16];   // g^(63 - n); scale g^(n - 15), 0 below n = 15
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n16 = lane & 15, quad = lane >> 4;
    const int BH = a.B * a.H;
    const int bh = blockIdx.x % BH, rest = blockIdx.x / BH, cb = rest % col_blocks, seg = rest / col_blocks;
    const int b = bh / a.H, h = bh - b * a.H;
    const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const int lo = seg * seg_len, hi = min(len, lo + seg_len);
    if (MODE != LIN_WHOLE && lo >= hi) return;
    const int col0 = cb * 64 * CT + wave * 16 * CT;   // first column of the wave
    const float g = a.decay[h];
    for (int i = threadIdx.x; i < LC + 16; i += 256) {
        const float p = power(g, i - 15 < 0 ? 0 : i - 15);
        ps[i] = i < 15 ? 0.f : a.scale * p;
        if (i >= 15 && i < 15 + LC) rw[LC - 1 - (i - 15)] = p;
    }
    const Minus minus;

    f32x4 M[RT][CT];
    const size_t tile = (size_t)bh * DK * a.dv;
    const size_t in_state = tile + (size_t)(4 * quad) * a.dv + col0 + n16;
    const float *from = MODE == LIN_WHOLE ? a.state_in : a.workspace + (size_t)seg * BH * DK * a.dv;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                M[rt][ct][r] = MODE != LIN_LOCAL && from && col0 + 16 * ct < a.dv
                                   ? from[in_state + (size_t)(16 * rt + r) * a.dv + 16 * ct]
                                   : 0.f;

    // A chunk's tokens fill rows 64 - cl .. 63 of LDS: weights then depend on
    // the row alone, and a chunk of fewer tokens has zeros in front.  Row 0 is
    // token r0 = c0 + cl - 64; a thread's 16-byte pieces are 256 apart.
    u32x4 kr[KP], qr[MODE == LIN_LOCAL ? 1 : KP], vr[VP];
    const size_t kstep = (size_t)BH * DK, vstep = (size_t)BH * a.dv;
    constexpr int KROWS = 256 / (DK / 8), VROWS = 256 / (CB / 8);   // rows of a pass over the pieces
    const int krow = threadIdx.x / (DK / 8), vrow = threadIdx.x / (CB / 8);
    const int kcol = threadIdx.x % (DK / 8) * 8, vcol = threadIdx.x % (CB / 8) * 8;
    const uint32_t kat = 2 * ((uint32_t)krow * (uint32_t)kstep + kcol);
    const int vsrc = min(cb * CB + vcol, a.dv - 8);   // columns behind the last are never stored
    const uint32_t vat = 2 * ((uint32_t)vrow * (uint32_t)vstep + vsrc);
    auto fetch = [&](int r0) {
        if (r0 >= lo) {   // wave-uniform rows and 32-bit places in them
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                const size_t row = (size_t)(r0 + KROWS * i) * kstep + (size_t)bh * DK;
                kr[i] = *(const u32x4 *)at((const uint16_t *)a.k + row, kat);
                if constexpr (MODE != LIN_LOCAL) qr[i] = *(const u32x4 *)at((const uint16_t *)a.q + row, kat);
            }
#pragma unroll
            for (int i = 0; i < VP; ++i)
                vr[i] = *(const u32x4 *)at((const uint16_t *)a.v + (size_t)(r0 + VROWS * i) * vstep + (size_t)bh * a.dv, vat);
        } else {          // fewer than 64 tokens in all: the rows in front repeat the first
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                const size_t from = (size_t)max(r0 + KROWS * i + krow, lo) * kstep + (size_t)bh * DK + kcol;
                kr[i] = *(const u32x4 *)((const uint16_t *)a.k + from);
                if constexpr (MODE != LIN_LOCAL) qr[i] = *(const u32x4 *)((const uint16_t *)a.q + from);
            }
#pragma unroll
            for (int i = 0; i < VP; ++i)
                vr[i] = *(const u32x4 *)((const uint16_t *)a.v + (size_t)max(r0 + VROWS * i + vrow, lo) * vstep +
                                         (size_t)bh * a.dv + vsrc);
        }
    };
    auto put = [&](int skip) {   // rows below `skip` are zeros
        if (skip) {
            const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < KP; ++i)
                if (KROWS * i + krow < skip) kr[i] = zero, qr[MODE == LIN_LOCAL ? 0 : i] = zero;
#pragma unroll
            for (int i = 0; i < VP; ++i)
                if (VROWS * i + vrow < skip) vr[i] = zero;
        }
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            *(u32x4 *)&kx[KROWS * i + krow][kcol] = kr[i];
            if constexpr (MODE != LIN_LOCAL) *(u32x4 *)&qx[KROWS * i + krow][kcol] = qr[i];
        }
#pragma unroll
        for (int i = 0; i < VP; ++i) *(u32x4 *)&vx[VROWS * i + vrow][vcol] = vr[i];
    };
    // operand of row `row`: k-slots of slice ks, whose elements lie in the row
    auto row_frag = [&](const uint16_t (*m)[ROW], int row, int ks) {
        // volatile: joined into one paired read the two take twice as long (bank
        // conflicts between the halves)
        typedef const volatile __attribute__((address_space(3))) u32x2 *local;
        const u32x2 x = *(local)&m[row][32 * ks + 4 * quad], y = *(local)&m[row][32 * ks + 16 + 4 * quad];
        return __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
    };
    // operand of column c + lane % 16: k-slots are the tokens of slice ks
    auto col_frag = [&](auto &m, int c, int ks) {
        typedef __attribute__((address_space(3))) s16x4 *local;
        s16x4 x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = 32 * ks + 16 * i + 4 * quad + (n16 >> 2);
            x[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((local)&m[row][c + (n16 & 3) * 4]);
        }
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(bf16x8, s16x8{x[0][0], x[0][1], x[0][2], x[0][3], x[1][0], x[1][1], x[1][2], x[1][3]});
    };

    if constexpr (MODE != LIN_LOCAL) {   // halves of the diagonal slices that lie above the diagonal
        if (wave < 3) {
            *((u32x2 *)&px[wave][score_slice(0, 0)][lane] + 1) = u32x2{0, 0};
            *((u32x2 *)&px[wave][score_slice(2, 1)][lane] + 1) = u32x2{0, 0};
        }
    }
    if (lo < hi) {
        const int skip = max(LC - (hi - lo), 0);
        fetch(lo - skip);
        put(skip);
    }
    local_barrier();
    for (int c0 = lo; c0 < hi; c0 += LC) {
        const int cl = min(LC, hi - c0), skip = LC - cl, r0 = c0 - skip;
        const bool more = c0 + LC < hi;
        const int skip2 = max(LC - (hi - c0 - LC), 0);   // of the next chunk
        if (more) fetch(c0 + LC - skip2);
        f32x4 o[4][CT];
        if constexpr (MODE != LIN_LOCAL) {
            // weighted scores, transposed: the ten tiles (i, j) at or below the
            // diagonal, (3, 0..2), (2, 0..2), (1, 0..1) and (0, 0), (3, 3) to the
            // four waves, so that a wave's tiles share their operands
            const int i0 = wave == 3 ? 3 : 3 - wave, i2 = wave == 2 ? 0 : i0;
            f32x4 sc[3];
#pragma unroll
            for (int it = 0; it < 3; ++it) sc[it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const bf16x8 q0 = row_frag(qx, 16 * i0 + n16, ks);
                if (wave == 3) {
                    sc[0] = mfma_bf16_k32(row_frag(kx, 48 + n16, ks), q0, sc[0]);
                } else {
                    const bf16x8 k0 = row_frag(kx, n16, ks);
                    sc[0] = mfma_bf16_k32(k0, q0, sc[0]);
                    sc[1] = mfma_bf16_k32(row_frag(kx, 16 + n16, ks), q0, sc[1]);
                    if (wave == 2)
                        sc[2] = mfma_bf16_k32(k0, row_frag(qx, n16, ks), sc[2]);
                    else
                        sc[2] = mfma_bf16_k32(row_frag(kx, 32 + n16, ks), q0, sc[2]);
                }
            }
#pragma unroll
            for (int it = 0; it < 3; ++it) {
                if (wave == 3 && it > 0) break;
                const int i = it == 2 ? i2 : i0, j = wave == 3 ? 3 : it == 2 && wave == 2 ? 0 : it;
                const float *w = ps + 15 + 16 * (i - j) + n16 - 4 * quad;
                float x[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = sc[it][r] * w[-r];
                uint32_t p[3][2];
                split3<2>(x, p, minus);
#pragma unroll
                for (int part = 0; part < 3; ++part)
                    *((u32x2 *)&px[part][score_slice(i, j >> 1)][lane] + (j & 1)) = u32x2{p[part][0], p[part][1]};
            }
            // Q M; the parts outermost, so that no product waits for the one before it
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) o[i][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
            bf16x8 qf[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) qf[0][i] = row_frag(qx, 16 * i + n16, 0);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if (ks + 1 < KS) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) qf[(ks + 1) & 1][i] = row_frag(qx, 16 * i + n16, ks + 1);
                }
                uint32_t m[CT][3][4];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = M[2 * ks + (e >> 2)][ct][e & 3];
                    split3<4>(x, m[ct], minus);
                }
#pragma unroll
                for (int part = 2; part >= 0; --part)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct)
                            o[i][ct] = mfma_bf16_k32(operand(m[ct][part]), qf[ks & 1][i], o[i][ct]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = ps[max(16 + 16 * i + n16 - skip, 0)];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) o[i][ct] *= w;
            }
            local_barrier();   // the scores of all waves are there
        }
        bf16x8 vf[2][CT];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) vf[ks][ct] = col_frag(vx, wave * 16 * CT + 16 * ct, ks);
        if constexpr (MODE != LIN_LOCAL) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int part = 2; part >= 0; --part)
#pragma unroll
                    for (int i = 2 * ks; i < 4; ++i) {
                        const bf16x8 pf = __builtin_bit_cast(bf16x8, px[part][score_slice(i, ks)][lane]);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) o[i][ct] = mfma_bf16_k32(vf[ks][ct], pf, o[i][ct]);
                    }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (16 * i + n16 >= skip) {
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        if (col0 + 16 * ct < a.dv)
                            *(f32x4 *)at(a.out + (long long)(r0 + 16 * i) * (long long)vstep + (size_t)bh * a.dv + col0 + 16 * ct,
                                         4 * ((uint32_t)n16 * (uint32_t)vstep + 4 * quad)) = o[i][ct];
                }
            }
        }
        if (more || MODE != LIN_OUTPUTS) {
            const float gc = cl == LC ? rw[0] * g : rw[LC - 1 - cl];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) M[rt][ct] *= gc;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                uint32_t vp[CT][3][4];
                const f32x4 w0 = *(const f32x4 *)&rw[32 * ks + 4 * quad], w1 = *(const f32x4 *)&rw[32 * ks + 16 + 4 * quad];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const u32x4 v = __builtin_bit_cast(u32x4, vf[ks][ct]);
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = (e & 1 ? hi_f32(v[e >> 1]) : lo_f32(v[e >> 1])) * (e < 4 ? w0[e] : w1[e & 3]);
                    split3<4>(x, vp[ct], minus);
                }
#pragma unroll
                for (int rt = 0; rt < RT; rt += 2) {
                    const bf16x8 kf[2] = {col_frag(kx, 16 * rt, ks), col_frag(kx, 16 * rt + 16, ks)};
#pragma unroll
                    for (int part = 2; part >= 0; --part)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct)
                                M[rt + x][ct] = mfma_bf16_k32(kf[x], operand(vp[ct][part]), M[rt + x][ct]);
                }
            }
        }
        if (more) {
            local_barrier();   // every wave is done with this chunk
            put(skip2);
            local_barrier();
        }
    }
    if constexpr (MODE != LIN_OUTPUTS) {
        float *to = MODE == LIN_WHOLE ? a.state_out : a.workspace + (size_t)seg * BH * DK * a.dv;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (col0 + 16 * ct < a.dv) to[in_state + (size_t)(16 * rt + r) * a.dv + 16 * ct] = M[rt][ct][r];
    }
}

// float32 inputs: the same chunk algebra on float32 matrix products (16 x 16 x 4),
// 32 tokens at a time.  Their k-slot is the lane group: with group x as row 4 x + r of a
// 16-row tile, register r of an accumulator tile is an operand as it stands.
// Bound by the matrix rate of float32 (a sixteenth of bf16): 128 states of 128 x 128
// over 2048 tokens take 293 us (72 TFLOP/s), token by token 2630 us.  Calls of 17 to 33
// tokens and 1024 states lose up to a tenth (46.6 us, 41.8 us), with fewer states they
// gain (11.6 us, 19.5 us), so the switch stands at 16 tokens as for bf16.
template <int DK, int CT, int MODE>
__global__ void __launch_bounds__(256, 2) linear_chunk_f32_kernel(LinearArgs a, int col_blocks, int segs, int seg_len) {
    constexpr int C = 32, RT = DK / 16, CB = 64 * CT;
    constexpr int KP = C * (DK / 4) / 256, VP = C * (CB / 4) / 256;   // 16-byte pieces a thread moves
    constexpr int ROW = DK + 4, VROW = CB + 4;
    __shared__ __align__(16) float kx[C][ROW], qx[MODE == LIN_LOCAL ? 1 : C][ROW], vx[C][VROW];
    __shared__ f32x4 px[3][MODE == LIN_LOCAL ? 1 : 64];               // weighted scores (0, 0), (1, 0), (1, 1)
    __shared__ __align__(16) float rw[C], ps[C + 16];
    const float *const K = (const float *)a.k, *const Q = (const float *)a.q, *const V = (const float *)a.v;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n16 = lane & 15, quad = lane >> 4;
    const int BH = a.B * a.H;
    const int bh = blockIdx.x % BH, rest = blockIdx.x / BH, cb = rest % col_blocks, seg = rest / col_blocks;
    const int b = bh / a.H, h = bh - b * a.H;
    const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const int lo = seg * seg_len, hi = min(len, lo + seg_len);
    if (MODE != LIN_WHOLE && lo >= hi) return;
    const int col0 = cb * CB + wave * 16 * CT;
    const float g = a.decay[h];
    for (int i = threadIdx.x; i < C + 16; i += 256) {
        const float p = power(g, i - 15 < 0 ? 0 : i - 15);
        ps[i] = i < 15 ? 0.f : a.scale * p;
        if (i >= 15 && i < 15 + C) rw[C - 1 - (i - 15)] = p;
    }
    f32x4 M[RT][CT];
    const size_t in_state = (size_t)bh * DK * a.dv + (size_t)(4 * quad) * a.dv + col0 + n16;
    const float *from = MODE == LIN_WHOLE ? a.state_in : a.workspace + (size_t)seg * BH * DK * a.dv;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                M[rt][ct][r] = MODE != LIN_LOCAL && from && col0 + 16 * ct < a.dv
                                   ? from[in_state + (size_t)(16 * rt + r) * a.dv + 16 * ct]
                                   : 0.f;

    // tokens fill the last rows of a chunk, as above
    f32x4 kr[KP], qr[MODE == LIN_LOCAL ? 1 : KP], vr[VP];
    const size_t kstep = (size_t)BH * DK, vstep = (size_t)BH * a.dv;
    auto fetch = [&](int r0) {
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            const int u = threadIdx.x + 256 * i, row = u / (DK / 4), at = u % (DK / 4) * 4;
            const size_t from = (size_t)max(r0 + row, lo) * kstep + (size_t)bh * DK + at;
            kr[i] = *(const f32x4 *)(K + from);
            if constexpr (MODE != LIN_LOCAL) qr[i] = *(const f32x4 *)(Q + from);
        }
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            const int u = threadIdx.x + 256 * i, row = u / (CB / 4), at = cb * CB + u % (CB / 4) * 4;
            vr[i] = *(const f32x4 *)(V + (size_t)max(r0 + row, lo) * vstep + (size_t)bh * a.dv + min(at, a.dv - 4));
        }
    };
    auto put = [&](int skip) {
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            const int u = threadIdx.x + 256 * i, row = u / (DK / 4), at = u % (DK / 4) * 4;
            *(f32x4 *)&kx[row][at] = row < skip ? zero : kr[i];
            if constexpr (MODE != LIN_LOCAL) *(f32x4 *)&qx[row][at] = row < skip ? zero : qr[i];
        }
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            const int u = threadIdx.x + 256 * i, row = u / (CB / 4);
            *(f32x4 *)&vx[row][u % (CB / 4) * 4] = row < skip ? zero : vr[i];
        }
    };
    if (lo < hi) {
        const int skip = max(C - (hi - lo), 0);
        fetch(lo - skip);
        put(skip);
    }
    local_barrier();
    for (int c0 = lo; c0 < hi; c0 += C) {
        const int cl = min(C, hi - c0), skip = C - cl, r0 = c0 - skip;
        const bool more = c0 + C < hi;
        const int skip2 = max(C - (hi - c0 - C), 0);
        if (more) fetch(c0 + C - skip2);
        f32x4 o[2][CT];
        if constexpr (MODE != LIN_LOCAL) {
            if (wave < 3) {   // tile (i, j) of the weighted scores, transposed
                const int i = wave > 0, j = wave > 1;
                f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const f32x4 kf = *(const f32x4 *)&kx[16 * j + n16][16 * rt + 4 * quad];
                    const f32x4 qf = *(const f32x4 *)&qx[16 * i + n16][16 * rt + 4 * quad];
#pragma unroll
                    for (int r = 0; r < 4; ++r) s = mfma_f32_k4(kf[r], qf[r], s);
                }
                const float *w = ps + 15 + 16 * (i - j) + n16 - 4 * quad;
#pragma unroll
                for (int r = 0; r < 4; ++r) s[r] *= w[-r];
                px[wave][lane] = s;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) o[i][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                f32x4 qf[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) qf[i] = *(const f32x4 *)&qx[16 * i + n16][16 * rt + 4 * quad];
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) o[i][ct] = mfma_f32_k4(M[rt][ct][r], qf[i][r], o[i][ct]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float w = ps[max(16 + 16 * i + n16 - skip, 0)];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) o[i][ct] *= w;
            }
            local_barrier();   // the scores of all waves are there
        }
        const float gc = cl == C ? rw[0] * g : rw[C - 1 - cl];
        if (more || MODE != LIN_OUTPUTS) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) M[rt][ct] *= gc;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            f32x4 p[2];   // of query tiles 0 and 1; keys 16..31 reach only the second
            if constexpr (MODE != LIN_LOCAL) p[0] = px[0][lane], p[1] = px[1 + j][lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * j + 4 * quad + r;
                float v[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) v[ct] = vx[t][wave * 16 * CT + 16 * ct + n16];
                if constexpr (MODE != LIN_LOCAL) {
#pragma unroll
                    for (int i = j; i < 2; ++i)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) o[i][ct] = mfma_f32_k4(v[ct], p[i][r], o[i][ct]);
                }
                if (more || MODE != LIN_OUTPUTS) {
                    const float w = rw[t];
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const float kk = kx[t][16 * rt + n16];
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) M[rt][ct] = mfma_f32_k4(kk, v[ct] * w, M[rt][ct]);
                    }
                }
            }
        }
        if constexpr (MODE != LIN_LOCAL) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (16 * i + n16 < skip) continue;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    if (col0 + 16 * ct < a.dv)
                        *(f32x4 *)(a.out + (size_t)(r0 + 16 * i + n16) * vstep + (size_t)bh * a.dv + col0 + 16 * ct + 4 * quad) = o[i][ct];
            }
        }
        if (more) {
            local_barrier();
            put(skip2);
            local_barrier();
        }
    }
    if constexpr (MODE != LIN_OUTPUTS) {
        float *to = MODE == LIN_WHOLE ? a.state_out : a.workspace + (size_t)seg * BH * DK * a.dv;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (col0 + 16 * ct < a.dv) to[in_state + (size_t)(16 * rt + r) * a.dv + 16 * ct] = M[rt][ct][r];
    }
}

// The states before each segment from those that the segments leave alone,
// in place in the workspace, and the state behind the last token
__global__ void __launch_bounds__(256) linear_prefix_kernel(LinearArgs a, int segs, int seg_len, int blocks) {
    const int bh = blockIdx.x / blocks, b = bh / a.H, h = bh - b * a.H;
    const size_t i = ((size_t)(blockIdx.x - bh * blocks) * 256 + threadIdx.x) * 4, size = (size_t)a.dk * a.dv;
    if (i >= size) return;
    const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const size_t step = (size_t)a.B * a.H * size;
    float *w = a.workspace + bh * size + i;
    f32x4 M = a.state_in ? *(const f32x4 *)(a.state_in + bh * size + i) : f32x4{0.f, 0.f, 0.f, 0.f};
    const float whole = power(a.decay[h], seg_len);
    const int used = (len + seg_len - 1) / seg_len;
    constexpr int N = 8;   // segments in flight
    for (int s0 = 0; s0 < used; s0 += N) {
        f32x4 x[N];
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = *(const f32x4 *)(w + (size_t)min(s0 + j, used - 1) * step);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int s = s0 + j;
            if (s >= used) break;
            *(f32x4 *)(w + (size_t)s * step) = M;
            const int n = min(len - s * seg_len, seg_len);
            M = M * (n == seg_len ? whole : power(a.decay[h], n)) + x[j];
        }
    }
    *(f32x4 *)(a.state_out + bh * size + i) = M;
}

// How a prompt is cut: segments of whole chunks where (sequence, head, column
// block) alone would leave units idle
struct LinearPlan {
    bool chunked;
    int ct, col_blocks, segs, seg_len;
};
LinearPlan linear_plan(int B, int H, int dk, int dv, int T, int bf16) {
    // (the bf16 kernel's offsets within a chunk have 32 bits)
    LinearPlan p{T > 16 && (double)B * H * std::max(dk, dv) * 64 < 4294967296.0, dv <= 64 ? 1 : 2, 1, 1, T};
    if (!p.chunked) return p;
    const long long states = (long long)B * H, wide = states * ((dv + 127) / 128), chunks = (T + LC - 1) / LC;
    // a segment reads K and V twice and moves 8 d_k d_v bytes of states, in three launches
    // instead of one: at least two chunks of it and four of them, and only until two
    // workgroups a unit are there, or three where the states are half as large
    // (16 states of 16384 tokens, d_k = 128: 146 us with 512 workgroups, 172 us with 768
    // and 165 us with 256 when chosen; 84 states of up to 1999 tokens, d_k = 64: 64 us with
    // 512, 55 us with 768; 16 states of 1024 tokens: 25 us with two chunks, 30 us with four;
    // 128 states of 256 tokens: 27 us in one segment, 37 us in two)
    auto segments = [&](long long groups) {
        const long long want = groups >= 256 ? 1 : (dk == 64 ? 768 : 512) / groups;
        return chunks < 8 ? 1 : std::min(want, chunks / 2);
    };
    // half the columns a workgroup where units would idle otherwise, or where that fills
    // them in place of a few segments (128 states of 256 tokens: 20 us against 27; of
    // 1024: 60 against 80; d_k = 64, 225 states of 3316 tokens: 198 us against 285 in three
    // segments, 176 of 1024 58 against 73 in four, but 176 of up to 4096 207 against 180).
    // float32: wherever units are not all busy, as its chunks are bound by a wave's
    // products (128 states of 128 x 128: 2048 tokens 293 us against 323; 1024
    // states of 256 tokens 252 against 220, so not there)
    if (wide < 256 && (!bf16 || (wide >= 128 && segments(wide) <= (chunks < 32 ? 4 : 3)) || wide * segments(wide) < 256)) p.ct = 1;
    p.col_blocks = (dv + 64 * p.ct - 1) / (64 * p.ct);
    const long long segs = segments(states * p.col_blocks);
    p.seg_len = (int)((chunks + segs - 1) / segs) * LC;
    p.segs = (T + p.seg_len - 1) / p.seg_len;
    return p;
}

template <int DK, int CT, int MODE>
void launch_chunk(const LinearArgs &a, const LinearPlan &p, int bf16, hipStream_t s) {
    const dim3 grid((unsigned)((long long)a.B * a.H * p.col_blocks * p.segs));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, p.col_blocks, p.segs, p.seg_len);
    };
    bf16 ? go(linear_chunk_kernel<DK, CT, MODE>) : go(linear_chunk_f32_kernel<DK, CT, MODE>);
}

template <int DK, int CT>
void launch_chunks(const LinearArgs &a, const LinearPlan &p, int bf16, hipStream_t s) {
    if (p.segs == 1) return launch_chunk<DK, CT, LIN_WHOLE>(a, p, bf16, s);
    const int blocks = (a.dk * a.dv / 4 + 255) / 256;
    launch_chunk<DK, CT, LIN_LOCAL>(a, p, bf16, s);
    hipLaunchKernelGGL(linear_prefix_kernel, dim3((unsigned)((long long)a.B * a.H * blocks)), dim3(256), 0, s, a, p.segs,
                       p.seg_len, blocks);
    launch_chunk<DK, CT, LIN_OUTPUTS>(a, p, bf16, s);
}

}  // namespace

uint64_t linear_attn_workspace(int B, int H, int dk, int dv, int T, int bf16) {
    const LinearPlan p = linear_plan(B, H, dk, dv, T, bf16);
    return p.segs == 1 ? 0 : (uint64_t)p.segs * B * H * dk * dv * 4;
}

hipError_t launch_linear_attn(const LinearArgs &a, int bf16, hipStream_t s) {
    const LinearPlan p = linear_plan(a.B, a.H, a.dk, a.dv, a.T, bf16);
    if (p.chunked) {
        if (a.dk == 128)
            p.ct == 1 ? launch_chunks<128, 1>(a, p, bf16, s) : launch_chunks<128, 2>(a, p, bf16, s);
        else
            p.ct == 1 ? launch_chunks<64, 1>(a, p, bf16, s) : launch_chunks<64, 2>(a, p, bf16, s);
        return hipGetLastError();
    }
    if (bf16) return a.dk == 128 ? launch_step<uint16_t, 128>(a, s) : launch_step<uint16_t, 64>(a, s);
    return a.dk == 128 ? launch_step<float, 128>(a, s) : launch_step<float, 64>(a, s);
}

}  // namespace pace
