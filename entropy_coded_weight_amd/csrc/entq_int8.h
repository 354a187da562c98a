// entq_int8.h -- what the kernels of the int8 products share: argument
// blocks, conversions, activations and the epilogue that turns a tile's
// integer sums into results or gradients.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "entq.h"

namespace entq {

// What a kernel computes from acc_w[m][n] = sum_k x[m][k] w[n][k]:
//   kFwd       y = acc sx sw                       (one weight)
//   kGated     y = act(g) u                        (two weights)
//   kBwd       sums over m of dy acc sx, and dy sw in bf16 (F16's: narrow_row)
//   kGatedBwd  the same for dg and du              (two weights; in fp32 for F16)
enum Int8Mode { kFwd = 0, kGated = 1, kBwd = 2, kGatedBwd = 3 };

struct Int8Args {
    const int8_t *x;        // [M][ldx]; activations themselves where x_type is not ENTQ_I8
    const int8_t *w[2];     // [N][ldw]
    const float *sx;        // [M]
    const float *sw[2];     // [N]
    uint64_t ldx, ldw[2];
    uint32_t M, N, K;
    int x_type;             // only the few-token kernel takes other than ENTQ_I8
    int act;
    void *y;                // forward: the result; backward: the incoming gradient
    int type;               // its entq_eltype
    uint64_t ldy;
    uint16_t *d[2];         // backward: 16-bit scaled gradients [M][ldd], or null; F16's are narrow_row's
    float *wide[2];         // gated backward of F16: the scaled gradients [M][ldd] before, or null
    float *back;            // backward of F16: [M], what undoes a row's power of two
    uint64_t ldd;           // a multiple of 64; columns N..ldd-1 are written as 0
    float *part[2];         // backward: partial column sums [token blocks][N], or null
    uint32_t splits;        // of K; above 1, integer sums go to
    int32_t *sums;          // [splits][weights][M][N rounded up to 4]
    bool narrows;           // kBwd: workgroups after the tiles run narrow_row
};

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// An fp32 value rounded to 16 bits. The value is an fp32 register first: a
// product's rounding to F16 would else be fused into a mixed-precision
// instruction in some kernels and not in others, with other last bits.
__device__ __forceinline__ uint16_t bits16(float v, bool f16) {
    asm("" : "+v"(v));
    return f16 ? __builtin_bit_cast(uint16_t, (_Float16)v) : __builtin_bit_cast(uint16_t, (__bf16)v);
}

__device__ __forceinline__ float from16(uint16_t b, bool f16) {
    return f16 ? (float)__builtin_bit_cast(_Float16, b) : __builtin_bit_cast(float, (uint32_t)b << 16);
}

// 16 and 8 bytes at any address: the hardware takes unaligned vector accesses.
struct __attribute__((packed)) any16 { v4i v; };
struct __attribute__((packed)) any8 { v2i v; };
struct __attribute__((packed)) any4 { int v; };

// Codes k..k+15 of a row of K codes at any address, zeros past its end.
__device__ __forceinline__ v4i load16_any(const int8_t *row, uint32_t k, uint32_t K) {
    if (k + 16 <= K) return ((const any16 *)(row + k))->v;
    if (k >= K) return v4i{0, 0, 0, 0};
    if (K >= 16) {  // the row's last 16 codes, moved down
        const v4i v = ((const any16 *)(row + K - 16))->v;
        uint64_t lo = (uint32_t)v[0] | (uint64_t)(uint32_t)v[1] << 32;
        uint64_t hi = (uint32_t)v[2] | (uint64_t)(uint32_t)v[3] << 32;
        const uint32_t shift = 8 * (16 - (K - k));  // 8 .. 120
        if (shift >= 64) {
            lo = hi >> (shift - 64);
            hi = 0;
        } else {
            lo = lo >> shift | hi << (64 - shift);
            hi >>= shift;
        }
        return v4i{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
    }
    uint32_t b[4] = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t i = 0; i < 15; ++i)
        if (k + i < K) b[i / 4] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i % 4));
    return v4i{(int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// Row quantisation (entq_quantize_rows): element i of a 16-byte piece of
// activations, and from the bits of a row's largest magnitude (as integers
// infinities and NaNs come out on top) its scale and codes.
template <int TYPE>
__device__ __forceinline__ float act_of(v4i piece, int i) {
    if (TYPE == ENTQ_F32) return __int_as_float(piece[i]);
    return from16((uint16_t)((uint32_t)piece[i / 2] >> (16 * (i % 2))), TYPE == ENTQ_F16);
}

constexpr float kMinScale = 0x1p-100f;  // its inverse is finite

struct Quantizer {
    float scale, inv;
    bool finite;
    __device__ explicit Quantizer(uint32_t big) {
        finite = big < 0x7F800000u;
        const float s = fmaxf(__uint_as_float(big) * (float)(1.0 / 127), kMinScale);
        inv = 1.0f / s;
        scale = finite ? s : __uint_as_float(0x7FC00000u);
    }
    __device__ uint32_t code(float v) const {
        return finite ? (uint32_t)(int)fminf(fmaxf(rintf(v * inv), -127.0f), 127.0f) & 0xFFu : 0u;
    }
    template <int TYPE>
    __device__ uint32_t code4(v4i piece, int first) const {
        return code(act_of<TYPE>(piece, first)) | code(act_of<TYPE>(piece, first + 1)) << 8 |
               code(act_of<TYPE>(piece, first + 2)) << 16 | code(act_of<TYPE>(piece, first + 3)) << 24;
    }
};

template <int TYPE>
__device__ __forceinline__ float load_act(const void *x, uint64_t at) {
    if (TYPE == ENTQ_F32) return ((const float *)x)[at];
    return from16(((const uint16_t *)x)[at], TYPE == ENTQ_F16);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int o = 32; o; o /= 2) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}

// act(v) of 4 values and, with GRAD, act'(v). exp is the hardware's 2^x after
// a product with log2 e (relative error about 1e-7 times the exponent, which
// is small where the result is not), 1 / x the hardware's (1 ulp). The choice
// of activation is made once for the 4 values, whose chains then overlap.
template <bool GRAD>
__device__ __forceinline__ void activate4(int act, const float (&x)[4], float (&r)[4], float (&grad)[4]) {
    if (act == ENTQ_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = x[i], p = __builtin_amdgcn_rcpf(1.0f + __expf(-v));
            r[i] = v * p;
            if (GRAD) grad[i] = p * (1.0f + v * (1.0f - p));
        }
    } else if (act == ENTQ_ACT_GELU) {
        // The normal distribution's tail Q(|v|) = exp(-v^2 / 2) t P(t), t = 1 / (1
        // + c |v|), with c and the polynomial P fitted here for the least
        // relative error over |v| <= 15 (1.0e-7): far below 0, where gelu is v
        // Q, an absolute error would be all there is. The gradient needs the
        // exponential anyway.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = x[i], e = __expf(-0.5f * v * v);
            const float t = __builtin_amdgcn_rcpf(1.0f + 0.30567637f * fabsf(v));
            float q = 0.036590103f;
            q = q * t - 0.15143743f;
            q = q * t + 0.18141808f;
            q = q * t - 0.034611415f;
            q = q * t + 0.11938832f;
            q = q * t + 0.10406668f;
            q = q * t + 0.12267242f;
            q = (q * t + 0.12191331f) * t * e;
            const float p = v >= 0.0f ? 1.0f - q : q;
            r[i] = v * p;
            if (GRAD) grad[i] = p + v * 0.39894228040143268f * e;
        }
    } else if (act == ENTQ_ACT_GELU_TANH) {
        // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = x[i], z2 = 1.5957691216057308f * (v + 0.044715f * v * v * v);
            const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-z2));
            r[i] = v * p;
            // (far out p (1 - p) is 0, where v^2 may be beyond fp32)
            const float w = __builtin_amdgcn_fmed3f(v, -64.0f, 64.0f);
            if (GRAD) grad[i] = p + w * p * (1.0f - p) * 1.5957691216057308f * (1.0f + 0.134145f * w * w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // a NaN stays one
            r[i] = x[i] > 0.0f ? x[i] : x[i] != x[i] ? x[i] : 0.0f;
            if (GRAD) grad[i] = x[i] > 0.0f ? 1.0f : 0.0f;
        }
    }
}

// The scales of channels n..n+3, 0 beyond N.
template <int MODE>
__device__ __forceinline__ void load_scales(const Int8Args &a, uint32_t n, float (&scale)[2][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = n + i < a.N;
        scale[0][i] = in ? a.sw[0][n + i] : 0.0f;
        scale[1][i] = in && (MODE == kGated || MODE == kGatedBwd) ? a.sw[1][n + i] : 0.0f;
    }
}

// The incoming gradient (4 values of 16 bits) at token m, channels n..n+3.
__device__ __forceinline__ uint2 load_grad4(const Int8Args &a, uint32_t m, uint32_t n) {
    if (m >= a.M || n >= a.N) return make_uint2(0, 0);
    const uint16_t *y = (const uint16_t *)a.y + (uint64_t)m * a.ldy + n;
    if (n + 4 <= a.N) {
        const v2i v = ((const any8 *)y)->v;
        return make_uint2((uint32_t)v[0], (uint32_t)v[1]);
    }
    uint32_t b[4] = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
        if (n + i < a.N) b[i] = y[i];
    return make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
}

// The results for token m (of scale sx) and the 4 channels n..n+3 (n a multiple of 4), or
// the gradients, whose contributions to the channel sums are added to sg, su.
// Channels of N and beyond are not stored; in a backward pass a token of M
// and beyond adds nothing.
template <int MODE>
__device__ __forceinline__ void epilogue4(const Int8Args &a, float sx, const float (&scale)[2][4], uint32_t m,
                                          uint32_t n, v4i ag, v4i au, uint2 dy4, float (&sg)[4],
                                          float (&su)[4]) {
    constexpr bool kTwo = MODE == kGated || MODE == kGatedBwd;
    constexpr bool kBack = MODE == kBwd || MODE == kGatedBwd;
    if (m >= a.M || n >= (kBack ? (uint32_t)a.ldd : a.N)) return;
    if constexpr (!kBack) {
        const bool whole = n + 4 <= a.N;
        const uint64_t at = (uint64_t)m * a.ldy + n;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ((float)ag[i] * sx) * scale[0][i];
        if (kTwo) {
            float r[4], none[4];
            activate4<false>(a.act, v, r, none);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = r[i] * (((float)au[i] * sx) * scale[1][i]);
        }
        if (a.type == ENTQ_F32) {
            float *y = (float *)a.y + at;
            if (whole) {
                ((any16 *)y)->v = __builtin_bit_cast(v4i, v4f{v[0], v[1], v[2], v[3]});
            } else {
                for (int i = 0; i < 4; ++i)
                    if (n + i < a.N) y[i] = v[i];
            }
        } else {
            const bool f16 = a.type == ENTQ_F16;
            uint16_t *y = (uint16_t *)a.y + at;
            uint16_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = bits16(v[i], f16);
            if (whole) {
                ((any8 *)y)->v = v2i{(int)(b[0] | (uint32_t)b[1] << 16), (int)(b[2] | (uint32_t)b[3] << 16)};
            } else {
                for (int i = 0; i < 4; ++i)
                    if (n + i < a.N) y[i] = b[i];
            }
        }
    } else {
        const bool f16 = a.type == ENTQ_F16;
        float d[2][4];
        float g0[4], u0[4], g[4], act[4], grad[4];  // g0, u0: before the channel's scale
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g0[i] = (float)ag[i] * sx;
            u0[i] = (float)au[i] * sx;
            g[i] = g0[i] * scale[0][i];
        }
        if (kTwo) activate4<true>(a.act, g, act, grad);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float dy = from16((uint16_t)((i < 2 ? dy4.x : dy4.y) >> (16 * (i % 2))), f16);
            // (beyond N: dy and the scales are 0, so d is 0, or NaN in a row
            // whose dX is NaN anyway; the sums are not used)
            const float dg = kTwo ? dy * (u0[i] * scale[1][i]) * grad[i] : dy;
            sg[i] += dg * g0[i];
            d[0][i] = dg * scale[0][i];
            if (kTwo) {
                const float du = dy * act[i];
                su[i] += du * u0[i];
                d[1][i] = du * scale[1][i];
            }
        }
        const uint64_t to = (uint64_t)m * a.ldd + n;
        if (kTwo && a.wide[0]) {
#pragma unroll
            for (int t = 0; t < 2; ++t) *(v4f *)(a.wide[t] + to) = v4f{d[t][0], d[t][1], d[t][2], d[t][3]};
        } else if (a.d[0] && !f16) {
#pragma unroll
            for (int t = 0; t < (kTwo ? 2 : 1); ++t) {
                uint16_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = bits16(d[t][i], false);
                *(uint2 *)(a.d[t] + to) = make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
            }
        }
    }
}

// Channel sums out of the token blocks' partial sums, added in block order.
struct SumArgs {
    const float *part[2];
    float *out[2];          // or null
    uint32_t rows, n;
};
constexpr uint32_t kSumThreads = 256;
inline uint32_t sum_blocks(const SumArgs &a) { return a.rows ? 2 * ((a.n + kSumThreads - 1) / kSumThreads) : 0; }
__device__ __forceinline__ void sum_parts_block(const SumArgs &a, uint32_t block) {
    const uint32_t half = (a.n + kSumThreads - 1) / kSumThreads, t = block >= half;
    const uint32_t i = (block - t * half) * kSumThreads + threadIdx.x;
    const float *p = t ? a.part[1] : a.part[0];
    float *out = t ? a.out[1] : a.out[0];
    if (i >= a.n || !out) return;
    float s = 0.0f;
#pragma unroll 8
    for (uint32_t b = 0; b < a.rows; ++b) s += p[(uint64_t)b * a.n + i];
    out[i] = s;
}

// dX = sum over the weights t of d[t] . W_t, a product along the channels.
struct GradArgs {
    const uint16_t *d[2];   // [M][ldd], zero beyond column N
    const int8_t *w[2];     // [N][ldw]
    uint64_t ldd, ldw[2];
    uint32_t M, N, K;       // N channels; K: the weights' columns, a multiple of 16
    uint32_t cols;          // of the result, K or up to 15 fewer
    uint32_t splits;        // of the sum; above 1, partial sums go to parts
    float *parts;           // [splits][M][K]
    int n_w;                // 1 or 2
    bool f16;
    void *dx;               // [M][lddx], bf16 or f16
    uint64_t lddx;
    const float *back;      // F16: [M], what row m of the result is multiplied with
    SumArgs sums;           // channel sums to finish in the same launch (rows 0: none)
};

// The choice between tile sizes and splits of the sum is made by what each
// would take, in us: `step` for one step of a workgroup's sum with one and
// with two workgroups on a CU (256-token tiles fill one), `tile` for a tile's
// end, the weights' bytes at `bytes_us`, and for a split sum a second launch
// that adds partial results. The constants are fitted to times measured on
// MI355X (1 .. 2,048 tokens, sides 512 .. 32,000) with every tile and 1 .. 24
// splits, as graphs of launches; `second` has 2 us more for what a second
// launch costs outside a graph. Over 284 shapes measured afterwards the choice
// is on average 1.2 % slower than the best variant of each shape, more than
// 10 % for 9 of them, 30 % at most.
struct TileCost {
    uint32_t tokens, width; // of a tile; width: weight rows, or columns of dX
    float step[2], tile;
};
struct SplitCost {
    float launch, bytes_us, second, per_split, per_value;
};
inline float tile_cost(const TileCost &t, const SplitCost &c, uint32_t tiles, uint32_t steps, uint32_t splits,
                       uint64_t weight_bytes, uint64_t results) {
    const uint32_t slots = t.tokens == 256 ? 256 : 512, groups = tiles * splits;
    const uint32_t full = groups / slots, rest = groups % slots;
    const float work = (float)((steps + splits - 1) / splits) *
                           (full * t.step[1] + (rest == 0 ? 0.0f : t.step[rest > 256])) +
                       t.tile * (full + (rest > 0));
    const float memory = weight_bytes / c.bytes_us;
    float us = c.launch + (work > memory ? work : memory);
    if (splits > 1) us += c.second + splits * (c.per_split + c.per_value * results);
    return us;
}
// The cheapest kind of tile and split for M tokens and a width.
struct TileChoice {
    int kind;
    uint32_t splits;
    float us;
};
template <int KINDS>
TileChoice cheapest_tile(const TileCost (&kinds)[KINDS], const SplitCost &c, uint32_t M, uint64_t width,
                         uint32_t steps, uint64_t weight_bytes, uint64_t results) {
    TileChoice best{-1, 1, 0.0f};
    for (int kind = 0; kind < KINDS; ++kind) {
        const TileCost &t = kinds[kind];
        const uint64_t n = (uint64_t)((M + t.tokens - 1) / t.tokens) * ((width + t.width - 1) / t.width);
        for (uint32_t s : {1u, 2u, 3u, 4u, 6u, 8u, 12u, 16u, 24u}) {
            if (s > 1 && (s > steps || n * s > 1100)) break;
            const float us = tile_cost(t, c, (uint32_t)(n > 0x7FFFFFFF ? 0x7FFFFFFF : n), steps, s, weight_bytes,
                                       results);
            if (best.kind < 0 || us < best.us) best = {kind, s, us};
        }
    }
    return best;
}

// How a product runs.
struct Int8Plan {
    bool few;               // the few-token kernel; else tiles:
    bool quantizes;         // the few-token kernel quantises the activations itself
    uint32_t splits;        // of K; above 1 the sums pass through memory
    int kind;               // of tile
    uint32_t part_rows;     // rows of Int8Args::part
};
Int8Plan int8_plan(Int8Mode mode, int x_type, uint32_t M, uint32_t N, uint32_t K);

// Row m of the scaled gradients in F16 (a.d) and what undoes its power of two
// (a.back[m]): dy sw, or with TWO the rows of a.wide. fp32 holds these values
// and F16 does not (its normal range spans 2^30): the power of two brings the
// largest of the row, over both weights, into [2^14, 2^15), so none overflows,
// those within 2^-28 of the largest keep 11 bits and those below are rounded
// to steps of 2^-38 of it. A row with an infinity or a NaN takes the power
// that fits every finite fp32 value. One workgroup of up to 16 waves, which
// gives 64 bytes of LDS; a thread keeps its first HELD groups of 4 channels in
// registers and reads the others twice.
template <bool TWO, int HELD>
__device__ __forceinline__ void narrow_row(const Int8Args &a, uint32_t m, uint32_t *top) {
    const uint32_t per = (uint32_t)(a.ldd / 4), all = TWO ? 2 * per : per;
    auto read = [&](uint32_t q) {
        const uint32_t t = TWO && q >= per, n = 4 * (q - t * per);
        if (TWO) return *(const v4f *)((t ? a.wide[1] : a.wide[0]) + (uint64_t)m * a.ldd + n);
        const uint2 g = load_grad4(a, m, n);
        v4f scale = {0, 0, 0, 0};
        if (n + 4 <= a.N)
            scale = __builtin_bit_cast(v4f, ((const any16 *)(a.sw[0] + n))->v);
        else
            for (uint32_t i = 0; i < 3; ++i)
                if (n + i < a.N) scale[i] = a.sw[0][n + i];
        // (beyond N both are 0)
        return v4f{from16((uint16_t)g.x, true) * scale[0], from16((uint16_t)(g.x >> 16), true) * scale[1],
                   from16((uint16_t)g.y, true) * scale[2], from16((uint16_t)(g.y >> 16), true) * scale[3]};
    };
    uint32_t big = 0;
    auto take = [&](v4f v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) big = max(big, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    };
    v4f held[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const uint32_t q = i * blockDim.x + threadIdx.x;
        held[i] = q < all ? read(q) : v4f{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i) take(held[i]);
    for (uint32_t q = HELD * blockDim.x + threadIdx.x; q < all; q += blockDim.x) take(read(q));
    big = wave_max(big);
    if (threadIdx.x % 64 == 0) top[threadIdx.x / 64] = big;
    __syncthreads();
    for (uint32_t i = 0; i < blockDim.x / 64; ++i) big = max(big, top[i]);
    // (at most 2^126, whose inverse is a normal number)
    const int up = big >= 0x7F800000u ? -113 : big ? 14 - max(-112, (int)(big >> 23) - 127) : 0;
    const float by = __uint_as_float((uint32_t)(127 + up) << 23);
    if (threadIdx.x == 0) a.back[m] = __uint_as_float((uint32_t)(127 - up) << 23);
    auto put = [&](uint32_t q, v4f v) {
        const uint32_t t = TWO && q >= per;
        uint16_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = bits16(v[i] * by, true);
        *(uint2 *)((t ? a.d[1] : a.d[0]) + (uint64_t)m * a.ldd + 4 * (q - t * per)) =
            make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const uint32_t q = i * blockDim.x + threadIdx.x;
        if (q < all) put(q, held[i]);
    }
    for (uint32_t q = HELD * blockDim.x + threadIdx.x; q < all; q += blockDim.x) put(q, read(q));
}

// Whether a launch's threads can be counted in 32 bits, as HIP requires.
inline bool launchable(uint64_t groups, uint32_t threads) { return groups && groups * threads < 1ull << 32; }

// Launchers; each returns an entq_status (ENTQ_EINVAL for more workgroups
// than one launch holds). Rows of x and w must start at
// multiples of 16 bytes, strides below 2^23, K be a multiple of 16.
bool few_quantizes(uint32_t M, uint32_t K);
int launch_int8_few(Int8Mode mode, const Int8Args &a, hipStream_t s);
int launch_int8_product(Int8Mode mode, const Int8Plan &p, const Int8Args &a, hipStream_t s);

struct GradPlan {
    int kind;               // of tile
    uint32_t splits;
};
GradPlan grad_plan(uint32_t M, uint32_t N, uint32_t K, int n_w);
int launch_grad_product(const GradPlan &p, const GradArgs &a, hipStream_t s);

}  // namespace entq
