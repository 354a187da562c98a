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
//   kBwd       sums over m of dy acc sx, and dy sw in 16 bits
//   kGatedBwd  the same for dg and du              (two weights)
enum Int8Mode { kFwd = 0, kGated = 1, kBwd = 2, kGatedBwd = 3 };

struct Int8Args {
    const int8_t *x;        // [M][ldx]
    const int8_t *w[2];     // [N][ldw]
    const float *sx;        // [M]
    const float *sw[2];     // [N]
    uint64_t ldx, ldw[2];
    uint32_t M, N, K;
    int act;
    void *y;                // forward: the result; backward: the incoming gradient
    int type;               // its entq_eltype
    bool vec;               // y's rows start at multiples of 4 elements (address and stride)
    uint64_t ldy;
    uint16_t *d[2];         // backward: 16-bit scaled gradients [M][ldd], or null
    uint64_t ldd;           // a multiple of 64; columns N..ldd-1 are written as 0
    float *part[2];         // backward: partial column sums [token blocks][N], or null
    const float *norm;      // F16 backward: the power of two that multiplies sw, then its inverse
};

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint16_t bits16(float v, bool f16) {
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
    uint32_t b[4] = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t i = 0; i < 15; ++i)
        if (k + i < K) b[i / 4] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i % 4));
    return v4i{(int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// act(v) and, for the backward pass, act'(v). exp is the hardware's 2^x after
// a product with log2 e (relative error about 1e-7 times the exponent, which
// is small where the result is not), 1 / x the hardware's (1 ulp).
__device__ __forceinline__ float act_and_grad(int act, float v, float &grad) {
    if (act == ENTQ_ACT_SILU) {
        const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-v));
        grad = p * (1.0f + v * (1.0f - p));
        return v * p;
    }
    if (act == ENTQ_ACT_GELU) {
        const float p = 0.5f * (1.0f + erff(v * 0.70710678118654752f));
        grad = p + v * 0.39894228040143268f * __expf(-0.5f * v * v);
        return v * p;
    }
    if (act == ENTQ_ACT_GELU_TANH) {
        // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
        const float z2 = 1.5957691216057308f * (v + 0.044715f * v * v * v);
        const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-z2));
        grad = p + v * p * (1.0f - p) * 1.5957691216057308f * (1.0f + 0.134145f * v * v);
        return v * p;
    }
    // a NaN stays one
    grad = v > 0.0f ? 1.0f : 0.0f;
    return v > 0.0f ? v : v != v ? v : 0.0f;
}

__device__ __forceinline__ float act_only(int act, float v) {
    float grad;
    return act_and_grad(act, v, grad);
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

// The results for token m and the 4 channels n..n+3 (n a multiple of 4), or
// the gradients, whose contributions to the channel sums are added to sg, su.
// Channels of N and beyond are not stored; in a backward pass a token of M
// and beyond adds nothing.
template <int MODE>
__device__ __forceinline__ void epilogue4(const Int8Args &a, const float (&scale)[2][4], float norm, uint32_t m,
                                          uint32_t n, v4i ag, v4i au, float (&sg)[4], float (&su)[4]) {
    constexpr bool kTwo = MODE == kGated || MODE == kGatedBwd;
    constexpr bool kBack = MODE == kBwd || MODE == kGatedBwd;
    if (m >= a.M || n >= (kBack ? (uint32_t)a.ldd : a.N)) return;
    const bool whole = n + 4 <= a.N;
    const float sx = a.sx[m];
    const uint64_t at = (uint64_t)m * a.ldy + n;
    if constexpr (!kBack) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = ((float)ag[i] * sx) * scale[0][i];
            if (kTwo) v[i] = act_only(a.act, v[i]) * (((float)au[i] * sx) * scale[1][i]);
        }
        if (a.type == ENTQ_F32) {
            float *y = (float *)a.y + at;
            if (whole && a.vec) {
                *(v4f *)y = v4f{v[0], v[1], v[2], v[3]};
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
            if (whole && a.vec) {
                *(uint2 *)y = make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
            } else {
                for (int i = 0; i < 4; ++i)
                    if (n + i < a.N) y[i] = b[i];
            }
        }
    } else {
        const bool f16 = a.type == ENTQ_F16;
        const uint16_t *y = (const uint16_t *)a.y + at;
        uint16_t b[4] = {0, 0, 0, 0};
        if (whole && a.vec) {
            const uint2 v = *(const uint2 *)y;
            b[0] = (uint16_t)v.x, b[1] = (uint16_t)(v.x >> 16);
            b[2] = (uint16_t)v.y, b[3] = (uint16_t)(v.y >> 16);
        } else {
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N) b[i] = y[i];
        }
        uint16_t d[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float dy = from16(b[i], f16);
            const float g0 = (float)ag[i] * sx;  // before the channel's scale
            const bool in = n + i < a.N;
            if (!kTwo) {
                if (in) sg[i] += dy * g0;
                d[0][i] = in ? bits16(dy * (scale[0][i] * norm), f16) : 0;
            } else {
                const float u0 = (float)au[i] * sx;
                float grad;
                const float act = act_and_grad(a.act, g0 * scale[0][i], grad);
                const float dg = dy * (u0 * scale[1][i]) * grad, du = dy * act;
                if (in) {
                    sg[i] += dg * g0;
                    su[i] += du * u0;
                }
                d[0][i] = in ? bits16(dg * (scale[0][i] * norm), f16) : 0;
                d[1][i] = in ? bits16(du * (scale[1][i] * norm), f16) : 0;
            }
        }
        if (a.d[0]) {
            const uint64_t to = (uint64_t)m * a.ldd + n;
#pragma unroll
            for (int t = 0; t < (kTwo ? 2 : 1); ++t)
                *(uint2 *)(a.d[t] + to) = make_uint2(d[t][0] | (uint32_t)d[t][1] << 16,
                                                     d[t][2] | (uint32_t)d[t][3] << 16);
        }
    }
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
    bool vec;               // dx's rows start at multiples of 4 elements
    const float *norm;      // F16: result times norm[1]; or null
};

// How a product runs.
struct Int8Plan {
    int tile;               // tokens of a tile
    uint32_t part_rows;     // rows of Int8Args::part
};
Int8Plan int8_plan(Int8Mode mode, uint32_t M, uint32_t N, uint32_t K);

// Launchers; each returns an entq_status. Rows of x and w must start at
// multiples of 16 bytes, strides below 2^23, K be a multiple of 16.
int launch_int8_product(Int8Mode mode, const Int8Plan &p, const Int8Args &a, hipStream_t s);

struct GradPlan {
    int tile;
    uint32_t splits;
};
GradPlan grad_plan(uint32_t M, uint32_t N, uint32_t K, int n_w);
int launch_grad_product(const GradPlan &p, const GradArgs &a, hipStream_t s);

}  // namespace entq
