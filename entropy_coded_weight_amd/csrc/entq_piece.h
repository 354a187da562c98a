// entq_piece.h -- rows of activations in pieces of 16 bytes, and sums over a
// workgroup, as the norms and the distillation loss use them.
#pragma once

#include "entq_int8.h"

namespace entq {

// Values of a 16-byte piece.
template <int TYPE>
constexpr int kPer = TYPE == ENTQ_F32 ? 4 : 8;

typedef v4i __attribute__((aligned(1))) any_v4i;

// Whether piece p of a row of n values is whole.
template <int TYPE>
__device__ __forceinline__ bool whole_piece(uint32_t p, uint32_t n) {
    return (p + 1) * kPer<TYPE> <= n;
}
// A whole piece at any address. (A row has fewer than 2^32 bytes: offsets of 32
// bits beside a base that is the same for the wave take half the address
// registers.)
__device__ __forceinline__ v4i load_whole(const void *row, uint32_t p) {
    return ((const any16 *)((const uint8_t *)row + p * 16))->v;
}
__device__ __forceinline__ void store_whole(void *row, uint32_t p, v4i v) {
    ((any16 *)((uint8_t *)row + p * 16))->v = v;
}
// A row's last piece, which it does not fill, or one behind it: zeros there.
template <int TYPE>
__device__ __forceinline__ v4i load_rest(const void *row, uint32_t p, uint32_t n) {
    const uint32_t c = p * kPer<TYPE>;
    v4i v = {0, 0, 0, 0};
    if (c >= n) return v;
#pragma unroll
    for (int i = 0; i < kPer<TYPE> - 1; ++i) {
        if (c + i >= n) continue;
        if (TYPE == ENTQ_F32)
            v[i] = ((const int *)row)[c + i];
        else
            v[i / 2] |= (int)((uint32_t)((const uint16_t *)row)[c + i] << (16 * (i % 2)));
    }
    return v;
}
template <int TYPE>
__device__ __forceinline__ void store_rest(void *row, uint32_t p, uint32_t n, v4i v) {
    const uint32_t c = p * kPer<TYPE>;
#pragma unroll
    for (int i = 0; i < kPer<TYPE> - 1; ++i) {
        if (c + i >= n) continue;
        if (TYPE == ENTQ_F32)
            ((int *)row)[c + i] = v[i];
        else
            ((uint16_t *)row)[c + i] = (uint16_t)((uint32_t)v[i / 2] >> (16 * (i % 2)));
    }
}
template <int TYPE>
__device__ __forceinline__ v4i load_piece(const void *row, uint32_t p, uint32_t n) {
    return whole_piece<TYPE>(p, n) ? load_whole(row, p) : load_rest<TYPE>(row, p, n);
}
template <int TYPE>
__device__ __forceinline__ void store_piece(void *row, uint32_t p, uint32_t n, v4i v) {
    if (whole_piece<TYPE>(p, n))
        store_whole(row, p, v);
    else
        store_rest<TYPE>(row, p, n, v);
}

// The values rounded to the type, as a piece.
template <int TYPE>
__device__ __forceinline__ v4i pack(const float (&f)[kPer<TYPE>]) {
    v4i v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == ENTQ_F32)
            v[i] = __float_as_int(f[i]);
        else
            v[i] = (int)(bits16(f[2 * i], TYPE == ENTQ_F16) | (uint32_t)bits16(f[2 * i + 1], TYPE == ENTQ_F16) << 16);
    }
    return v;
}

// Values c.. of a vector of n fp32 values for piece p, zeros past its end.
template <int TYPE>
__device__ __forceinline__ void load_floats(const float *w, uint32_t p, uint32_t n, float (&f)[kPer<TYPE>]) {
    const uint32_t c = p * kPer<TYPE>;
    if (c + kPer<TYPE> <= n) {
#pragma unroll
        for (int h = 0; h < kPer<TYPE> / 4; ++h) {
            const v4i v = ((const any16 *)(w + c + 4 * h))->v;
#pragma unroll
            for (int i = 0; i < 4; ++i) f[4 * h + i] = __int_as_float(v[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kPer<TYPE>; ++i) f[i] = c + i < n ? w[c + i] : 0.0f;
}

// A lane's value plus that of the lane that CTRL names in its row of 16.
template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// The sum of each row of 16 lanes, in all of them: lanes 1 and 2 away, then the
// mirrored half row and row.
__device__ __forceinline__ double row16_sum(double v) {
    v = add_dpp<0xB1>(v);
    v = add_dpp<0x4E>(v);
    v = add_dpp<0x141>(v);
    return add_dpp<0x140>(v);
}

// The sum of a wave's lanes, in all of them.
__device__ __forceinline__ double wave_sum(double v) {
    v = row16_sum(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// The greatest of a wave's values, all lanes active: as row16_sum, then the
// rows' own.
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t greatest(uint32_t v) {
    v = max_dpp<0x140>(max_dpp<0x141>(max_dpp<0x4E>(max_dpp<0xB1>(v))));
    const uint32_t r[4] = {(uint32_t)__builtin_amdgcn_readlane(v, 0), (uint32_t)__builtin_amdgcn_readlane(v, 16),
                           (uint32_t)__builtin_amdgcn_readlane(v, 32), (uint32_t)__builtin_amdgcn_readlane(v, 48)};
    return max(max(r[0], r[1]), max(r[2], r[3]));
}

// 1 / sqrt(v) of a positive 64-bit value, rounded to fp32 (0 for an infinity):
// the hardware's estimate and one step of Newton's method.
__device__ __forceinline__ float rsqrt64(double v) {
    const double r = __builtin_amdgcn_rsq(v);
    return (float)(v < __builtin_inf() ? r * (1.5 - 0.5 * v * r * r) : r);
}

}  // namespace entq
