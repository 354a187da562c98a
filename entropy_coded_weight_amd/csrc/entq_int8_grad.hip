// entq_int8_grad.hip -- dX = d . W for 16-bit gradients d [M][N] and int8
// codes W [N][K]: a product along the weights' rows.
#include "entq_int8.h"

namespace entq {
namespace {

constexpr uint32_t kTile = 64;

template <bool F16>
__global__ __launch_bounds__(256) void grad_product(GradArgs a) {
    __shared__ uint16_t ds[kTile][kTile + 8], wt[kTile][kTile + 8];  // wt: column of W, channel
    const uint32_t t = threadIdx.x, lane = t % 64, wave = t / 64;
    const uint32_t k0 = blockIdx.x * kTile, m0 = blockIdx.y * kTile;
    v4f acc[4] = {};
    for (int w = 0; w < a.n_w; ++w) {
        for (uint32_t n0 = 0; n0 < a.N; n0 += kTile) {
#pragma unroll
            for (uint32_t i = t; i < kTile * kTile / 4; i += 256) {
                const uint32_t r = i / 16, c = i % 16 * 4;
                *(uint2 *)&ds[r][c] = m0 + r < a.M
                                          ? *(const uint2 *)(a.d[w] + (m0 + r) * a.ldd + n0 + c)
                                          : make_uint2(0, 0);
            }
#pragma unroll
            for (uint32_t i = t; i < kTile * kTile; i += 256) {
                const uint32_t r = i / 64, c = i % 64;
                const bool in = n0 + r < a.N && k0 + c < a.K;
                wt[c][r] = bits16(in ? (float)a.w[w][(n0 + r) * a.ldw[w] + k0 + c] : 0.0f, F16);
            }
            __syncthreads();
#pragma unroll
            for (uint32_t s = 0; s < kTile; s += 32) {
                const v4i wf = *(const v4i *)&wt[wave * 16 + lane % 16][s + lane / 16 * 8];
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const v4i df = *(const v4i *)&ds[f * 16 + lane % 16][s + lane / 16 * 8];
                    if (F16)
                        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            __builtin_bit_cast(f16x8, wf), __builtin_bit_cast(f16x8, df), acc[f], 0,
                            0, 0);
                    else
                        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, wf), __builtin_bit_cast(bf16x8, df), acc[f],
                            0, 0, 0);
                }
            }
            __syncthreads();
        }
    }
    const float back = a.norm ? a.norm[1] : 1.0f;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
        const uint32_t m = m0 + f * 16 + lane % 16, k = k0 + wave * 16 + lane / 16 * 4;
        if (m >= a.M) continue;
        uint16_t *to = (uint16_t *)a.dx + m * a.lddx + k;
        for (int i = 0; i < 4; ++i)
            if (k + i < a.K) to[i] = bits16(acc[f][i] * back, F16);
    }
}

}  // namespace

int launch_grad_product(const GradArgs &a, hipStream_t s) {
    const dim3 grid((a.K + kTile - 1) / kTile, (a.M + kTile - 1) / kTile);
    if (a.f16)
        grad_product<true><<<grid, 256, 0, s>>>(a);
    else
        grad_product<false><<<grid, 256, 0, s>>>(a);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

}  // namespace entq
