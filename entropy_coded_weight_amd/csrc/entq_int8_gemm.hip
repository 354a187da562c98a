// entq_int8_gemm.hip -- products of int8 activation codes with int8 weight
// codes, with the epilogues of the forward and backward calls.
#include "entq_int8.h"

namespace entq {
namespace {

constexpr uint32_t kTile = 64;  // tokens and channels of a workgroup's tile

// 16 codes of row r, columns k..k+15; zeros outside the matrix.
__device__ __forceinline__ v4i load16(const int8_t *p, uint64_t ld, uint32_t r, uint32_t rows,
                                      uint32_t k, uint32_t K) {
    v4i v = {0, 0, 0, 0};
    if (r >= rows || k >= K) return v;
    const int8_t *q = p + (uint64_t)r * ld + k;
    if (k + 16 <= K && (uintptr_t)q % 16 == 0) return *(const v4i *)q;
    uint32_t b[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (k + i < K) b[i / 4] |= (uint32_t)(uint8_t)q[i] << (8 * (i % 4));
    return v4i{(int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

template <int MODE>
__global__ __launch_bounds__(256) void int8_product(Int8Args a) {
    constexpr int kW = MODE == kGated || MODE == kGatedBwd ? 2 : 1;
    constexpr bool kBack = MODE == kBwd || MODE == kGatedBwd;
    __shared__ v4i xs[kTile][5], ws[kW][kTile][5];
    const uint32_t t = threadIdx.x, lane = t % 64, wave = t / 64;
    const uint32_t n0 = blockIdx.x * kTile, m0 = blockIdx.y * kTile;
    const uint32_t row = t / 4, chunk = t % 4;
    v4i acc[kW][4] = {};
    for (uint32_t k0 = 0; k0 < a.K; k0 += 64) {
        xs[row][chunk] = load16(a.x, a.ldx, m0 + row, a.M, k0 + 16 * chunk, a.K);
#pragma unroll
        for (int w = 0; w < kW; ++w)
            ws[w][row][chunk] = load16(a.w[w], a.ldw[w], n0 + row, a.N, k0 + 16 * chunk, a.K);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            const v4i wf = ws[w][wave * 16 + lane % 16][lane / 16];
#pragma unroll
            for (int f = 0; f < 4; ++f)
                acc[w][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                    wf, xs[f * 16 + lane % 16][lane / 16], acc[w][f], 0, 0, 0);
        }
        __syncthreads();
    }
    const uint32_t n = n0 + wave * 16 + lane / 16 * 4;
    float sg[4] = {}, su[4] = {};
#pragma unroll
    for (int f = 0; f < 4; ++f)
        epilogue4<MODE>(a, m0 + f * 16 + lane % 16, n, acc[0][f], acc[kW - 1][f], sg, su);
    if constexpr (kBack) {
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            if (!a.part[w]) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float s = w ? su[i] : sg[i];
#pragma unroll
                for (int o = 1; o < 16; o *= 2) s += __shfl_xor(s, o);
                if (lane % 16 == 0 && n + i < a.N)
                    a.part[w][(uint64_t)blockIdx.y * a.N + n + i] = s;
            }
        }
    }
}

}  // namespace

uint32_t int8_token_blocks(uint32_t M) { return (M + kTile - 1) / kTile; }

int launch_int8_product(Int8Mode mode, const Int8Args &a, hipStream_t s) {
    const uint32_t cols = mode == kBwd || mode == kGatedBwd ? (uint32_t)a.ldd : a.N;
    const dim3 grid((cols + kTile - 1) / kTile, int8_token_blocks(a.M));
    if (mode == kFwd) int8_product<kFwd><<<grid, 256, 0, s>>>(a);
    if (mode == kGated) int8_product<kGated><<<grid, 256, 0, s>>>(a);
    if (mode == kBwd) int8_product<kBwd><<<grid, 256, 0, s>>>(a);
    if (mode == kGatedBwd) int8_product<kGatedBwd><<<grid, 256, 0, s>>>(a);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

}  // namespace entq
