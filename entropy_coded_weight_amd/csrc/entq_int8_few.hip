// entq_int8_few.hip -- the int8 products for few tokens, where the weights'
// bytes are what there is to do: they go from memory straight to registers.
#include <algorithm>

#include "entq_int8.h"

namespace entq {
namespace {

constexpr int kFewWaves = 8;

// Bytes of a token's codes in LDS: whole blocks.
__host__ __device__ constexpr uint32_t few_codes(uint32_t K) { return (K + 127) / 128 * 128; }

// A workgroup computes 16 channels (of both weights, gated) for MT groups of
// 16 tokens; its 8 waves take the 128-code blocks of K in turn, four of them in
// flight, and add their sums up in LDS. Lane l reads codes 32 (l / 16) .. + 31
// of a block of row l % 16, for weights and tokens alike: a wave's two loads
// cover 16 whole 128-byte lines, and the order of K inside a block does not
// matter to the sum. Rows may lie at any address. Every weight byte is read
// once, so the bound is memory: one token takes 15.0 us for 8192 x 8192 (67
// MB, 4.5 TB/s with the launch in it), 45 us for 8192 x 28672 (5.2 TB/s), 81 us
// for gated 28672 x 8192 (5.8 TB/s; a copy reaches 4.7 TB/s of reads and
// writes). With 16 tokens the activations are as many bytes again out of the
// L2, and 64-token tiles win where the bytes count. 32 channels a workgroup
// (half the activation reads, half the workgroups) took 21.1 us and 111 us
// where this takes 17.5 and 86 (both with the quantiser), 16 waves the same
// for one weight and 5-10 % more for two.
//
// XT other than ENTQ_I8: one token, whose activations every workgroup
// quantises for itself into its LDS while the first weights are on their way.
template <int MODE, int MT, int XT>
__global__ __launch_bounds__(64 * kFewWaves) void int8_few(Int8Args a) {
    constexpr bool kTwo = MODE == kGated || MODE == kGatedBwd;
    constexpr bool kBack = MODE == kBwd || MODE == kGatedBwd;
    constexpr int NW = kTwo ? 2 : 1, kSums = NW * MT;
    constexpr int kDepth = kSums >= 8 ? 2 : 4;  // blocks in flight
    __shared__ v4i sums[kFewWaves][kSums][64];
    extern __shared__ __attribute__((aligned(16))) int8_t codes[];  // the token's, XT not ENTQ_I8
    __shared__ uint32_t top[kFewWaves];
    float own_scale = 0.0f;
    const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t n0 = blockIdx.x * 16, kc = lane / 16 * 32;

    const int8_t *w[NW], *x[MT];
#pragma unroll
    for (int t = 0; t < NW; ++t) w[t] = a.w[t] + (uint64_t)min(n0 + lane % 16, a.N - 1) * a.ldw[t] + kc;
#pragma unroll
    for (int g = 0; g < MT; ++g)
        x[g] = XT == ENTQ_I8 ? a.x + (uint64_t)min(g * 16 + lane % 16, a.M - 1) * a.ldx + kc
                             : codes + kc;

    v4i acc[NW][MT] = {};
    struct Block {
        v4i w[NW][2], x[MT][2];
    };
    auto load = [&](Block &b, uint32_t k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int t = 0; t < NW; ++t) b.w[t][h] = ((const any16 *)(w[t] + k + 16 * h))->v;
#pragma unroll
            for (int g = 0; g < MT; ++g)
                if (XT == ENTQ_I8) b.x[g][h] = ((const any16 *)(x[g] + k + 16 * h))->v;
        }
    };
    auto own_codes = [&](Block &b, uint32_t k) {  // (right before their use)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < MT; ++g)
                if (XT != ENTQ_I8) b.x[g][h] = *(const v4i *)(x[g] + k + 16 * h);
    };
    auto multiply = [&](const Block &b) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < NW; ++t)
#pragma unroll
                for (int g = 0; g < MT; ++g)
                    acc[t][g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b.w[t][h], b.x[g][h], acc[t][g], 0, 0, 0);
    };
    const uint32_t blocks = a.K / 128;  // whole ones
    const uint32_t mine = blocks > wave ? (blocks - wave + kFewWaves - 1) / kFewWaves : 0;
    Block b[kDepth];
    auto at = [&](uint32_t i) { return (i * kFewWaves + wave) * 128; };
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        if ((uint32_t)d < mine) load(b[d], at(d));
    if constexpr (XT != ENTQ_I8) {
        constexpr int kPer = XT == ENTQ_F32 ? 4 : 8, kThreads = 64 * kFewWaves;
        auto piece = [&](uint32_t p) { return ((const any16 *)((const uint8_t *)a.x + p * 16))->v; };
        const uint32_t full = a.K / kPer, rest = full * kPer + threadIdx.x;
        uint32_t big = 0;
#pragma unroll 4
        for (uint32_t p = threadIdx.x; p < full; p += kThreads) {
            const v4i v = piece(p);
#pragma unroll
            for (int e = 0; e < kPer; ++e) big = max(big, __float_as_uint(act_of<XT>(v, e)) & 0x7FFFFFFFu);
        }
        if (rest < a.K) big = max(big, __float_as_uint(load_act<XT>(a.x, rest)) & 0x7FFFFFFFu);
        big = wave_max(big);
        if (lane == 0) top[wave] = big;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < kFewWaves; ++v) big = max(big, top[v]);
        const Quantizer z(big);
        own_scale = z.scale;
#pragma unroll 4
        for (uint32_t p = threadIdx.x; p < full; p += kThreads) {
            const v4i v = piece(p);
            if constexpr (kPer == 8)
                *(v2i *)(codes + p * 8) = v2i{(int)z.code4<XT>(v, 0), (int)z.code4<XT>(v, 4)};
            else
                *(int *)(codes + p * 4) = (int)z.code4<XT>(v, 0);
        }
        if (rest < a.K) codes[rest] = (int8_t)z.code(load_act<XT>(a.x, rest));
        for (uint32_t c = a.K + threadIdx.x; c < few_codes(a.K); c += kThreads) codes[c] = 0;
        __syncthreads();
    }
    uint32_t i = 0;
    for (; i + 2 * kDepth <= mine; i += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            own_codes(b[d], at(i + d));
            multiply(b[d]);
            load(b[d], at(i + d + kDepth));
        }
    }
    for (; i < mine; i += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            if (i + d < mine) {
                own_codes(b[d], at(i + d));
                multiply(b[d]);
            }
            if (i + d + kDepth < mine) load(b[d], at(i + d + kDepth));
        }
    }
    if (a.K % 128 && wave == blocks % kFewWaves) {
        Block e;
        const uint32_t k = blocks * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int t = 0; t < NW; ++t) e.w[t][h] = load16_any(w[t] - kc, k + kc + 16 * h, a.K);
#pragma unroll
            for (int g = 0; g < MT; ++g)
                if (XT == ENTQ_I8) e.x[g][h] = load16_any(x[g] - kc, k + kc + 16 * h, a.K);
        }
        own_codes(e, k);
        multiply(e);
    }

#pragma unroll
    for (int t = 0; t < NW; ++t)
#pragma unroll
        for (int g = 0; g < MT; ++g) sums[wave][t * MT + g][lane] = acc[t][g];
    __syncthreads();
    if (wave < MT) {
        const uint32_t g = wave;
        v4i s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < kFewWaves; ++v) {
            s0 += sums[v][g][lane];
            if (kTwo) s1 += sums[v][MT + g][lane];
        }
        const uint32_t n = n0 + lane / 16 * 4;
        float scale[2][4], sg[4] = {}, su[4] = {};
        load_scales<MODE>(a, n, scale);
        const uint32_t m = g * 16 + lane % 16;
        const float sx = XT == ENTQ_I8 ? a.sx[min(m, a.M - 1)] : own_scale;
        const uint2 dy4 = kBack ? load_grad4(a, m, n) : make_uint2(0, 0);
        epilogue4<MODE>(a, sx, scale, m, n, s0, s1, dy4, sg, su);
        if constexpr (kBack) {
#pragma unroll
            for (int t = 0; t < NW; ++t) {
                if (!a.part[t]) continue;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float s = t ? su[c] : sg[c];
#pragma unroll
                    for (int o = 1; o < 16; o *= 2) s += __shfl_xor(s, o);
                    if (lane % 16 == 0 && n + c < a.N) a.part[t][(uint64_t)g * a.N + n + c] = s;
                }
            }
        }
    }
}

template <int MT, int XT>
int launch_few(Int8Mode mode, const Int8Args &a, hipStream_t s) {
    const uint32_t cols = mode == kBwd || mode == kGatedBwd ? (uint32_t)a.ldd : a.N;
    constexpr int kThreads = 64 * kFewWaves;
    const dim3 grid(cols / 16 + (cols % 16 != 0));
    if (!launchable(grid.x, kThreads)) return ENTQ_EINVAL;
    const uint32_t lds = XT == ENTQ_I8 ? 0 : few_codes(a.K);
    if (mode == kFwd) int8_few<kFwd, MT, XT><<<grid, kThreads, lds, s>>>(a);
    if (mode == kGated) int8_few<kGated, MT, XT><<<grid, kThreads, lds, s>>>(a);
    if constexpr (XT == ENTQ_I8) {
        if (mode == kBwd) int8_few<kBwd, MT, XT><<<grid, kThreads, lds, s>>>(a);
        if (mode == kGatedBwd) int8_few<kGatedBwd, MT, XT><<<grid, kThreads, lds, s>>>(a);
    }
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

}  // namespace

// One token, whose codes fit a share of the LDS. Measured against a launch of
// the quantiser before over sides of 512 .. 32,000 x 1,024 .. 32,768 (bf16,
// us): product 1024 x 1024 3.9 / 5.1, 8192 x 8192 17.1 / 18.0, 28672 x 8192
// 44.6 / 46.8, gated 28672 x 8192 84.1 / 86.2; it loses at most 4 %, where
// there are many channels of many columns (28672 x 32768 189 / 182). For several
// tokens it does not pay (4: 21.3 / 18.7).
bool few_quantizes(uint32_t M, uint32_t K) { return M == 1 && K <= 32768; }

int launch_int8_few(Int8Mode mode, const Int8Args &a, hipStream_t s) {
    if (a.x_type == ENTQ_BF16) return launch_few<1, ENTQ_BF16>(mode, a, s);
    if (a.x_type == ENTQ_F16) return launch_few<1, ENTQ_F16>(mode, a, s);
    if (a.x_type == ENTQ_F32) return launch_few<1, ENTQ_F32>(mode, a, s);
    if (a.M <= 16) return launch_few<1, ENTQ_I8>(mode, a, s);
    if (a.M <= 32) return launch_few<2, ENTQ_I8>(mode, a, s);
    return launch_few<4, ENTQ_I8>(mode, a, s);
}

}  // namespace entq
