// entq_int8_grad.hip -- dX = sum over the weights of d . W for 16-bit
// gradients d [M][N] and int8 codes W [N][K]: a product along the weights'
// rows.
#include <algorithm>

#include "entq_int8_tile.h"

namespace entq {
namespace {

// 8 codes (two dwords) as 8 values of 16 bits; every code is exact in both
// types.
template <bool F16>
__device__ __forceinline__ v2i widen4(int codes) {
    v2i r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (F16) {
            // 0x6400 | u is 1024 + u for a byte u; u = code + 128
            const uint32_t u = (uint32_t)codes ^ 0x80808080u;
            const uint32_t h = __builtin_amdgcn_perm(0x64646464u, u, i ? 0x04030402u : 0x04010400u);
            typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
            r[i] = __builtin_bit_cast(int, __builtin_bit_cast(f16x2, h) - f16x2{(_Float16)1152.0f, (_Float16)1152.0f});
        } else {
            const float lo = (float)(int8_t)(codes >> (16 * i)), hi = (float)(int8_t)(codes >> (16 * i + 8));
            r[i] = (int)__builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
        }
    }
    return r;
}

// A workgroup of 4 waves (WM x WN) computes BM tokens x BK columns. The sum
// goes by in steps of 64 channels, the first weight's and then the second's;
// S steps are kept in LDS. The weights stay int8 until they are in registers:
// a transposing LDS read gives a lane 8 consecutive channels of its column,
// which it widens to 16 bits (12 vector instructions per 8 codes, beside the
// products of the fragments before). In the 256 x 256 kind the waves divide the
// columns, not the tokens, so that each code is widened once a workgroup; in
// the smaller kinds, 2 x 2 waves, it is widened twice.
//
// What bounds it: at 2048 x 28672 x 8192 (two weights, 1.92 TFLOP) it takes
// 1.40 to 1.44 ms, 1.35 PFLOP/s (the library's bf16 product of 8192 a side
// reaches 1.5); the matrix units are busy three quarters of the cycles, at 1.5
// GHz (of 2.4): power.
// Measured there for the whole backward call, waves as 2 x 2: 2240 us, 1 x 4
// (here): 2222, 8 waves as 2 x 4: 2295 against 2273. LDS reads meet no bank
// conflicts. Splitting the sum (partial sums in fp32, added in order) serves few
// tokens: 16 tokens, 8192 x 8192 27.9 us in 4 parts, 28.9 in 8.
template <bool F16, int BM, int BK, int WM, int WN, int S>
__global__ __launch_bounds__(256) void grad_tiles(GradArgs a, uint32_t nb_m, uint32_t nb_k) {
    constexpr int FM = BM / WM / 32, FN = BK / WN / 32;
    constexpr int kLoadsD = BM / 32, kLoadsW = BK / 64, kLoads = kLoadsD + kLoadsW;
    constexpr uint32_t kStageD = BM * kRowBytes, kStageW = 64 * BK;
    constexpr uint32_t kChunks = BK / 16, kRowsW = 64 / kChunks;  // of a weight row; of a wave's load
    constexpr int kFlying = (S - 2) * kLoads;
    static_assert(WM * WN == 4 && (BK == 256 || BK == 128), "");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S * (kStageD + kStageW)];
    // 16-byte chunk c of row r lies at c ^ twist(r): the 16 chunks that 32
    // lanes read at once (8 rows, 2 neighbouring columns chunks) fill all banks
    auto twist = [](uint32_t r) { return BK == 256 ? 2 * (r % 8) : 2 * (r / 2 % 4); };

    // the workgroups after the tiles finish the channel sums of the kernel before
    if (blockIdx.x >= nb_m * nb_k) {
        if (blockIdx.y == 0) sum_parts_block(a.sums, blockIdx.x - nb_m * nb_k);
        return;
    }
    const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t wm = wave % WM, wn = wave / WM;
    uint32_t tm, tk;
    tile_of(blockIdx.x, nb_m, nb_k, tm, tk);
    const uint32_t m0 = tm * BM, k0 = tk * BK;

    const uint32_t per = (uint32_t)(a.ldd / 64);  // steps of one weight
    const uint32_t total = a.n_w * per;
    const uint32_t first = (uint32_t)((uint64_t)total * blockIdx.y / a.splits);
    const uint32_t steps = (uint32_t)((uint64_t)total * (blockIdx.y + 1) / a.splits) - first;

    uint32_t doff[kLoadsD], wrow[kLoadsW], wcol[kLoadsW];
#pragma unroll
    for (int i = 0; i < kLoadsD; ++i)
        doff[i] = min(8 * (4 * i + wave) + lane / 8, a.M - 1 - m0) * (uint32_t)a.ldd * 2 +
                  16 * ((lane % 8) ^ swizzle(8 * wave + lane / 8));
#pragma unroll
    for (int i = 0; i < kLoadsW; ++i) {
        wrow[i] = (4 * i + wave) * kRowsW + lane / kChunks;
        const uint32_t c = 16 * ((lane % kChunks) ^ twist(wrow[i]));
        wcol[i] = k0 + c < a.K ? k0 + c : 0;  // beyond the columns: results not stored
    }
    const uint16_t *dbase[2] = {a.d[0] + (uint64_t)m0 * a.ldd, a.d[1] + (uint64_t)m0 * a.ldd};
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds));
    const uint32_t ldsw = lds0 + S * kStageD;
    // load j of step `step` (of this split) into a slot, weights first
    auto load_one = [&](int j, uint32_t step, uint32_t slot) {
        const uint32_t s = first + step, t = s >= per ? 1 : 0, n = (s - t * per);
        if (j < kLoadsW) {
            // beyond the channels the last one's codes: d is 0 there
            const uint32_t off = __umul24(min(wrow[j], a.N - 1 - n * 64), (uint32_t)(t ? a.ldw[1] : a.ldw[0])) + wcol[j];
            load_lds16((t ? a.w[1] : a.w[0]) + (uint64_t)n * 64 * (t ? a.ldw[1] : a.ldw[0]), off,
                       ldsw + slot * kStageW + (4 * j + wave) * 1024);
        } else {
            load_lds16((t ? dbase[1] : dbase[0]) + n * 64, doff[j - kLoadsW],
                       lds0 + slot * kStageD + (4 * (j - kLoadsW) + wave) * 1024);
        }
    };

    v16f acc[FN][FM] = {};
    v4i df[2][FM], wf[2][FN];
    v2i raw[FN];
    const uint32_t drow = lds0 + (wm * (BM / WM) + lane % 32) * kRowBytes;
    const uint32_t wr = lane / 32 * 8 + lane % 16 / 2;  // the row whose bytes this lane names
    uint32_t wat[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f)
        wat[f] = ldsw + wr * BK + 16 * ((wn * FN * 2 + f * 2 + lane / 16 % 2) ^ twist(wr)) + lane % 2 * 8;
    auto fetch_one = [&](int set, uint32_t slot, int sub, int j) {
        if (j < FN)
            raw[j] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (__attribute__((address_space(3))) v2i *)(uintptr_t)(wat[j] + slot * kStageW + sub * 16 * BK));
        else
            df[set][j - FN] = read_lds16(drow + slot * kStageD +
                                         16 * ((2 * sub + lane / 32) ^ swizzle(lane % 32)) +
                                         (j - FN) * 32 * kRowBytes);
    };
    auto widen_one = [&](int set, int j) {  // half a fragment
        const v2i w = widen4<F16>(raw[j / 2][j % 2]);
        wf[set][j / 2][2 * (j % 2)] = w[0];
        wf[set][j / 2][2 * (j % 2) + 1] = w[1];
    };
    // 16 channels: the products of one fragment set, beside them the reads
    // (first half) and the widening (second half) of the next set and, with
    // part >= 0, that part of a later step's loads.
    auto quarter = [&](int set, uint32_t slot, int sub, int part, uint32_t step, uint32_t to) {
        constexpr int kMul = FN * FM, kFetch = FN + FM, kWiden = 2 * FN, kHalf = (kMul + 1) / 2;
#pragma unroll
        for (int i = 0; i < kMul; ++i) {
            if (i < kHalf) {
#pragma unroll
                for (int j = i * kFetch / kHalf; j < (i + 1) * kFetch / kHalf; ++j) fetch_one(set ^ 1, slot, sub, j);
            }
            if (part >= 0) {
                const int f = part * kMul + i;
#pragma unroll
                for (int j = f * kLoads / (4 * kMul); j < (f + 1) * kLoads / (4 * kMul); ++j) load_one(j, step, to);
            }
            if (F16)
                acc[i / FM][i % FM] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                    __builtin_bit_cast(f16x8, wf[set][i / FM]), __builtin_bit_cast(f16x8, df[set][i % FM]),
                    acc[i / FM][i % FM], 0, 0, 0);
            else
                acc[i / FM][i % FM] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    __builtin_bit_cast(bf16x8, wf[set][i / FM]), __builtin_bit_cast(bf16x8, df[set][i % FM]),
                    acc[i / FM][i % FM], 0, 0, 0);
            if (i >= kMul - kHalf) {
                const int h = i - (kMul - kHalf);
#pragma unroll
                for (int j = h * kWiden / kHalf; j < (h + 1) * kWiden / kHalf; ++j) widen_one(set ^ 1, j);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto after = [](uint32_t slot) { return slot + 1 == S ? 0 : slot + 1; };

    for (uint32_t i = 0; i < (uint32_t)S && i < steps; ++i)
#pragma unroll
        for (int j = 0; j < kLoads; ++j) load_one(j, i, i);
    if (steps >= S)
        wait_loads_and_meet<(S - 1) * kLoads>();
    else
        wait_loads_and_meet<0>();
#pragma unroll
    for (int j = 0; j < FN + FM; ++j) fetch_one(0, 0, 0, j);
#pragma unroll
    for (int j = 0; j < 2 * FN; ++j) widen_one(0, j);
    uint32_t step = 0, slot = 0;
    quarter(0, 0, 1, -1, 0, 0);
    quarter(1, 0, 2, -1, 0, 0);
    quarter(0, 0, 3, -1, 0, 0);
    if (steps >= S)
        wait_loads_and_meet<kFlying>();
    else
        wait_loads_and_meet<0>();
    // `step` is read except for its last quarter, which is in registers; the
    // next step has landed
    for (; step + S < steps; ++step) {
        const uint32_t next = after(slot);
        quarter(1, next, 0, 0, step + S, slot);
        quarter(0, next, 1, 1, step + S, slot);
        quarter(1, next, 2, 2, step + S, slot);
        quarter(0, next, 3, 3, step + S, slot);
        wait_loads_and_meet<kFlying>();
        slot = next;
    }
#pragma unroll 1
    for (; step + 1 < steps; ++step) {
        slot = after(slot);
        quarter(1, slot, 0, -1, 0, 0);
        quarter(0, slot, 1, -1, 0, 0);
        quarter(1, slot, 2, -1, 0, 0);
        quarter(0, slot, 3, -1, 0, 0);
        wait_loads_and_meet<0>();
    }
    quarter(1, slot, 0, -1, 0, 0);  // (what it reads is not used)

    float back[FM];
#pragma unroll
    for (int g = 0; g < FM; ++g)
        back[g] = F16 && a.splits == 1 ? a.back[min(m0 + wm * (BM / WM) + g * 32 + lane % 32, a.M - 1)] : 1.0f;
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int g = 0; g < FM; ++g) {
            const uint32_t m = m0 + wm * (BM / WM) + g * 32 + lane % 32;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t k = k0 + wn * (BK / WN) + f * 32 + q * 8 + lane / 32 * 4;
                const v4f v = {acc[f][g][4 * q], acc[f][g][4 * q + 1], acc[f][g][4 * q + 2], acc[f][g][4 * q + 3]};
                if (m >= a.M || k >= a.K) continue;
                if (a.splits > 1) {
                    *(v4f *)(a.parts + ((uint64_t)blockIdx.y * a.M + m) * a.K + k) = v;
                    continue;
                }
                uint16_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = bits16(v[i] * back[g], F16);
                uint16_t *to = (uint16_t *)a.dx + (uint64_t)m * a.lddx + k;
                if (k + 4 <= a.cols) {
                    ((any8 *)to)->v = v2i{(int)(b[0] | (uint32_t)b[1] << 16), (int)(b[2] | (uint32_t)b[3] << 16)};
                } else {
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i)
                        if (k + i < a.cols) to[i] = b[i];
                }
            }
        }
}

// dX from the splits' partial sums, added in order.
__global__ __launch_bounds__(256) void grad_sum(GradArgs a) {
    const uint32_t k = 4 * (blockIdx.x * 256 + threadIdx.x);
    if (k >= a.K) return;
    for (uint64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
        const float back = a.f16 ? a.back[m] : 1.0f;
        v4f v = {0, 0, 0, 0};
#pragma unroll 4
        for (uint32_t s = 0; s < a.splits; ++s) v += *(const v4f *)(a.parts + ((uint64_t)s * a.M + m) * a.K + k);
        for (uint32_t i = 0; i < 4; ++i)
            if (k + i < a.cols) ((uint16_t *)a.dx)[m * a.lddx + k + i] = bits16(v[i] * back, a.f16);
    }
}

template <int BM, int BK, int WM, int WN, int S>
int launch_tiles(const GradArgs &a, hipStream_t s) {
    const uint32_t nb_m = (a.M + BM - 1) / BM, nb_k = (a.K + BK - 1) / BK;
    if (!launchable(((uint64_t)nb_m * nb_k + sum_blocks(a.sums)) * a.splits, 256)) return ENTQ_EINVAL;
    const dim3 grid(nb_m * nb_k + sum_blocks(a.sums), a.splits);
    if (a.f16)
        grad_tiles<true, BM, BK, WM, WN, S><<<grid, 256, 0, s>>>(a, nb_m, nb_k);
    else
        grad_tiles<false, BM, BK, WM, WN, S><<<grid, 256, 0, s>>>(a, nb_m, nb_k);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

}  // namespace

// tokens x columns of the kinds of tiles
static const TileCost kTiles[3] = {{64, 128, {0.542f, 0.857f}, 0.0f},
                                   {128, 128, {0.625f, 1.13f}, 0.0f},
                                   {256, 256, {1.32f, 1.64f}, 1.9f}};
static const SplitCost kSplits = {6.6f, 9.2e6f, 3.5f, 0.125f, 1.54e-6f};

GradPlan grad_plan(uint32_t M, uint32_t N, uint32_t K, int n_w) {
    const TileChoice t = cheapest_tile(kTiles, kSplits, M, K, n_w * ((N + 63) / 64), (uint64_t)n_w * N * K,
                                       (uint64_t)M * K);
    return {t.kind, t.splits};
}

int launch_grad_product(const GradPlan &p, const GradArgs &a, hipStream_t s) {
    const int r = p.kind == 0   ? launch_tiles<64, 128, 2, 2, 3>(a, s)
                  : p.kind == 1 ? launch_tiles<128, 128, 2, 2, 3>(a, s)
                                : launch_tiles<256, 256, 1, 4, 3>(a, s);
    if (r != ENTQ_OK || p.splits == 1) return r;
    grad_sum<<<dim3((a.K / 4 + 255) / 256, std::min(a.M, 65535u)), 256, 0, s>>>(a);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

}  // namespace entq
