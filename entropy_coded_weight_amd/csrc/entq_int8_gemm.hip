// entq_int8_gemm.hip -- products of int8 activation codes with int8 weight
// codes, with the epilogues of the forward and backward calls.
#include <algorithm>

#include "entq_int8_tile.h"

namespace entq {
namespace {

// Where a split's sums of token m, channels n..n+3 and weight t go.
template <bool TWO>
__device__ __forceinline__ int32_t *part_sums(const Int8Args &a, uint32_t split, uint32_t t, uint32_t m, uint32_t n) {
    const uint64_t wide = (a.N + 3) / 4 * 4;
    return a.sums + (((uint64_t)split * (TWO ? 2 : 1) + t) * a.M + m) * wide + n;
}

// A workgroup of WM x WN waves computes BM tokens x BN weight rows; a
// gated tile's rows alternate 32 of gate and 32 of up, so that a lane's
// fragments hold both sums of a channel. K goes by in steps of 128 codes.
// Weights are the matrix instruction's first operand: a lane's results are 4
// consecutive channels of one token.
//
// SX and SW steps of the two operands are kept in LDS (SX = SW or SW + 1).
// Once a step is read by every wave its place is loaded again, a quarter of
// the loads beside each quarter step of products: a CU takes about 24 cycles
// per load instruction, and loads that wait for their turn hold up the
// wave's products. A wave's fragments for a quarter step are read during the
// one before, so one barrier a step is all that the waves wait for.
//
// What bounds it: for many tokens the matrix units and the card's power. At
// 4096 x 8192 x 28672 the 256-token tiles keep the matrix units busy 74 % of
// the cycles at 1.7 GHz (of 2.4) and take 0.70 to 0.72 ms, 2.7 POP/s (the
// library's int8 product reaches 2.6); busier kernels ran at lower clocks. For up to some
// 200 tokens the weights' bytes: 32000 x 8192 with 16 tokens 50 to 61 us with
// the quantiser, 4.3 to 5.3 TB/s. Steps: one after the other, alone the compiler reads
// each fragment right before its use (gated 4096 x 28672 x 8192 2.65 ms); fixed
// order 1.76; five half-stages of 32 KB with the loads spread 1.73 (product
// 0.81 -> 0.74); epilogue through LDS with its scales read ahead and one choice
// of activation per 4 values 1.56; bands of 4 tiles 1.55. Steps of 64 codes in 4
// or 5 stages: 1.90 (a load instruction then touches twice the lines).
template <int MODE, int BM, int BN, int WM, int WN, int SX, int SW>
__global__ __launch_bounds__(64 * WM * WN) void int8_tiles(Int8Args a, uint32_t nb_m, uint32_t nb_n) {
    constexpr bool kTwo = MODE == kGated || MODE == kGatedBwd;
    constexpr bool kBack = MODE == kBwd || MODE == kGatedBwd;
    constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
    constexpr int kWaves = WM * WN, kLoadsX = BM / 8 / kWaves, kLoadsW = BN / 8 / kWaves;  // of a wave and step
    constexpr uint32_t kStageX = BM * kRowBytes, kStageW = BN * kRowBytes;
    constexpr uint32_t kLds = SX * kStageX + SW * kStageW;
    constexpr uint32_t kChannels = kTwo ? BN / 2 : BN;
    // loads that may be in flight while the next step is read: those issued
    // after the last one of that step
    constexpr int kFlying = (SX - SW) * kLoadsX + (SW - 2) * (kLoadsX + kLoadsW);
    static_assert((!kTwo || FN % 2 == 0) && (SX == SW || SX == SW + 1), "");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];

    if (MODE == kBwd && blockIdx.x >= nb_m * nb_n) {  // a workgroup after the tiles: one token
        const uint32_t m = (blockIdx.x - nb_m * nb_n) * a.splits + blockIdx.y;
        if (m < a.M) narrow_row<false, 4>(a, m, (uint32_t *)lds);
        return;
    }
    const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t wm = wave % WM, wn = wave / WM;
    uint32_t tm, tn;
    tile_of(blockIdx.x, nb_m, nb_n, tm, tn);
    const uint32_t m0 = tm * BM, n0 = tn * kChannels;

    // This wave's loads: rows 8 (4 i + wave) .. + 7 of a tile. Lane l fills
    // position l % 8 of row l / 8.
    const uint32_t kc = 16 * ((lane % 8) ^ swizzle(8 * wave + lane / 8));
    uint32_t xoff[kLoadsX], woff[kLoadsW];
    // this split's steps
    const uint32_t all = (a.K + 127) / 128, first = all * blockIdx.y / a.splits;
    const uint32_t steps = all * (blockIdx.y + 1) / a.splits - first, K = a.K - first * 128;
    const int8_t *xbase = a.x + (uint64_t)m0 * a.ldx + first * 128;
    const int8_t *wbase0 = a.w[0] + (uint64_t)n0 * a.ldw[0] + first * 128;
    const int8_t *wbase1 = kTwo ? a.w[1] + (uint64_t)n0 * a.ldw[1] + first * 128 : wbase0;
#pragma unroll
    for (int i = 0; i < kLoadsX; ++i)
        xoff[i] = min(8 * (kWaves * i + wave) + lane / 8, a.M - 1 - m0) * (uint32_t)a.ldx + kc;
#pragma unroll
    for (int i = 0; i < kLoadsW; ++i) {
        const uint32_t r = 8 * (kWaves * i + wave), c = kTwo ? r / 64 * 32 + r % 32 : r;
        woff[i] = min(c + lane / 8, a.N - 1 - n0) * (uint32_t)(kTwo && r / 32 % 2 ? a.ldw[1] : a.ldw[0]) + kc;
    }
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds));
    const uint32_t ldsw = lds0 + SX * kStageX;
    auto load_x = [&](int i, uint32_t step, uint32_t slot) {
        load_lds16(xbase + step * 128, xoff[i], lds0 + slot * kStageX + (kWaves * i + wave) * 1024);
    };
    auto load_w = [&](int i, uint32_t step, uint32_t slot) {
        const int8_t *base = kTwo && (kWaves * i + wave) / 4 % 2 ? wbase1 : wbase0;
        load_lds16(base + step * 128, woff[i], ldsw + slot * kStageW + (kWaves * i + wave) * 1024);
    };
    // A whole step's loads; past the rows' end tokens are zeros and weights
    // whatever is there.
    auto load_step_x = [&](uint32_t step, uint32_t slot) {
        const bool in = step * 128 + kc < K;
#pragma unroll
        for (int i = 0; i < kLoadsX; ++i) {
            if (in)
                load_x(i, step, slot);
            else
                *(v4i *)(lds + slot * kStageX + (kWaves * i + wave) * 1024 + lane * 16) = v4i{0, 0, 0, 0};
        }
    };
    auto load_step_w = [&](uint32_t step, uint32_t slot) {
        if (step * 128 + kc < K) {
#pragma unroll
            for (int i = 0; i < kLoadsW; ++i) load_w(i, step, slot);
        }
    };

    v16i acc[FN][FM] = {};
    v4i xf[2][FM], wf[2][FN];
    const uint32_t xrow = lds0 + (wm * (BM / WM) + lane % 32) * kRowBytes;
    const uint32_t wrow = ldsw + (wn * (BN / WN) + lane % 32) * kRowBytes;
    // fragment j of a quarter step: in the order in which they are needed
    auto fetch_one = [&](int set, uint32_t sx, uint32_t sw, int sub, int j) {
        const uint32_t c = 16 * ((2 * sub + lane / 32) ^ swizzle(lane % 32));
        if (j == 0 || j > FM)
            wf[set][j ? j - FM : 0] = read_lds16(wrow + sw * kStageW + c + (j ? j - FM : 0) * 32 * kRowBytes);
        else
            xf[set][j - 1] = read_lds16(xrow + sx * kStageX + c + (j - 1) * 32 * kRowBytes);
    };
    // A quarter step: the products of one fragment set, between them the
    // reads of the next set (quarter `sub` of slots sx, sw) and, with part >=
    // 0, that part of the loads of steps tw and tx into slots lw and lx. The
    // order is fixed: left alone, the compiler reads each fragment right
    // before its use and waits for it.
    auto quarter = [&](int set, uint32_t sx, uint32_t sw, int sub, int part, uint32_t tx, uint32_t tw, uint32_t lx,
                       uint32_t lw) {
        constexpr int kMul = FN * FM, kFetch = FN + FM, kLoads = kLoadsX + kLoadsW;
#pragma unroll
        for (int i = 0; i < kMul; ++i) {
#pragma unroll
            for (int j = i * kFetch / kMul; j < (i + 1) * kFetch / kMul; ++j) fetch_one(set ^ 1, sx, sw, sub, j);
            if (part >= 0) {
                const int f = part * kMul + i;
#pragma unroll
                for (int j = f * kLoads / (4 * kMul); j < (f + 1) * kLoads / (4 * kMul); ++j) {
                    if (j < kLoadsW)
                        load_w(j, tw, lw);
                    else
                        load_x(j - kLoadsW, tx, lx);
                }
            }
            acc[i / FM][i % FM] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[set][i / FM], xf[set][i % FM],
                                                                        acc[i / FM][i % FM], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto after = [](uint32_t slot, uint32_t slots) { return slot + 1 == slots ? 0 : slot + 1; };

    for (uint32_t i = 0; i < SX; ++i) {
        if (i < steps) load_step_x(i, i);
        if (i < SW && i < steps) load_step_w(i, i);
    }
    // (the last step's loads may be fewer than kLoads: waits that could meet
    // them in flight are for all)
    if (steps > SX)
        wait_loads_and_meet<(SX - 1) * kLoadsX + (SW - 1) * kLoadsW>();
    else
        wait_loads_and_meet<0>();
#pragma unroll
    for (int j = 0; j < FN + FM; ++j) fetch_one(0, 0, 0, 0, j);
    uint32_t step = 0, sx = 0, sw = 0;
    quarter(0, 0, 0, 1, -1, 0, 0, 0, 0);
    quarter(1, 0, 0, 2, -1, 0, 0, 0, 0);
    quarter(0, 0, 0, 3, -1, 0, 0, 0, 0);
    if (steps > SX)
        wait_loads_and_meet<kFlying>();
    else
        wait_loads_and_meet<0>();
    // `step` is read except for its last quarter, which is in registers; the
    // next step has landed
    for (; step + SX + 1 < steps; ++step) {
        const uint32_t nx = after(sx, SX), nw = after(sw, SW), tx = step + SX, tw = step + SW;
        quarter(1, nx, nw, 0, 0, tx, tw, sx, sw);
        quarter(0, nx, nw, 1, 1, tx, tw, sx, sw);
        quarter(1, nx, nw, 2, 2, tx, tw, sx, sw);
        quarter(0, nx, nw, 3, 3, tx, tw, sx, sw);
        wait_loads_and_meet<kFlying>();
        sx = nx;
        sw = nw;
    }
#pragma unroll 1
    for (; step + 1 < steps; ++step) {
        const uint32_t nx = after(sx, SX), nw = after(sw, SW);
        if (step + SW < steps) load_step_w(step + SW, sw);
        if (step + SX < steps) load_step_x(step + SX, sx);
        quarter(1, nx, nw, 0, -1, 0, 0, 0, 0);
        quarter(0, nx, nw, 1, -1, 0, 0, 0, 0);
        quarter(1, nx, nw, 2, -1, 0, 0, 0, 0);
        quarter(0, nx, nw, 3, -1, 0, 0, 0, 0);
        wait_loads_and_meet<0>();
        sx = nx;
        sw = nw;
    }
    // The sums pass through LDS, 32 tokens of this wave at a time, so that
    // neighbouring lanes then hold neighbouring channels of one token. Those
    // tokens' scales and incoming gradients are read one such group ahead, and
    // through LDS too, into a loop short enough for the instruction cache.
    constexpr uint32_t kRow = FN * 128 + 16;                  // bytes of a token's sums; 16 spread the banks
    constexpr uint32_t kQuads = FN * 8 / (kTwo ? 2 : 1);      // groups of 4 channels
    constexpr uint32_t kTokens = 64 / kQuads;                 // that the wave handles at once
    constexpr uint32_t kTurns = 32 / kTokens;
    constexpr uint32_t kArea = 32 * kRow + (kBack ? kTurns * 512 : 0) + 128;
    static_assert(kWaves * kArea <= kLds, "");
    const uint32_t quad = lane % kQuads, r = wn * (BN / WN) + (kTwo ? quad / 8 * 64 : 0);
    const uint32_t n = n0 + (kTwo ? r / 2 + quad % 8 * 4 : r + quad * 4);
    const uint32_t at = kTwo ? quad / 8 * 256 + quad % 8 * 16 : quad * 16;
    const uint32_t mw = m0 + wm * (BM / WM);
    float sx32;
    uint2 dy4[kBack ? kTurns : 1];
    auto read_ahead = [&](int g) {
        if (a.splits > 1) return;
        sx32 = a.sx[min(mw + g * 32 + lane % 32, a.M - 1)];
        if (kBack) {
#pragma unroll
            for (uint32_t i = 0; i < kTurns; ++i) dy4[i] = load_grad4(a, mw + g * 32 + i * kTokens + lane / kQuads, n);
        }
    };
    read_ahead(0);
    float scale[2][4], sg[4] = {}, su[4] = {};
    load_scales<MODE>(a, n, scale);
#pragma unroll
    for (int i = 0; i < FN * FM; ++i)
        acc[i / FM][i % FM] =
            __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[1][i / FM], xf[1][i % FM], acc[i / FM][i % FM], 0, 0, 0);

    __syncthreads();
    uint8_t *mine = lds + wave * kArea;
    float *const sx_at = (float *)(mine + 32 * kRow);
    uint2 *const dy_at = (uint2 *)(mine + 32 * kRow + 128);
#pragma unroll
    for (int g = 0; g < FM; ++g) {
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(v4i *)(mine + lane % 32 * kRow + f * 128 + q * 32 + lane / 32 * 16) =
                    v4i{acc[f][g][4 * q], acc[f][g][4 * q + 1], acc[f][g][4 * q + 2], acc[f][g][4 * q + 3]};
        if (a.splits == 1) {
            sx_at[lane % 32] = sx32;
            if (kBack) {
#pragma unroll
                for (uint32_t i = 0; i < kTurns; ++i) dy_at[i * 64 + lane] = dy4[i];
            }
        }
        if (g + 1 < FM) read_ahead(g + 1);
#pragma unroll 1
        for (uint32_t i = 0; i < kTurns; ++i) {
            const uint32_t t = i * kTokens + lane / kQuads, m = mw + g * 32 + t;
            const uint8_t *p = mine + t * kRow + at;
            const v4i s0 = *(const v4i *)p, s1 = *(const v4i *)(p + (kTwo ? 128 : 0));
            if (a.splits > 1) {
                if (m < a.M && n < a.N) {
                    *(v4i *)part_sums<kTwo>(a, blockIdx.y, 0, m, n) = s0;
                    if (kTwo) *(v4i *)part_sums<kTwo>(a, blockIdx.y, 1, m, n) = s1;
                }
            } else {
                epilogue4<MODE>(a, sx_at[t], scale, m, n, s0, s1,
                                kBack ? dy_at[i * 64 + lane] : make_uint2(0, 0), sg, su);
            }
        }
    }
    if (kBack && a.splits == 1) {
#pragma unroll
        for (int w = 0; w < (kTwo ? 2 : 1); ++w) {
            if (!a.part[w]) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float s = w ? su[i] : sg[i];
#pragma unroll
                for (uint32_t o = kQuads; o < 64; o *= 2) s += __shfl_xor(s, o);
                if (lane < kQuads && n + i < a.N) a.part[w][(uint64_t)(tm * WM + wm) * a.N + n + i] = s;
            }
        }
    }
}

// Adds the splits' sums up (integers: in any order the same) and finishes
// them. A workgroup: 256 channels (a wave's lanes 4 each), its 4 waves a
// token each.
template <int MODE>
__global__ __launch_bounds__(256) void int8_finish(Int8Args a) {
    constexpr bool kTwo = MODE == kGated || MODE == kGatedBwd;
    constexpr bool kBack = MODE == kBwd || MODE == kGatedBwd;
    __shared__ float waves[4][2][4][64];
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const uint32_t n = blockIdx.x * 256 + lane * 4;
    float scale[2][4], sg[4] = {}, su[4] = {};
    load_scales<MODE>(a, n, scale);
    const uint32_t m = blockIdx.y * 4 + wave;
    v4i s[2] = {};
    if (m < a.M && n < a.N) {
#pragma unroll 4
        for (uint32_t k = 0; k < a.splits; ++k) {
            s[0] += *(const v4i *)part_sums<kTwo>(a, k, 0, m, n);
            if (kTwo) s[1] += *(const v4i *)part_sums<kTwo>(a, k, 1, m, n);
        }
    }
    epilogue4<MODE>(a, a.sx[min(m, a.M - 1)], scale, m, n, s[0], s[1],
                    kBack ? load_grad4(a, m, n) : make_uint2(0, 0), sg, su);
    if constexpr (kBack) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            waves[wave][0][i][lane] = sg[i];
            waves[wave][1][i][lane] = su[i];
        }
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int t = 0; t < (kTwo ? 2 : 1); ++t) {
            if (!a.part[t]) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float s = waves[0][t][i][lane];
#pragma unroll
                for (int w = 1; w < 4; ++w) s += waves[w][t][i][lane];
                if (n + i < a.N) a.part[t][(uint64_t)blockIdx.y * a.N + n + i] = s;
            }
        }
    }
}

// WNB: waves along the weight rows where the epilogue is long (two waves on a
// SIMD cover each other's), WN for the plain product. Measured for 256-token
// tiles, 4 and 8 waves: product 4096 x 8192 x 28672 750 and 785 us (a wave's
// fragments serve fewer products, more LDS reads), gated 4096 x 28672 x 8192
// 1605 and 1596, product back 2048 x 8192 x 8192 329 and 322.
template <int BM, int BN, int WM, int WN, int WNB, int SX, int SW>
int launch_tiles(Int8Mode mode, const Int8Args &a, hipStream_t s) {
    const bool two = mode == kGated || mode == kGatedBwd;
    const uint32_t cols = mode == kBwd || mode == kGatedBwd ? (uint32_t)a.ldd : a.N;
    const uint32_t ch = two ? BN / 2 : BN;
    const uint32_t nb_m = (a.M + BM - 1) / BM, nb_n = (cols + ch - 1) / ch;
    constexpr int kOne = 64 * WM * WN, kLong = 64 * WM * WNB;
    const uint64_t groups = (uint64_t)nb_m * nb_n + (a.narrows ? (a.M + a.splits - 1) / a.splits : 0);
    if (!launchable(groups * a.splits, kLong)) return ENTQ_EINVAL;
    const dim3 grid((uint32_t)groups, a.splits);
    if (mode == kFwd) int8_tiles<kFwd, BM, BN, WM, WN, SX, SW><<<grid, kOne, 0, s>>>(a, nb_m, nb_n);
    if (mode == kGated) int8_tiles<kGated, BM, BN, WM, WNB, SX, SW><<<grid, kLong, 0, s>>>(a, nb_m, nb_n);
    if (mode == kBwd) int8_tiles<kBwd, BM, BN, WM, WNB, SX, SW><<<grid, kLong, 0, s>>>(a, nb_m, nb_n);
    if (mode == kGatedBwd) int8_tiles<kGatedBwd, BM, BN, WM, WNB, SX, SW><<<grid, kLong, 0, s>>>(a, nb_m, nb_n);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

void launch_finish(Int8Mode mode, const Int8Args &a, hipStream_t s) {
    const uint32_t cols = mode == kBwd || mode == kGatedBwd ? (uint32_t)a.ldd : a.N;
    const dim3 grid((cols + 255) / 256, (a.M + 3) / 4);
    if (mode == kFwd) int8_finish<kFwd><<<grid, 256, 0, s>>>(a);
    if (mode == kGated) int8_finish<kGated><<<grid, 256, 0, s>>>(a);
    if (mode == kBwd) int8_finish<kBwd><<<grid, 256, 0, s>>>(a);
    if (mode == kGatedBwd) int8_finish<kGatedBwd><<<grid, 256, 0, s>>>(a);
}

}  // namespace

// tokens x weight rows of the kinds of tiles. (64 x 64 tiles were measured
// too: 0.2 % better on average, not kept.)
static const TileCost kTiles[3] = {{64, 128, {0.427f, 0.81f}, 1.3f},
                                   {128, 128, {0.80f, 1.24f}, 1.5f},
                                   {256, 256, {1.58f, 1.63f}, 4.9f}};
static const SplitCost kSplits = {3.0f, 7.2e6f, 5.0f, 0.1f, 1.25e-6f};

Int8Plan int8_plan(Int8Mode mode, int x_type, uint32_t M, uint32_t N, uint32_t K) {
    const uint64_t n_w = mode == kGated || mode == kGatedBwd ? 2 : 1;
    const TileChoice t =
        cheapest_tile(kTiles, kSplits, M, n_w * N, (K + 127) / 128, n_w * N * K, n_w * M * (uint64_t)N);
    Int8Plan p{};
    p.kind = t.kind;
    p.splits = t.splits;
    if (M <= 64) {
        // The few-token kernel: limited by a wave's turns over K, all the more
        // the more groups of tokens it has, or by the weights' bytes. (At 1 and
        // 4 tokens it was the fastest, or within 6 %, for 13 of 14 shapes, but
        // 512 x 16384 takes 13.6 us where 16 splits take 10.4; at 16 it is
        // faster where the latency counts, 1024 x 1024 4.2 us against 7.0,
        // and slower where the bytes do, 32000 x 8192 66 us against 53.)
        const uint32_t groups = M <= 16 ? 1 : M <= 32 ? 2 : 4;
        const float rounds = 1 + 0.87f * ((n_w * N + 4095) / 4096 - 1);  // of workgroups on a CU
        const float turns = (K + 1023) / 1024 * (0.60f + 0.40f * groups) * rounds;
        const float memory = n_w * N * (float)K * (1 / 5.4e6f + 2.5e-8f * groups);
        p.few = M <= 4 || 3.4f + std::max(turns, memory) < t.us;
        if (p.few) {
            p.quantizes = x_type != ENTQ_I8 && few_quantizes(M, K);
            p.splits = 1;
            p.part_rows = groups;
            return p;
        }
    }
    const uint32_t tokens = kTiles[p.kind].tokens;
    p.part_rows = p.splits > 1 ? (M + 3) / 4 : (M + tokens - 1) / tokens * 2;
    return p;
}

int launch_int8_product(Int8Mode mode, const Int8Plan &p, const Int8Args &a, hipStream_t s) {
    if (p.few) return launch_int8_few(mode, a, s);
    const int r = p.kind == 0   ? launch_tiles<64, 128, 2, 2, 2, 3, 3>(mode, a, s)
                  : p.kind == 1 ? launch_tiles<128, 128, 2, 2, 2, 3, 2>(mode, a, s)
                                : launch_tiles<256, 256, 2, 2, 4, 3, 2>(mode, a, s);
    if (r != ENTQ_OK || a.splits == 1) return r;
    launch_finish(mode, a, s);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

}  // namespace entq
