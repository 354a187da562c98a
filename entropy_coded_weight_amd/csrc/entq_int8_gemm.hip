// entq_int8_gemm.hip -- products of int8 activation codes with int8 weight
// codes, with the epilogues of the forward and backward calls.
#include <algorithm>

#include "entq_int8_tile.h"

namespace entq {
namespace {

// A workgroup of 4 waves (WM x WN) computes BM tokens x BN weight rows; a
// gated tile's rows alternate 32 of gate and 32 of up, so that a lane's
// fragments hold both sums of a channel. K goes by in steps of 128 codes in
// two LDS stages. Weights are the matrix instruction's first operand: a lane's
// results are 4 consecutive channels of one token.
template <int MODE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(256) void int8_tiles(Int8Args a, uint32_t nb_m, uint32_t nb_n) {
    constexpr bool kTwo = MODE == kGated || MODE == kGatedBwd;
    constexpr bool kBack = MODE == kBwd || MODE == kGatedBwd;
    constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
    constexpr int kLoads = (BM + BN) / 32;  // of a wave and step: 8 rows each
    constexpr uint32_t kStage = (BM + BN) * kRowBytes;
    constexpr uint32_t kChannels = kTwo ? BN / 2 : BN;
    static_assert(WM * WN == 4 && (!kTwo || FN % 2 == 0), "");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];

    const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t wm = wave % WM, wn = wave / WM;
    uint32_t tm, tn;
    tile_of(blockIdx.x, nb_m, nb_n, 8, tm, tn);
    const uint32_t m0 = tm * BM, n0 = tn * kChannels;

    // This wave's loads: rows 8 (4 i + wave) .. + 7 of the stage, tokens first.
    // Lane l takes chunk (l % 8) ^ (l / 8) of row l / 8, which belongs at l.
    const uint32_t kc = 16 * ((lane % 8) ^ (lane / 8));
    uint32_t off[kLoads];
    const int8_t *base[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const uint32_t first = 8 * (4 * i + wave);
        if (4 * i * 8 < BM) {
            base[i] = a.x + (uint64_t)m0 * a.ldx;
            off[i] = min(first + lane / 8, a.M - 1 - m0) * (uint32_t)a.ldx + kc;
        } else {
            const uint32_t r = first - BM, t = kTwo ? r / 32 % 2 : 0;
            const uint32_t c = kTwo ? r / 64 * 32 + r % 32 : r;
            base[i] = a.w[t] + (uint64_t)n0 * a.ldw[t];
            off[i] = min(c + lane / 8, a.N - 1 - n0) * (uint32_t)a.ldw[t] + kc;
        }
    }
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds));
    const uint32_t steps = (a.K + 127) / 128;
    auto load_one = [&](int i, uint32_t step) {
        load_lds16(base[i] + step * 128, off[i], lds0 + (step & 1) * kStage + wave * 1024 + i * 4096);
    };
    auto load = [&](uint32_t step) {
        if (step * 128 + 128 <= a.K) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) load_one(i, step);
            return;
        }
        // past the row's end: tokens as zeros, weights as whatever is there
        const bool in = step * 128 + kc < a.K;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (in)
                load_one(i, step);
            else if (4 * i * 8 < BM)
                *(v4i *)(lds + (step & 1) * kStage + wave * 1024 + i * 4096 + lane * 16) = v4i{0, 0, 0, 0};
        }
    };

    v16i acc[FN][FM] = {};
    v4i xf[2][FM], wf[2][FN];
    const uint32_t xrow = lds0 + (wm * (BM / WM) + lane % 32) * kRowBytes;
    const uint32_t wrow = lds0 + (BM + wn * (BN / WN) + lane % 32) * kRowBytes;
    // fragment j of a quarter step: in the order in which they are needed
    auto fetch_one = [&](int set, uint32_t stage, int sub, int j) {
        const uint32_t c = stage * kStage + 16 * ((2 * sub + lane / 32) ^ (lane % 8));
        if (j == 0 || j > FM)
            wf[set][j ? j - FM : 0] = read_lds16(wrow + c + (j ? j - FM : 0) * 32 * kRowBytes);
        else
            xf[set][j - 1] = read_lds16(xrow + c + (j - 1) * 32 * kRowBytes);
    };
    // A quarter step: the products of one fragment set, with the next set's
    // reads and (LOAD) the loads of a later step between them. The order is
    // fixed: left alone, the compiler reads each fragment right before its
    // use and waits for it.
    auto quarter = [&](int set, bool fetch, uint32_t stage, int sub, bool loads, uint32_t step) {
        constexpr int kMul = FN * FM, kFetch = FN + FM;
#pragma unroll
        for (int i = 0; i < kMul; ++i) {
#pragma unroll
            for (int j = i * kFetch / kMul; j < (i + 1) * kFetch / kMul; ++j)
                if (fetch) fetch_one(set ^ 1, stage, sub, j);
#pragma unroll
            for (int j = i * kLoads / kMul; j < (i + 1) * kLoads / kMul; ++j)
                if (loads) load_one(j, step);
            acc[i / FM][i % FM] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[set][i / FM], xf[set][i % FM],
                                                                        acc[i / FM][i % FM], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    load(0);
    wait_loads_and_meet();
    if (steps > 1) load(1);
#pragma unroll
    for (int j = 0; j < FN + FM; ++j) fetch_one(0, 0, 0, j);
    uint32_t step = 0;
    for (; step + 3 < steps; ++step) {
        const uint32_t stage = step & 1;
        quarter(0, true, stage, 1, false, 0);
        quarter(1, true, stage, 2, false, 0);
        quarter(0, true, stage, 3, false, 0);
        // this stage is read, the next one has landed
        wait_loads_and_meet();
        quarter(1, true, stage ^ 1, 0, true, step + 2);
    }
#pragma unroll 1
    for (; step < steps; ++step) {
        const uint32_t stage = step & 1;
        quarter(0, true, stage, 1, false, 0);
        quarter(1, true, stage, 2, false, 0);
        quarter(0, true, stage, 3, false, 0);
        wait_loads_and_meet();
        if (step + 2 < steps) load(step + 2);
        quarter(1, true, stage ^ 1, 0, false, 0);  // (after the last step: read and not used)
    }

    // The sums pass through LDS, 32 tokens of this wave at a time, so that
    // neighbouring lanes then hold neighbouring channels of one token.
    constexpr uint32_t kRow = FN * 128 + 16;                  // bytes of a token's sums; 16 spread the banks
    constexpr uint32_t kQuads = FN * 8 / (kTwo ? 2 : 1);      // groups of 4 channels
    constexpr uint32_t kTokens = 64 / kQuads;                 // that the wave handles at once
    static_assert(4 * 32 * kRow <= 2 * kStage, "");
    __syncthreads();
    uint8_t *mine = lds + wave * 32 * kRow;
    const uint32_t quad = lane % kQuads, r = wn * (BN / WN) + (kTwo ? quad / 8 * 64 : 0);
    const uint32_t n = n0 + (kTwo ? r / 2 + quad % 8 * 4 : r + quad * 4);
    const uint32_t at = kTwo ? quad / 8 * 256 + quad % 8 * 16 : quad * 16;
    float sg[4] = {}, su[4] = {};
#pragma unroll
    for (int g = 0; g < FM; ++g) {
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(v4i *)(mine + lane % 32 * kRow + f * 128 + q * 32 + lane / 32 * 16) =
                    v4i{acc[f][g][4 * q], acc[f][g][4 * q + 1], acc[f][g][4 * q + 2], acc[f][g][4 * q + 3]};
#pragma unroll 1
        for (uint32_t t = lane / kQuads; t < 32; t += kTokens) {
            const uint8_t *p = mine + t * kRow + at;
            epilogue4<MODE>(a, m0 + wm * (BM / WM) + g * 32 + t, n, *(const v4i *)p,
                            *(const v4i *)(p + (kTwo ? 128 : 0)), sg, su);
        }
    }
    if constexpr (kBack) {
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

template <int BM, int BN, int WM, int WN>
void launch_tiles(Int8Mode mode, const Int8Args &a, hipStream_t s) {
    const bool two = mode == kGated || mode == kGatedBwd;
    const uint32_t cols = mode == kBwd || mode == kGatedBwd ? (uint32_t)a.ldd : a.N;
    const uint32_t ch = two ? BN / 2 : BN;
    const uint32_t nb_m = (a.M + BM - 1) / BM, nb_n = (cols + ch - 1) / ch;
    const dim3 grid(nb_m * nb_n);
    if (mode == kFwd) int8_tiles<kFwd, BM, BN, WM, WN><<<grid, 256, 0, s>>>(a, nb_m, nb_n);
    if (mode == kGated) int8_tiles<kGated, BM, BN, WM, WN><<<grid, 256, 0, s>>>(a, nb_m, nb_n);
    if (mode == kBwd) int8_tiles<kBwd, BM, BN, WM, WN><<<grid, 256, 0, s>>>(a, nb_m, nb_n);
    if (mode == kGatedBwd) int8_tiles<kGatedBwd, BM, BN, WM, WN><<<grid, 256, 0, s>>>(a, nb_m, nb_n);
}

}  // namespace

Int8Plan int8_plan(Int8Mode mode, uint32_t M, uint32_t N, uint32_t K) {
    Int8Plan p{};
    const char *f = getenv("ENTQ_TILE");
    p.tile = f ? atoi(f) : 256;
    p.part_rows = (M + p.tile - 1) / p.tile * 2;
    return p;
}

int launch_int8_product(Int8Mode mode, const Int8Plan &p, const Int8Args &a, hipStream_t s) {
    if (p.tile == 256) launch_tiles<256, 256, 2, 2>(mode, a, s);
    if (p.tile == 128) launch_tiles<128, 128, 2, 2>(mode, a, s);
    if (p.tile == 64) launch_tiles<64, 128, 2, 2>(mode, a, s);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

}  // namespace entq
