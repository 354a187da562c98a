// entq_moe.hip -- a mixture-of-experts layer on int8 codes for few tokens
// (entq_moe_few): router, choice, the experts' gated products, their down
// products and the weighted sum.
#include <algorithm>

#include "entq_piece.h"

namespace entq {
namespace {

constexpr uint32_t kTokens = ENTQ_MOE_MAX_TOKENS, kMaxExperts = ENTQ_MOE_MAX_EXPERTS;

struct MoeArgs {
    const void *x, *router;
    uint64_t ldx, ldr;
    uint32_t M, E, K, D, F, N;     // tokens, experts, chosen, width, hidden, results
    int act;
    bool normalize;
    const int8_t *w[3];            // gate, up, down of expert 0
    const float *sw[3];
    uint64_t ldw[3], stride[3], sstride[3];
    // the workspace
    uint64_t *tokens;              // [E]: a bit for each token that chose the expert
    int8_t *codes;                 // [M][ldc] of x
    float *sx;                     // [M]
    double *logits;                // [M][E]
    int8_t *place;                 // [E][M]: which of its token's choices the expert is, -1: none
    uint16_t *chosen;              // [M K]: a choice's expert
    float *share;                  // [M K]: the token's weight for its choice
    float *h;                      // [M K][F]
    int8_t *hcodes;                // [M K][ldh]
    float *factor;                 // [M K]: share times the scale of the codes
    uint64_t ldc, ldh;
    uint16_t *jobs;                // [most jobs][2 + columns]: expert, tokens, their rows
    uint32_t *count;               // of jobs
    uint32_t most;                 // of jobs there can be
    float *part;                   // [splits][M][N rounded up to 4]: sums of a part of the list
    uint32_t splits;
    // the results
    void *y;
    int y_type;
    uint64_t ldy;
    int32_t *experts;              // [M][K], or null
    float *weights;                // [M][K], or null
};

// Values c..c+7 of a row of n values of any type, zeros past its end.
template <int TYPE>
__device__ __forceinline__ void load8(const void *row, uint32_t c, uint32_t n, float (&f)[8]) {
#pragma unroll
    for (int h = 0; h < 8 / kPer<TYPE>; ++h) {
        const v4i v = load_piece<TYPE>(row, c / kPer<TYPE> + h, n);
#pragma unroll
        for (int i = 0; i < kPer<TYPE>; ++i) f[h * kPer<TYPE> + i] = act_of<TYPE>(v, i);
    }
}

// Rows of codes as the products read them: in segments of 16, padded with
// zeros to blocks of 128. Where a row of n codes ends inside a segment, that
// segment holds its last 16 codes instead, zeros for those of the segment
// before: then every lane can read 16 of a weight row's codes, from column
// min(segment, n - 16), without a branch and within the row. (Rows of fewer
// than 16 codes: one segment, read by load16_any.)
//
// 8 codes of such a row, from position `at` (a multiple of 8).
template <int TYPE>
__device__ __forceinline__ v2i segment_codes(const Quantizer &z, const void *row, uint32_t at, uint32_t n) {
    float f[8];
    const uint32_t segment = at / 16 * 16;
    if (segment + 16 <= n || n < 16 || segment >= n) {
        load8<TYPE>(row, at, n, f);
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            const uint32_t c = n - 16 + at % 16 + i;
            f[i] = c >= segment ? load_act<TYPE>(row, c) : 0.0f;
        }
    }
    uint32_t q[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i / 4] |= z.code(f[i]) << (8 * (i % 4));
    return v2i{(int)q[0], (int)q[1]};
}

// The codes and the scale of one row (the values of entq_quantize_rows); one
// workgroup.
template <int TYPE, int THREADS>
__device__ __forceinline__ float quantize_segments(const void *x, uint32_t n, int8_t *codes, uint32_t ldc) {
    __shared__ uint32_t top[THREADS / 64];
    uint32_t big = 0;
    for (uint32_t c = threadIdx.x * 8; c < n; c += THREADS * 8) {
        float f[8];
        load8<TYPE>(x, c, n, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) big = max(big, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    }
    big = greatest(big);
    if (threadIdx.x % 64 == 0) top[threadIdx.x / 64] = big;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) big = max(big, top[i]);
    const Quantizer z(big);
    for (uint32_t c = threadIdx.x * 8; c < ldc; c += THREADS * 8) *(v2i *)(codes + c) = segment_codes<TYPE>(z, x, c, n);
    return z.scale;
}

// Codes of segment k of a weight row of n codes (TINY: of fewer than 16).
template <bool TINY>
__device__ __forceinline__ v4i weight_segment(const int8_t *row, uint32_t k, uint32_t n) {
    if (TINY) return load16_any(row, k, n);
    return ((const any16 *)(row + min(k, n - 16)))->v;
}

// The router's logits, summed in 64 bits: which expert is chosen hangs on
// their order. A workgroup takes one expert and up to 8 tokens; those after
// them quantise a token each.
// (The router's type is a template's and not the loop's to look at: with the
// three loads of it in one kernel the compiler shared a token's offset with
// them and left it unset on the way of the third.)
constexpr uint32_t kRouteTokens = 8, kRouteThreads = 512;
template <int TYPE, int ROUTER>
__global__ __launch_bounds__(kRouteThreads) void moe_route(MoeArgs a) {
    const uint32_t groups = (a.M + kRouteTokens - 1) / kRouteTokens;
    if (blockIdx.x >= a.E * groups) {
        const uint32_t m = blockIdx.x - a.E * groups;
        const float s = quantize_segments<TYPE, kRouteThreads>((const uint8_t *)a.x + m * a.ldx * (TYPE == ENTQ_F32 ? 4 : 2), a.D,
                                                     a.codes + m * a.ldc, (uint32_t)a.ldc);
        if (threadIdx.x == 0) a.sx[m] = s;
        return;
    }
    __shared__ double part[kRouteThreads / 64][kRouteTokens];
    const uint32_t e = blockIdx.x / groups, m0 = blockIdx.x % groups * kRouteTokens;
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    if (m0 == 0 && threadIdx.x == 0) a.tokens[e] = 0;  // for the choice that comes next
    double sum[kRouteTokens] = {};
    const uint32_t all = (a.D + 7) / 8;
    for (uint32_t g = threadIdx.x; g < all; g += kRouteThreads) {
        float r[8], x[kRouteTokens][8];
        load8<ROUTER>((const uint8_t *)a.router + e * a.ldr * (ROUTER == ENTQ_F32 ? 4 : 2), g * 8, a.D, r);
#pragma unroll
        for (uint32_t i = 0; i < kRouteTokens; ++i)
            if (m0 + i < a.M)
                load8<TYPE>((const uint8_t *)a.x + (m0 + i) * a.ldx * (TYPE == ENTQ_F32 ? 4 : 2), g * 8, a.D, x[i]);
#pragma unroll
        for (uint32_t i = 0; i < kRouteTokens; ++i)
            if (m0 + i < a.M) {
#pragma unroll
                for (int c = 0; c < 8; ++c) sum[i] += (double)r[c] * (double)x[i][c];
            }
    }
#pragma unroll
    for (uint32_t i = 0; i < kRouteTokens; ++i) {
        if (m0 + i >= a.M) continue;
        sum[i] = row16_sum(sum[i]);
        sum[i] += __shfl_xor(sum[i], 16);
        sum[i] += __shfl_xor(sum[i], 32);
        if (lane == 0) part[wave][i] = sum[i];
    }
    __syncthreads();
    if (threadIdx.x < kRouteTokens && m0 + threadIdx.x < a.M) {
        double s = 0.0;
#pragma unroll
        for (uint32_t w = 0; w < kRouteThreads / 64; ++w) s += part[w][threadIdx.x];
        a.logits[(uint64_t)(m0 + threadIdx.x) * a.E + e] = s;
    }
}

// A total order of the logits: a NaN above all.
__device__ __forceinline__ uint64_t order_of(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    if (v != v) return ~0ull;
    return b >> 63 ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ void write_choice(const MoeArgs &a, uint32_t m, uint32_t expert, uint32_t place, float w) {
    const uint32_t r = m * a.K + place;
    a.share[r] = w;
    a.chosen[r] = (uint16_t)expert;
    if (a.experts) a.experts[r] = (int32_t)expert;
    if (a.weights) a.weights[r] = w;
}

// A token's choices, one workgroup a token and one thread an expert: its place
// is the number of experts before it (greater logits, or equal ones of lower
// index).
__global__ __launch_bounds__(kMaxExperts) void moe_choose(MoeArgs a) {
    __shared__ __attribute__((aligned(16))) uint64_t key[kMaxExperts];
    __shared__ double part[kMaxExperts / 64], most;
    const uint32_t m = blockIdx.x, t = threadIdx.x;
    const double mine = t < a.E ? a.logits[(uint64_t)m * a.E + t] : 0.0;
    const uint64_t k = order_of(mine);
    key[t] = t < a.E ? k : 0;  // (below every logit's)
    __syncthreads();
    uint32_t before = 0;
    for (uint32_t i = 0; i < a.E; i += 8) {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
            const uint64_t other = key[i + j];
            before += other > k || (other == k && i + j < t);
        }
    }
    if (t < a.E && before == 0) most = mine;
    __syncthreads();
    const bool in = t < a.E && before < a.K;
    const double p = t < a.E && (in || !a.normalize) ? exp(mine - most) : 0.0;
    double s = wave_sum(p);
    if (t % 64 == 0) part[t / 64] = s;
    __syncthreads();
    s = 0.0;
    for (uint32_t i = 0; i < (a.E + 63) / 64; ++i) s += part[i];
    if (t >= a.E) return;
    a.place[(uint64_t)t * a.M + m] = in ? (int8_t)before : -1;
    if (!in) return;
    atomicOr((unsigned long long *)&a.tokens[t], 1ull << m);
    write_choice(a, m, t, before, (float)(p / s));
}

// The same for up to kFewTokens tokens and 64 experts, inside the products that
// follow: every workgroup of theirs chooses for itself, a wave a token and a
// lane an expert, which takes 1 to 2 us of them and saves 4.7 for the launch
// between (1 token 102.4 -> 99.9 us, 4 tokens 48.6 -> 46.2). The
// greatest logit in turn, by its fp32 value, which has the order of the
// 64-bit ones; only where two have one fp32 value do those decide.
constexpr uint32_t kFewTokens = 4, kFewExperts = 64;
struct Choice {
    uint64_t experts[kFewTokens];              // a bit for each of the token's
    int8_t place[kFewTokens][kFewExperts];
};
__device__ __forceinline__ void choose_few(const MoeArgs &a, uint32_t lane, uint32_t m, bool write, Choice &c) {
    const bool real = lane < a.E;
    const double mine = real ? a.logits[m * a.E + lane] : 0.0;
    const uint32_t b = __float_as_uint((float)mine);
    const uint32_t key = !real ? 0 : mine != mine ? 0xFFFFFFFFu : b >> 31 ? ~b : b | 1u << 31;
    const uint64_t k = order_of(mine);
    int place = -1;
    double most = 0.0;
    for (uint32_t i = 0; i < a.K; ++i) {
        const uint32_t top = greatest(place < 0 ? key : 0);
        uint64_t best = __ballot(real && place < 0 && key == top);
        uint32_t at = __builtin_ctzll(best);
        for (best &= best - 1; best; best &= best - 1) {
            const uint32_t j = __builtin_ctzll(best);
            if (__shfl(k, (int)j) > __shfl(k, (int)at)) at = j;
        }
        if (lane == at) place = (int)i;
        if (i == 0) most = __shfl(mine, (int)at);
    }
    const bool in = place >= 0;
    const uint64_t chosen = __ballot(in);
    if (lane == 0) c.experts[m] = chosen;
    c.place[m][lane] = (int8_t)place;
    if (!write) return;
    const double p = real && (in || !a.normalize) ? exp(mine - most) : 0.0;
    const double s = wave_sum(p);
    if (in) write_choice(a, m, lane, (uint32_t)place, (float)(p / s));
}

// The products go by jobs: an expert and up to COLS of its tokens, in their
// order, each a column of the matrix instructions. (Most experts of a batch
// have a few of its tokens: with a column for every token the codes of x and h
// were two thirds of all loads, and 48 tokens took 428 us.)
//
// The jobs of the experts before each lane's (of 64 from e0), and their sum.
template <int COLS>
__device__ __forceinline__ uint32_t jobs_before(uint64_t tokens, uint32_t lane, uint32_t &all) {
    const uint32_t mine = ((uint32_t)__popcll(tokens) + COLS - 1) / COLS;
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const uint32_t v = (uint32_t)__shfl_up((int)sum, o);
        if (lane >= (uint32_t)o) sum += v;
    }
    all = (uint32_t)__shfl((int)sum, 63);
    return sum - mine;
}

struct Job {
    uint32_t expert;        // E: there is none
    uint32_t first;         // of the expert's tokens
    uint64_t tokens;        // of the expert
};
template <int COLS>
__device__ __forceinline__ Job nth_job(const MoeArgs &a, uint32_t nth, uint32_t lane) {
    for (uint32_t e = 0; e < a.E; e += 64) {
        const uint64_t tokens = e + lane < a.E ? a.tokens[e + lane] : 0;
        uint32_t all;
        const uint32_t before = jobs_before<COLS>(tokens, lane, all);
        if (nth < all) {
            const bool here = tokens && before <= nth && nth - before < ((uint32_t)__popcll(tokens) + COLS - 1) / COLS;
            const int at = __builtin_ctzll(__ballot(here));
            const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)tokens, at);
            const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(tokens >> 32), at);
            return {e + at, (nth - __builtin_amdgcn_readlane(before, at)) * COLS, (uint64_t)hi << 32 | lo};
        }
        nth -= all;
    }
    return {a.E, 0, 0};
}

// The nth expert of a choice for few tokens, which is a job.
__device__ __forceinline__ Job nth_job(const MoeArgs &a, uint32_t nth, uint32_t lane, const Choice &c) {
    uint64_t experts = 0;
    uint32_t tokens = 0;
    for (uint32_t m = 0; m < a.M; ++m) {
        const uint64_t of = c.experts[m];
        experts |= of;
        tokens |= (uint32_t)(of >> lane & 1) << m;
    }
    const uint32_t rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(experts >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)experts, 0));
    const uint64_t here = __ballot(tokens && rank == nth);
    if (!here) return {a.E, 0, 0};
    const uint32_t e = __builtin_ctzll(here);
    return {e, 0, (uint32_t)__builtin_amdgcn_readlane(tokens, e)};
}

// The token at a place of the set (its last one for places beyond).
__device__ __forceinline__ uint32_t token_at(uint64_t tokens, uint32_t place, uint32_t lane) {
    const uint32_t n = (uint32_t)__popcll(tokens);
    const uint32_t rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(tokens >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)tokens, 0));
    // lane r gets the rth token (the others' lanes are past the last one)
    const uint32_t to = tokens >> lane & 1 ? rank : n + (lane - rank);
    const int mine = __builtin_amdgcn_ds_permute((int)(to * 4), (int)lane);
    return (uint32_t)__shfl(mine, (int)min(place, n - 1));
}

// h = act(x gate^T) (x up^T) for a job: a workgroup takes 16 of the expert's
// channels, its waves blocks of 128 codes in turn, some of them on their way.
// Columns beyond the job's tokens read with its last one (the same cache
// lines, and no branch, so that no load waits for another); their sums go
// nowhere. WIDE, for more than 16 columns: each wave has 16 channels of its own
// and takes all blocks, so that a workgroup's way to its job is paid once for
// four times the channels, and its waves read the same codes of x.
// Bound by memory: one token, 2 experts of 5120 x 13824, in 57 us (5.0 TB/s), 48
// tokens, 64 experts of 5120 x 1728, 231 us (4.9 TB/s); with more columns an
// expert by the waits of a wave's blocks for each other (64 tokens, 4 experts of
// 4096 x 8192: 81 us, 3.3 TB/s).
template <int MT, int WAVES, bool TINY, bool FEW, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void moe_gated(MoeArgs a) {
    constexpr int kDepth = MT > 1 ? 2 : 4, kCols = 16 * MT, kSteps = WIDE ? 1 : WAVES;
    __shared__ v4i sums[WIDE ? 1 : WAVES][2 * MT][64];
    __shared__ Choice choice;
    const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t n0 = WIDE ? (blockIdx.x * WAVES + wave) * 16 : blockIdx.x * 16, kc = lane / 16 * 32;
    Job job;
    if constexpr (FEW) {
        static_assert(!FEW || WAVES == kFewTokens, "a wave for each token");
        const bool first = blockIdx.x == 0 && blockIdx.y == 0;
        if (wave < a.M) choose_few(a, lane, wave, first, choice);
        __syncthreads();
        if (first && wave == 0 && lane < a.E) {
            uint64_t tokens = 0;
            for (uint32_t m = 0; m < a.M; ++m) tokens |= (choice.experts[m] >> lane & 1) << m;
            a.tokens[lane] = tokens;
        }
        job = nth_job(a, blockIdx.y, lane, choice);
    } else {
        job = nth_job<kCols>(a, blockIdx.y, lane);
    }
    const uint32_t e = job.expert;
    if (e >= a.E || (WIDE && n0 >= a.F)) return;
    uint32_t x[MT], token[MT];
#pragma unroll
    for (int g = 0; g < MT; ++g) {
        token[g] = token_at(job.tokens, job.first + g * 16 + lane % 16, lane);
        x[g] = (uint32_t)(token[g] * a.ldc) + kc;
    }
    const uint64_t row = min(n0 + lane % 16, a.F - 1);
    const int8_t *w[2] = {a.w[0] + e * a.stride[0] + row * a.ldw[0], a.w[1] + e * a.stride[1] + row * a.ldw[1]};
    v4i acc[2][MT] = {};
    struct Block {
        v4i w[2][2], x[MT][2];
    };
    const uint32_t blocks = (a.D + 127) / 128, first = WIDE ? 0 : wave,
                   mine = blocks > first ? (blocks - first + kSteps - 1) / kSteps : 0;
    auto load = [&](Block &b, uint32_t i) {
        const uint32_t k = (i * kSteps + first) * 128;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int t = 0; t < 2; ++t) b.w[t][half] = weight_segment<TINY>(w[t], k + kc + 16 * half, a.D);
#pragma unroll
            for (int g = 0; g < MT; ++g) b.x[g][half] = *(const v4i *)(a.codes + (x[g] + k + 16 * half));
        }
    };
    auto multiply = [&](const Block &b) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int g = 0; g < MT; ++g)
                    acc[t][g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b.w[t][half], b.x[g][half], acc[t][g], 0, 0, 0);
    };
    Block b[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        if ((uint32_t)d < mine) load(b[d], d);
    uint32_t i = 0;
    for (; i + 2 * kDepth <= mine; i += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            multiply(b[d]);
            load(b[d], i + d + kDepth);
        }
    }
    for (; i < mine; i += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            if (i + d < mine) multiply(b[d]);
            if (i + d + kDepth < mine) load(b[d], i + d + kDepth);
        }
    }
    // 16 channels of 16 columns: their hidden values
    const uint32_t n = n0 + lane / 16 * 4;
    auto finish = [&](v4i s0, v4i s1, uint32_t group, uint32_t m) {
        if (job.first + group * 16 + lane % 16 >= (uint32_t)__popcll(job.tokens) || n >= a.F) return;
        const int32_t place = FEW ? choice.place[m][e] : a.place[(uint64_t)e * a.M + m];
        const float sx = a.sx[m];
        float g[4], u[4], r[4], none[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool there = n + i < a.F;
            g[i] = ((float)s0[i] * sx) * (there ? a.sw[0][e * a.sstride[0] + n + i] : 0.0f);
            u[i] = ((float)s1[i] * sx) * (there ? a.sw[1][e * a.sstride[1] + n + i] : 0.0f);
        }
        activate4<false>(a.act, g, r, none);
        float *h = a.h + ((uint64_t)m * a.K + place) * a.F + n;
        if (n + 4 <= a.F) {
            ((any16 *)h)->v = __builtin_bit_cast(v4i, v4f{r[0] * u[0], r[1] * u[1], r[2] * u[2], r[3] * u[3]});
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (n + i < a.F) h[i] = r[i] * u[i];
        }
    };
    if constexpr (WIDE) {
#pragma unroll
        for (int g = 0; g < MT; ++g) finish(acc[0][g], acc[1][g], g, token[g]);
    } else {
        static_assert(WAVES >= MT, "a wave for each 16 columns at the end");
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int g = 0; g < MT; ++g) sums[wave][t * MT + g][lane] = acc[t][g];
        __syncthreads();
        if (wave >= MT) return;
        v4i s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < WAVES; ++v) {
            s0 += sums[v][wave][lane];
            s1 += sums[v][MT + wave][lane];
        }
        uint32_t m = token[0];
#pragma unroll
        for (int g = 1; g < MT; ++g) m = wave == (uint32_t)g ? token[g] : m;
        finish(s0, s1, wave, m);
    }
}

// The hidden values' codes, and what a row's products are scaled with: its
// scale times the token's weight for the expert. Each row also enters itself
// into its job.
template <int COLS>
__global__ __launch_bounds__(1024) void moe_quantize(MoeArgs a) {
    const uint32_t r = blockIdx.x;
    const float s = quantize_segments<ENTQ_F32, 1024>(a.h + (uint64_t)r * a.F, a.F, a.hcodes + r * a.ldh, (uint32_t)a.ldh);
    if (threadIdx.x == 0) a.factor[r] = a.share[r] * s;
    if (threadIdx.x >= 64) return;
    const uint32_t lane = threadIdx.x, expert = a.chosen[r], m = r / a.K;
    uint32_t base = 0, job = 0;
    for (uint32_t e = 0; e < a.E; e += 64) {
        const uint64_t tokens = e + lane < a.E ? a.tokens[e + lane] : 0;
        uint32_t all;
        const uint32_t before = jobs_before<COLS>(tokens, lane, all);
        if (expert - e < 64) job = base + (uint32_t)__shfl((int)before, (int)(expert - e));
        base += all;
    }
    if (lane) return;
    if (r == 0) *a.count = base;
    const uint64_t tokens = a.tokens[expert];
    const uint32_t place = (uint32_t)__popcll(tokens & ((1ull << m) - 1)), n = (uint32_t)__popcll(tokens);
    uint16_t *entry = a.jobs + (job + place / COLS) * (2 + COLS);
    entry[2 + place % COLS] = (uint16_t)r;
    if (place % COLS == 0) {
        entry[0] = (uint16_t)expert;
        entry[1] = (uint16_t)min((uint32_t)COLS, n - place);
    }
}

// Results n..n+3 of token m.
__device__ __forceinline__ void store_result(const MoeArgs &a, uint32_t m, uint32_t n, v4f s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i >= a.N) continue;
        const uint64_t to = m * a.ldy + n + i;
        if (a.y_type == ENTQ_F32)
            ((float *)a.y)[to] = s[i];
        else
            ((uint16_t *)a.y)[to] = bits16(s[i], a.y_type == ENTQ_F16);
    }
}

// y = the sum over experts of share (h down^T): a workgroup takes 16 results
// of every token, and its part of a list of the blocks of 128 codes of all
// jobs, which its waves take in turn, so that the next job's codes are on their
// way while one's are multiplied; at a job's end a wave scales its integer sums
// and adds them to its tokens' fp32 sums in LDS. The list is split over
// workgroups (blockIdx.y), so that there are some for every CU, and moe_join
// adds the parts up. (Left to the workgroup that ends last it took 297 .. 583
// us where all of one token took 107: the fences that order it write back an
// XCD's whole L2.)
constexpr uint32_t kMostJobs = 64;  // of a part of the list
template <int MT, int WAVES, bool TINY>
__global__ __launch_bounds__(64 * WAVES) void moe_down(MoeArgs a) {
    constexpr int kDepth = MT > 1 ? 2 : 4, kCols = 16 * MT;
    extern __shared__ __attribute__((aligned(16))) uint8_t room[];
    const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), t = threadIdx.x;
    const uint32_t n0 = blockIdx.x * 16, kc = lane / 16 * 32;
    const uint32_t count = *a.count, blocks = (a.F + 127) / 128;
    // this workgroup's items of the list, and their jobs
    const uint32_t items = count * blocks, end = (uint32_t)((uint64_t)items * (blockIdx.y + 1) / a.splits);
    uint32_t item = (uint32_t)((uint64_t)items * blockIdx.y / a.splits);
    const uint32_t job0 = item / blocks, n_jobs = (end + blocks - 1) / blocks - job0;
    float *const sums = (float *)room;                              // [WAVES][M][16]
    float *const scale = sums + WAVES * a.M * 16;                   // [jobs][16]
    float *const factor = scale + kMostJobs * 16;                   // [jobs][columns]; 0 beyond the tokens
    uint16_t *const rows = (uint16_t *)(factor + kMostJobs * kCols);  // [jobs][columns]
    uint16_t *const expert = rows + kMostJobs * kCols;              // [jobs]
    for (uint32_t i = t; i < WAVES * a.M * 16; i += 64 * WAVES) sums[i] = 0.0f;
    for (uint32_t i = t; i < n_jobs * kCols; i += 64 * WAVES) {
        const uint16_t *entry = a.jobs + (job0 + i / kCols) * (2 + kCols);
        const uint32_t c = i % kCols, tokens = entry[1];
        rows[i] = entry[2 + min(c, tokens - 1)];
        factor[i] = c < tokens ? a.factor[rows[i]] : 0.0f;
        if (c == 0) expert[i / kCols] = entry[0];
    }
    for (uint32_t i = t; i < n_jobs * 16; i += 64 * WAVES) {
        const uint32_t e = a.jobs[(job0 + i / 16) * (2 + kCols)];
        scale[i] = n0 + i % 16 < a.N ? a.sw[2][e * a.sstride[2] + n0 + i % 16] : 0.0f;
    }
    __syncthreads();
    const uint64_t row = min(n0 + lane % 16, a.N - 1) * a.ldw[2];
    const uint32_t step_j = WAVES / blocks, step_b = WAVES % blocks;
    struct Block {
        v4i w[2], x[MT][2];
        uint32_t job;
    };
    item += wave;
    uint32_t job = item / blocks - job0, block = item % blocks;  // the next to load
    auto load = [&](Block &b) {
        b.job = job;
        const uint32_t e = __builtin_amdgcn_readfirstlane(expert[job]), k = block * 128 + kc;
        const int8_t *w = a.w[2] + e * a.stride[2] + row;
#pragma unroll
        for (int half = 0; half < 2; ++half) b.w[half] = weight_segment<TINY>(w, k + 16 * half, a.F);
#pragma unroll
        for (int g = 0; g < MT; ++g) {
            const int8_t *x = a.hcodes + rows[job * kCols + g * 16 + lane % 16] * a.ldh + k;
#pragma unroll
            for (int half = 0; half < 2; ++half) b.x[g][half] = *(const v4i *)(x + 16 * half);
        }
        item += WAVES;
        block += step_b;
        job += step_j;
        if (block >= blocks) {
            block -= blocks;
            ++job;
        }
    };
    v4i acc[MT] = {};
    auto finish = [&](uint32_t done) {
        const v4f s = *(const v4f *)(scale + done * 16 + lane / 16 * 4);
#pragma unroll
        for (int g = 0; g < MT; ++g) {
            const uint32_t c = done * kCols + g * 16 + lane % 16;
            const float f = factor[c];
            const bool last = g * 16 + lane % 16 > 0 && rows[c] == rows[c - 1];  // (beyond the tokens)
            if (!last) {
                v4f *to = (v4f *)(sums + (wave * a.M + rows[c] / a.K) * 16 + lane / 16 * 4);
                *to += v4f{(float)acc[g][0] * f * s[0], (float)acc[g][1] * f * s[1], (float)acc[g][2] * f * s[2],
                           (float)acc[g][3] * f * s[3]};
            }
            acc[g] = v4i{0, 0, 0, 0};
        }
    };
    Block b[kDepth];
    constexpr uint32_t kNone = 0xFFFFFFFFu;
    uint32_t current = item < end ? job : kNone;
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
        b[d].job = kNone;
        if (item < end) load(b[d]);
    }
    while (b[0].job != kNone) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            if (b[d].job == kNone) continue;
            if (b[d].job != current) {
                finish(current);
                current = b[d].job;
            }
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int g = 0; g < MT; ++g)
                    acc[g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[d].w[half], b[d].x[g][half], acc[g], 0, 0, 0);
            b[d].job = kNone;
            if (item < end) load(b[d]);
        }
    }
    if (current != kNone) finish(current);
    __syncthreads();
    for (uint32_t i = t; i < a.M * 4; i += 64 * WAVES) {
        v4f s = {0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < WAVES; ++v) s += *(const v4f *)(sums + (v * a.M * 4 + i) * 4);
        const uint32_t m = i / 4, at = n0 + i % 4 * 4;
        if (at >= a.N) continue;
        if (a.splits > 1)
            *(v4f *)(a.part + ((uint64_t)blockIdx.y * a.M + m) * ((a.N + 3) / 4 * 4) + at) = s;
        else
            store_result(a, m, at, s);
    }
}

// The results out of the parts' sums, in the order of the parts; four a thread.
__global__ __launch_bounds__(256) void moe_join(MoeArgs a) {
    const uint32_t n = 4 * (blockIdx.x * 256 + threadIdx.x), m = blockIdx.y;
    if (n >= a.N) return;
    const uint64_t step = (uint64_t)a.M * ((a.N + 3) / 4 * 4);
    const float *p = a.part + (uint64_t)m * ((a.N + 3) / 4 * 4) + n;
    v4f s = {0, 0, 0, 0};
#pragma unroll 4
    for (uint32_t i = 0; i < a.splits; ++i) s += *(const v4f *)(p + i * step);
    store_result(a, m, n, s);
}

// Parts of the list of blocks: some 5 workgroups for each of 256 CUs, and the
// jobs of a part (one more than its share, where it begins inside one) in LDS.
uint32_t splits_of(uint32_t results, uint32_t most) {
    const uint32_t fill = std::min(8u, 1280 / ((results + 15) / 16));
    return std::max(std::max(1u, fill), (most + kMostJobs - 3) / (kMostJobs - 2));
}

// Columns of a job: as many as the experts have tokens on average, times two.
// With 16, 32 and 64 of them, us: 8 tokens an expert (32 tokens, 2 of 8, 4096 x
// 8192) 180, 197, 219; 16 (64 tokens) 245, 217, 236; 32 (64 tokens, 2 of 4) 205,
// 174, 156; between the steps the choice is 5 % off at most (24 an expert, 48
// tokens, 2 of 4, 4096 x 4096: 104, 87, 91).
uint32_t columns_of(uint32_t tokens, uint32_t top_k, uint32_t experts) {
    const uint32_t average = tokens * top_k / experts;
    return tokens <= 16 || average <= 8 ? 16 : tokens <= 32 || average <= 16 ? 32 : 64;
}
uint32_t most_jobs(uint32_t tokens, uint32_t top_k, uint32_t experts, uint32_t columns) {
    const uint32_t rows = tokens * top_k;
    return std::min(rows, std::min(experts, rows) + rows / columns);
}

// Workgroups from which WIDE pays, 64 tokens, us with it and without: 8 experts of
// 4096 x 8192 215 and 224, 4096 x 4096 122 and 127, 4096 x 2048 (256 of them) 80.6
// and 80.8, 4 of 4096 x 1024 (64) 70 and 46.
constexpr uint32_t kWideGroups = 512;
template <int MT>
void launch_products(const MoeArgs &a, hipStream_t s) {
    constexpr int W = 4;
    const dim3 grid((a.F + 15) / 16, a.most), down((a.N + 15) / 16, a.splits);
    const bool few = a.M <= kFewTokens && a.E <= kFewExperts;
    if (!few) moe_choose<<<a.M, kMaxExperts, 0, s>>>(a);
    const dim3 wide((a.F + 16 * W - 1) / (16 * W), a.most);
    if (MT == 1 && few && a.D >= 16)
        moe_gated<1, W, false, true, false><<<grid, 64 * W, 0, s>>>(a);
    else if (MT == 1 && few)
        moe_gated<1, W, true, true, false><<<grid, 64 * W, 0, s>>>(a);
    else if (MT > 1 && a.D >= 16 && wide.x * std::min(a.E, a.most) >= kWideGroups)
        moe_gated<MT, W, false, false, (MT > 1)><<<wide, 64 * W, 0, s>>>(a);
    else if (a.D >= 16)
        moe_gated<MT, W, false, false, false><<<grid, 64 * W, 0, s>>>(a);
    else
        moe_gated<MT, W, true, false, false><<<grid, 64 * W, 0, s>>>(a);
    moe_quantize<16 * MT><<<a.M * a.K, 1024, 0, s>>>(a);
    const uint32_t lds = W * a.M * 64 + kMostJobs * (64 + 16 * MT * 6 + 2);
    if (a.F < 16)
        moe_down<MT, W, true><<<down, 64 * W, lds, s>>>(a);
    else
        moe_down<MT, W, false><<<down, 64 * W, lds, s>>>(a);
    if (a.splits > 1) moe_join<<<dim3((a.N + 1023) / 1024, a.M), 256, 0, s>>>(a);
}

uint32_t bytes_of(int t) { return t == ENTQ_F32 ? 4 : 2; }
bool float_type(int t) { return t == ENTQ_BF16 || t == ENTQ_F16 || t == ENTQ_F32; }

constexpr uint64_t kMostLd = 1ull << 40;

entq_status check(const entq_rows *x, const entq_experts *e) {
    if (!x || !e || x->reserved || e->reserved) return ENTQ_EINVAL;
    if (!float_type(x->type) || !float_type(e->router_type) || x->d_scales) return ENTQ_EINVAL;
    if (x->rows > kTokens || x->cols > ENTQ_INT8_MAX_COLS || x->ld < x->cols || x->ld > kMostLd) return ENTQ_EINVAL;
    if (!e->experts || e->experts > kMaxExperts || !e->top_k || e->top_k > e->experts ||
        e->top_k > ENTQ_MOE_MAX_TOP)
        return ENTQ_EINVAL;
    if (!x->cols || !e->hidden || !e->out || e->hidden > ENTQ_INT8_MAX_COLS || e->out > (1u << 22))
        return ENTQ_EINVAL;
    if (e->activation < ENTQ_ACT_SILU || e->activation > ENTQ_ACT_RELU || (e->normalize & ~1)) return ENTQ_EINVAL;
    if (e->ldrouter < x->cols || e->ldrouter > kMostLd || !e->d_router) return ENTQ_EINVAL;
    const uint64_t cols[3] = {x->cols, x->cols, e->hidden}, rows[3] = {e->hidden, e->hidden, e->out};
    for (int i = 0; i < 3; ++i) {
        if (!e->d_weights[i] || !e->d_scales[i] || e->ld[i] < cols[i] || e->ld[i] > kMostLd ||
            e->stride[i] > kMostLd || e->scale_stride[i] > kMostLd)
            return ENTQ_EINVAL;
        if (e->experts > 1 && (e->stride[i] < (rows[i] - 1) * e->ld[i] + cols[i] || e->scale_stride[i] < rows[i]))
            return ENTQ_EINVAL;
        if ((uintptr_t)e->d_scales[i] % 4) return ENTQ_EALIGN;
    }
    if (x->rows && !x->d_data) return ENTQ_EINVAL;
    if ((uintptr_t)x->d_data % bytes_of(x->type) || (uintptr_t)e->d_router % bytes_of(e->router_type))
        return ENTQ_EALIGN;
    return ENTQ_OK;
}

// The workspace in order; with base null it only counts.
uint64_t lay_out(const entq_rows &x, const entq_experts &e, uint8_t *base, MoeArgs &a) {
    uint64_t used = 0;
    const auto take = [&](auto *&p, uint64_t n) {
        p = base ? (std::remove_reference_t<decltype(p)>)(base + used) : nullptr;
        used += (n * sizeof(*p) + 255) / 256 * 256;
    };
    const uint64_t M = x.rows, rows = M * e.top_k;
    a.ldc = (x.cols + 127ull) / 128 * 128;
    a.ldh = (e.hidden + 127ull) / 128 * 128;
    take(a.tokens, e.experts);
    take(a.codes, M * a.ldc);
    take(a.sx, M);
    take(a.logits, M * e.experts);
    take(a.place, M * e.experts);
    take(a.chosen, rows);
    take(a.share, rows);
    take(a.h, rows * e.hidden);
    take(a.hcodes, rows * a.ldh);
    take(a.factor, rows);
    const uint32_t columns = columns_of(x.rows, e.top_k, e.experts);
    a.most = most_jobs(x.rows, e.top_k, e.experts, columns);
    a.splits = splits_of(e.out, a.most);
    take(a.jobs, a.most * (2 + columns));
    take(a.count, 1);
    take(a.part, a.splits > 1 ? a.splits * M * ((e.out + 3) / 4 * 4) : 0);
    return used;
}

}  // namespace
}  // namespace entq

using namespace entq;

extern "C" {

uint64_t entq_moe_few_workspace_bytes(const entq_rows *x, const entq_experts *e) {
    MoeArgs a{};
    return check(x, e) == ENTQ_OK ? lay_out(*x, *e, nullptr, a) : 0;
}

entq_status entq_moe_few(const entq_rows *x, const entq_experts *e, void *d_y, int y_type, uint64_t ldy,
                         int32_t *d_experts, float *d_weights, void *d_workspace, uint64_t workspace_bytes,
                         void *stream) {
    entq_status st = check(x, e);
    if (st != ENTQ_OK) return st;
    if (!float_type(y_type) || ldy < e->out || ldy > kMostLd || (x->rows && !d_y)) return ENTQ_EINVAL;
    if ((uintptr_t)d_y % bytes_of(y_type) || (uintptr_t)d_experts % 4 || (uintptr_t)d_weights % 4) return ENTQ_EALIGN;
    if (!x->rows) return ENTQ_OK;
    MoeArgs a{};
    if (!d_workspace || workspace_bytes < lay_out(*x, *e, nullptr, a)) return ENTQ_EWORKSPACE;
    if ((uintptr_t)d_workspace % 256) return ENTQ_EALIGN;
    lay_out(*x, *e, (uint8_t *)d_workspace, a);
    a.x = x->d_data;
    a.ldx = x->ld;
    a.router = e->d_router;
    a.ldr = e->ldrouter;
    a.M = x->rows;
    a.E = e->experts;
    a.K = e->top_k;
    a.D = x->cols;
    a.F = e->hidden;
    a.N = e->out;
    a.act = e->activation;
    a.normalize = e->normalize;
    for (int i = 0; i < 3; ++i) {
        a.w[i] = e->d_weights[i];
        a.sw[i] = e->d_scales[i];
        a.ldw[i] = e->ld[i];
        a.stride[i] = e->stride[i];
        a.sstride[i] = e->scale_stride[i];
    }
    a.y = d_y;
    a.y_type = y_type;
    a.ldy = ldy;
    a.experts = d_experts;
    a.weights = d_weights;
    const hipStream_t s = (hipStream_t)stream;
    const uint32_t route = a.E * ((a.M + kRouteTokens - 1) / kRouteTokens) + a.M;
    const auto go = [&](auto type) {
        constexpr int T = decltype(type)::value;
        if (e->router_type == ENTQ_BF16) moe_route<T, ENTQ_BF16><<<route, kRouteThreads, 0, s>>>(a);
        if (e->router_type == ENTQ_F16) moe_route<T, ENTQ_F16><<<route, kRouteThreads, 0, s>>>(a);
        if (e->router_type == ENTQ_F32) moe_route<T, ENTQ_F32><<<route, kRouteThreads, 0, s>>>(a);
    };
    if (x->type == ENTQ_BF16) go(std::integral_constant<int, ENTQ_BF16>());
    if (x->type == ENTQ_F16) go(std::integral_constant<int, ENTQ_F16>());
    if (x->type == ENTQ_F32) go(std::integral_constant<int, ENTQ_F32>());
    const uint32_t columns = columns_of(a.M, a.K, a.E);
    if (columns == 16) launch_products<1>(a, s);
    if (columns == 32) launch_products<2>(a, s);
    if (columns == 64) launch_products<4>(a, s);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

}  // extern "C"
