// entq_moe.hip -- a mixture-of-experts layer on int8 codes for few tokens
// (entq_moe_few): router, choice, the experts' gated products, their down
// products and the weighted sum.
#include <algorithm>

#include "entq_piece.h"

namespace entq {
namespace {

constexpr int kWavesMoe = 8;
constexpr uint32_t kTokens = ENTQ_MOE_MAX_TOKENS, kMaxExperts = ENTQ_MOE_MAX_EXPERTS;

struct MoeArgs {
    const void *x, *router;
    uint64_t ldx, ldr;
    int x_type, router_type;
    uint32_t M, E, K, D, F, N;     // tokens, experts, chosen, width, hidden, results
    int act;
    bool normalize;
    const int8_t *w[3];            // gate, up, down of expert 0
    const float *sw[3];
    uint64_t ldw[3], stride[3], sstride[3];
    // the workspace
    int8_t *codes;                 // [M][ldc] of x
    float *sx;                     // [M]
    double *logits;                // [M][E]
    int32_t *place;                // [E][M]: which of its token's choices the expert is, -1: none
    float *share;                  // [E][M]
    float *h;                      // [M K][F]
    int8_t *hcodes;                // [M K][ldh]
    float *sh;                     // [M K]
    uint64_t ldc, ldh;
    // the results
    void *y;
    int y_type;
    uint64_t ldy;
    int32_t *experts;              // [M][K], or null
    float *weights;                // [M][K], or null
};

__device__ __forceinline__ float value(const void *p, int type, uint64_t at) {
    return type == ENTQ_F32 ? ((const float *)p)[at] : from16(((const uint16_t *)p)[at], type == ENTQ_F16);
}

// The router's logits, summed in 64 bits: which expert is chosen hangs on
// their order. One workgroup per expert and 8 tokens.
__global__ __launch_bounds__(256) void moe_route(MoeArgs a) {
    __shared__ double part[4][8];
    const uint32_t e = blockIdx.x, m0 = blockIdx.y * 8, lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    double sum[8] = {};
    for (uint32_t c = threadIdx.x; c < a.D; c += 256) {
        const double r = value(a.router, a.router_type, e * a.ldr + c);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
            if (m0 + i < a.M) sum[i] += r * (double)value(a.x, a.x_type, (m0 + i) * a.ldx + c);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        sum[i] = wave_sum(sum[i]);
        if (lane == 0) part[wave][i] = sum[i];
    }
    __syncthreads();
    if (threadIdx.x < 8 && m0 + threadIdx.x < a.M)
        a.logits[(uint64_t)(m0 + threadIdx.x) * a.E + e] =
            part[0][threadIdx.x] + part[1][threadIdx.x] + part[2][threadIdx.x] + part[3][threadIdx.x];
}

// A total order of the logits: a NaN above all.
__device__ __forceinline__ uint64_t order_of(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    if (v != v) return ~0ull;
    return b >> 63 ? ~b : b | 1ull << 63;
}

// A token's choices, one workgroup a token: an expert's place is the number
// of experts before it (greater logits, or equal ones of lower index).
__global__ __launch_bounds__(256) void moe_choose(MoeArgs a) {
    __shared__ uint64_t key[kMaxExperts];
    __shared__ double part[4];
    const uint32_t m = blockIdx.x, t = threadIdx.x;
    const double *l = a.logits + (uint64_t)m * a.E;
    const double mine = t < a.E ? l[t] : 0.0;
    if (t < a.E) key[t] = order_of(mine);
    __syncthreads();
    uint32_t before = 0;
    double most = -INFINITY;
    for (uint32_t i = 0; i < a.E; ++i) {
        if (t < a.E) before += key[i] > key[t] || (key[i] == key[t] && i < t);
        const double v = l[i];
        most = v > most || v != v ? v : most;
    }
    const bool in = t < a.E && before < a.K;
    const double p = t < a.E ? exp(mine - most) : 0.0;
    double s = wave_sum(in || !a.normalize ? p : 0.0);
    if (t % 64 == 0) part[t / 64] = s;
    __syncthreads();
    s = part[0] + part[1] + part[2] + part[3];
    if (t >= a.E) return;
    const float w = (float)(p / s);
    a.place[(uint64_t)t * a.M + m] = in ? (int32_t)before : -1;
    a.share[(uint64_t)t * a.M + m] = in ? w : 0.0f;
    if (!in) return;
    if (a.experts) a.experts[(uint64_t)m * a.K + before] = (int32_t)t;
    if (a.weights) a.weights[(uint64_t)m * a.K + before] = w;
}

// Codes k..k+15 (of a lane's row) of a block that may pass the row's end.
__device__ __forceinline__ v4i load_codes(const int8_t *row, uint32_t k, uint32_t K, bool whole) {
    return whole ? ((const any16 *)(row + k))->v : load16_any(row, k, K);
}

// h = act(x gate^T) (x up^T) for the tokens of one expert: a workgroup takes
// 16 of its channels, its waves blocks of 128 codes in turn. Every token has
// its column of the matrix instruction; those that did not choose the expert
// load nothing.
template <int MT>
__global__ __launch_bounds__(64 * kWavesMoe) void moe_gated(MoeArgs a) {
    __shared__ v4i sums[kWavesMoe][2 * MT][64];
    const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t e = blockIdx.y, n0 = blockIdx.x * 16, kc = lane / 16 * 32;
    int32_t place[MT];
    bool any = false;
#pragma unroll
    for (int g = 0; g < MT; ++g) {
        const uint32_t m = g * 16 + lane % 16;
        place[g] = m < a.M ? a.place[(uint64_t)e * a.M + m] : -1;
        any |= place[g] >= 0;
    }
    if (!__any(any)) return;
    const uint64_t row = min(n0 + lane % 16, a.F - 1);
    const int8_t *wg = a.w[0] + e * a.stride[0] + row * a.ldw[0], *wu = a.w[1] + e * a.stride[1] + row * a.ldw[1];
    v4i acc[2][MT] = {};
    const uint32_t blocks = (a.D + 127) / 128;
    for (uint32_t b = wave; b < blocks; b += kWavesMoe) {
        const bool whole = b * 128 + 128 <= a.D;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t k = b * 128 + kc + 16 * half;
            const v4i g0 = load_codes(wg, k, a.D, whole), u0 = load_codes(wu, k, a.D, whole);
#pragma unroll
            for (int g = 0; g < MT; ++g) {
                v4i xv = {0, 0, 0, 0};
                if (place[g] >= 0) xv = *(const v4i *)(a.codes + (g * 16 + lane % 16) * a.ldc + k);
                acc[0][g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(g0, xv, acc[0][g], 0, 0, 0);
                acc[1][g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(u0, xv, acc[1][g], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int g = 0; g < MT; ++g) sums[wave][t * MT + g][lane] = acc[t][g];
    __syncthreads();
    if (wave >= MT) return;
    v4i s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < kWavesMoe; ++v) {
        s0 += sums[v][wave][lane];
        s1 += sums[v][MT + wave][lane];
    }
    const uint32_t m = wave * 16 + lane % 16, n = n0 + lane / 16 * 4;
    const int32_t at = m < a.M ? a.place[(uint64_t)e * a.M + m] : -1;
    if (at < 0 || n >= a.F) return;
    const float sx = a.sx[m];
    float g[4], u[4], r[4], none[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = n + i < a.F;
        g[i] = ((float)s0[i] * sx) * (in ? a.sw[0][e * a.sstride[0] + n + i] : 0.0f);
        u[i] = ((float)s1[i] * sx) * (in ? a.sw[1][e * a.sstride[1] + n + i] : 0.0f);
    }
    activate4<false>(a.act, g, r, none);
    float *h = a.h + ((uint64_t)m * a.K + at) * a.F + n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < a.F) h[i] = r[i] * u[i];
}

// y = the sum over experts of share (h down^T): a workgroup takes 16 results
// of every token and goes over the experts in use in their order.
template <int MT>
__global__ __launch_bounds__(64 * kWavesMoe) void moe_down(MoeArgs a) {
    __shared__ v4f sums[kWavesMoe][MT][64];
    const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t n0 = blockIdx.x * 16, kc = lane / 16 * 32, n = n0 + lane / 16 * 4;
    const uint64_t row = min(n0 + lane % 16, a.N - 1);
    float total[MT][4] = {};
    const uint32_t blocks = (a.F + 127) / 128;
    for (uint32_t e = 0; e < a.E; ++e) {
        int32_t place[MT];
        bool any = false;
#pragma unroll
        for (int g = 0; g < MT; ++g) {
            const uint32_t m = g * 16 + lane % 16;
            place[g] = m < a.M ? a.place[(uint64_t)e * a.M + m] : -1;
            any |= place[g] >= 0;
        }
        if (!__any(any)) continue;
        const int8_t *w = a.w[2] + e * a.stride[2] + row * a.ldw[2];
        v4i acc[MT] = {};
        for (uint32_t b = wave; b < blocks; b += kWavesMoe) {
            const bool whole = b * 128 + 128 <= a.F;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t k = b * 128 + kc + 16 * half;
                const v4i wv = load_codes(w, k, a.F, whole);
#pragma unroll
                for (int g = 0; g < MT; ++g) {
                    v4i hv = {0, 0, 0, 0};
                    if (place[g] >= 0)
                        hv = *(const v4i *)(a.hcodes + ((uint64_t)(g * 16 + lane % 16) * a.K + place[g]) * a.ldh + k);
                    acc[g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, hv, acc[g], 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int g = 0; g < MT; ++g) {
            if (place[g] < 0) continue;
            const uint32_t m = g * 16 + lane % 16;
            const float f = a.share[(uint64_t)e * a.M + m] * a.sh[(uint64_t)m * a.K + place[g]];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                total[g][i] += (float)acc[g][i] * f * (n + i < a.N ? a.sw[2][e * a.sstride[2] + n + i] : 0.0f);
        }
    }
#pragma unroll
    for (int g = 0; g < MT; ++g) sums[wave][g][lane] = v4f{total[g][0], total[g][1], total[g][2], total[g][3]};
    __syncthreads();
    if (wave >= MT) return;
    v4f s = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < kWavesMoe; ++v) s += sums[v][wave][lane];
    const uint32_t m = wave * 16 + lane % 16;
    if (m >= a.M) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i >= a.N) continue;
        const uint64_t at = m * a.ldy + n + i;
        if (a.y_type == ENTQ_F32)
            ((float *)a.y)[at] = s[i];
        else
            ((uint16_t *)a.y)[at] = bits16(s[i], a.y_type == ENTQ_F16);
    }
}

template <int MT>
void launch_products(const MoeArgs &a, hipStream_t s) {
    moe_gated<MT><<<dim3((a.F + 15) / 16, a.E), 64 * kWavesMoe, 0, s>>>(a);
    quantize_padded({a.h, a.F, nullptr, a.M * a.K, a.F, ENTQ_F32, 0}, a.hcodes, a.ldh, a.sh, s);
    moe_down<MT><<<(a.N + 15) / 16, 64 * kWavesMoe, 0, s>>>(a);
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
    take(a.codes, M * a.ldc);
    take(a.sx, M);
    take(a.logits, M * e.experts);
    take(a.place, M * e.experts);
    take(a.share, M * e.experts);
    take(a.h, rows * e.hidden);
    take(a.hcodes, rows * a.ldh);
    take(a.sh, rows);
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
    a.x_type = x->type;
    a.router = e->d_router;
    a.ldr = e->ldrouter;
    a.router_type = e->router_type;
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
    if ((st = quantize_padded(*x, a.codes, a.ldc, a.sx, s)) != ENTQ_OK) return st;
    moe_route<<<dim3(a.E, (a.M + 7) / 8), 256, 0, s>>>(a);
    moe_choose<<<a.M, 256, 0, s>>>(a);
    const uint32_t groups = (a.M + 15) / 16;
    if (groups == 1) launch_products<1>(a, s);
    if (groups == 2) launch_products<2>(a, s);
    if (groups > 2) launch_products<4>(a, s);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

}  // extern "C"
