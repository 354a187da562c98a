// entq_distill.hip -- the distillation loss from a teacher's top logits, and
// the gradient of the student's logits (entq_distill_loss, _backward).
#include <algorithm>
#include <cmath>

#include "entq_piece.h"

namespace entq {
namespace {

// With z = logits / T, L = log sum_v exp z_v and the teacher's p over its top
// entries (their softmax; or, with the log-sum lse over all its classes, p_j =
// exp(t_j / T - lse), the rest pt = max(0, 1 - sum p) being the tail's):
//   loss = sum_j p_j (log p_j - z_j + L)  [+ pt (log pt - Lt + L)]
//   dL/dz_v = q_v - sum_{j of v} p_j,   q_v = exp(z_v - L)
// Lt is the log-sum over the classes outside the top entries, whose gradient
// with a tail is q_v - pt exp(z_v - Lt) = exp(z_v - Lt) (qt - pt), qt = exp(Lt
// - L). Lt comes from a sum over those classes alone (a bit for each class
// marks the others): L minus the top entries would lose it to cancellation
// where the student is sure.
struct DistillArgs {
    const void *logits, *teacher, *index;
    const float *lse, *weight, *dloss;
    float *loss;            // or null
    void *dlogits;          // or null
    uint64_t ld, ldt, ldi, ldd;
    uint32_t M, V, K;
    int teacher_type;
    bool wide;              // 64-bit indices
    float scale;            // log2(e) / T: logits times it are exponents of 2
    double inv_t;           // 1 / T
};

constexpr uint32_t kMaxTop = ENTQ_DISTILL_MAX_TOP;

__device__ __forceinline__ float read_teacher(const DistillArgs &a, uint64_t at) {
    return a.teacher_type == ENTQ_F32 ? ((const float *)a.teacher)[at]
                                      : from16(((const uint16_t *)a.teacher)[at], a.teacher_type == ENTQ_F16);
}

__device__ __forceinline__ float wave_maxf(float v) {
#pragma unroll
    for (int o = 32; o; o /= 2) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ float wave_sumf(float v) {
#pragma unroll
    for (int o = 32; o; o /= 2) v += __shfl_xor(v, o);
    return v;
}

// One workgroup per token, which reads the row twice (three times with the
// gradient), the second time out of the L2.
template <int TYPE, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void distill_rows(DistillArgs a, uint32_t row0) {
    constexpr int kP = kPer<TYPE>, kThreads = 64 * WAVES;
    extern __shared__ uint32_t marks[];  // with a tail: a bit for each class of the top entries
    __shared__ float part[WAVES], part2[WAVES];
    __shared__ int32_t where[kMaxTop];   // an entry's class, -1: none
    __shared__ float mass[kMaxTop];      // the teacher's p of it
    __shared__ float common[2];
    __shared__ double log_sum;
    const uint64_t m = (uint64_t)row0 + blockIdx.x;
    const uint32_t t = threadIdx.x, lane = t % 64, wave = t / 64;
    const uint32_t pieces = (a.V + kP - 1) / kP;
    const uint8_t *row = (const uint8_t *)a.logits + m * a.ld * (TYPE == ENTQ_F32 ? 4 : 2);
    uint8_t *grad = (uint8_t *)a.dlogits + m * a.ldd * (TYPE == ENTQ_F32 ? 4 : 2);
    const float weight = a.weight ? a.weight[m] : 1.0f;
    if (weight == 0.0f) {  // whatever the row holds
        if (a.loss && t == 0) a.loss[m] = 0.0f;
        if (a.dlogits)
            for (uint32_t p = t; p < pieces; p += kThreads) store_piece<TYPE>(grad, p, a.V, v4i{0, 0, 0, 0});
        return;
    }
    const bool tail = a.lse != nullptr;
    if (tail) {
        for (uint32_t i = t; i < (a.V + 31) / 32; i += kThreads) marks[i] = 0;
        __syncthreads();
    }
    bool bad = false;  // an index beyond the classes
    for (uint32_t j = t; j < a.K; j += kThreads) {
        const int64_t i = a.wide ? ((const int64_t *)a.index)[m * a.ldi + j] : ((const int32_t *)a.index)[m * a.ldi + j];
        bad |= i >= (int64_t)a.V;
        const bool in = i >= 0 && i < (int64_t)a.V;
        where[j] = in ? (int32_t)i : -1;
        if (tail && in) atomicOr(&marks[(uint32_t)i / 32], 1u << ((uint32_t)i % 32));
    }
    bad = __syncthreads_or(bad);
    auto marked = [&](uint32_t p) -> uint32_t {  // the piece's classes of the top entries
        if (!tail) return 0;
        const uint32_t c = p * kP;
        return (marks[c / 32] >> (c % 32)) & ((1u << kP) - 1);
    };
    // the largest logit outside the marked classes; exponents are differences
    // from it, which the logits' own sizes do not blur
    float top = -INFINITY;
    for (uint32_t p = t; p < pieces; p += kThreads) {
        const v4i v = load_piece<TYPE>(row, p, a.V);
        const uint32_t out = marked(p);
#pragma unroll
        for (int i = 0; i < kP; ++i)
            if (p * kP + i < a.V && !(out >> i & 1)) top = fmaxf(top, act_of<TYPE>(v, i));
    }
    top = wave_maxf(top);
    if (lane == 0) part[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = fmaxf(top, part[w]);
    const float from = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (uint32_t p = t; p < pieces; p += kThreads) {
        const v4i v = load_piece<TYPE>(row, p, a.V);
        const uint32_t out = marked(p);
#pragma unroll
        for (int i = 0; i < kP; ++i)
            if (p * kP + i < a.V && !(out >> i & 1)) sum += exp2f((act_of<TYPE>(v, i) - from) * a.scale);
    }
    sum = wave_sumf(sum);
    if (lane == 0) part2[wave] = sum;
    __syncthreads();
    // The few entries: one wave, in 64 bits, since the loss is a small difference of their terms.
    if (wave == 0) {
        double total = 0.0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) total += part2[w];
        const double lt = from * a.inv_t + log(total);  // outside the marks
        // the teacher's log-sum
        double most = -INFINITY, lse = 0.0;
        if (!tail) {
            for (uint32_t j = lane; j < a.K; j += 64)
                if (where[j] >= 0) {
                    const double v = read_teacher(a, m * a.ldt + j) * a.inv_t;
                    most = v > most || v != v ? v : most;
                }
            for (int o = 32; o; o /= 2) {
                const double v = __shfl_xor(most, o);
                most = v > most || v != v ? v : most;
            }
            double s = 0.0;
            for (uint32_t j = lane; j < a.K; j += 64)
                if (where[j] >= 0) s += exp(read_teacher(a, m * a.ldt + j) * a.inv_t - most);
            lse = most + log(wave_sum(s));
        } else {
            lse = a.lse[m];
        }
        // the student's log-sum
        double l = lt;
        uint32_t distinct = 0;
        if (tail) {
            double peak = -INFINITY;
            for (uint32_t j = lane; j < a.K; j += 64)
                if (where[j] >= 0) {
                    const double z = load_act<TYPE>(row, (uint32_t)where[j]) * a.inv_t;
                    peak = z > peak || z != z ? z : peak;
                }
            for (int o = 32; o; o /= 2) {
                const double v = __shfl_xor(peak, o);
                peak = v > peak || v != v ? v : peak;
            }
            peak = lt > peak || lt != lt ? lt : peak;
            double s = 0.0;
            for (uint32_t j = lane; j < a.K; j += 64) {
                if (where[j] < 0) continue;
                bool first = true;  // of its class
                for (uint32_t i = 0; i < j; ++i) first &= where[i] != where[j];
                if (!first) continue;
                ++distinct;
                s += exp(load_act<TYPE>(row, (uint32_t)where[j]) * a.inv_t - peak);
            }
            s = wave_sum(s) + exp(lt - peak);
            l = peak + log(s);
            for (int o = 32; o; o /= 2) distinct += __shfl_xor(distinct, o);
        }
        double loss = 0.0, all = 0.0;
        bool any = false;
        for (uint32_t j = lane; j < a.K; j += 64) {
            if (where[j] < 0) {
                mass[j] = 0.0f;
                continue;
            }
            any = true;
            const double logp = read_teacher(a, m * a.ldt + j) * a.inv_t - lse;
            const double p = exp(logp), z = load_act<TYPE>(row, (uint32_t)where[j]) * a.inv_t;
            mass[j] = (float)p;
            all += p;
            if (!(p == 0.0)) loss += p * (logp - z + l);
        }
        loss = wave_sum(loss);
        all = wave_sum(all);
        any = __any(any);
        double factor = exp(lt - l);  // the student's mass outside the marks
        if (!any) {
            loss = 0.0;
            factor = 0.0;
        } else if (tail) {
            double pt = fmax(0.0, 1.0 - all);
            if (distinct == a.V) pt = 0.0;
            if (pt > 0.0) loss += pt * (log(pt) - lt + l);
            factor -= pt;
        }
        if (bad) loss = factor = NAN;
        if (lane == 0) {
            if (a.loss) a.loss[m] = (float)(loss * weight);
            const double by = (double)weight * (a.dloss ? a.dloss[m] : 1.0f) * a.inv_t;
            common[0] = factor == 0.0 ? 0.0f : (float)(factor / total * by);
            common[1] = (float)by;
            log_sum = l;
        }
    }
    if (!a.dlogits) return;
    __syncthreads();
    const float factor = common[0], by = common[1];
    const double l = log_sum;
    for (uint32_t p = t; p < pieces; p += kThreads) {
        const v4i v = load_piece<TYPE>(row, p, a.V);
        float g[kP];
#pragma unroll
        for (int i = 0; i < kP; ++i)
            g[i] = factor == 0.0f ? 0.0f : factor * exp2f((act_of<TYPE>(v, i) - from) * a.scale);
        store_piece<TYPE>(grad, p, a.V, pack<TYPE>(g));
    }
    __syncthreads();
    // the entries' classes again, each by its first entry
    for (uint32_t j = t; j < a.K; j += kThreads) {
        if (where[j] < 0) continue;
        bool first = true;
        float p = 0.0f;
        for (uint32_t i = 0; i < a.K; ++i)
            if (where[i] == where[j]) {
                first &= i >= j;
                p += mass[i];
            }
        if (!first) continue;
        const uint32_t c = (uint32_t)where[j];
        const double z = load_act<TYPE>(row, c) * a.inv_t;
        const float g = bad ? NAN : by * ((float)exp(z - l) - p);
        if (TYPE == ENTQ_F32)
            ((float *)grad)[c] = g;
        else
            ((uint16_t *)grad)[c] = bits16(g, TYPE == ENTQ_F16);
    }
}

template <int TYPE>
int launch_distill(const DistillArgs &a, hipStream_t s) {
    constexpr uint32_t kMost = 1u << 20;  // a launch's threads stay below 2^32
    const uint32_t lds = a.lse ? (a.V + 31) / 32 * 4 : 0;
    for (uint64_t r = 0; r < a.M; r += kMost)
        distill_rows<TYPE, 16><<<(uint32_t)std::min<uint64_t>(kMost, a.M - r), 1024, lds, s>>>(a, (uint32_t)r);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

uint32_t bytes_of(int t) { return t == ENTQ_F32 ? 4 : 2; }

bool float_type(int t) { return t == ENTQ_BF16 || t == ENTQ_F16 || t == ENTQ_F32; }

entq_status check(const entq_distill *d) {
    if (!d || d->reserved) return ENTQ_EINVAL;
    if (!float_type(d->type) || !float_type(d->teacher_type)) return ENTQ_EINVAL;
    if (d->index_bytes != 4 && d->index_bytes != 8) return ENTQ_EINVAL;
    if (d->rows > 0x7FFFFFFFu || !d->classes || d->classes > ENTQ_DISTILL_MAX_CLASSES) return ENTQ_EINVAL;
    if (!d->top || d->top > ENTQ_DISTILL_MAX_TOP) return ENTQ_EINVAL;
    constexpr uint64_t most = 1ull << 40;
    if (d->ldlogits < d->classes || d->ldindex < d->top || d->ldteacher < d->top || d->ldlogits > most ||
        d->ldindex > most || d->ldteacher > most)
        return ENTQ_EINVAL;
    if (!(d->temperature > 0.0f) || !std::isfinite(d->temperature)) return ENTQ_EINVAL;
    if (!(d->temperature >= 1e-4f && d->temperature <= 1e4f)) return ENTQ_EINVAL;
    if (d->rows && (!d->d_logits || !d->d_index || !d->d_teacher)) return ENTQ_EINVAL;
    if ((uintptr_t)d->d_logits % bytes_of(d->type) || (uintptr_t)d->d_teacher % bytes_of(d->teacher_type) ||
        (uintptr_t)d->d_index % d->index_bytes || (uintptr_t)d->d_lse % 4 || (uintptr_t)d->d_weight % 4)
        return ENTQ_EALIGN;
    return ENTQ_OK;
}

entq_status run(const entq_distill &d, float *loss, const float *dloss, void *dlogits, uint64_t ldd, hipStream_t s) {
    if (!d.rows) return ENTQ_OK;
    DistillArgs a{};
    a.logits = d.d_logits;
    a.teacher = d.d_teacher;
    a.index = d.d_index;
    a.lse = d.d_lse;
    a.weight = d.d_weight;
    a.dloss = dloss;
    a.loss = loss;
    a.dlogits = dlogits;
    a.ld = d.ldlogits;
    a.ldt = d.ldteacher;
    a.ldi = d.ldindex;
    a.ldd = ldd;
    a.M = d.rows;
    a.V = d.classes;
    a.K = d.top;
    a.teacher_type = d.teacher_type;
    a.wide = d.index_bytes == 8;
    a.inv_t = 1.0 / d.temperature;
    a.scale = (float)(1.44269504088896340736 / d.temperature);
    return (entq_status)(d.type == ENTQ_BF16  ? launch_distill<ENTQ_BF16>(a, s)
                         : d.type == ENTQ_F16 ? launch_distill<ENTQ_F16>(a, s)
                                              : launch_distill<ENTQ_F32>(a, s));
}

}  // namespace
}  // namespace entq

extern "C" {

entq_status entq_distill_loss(const entq_distill *d, float *d_loss, void *stream) {
    const entq_status st = entq::check(d);
    if (st != ENTQ_OK) return st;
    if (d->rows && !d_loss) return ENTQ_EINVAL;
    if ((uintptr_t)d_loss % 4) return ENTQ_EALIGN;
    return entq::run(*d, d_loss, nullptr, nullptr, d->classes, (hipStream_t)stream);
}

entq_status entq_distill_backward(const entq_distill *d, const float *d_dloss, void *d_dlogits, uint64_t lddlogits,
                                  float *d_loss, void *stream) {
    const entq_status st = entq::check(d);
    if (st != ENTQ_OK) return st;
    if ((d->rows && !d_dlogits) || lddlogits < d->classes || lddlogits > (1ull << 40)) return ENTQ_EINVAL;
    if ((uintptr_t)d_dlogits % entq::bytes_of(d->type) || (uintptr_t)d_dloss % 4 || (uintptr_t)d_loss % 4)
        return ENTQ_EALIGN;
    return entq::run(*d, d_loss, d_dloss, d_dlogits, lddlogits, (hipStream_t)stream);
}

}  // extern "C"
