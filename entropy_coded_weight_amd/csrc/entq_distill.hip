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
//   dloss/dz_v = all q_v - sum_{j of v} p_j,   q_v = exp(z_v - L),   all = sum p [+ pt]
// (all is 1 unless sum p is above 1, or below it with entries that cover every
// class: what a rounded lse or teacher and a class with two entries leave.) Lt
// is the log-sum over the classes outside the top entries, whose gradient with
// a tail is all q_v - pt exp(z_v - Lt) = exp(z_v - Lt) (all qt - pt), qt =
// exp(Lt - L). Lt comes from a sum over those classes alone (a bit for each
// class marks the others): L minus the top entries would lose it to
// cancellation where the student is sure.
struct DistillArgs {
    const void *logits, *teacher, *index;
    const float *lse, *weight, *dloss;
    float *loss;            // or null
    void *dlogits;          // or null
    uint64_t ld, ldt, ldi, ldd;
    uint32_t M, V, K;
    int teacher_type;
    bool wide;              // 64-bit indices
    float scale;            // log2(e) / T rounded
    double scale64, inv_t;  // log2(e) / T, 1 / T
};

constexpr uint32_t kMaxTop = ENTQ_DISTILL_MAX_TOP;
constexpr double kLn2 = 0.693147180559945309417;

__device__ __forceinline__ float read_teacher(const DistillArgs &a, uint64_t at) {
    return a.teacher_type == ENTQ_F32 ? ((const float *)a.teacher)[at]
                                      : from16(((const uint16_t *)a.teacher)[at], a.teacher_type == ENTQ_F16);
}

__device__ __forceinline__ float wave_maxf(float v) {
#pragma unroll
    for (int o = 32; o; o /= 2) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ float scalar(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(v)));
}
__device__ __forceinline__ double scalar(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
// (a NaN wins)
__device__ __forceinline__ double wave_max64(double v) {
#pragma unroll
    for (int o = 32; o; o /= 2) {
        const double w = __shfl_xor(v, o);
        v = w > v || w != w ? w : v;
    }
    return v;
}

// Element i of a piece replaced by -infinity: a class that counts for nothing.
template <int TYPE>
__device__ __forceinline__ void remove(v4i &v, int i) {
    if (TYPE == ENTQ_F32) {
        v[i] = (int)0xFF800000u;
    } else {
        const uint32_t inf = TYPE == ENTQ_F16 ? 0xFC00u : 0xFF80u, shift = 16 * (i % 2);
        v[i / 2] = (int)(((uint32_t)v[i / 2] & ~(0xFFFFu << shift)) | inf << shift);
    }
}

// What the entries of a row come to. Logits count from the row's largest.
struct Entries {
    double terms;           // sum p (log p - z)
    double mass;            // sum p
    double top;             // with a tail: the student's sum over the entries' classes, from all's largest
    double back;            // and what takes the row's waves' sum there
    uint32_t distinct;      // of these classes
    bool any, bad, twice;   // an entry, an index beyond the classes, a class with two entries
};
struct EntryTable {
    int32_t where[kMaxTop]; // an entry's class, -1: none
    double mass[kMaxTop];   // the teacher's p of it
    double z2[kMaxTop];     // the student's exponent of it
    bool later[kMaxTop];    // an earlier entry has its class
};
// A lane's entries: lane, lane + 64, ...
constexpr int kOwn = kMaxTop / 64;
struct OwnEntries {
    int32_t at[kOwn];       // the class, -1: none, -2: beyond the classes
    float teacher[kOwn], logit[kOwn];
    double p[kOwn];
    bool first[kOwn];       // of its class
};
#define ENTQ_OWN_ENTRIES(i, j) \
    _Pragma("unroll") for (int i = 0; i < kOwn; ++i) if (const uint32_t j = i * 64 + lane; j < a.K)

__device__ __forceinline__ void load_entries(const DistillArgs &a, uint64_t m, uint32_t lane, OwnEntries &o) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) o.at[i] = -1;  // (no way leaves it unset)
    ENTQ_OWN_ENTRIES(i, j) {
        const int64_t c = a.wide ? ((const int64_t *)a.index)[m * a.ldi + j] : ((const int32_t *)a.index)[m * a.ldi + j];
        o.at[i] = c < 0 ? -1 : c < (int64_t)a.V ? (int32_t)c : -2;
        o.teacher[i] = read_teacher(a, m * a.ldt + j);
    }
}

// A row's entries, in 64 bits; one wave. First their classes, marked in `marks`
// when `marked` is called, and the teacher's side ...
template <int TYPE, class Marked>
__device__ __forceinline__ Entries teacher_side(const DistillArgs &a, uint64_t m, const void *row, uint32_t lane,
                                                OwnEntries &o, EntryTable &e, uint32_t *marks, Marked marked) {
    Entries f{};
    ENTQ_OWN_ENTRIES(i, j) {
        const bool in = o.at[i] >= 0;
        f.bad |= o.at[i] == -2;
        f.any |= in;
        e.where[j] = o.at[i];
        o.logit[i] = in ? load_act<TYPE>(row, (uint32_t)o.at[i]) : 0.0f;
        const uint32_t c = (uint32_t)o.at[i];
        if (in) f.twice |= atomicOr(&marks[c / 32], 1u << (c % 32)) >> (c % 32) & 1;
    }
    f.bad = __any(f.bad);
    f.any = __any(f.any);
    f.twice = __any(f.twice);
    marked();
    double most = -INFINITY;
    ENTQ_OWN_ENTRIES(i, j) {
        o.first[i] = o.at[i] >= 0;
        if (f.twice) {
            for (uint32_t k = 0; k < j; ++k) o.first[i] &= e.where[k] != o.at[i];
        }
        e.later[j] = !o.first[i];
        f.distinct += o.first[i];
        const double v = o.at[i] >= 0 ? o.teacher[i] * a.inv_t : -INFINITY;
        most = v > most || v != v ? v : most;
    }
#pragma unroll
    for (int w = 32; w; w /= 2) f.distinct += __shfl_xor(f.distinct, w);
    double lse;
    if (a.lse) {
        lse = a.lse[m];
    } else {
        most = wave_max64(most);
        double s = 0.0;
        ENTQ_OWN_ENTRIES(i, j) {
            if (o.at[i] >= 0) s += exp(o.teacher[i] * a.inv_t - most);
        }
        lse = most + log(wave_sum(s));
    }
    ENTQ_OWN_ENTRIES(i, j) {
        if (o.at[i] < 0) continue;
        const double logp = o.teacher[i] * a.inv_t - lse;
        o.p[i] = exp(logp);
        e.mass[j] = o.p[i];
        f.mass += o.p[i];
        if (!(o.p[i] == 0.0)) f.terms += o.p[i] * logp;
    }
    f.mass = wave_sum(f.mass);
    f.terms = wave_sum(f.terms);
    return f;
}

// ... then the student's, its logits counted from `from`.
__device__ __forceinline__ void student_side(const DistillArgs &a, uint32_t lane, double from, const OwnEntries &o,
                                             EntryTable &e, Entries &f) {
    double s = 0.0;
    ENTQ_OWN_ENTRIES(i, j) {
        const double z = o.at[i] >= 0 ? (o.logit[i] - from) * a.scale64 : -INFINITY;
        e.z2[j] = z;
        if (o.at[i] >= 0 && !(o.p[i] == 0.0)) s += o.p[i] * z;
    }
    f.terms -= wave_sum(s) * kLn2;
    if (!a.lse) return;
    s = 0.0;
    ENTQ_OWN_ENTRIES(i, j) {
        if (o.first[i]) s += exp2((o.logit[i] - from) * a.scale64);
    }
    f.top = wave_sum(s);
}

// One workgroup per token: WAVES waves for the row, and one for the entries,
// whose few terms are in 64 bits (the loss is a small difference of them) and
// come out while the row is read. VECS pieces a thread stay in registers, so
// that a row is read once for the loss and its gradient; VECS 0: any length,
// read two or three times, again out of the caches.
//
// The exponentials are the hardware's 2^x of one fused multiply-add. Of the
// sum: x scale + c with c = - (the largest logit) scale, differences from the
// largest, so that the exponents that count are small and have their bits, and
// its logarithm in 64 bits, since the loss is a small difference of that (with
// exponents from 64 down and the hardware's logarithm a loss of 0.01 was off by
// 5e-6 of it, and no faster). What rounding c does to all of them alike is put
// right in 64 bits. What is left in the logarithm of the sum is scale's own
// rounding, |scale / (log2(e) / T) - 1| E_q |z - max|, the factor at most 2^-24,
// and the exponents' roundings: over 32000 classes 3e-8 and 2e-8 at T = 1.5,
// 2.1e-7 and 2e-8 at 1.25. Without a tail that is the loss's error; with one the
// loss takes qt - pt of it, and was off by 7e-8 to 3e-7 of losses of 2.5e-4 to 0.4
// (T of 0.7 to 4). Of the gradients: x scale + c + 64, 2^64 above
// the smallest exponents that the hardware flushes, so that small ones are
// there, to 1e-6 of their values (without the 64 where the weight is so small
// that they would not be there anyway).
//
// Bound by memory where rows fill their variant: 4096 x 32000 bf16 in 46.7 us
// (5.6 TB/s of reads, part of them from the last-level cache: 32768 rows 383 us, 5.5 TB/s),
// with the gradient 107.6 us (4.9 TB/s; a copy reaches 5.1; 32768 rows 806 us), 515 x 50021
// f16 with it in 24.9 us. What carries that are waves: a workgroup has a multiple of 4 (with
// 9, one SIMD's three decide, and the first took 107 us), the entries have a
// wave to themselves (in a wave of the row their 64-bit registers come on top
// of the row's: 54.7 and 127.4 us), and the registers are held to 80 and 64
// for 3 and 4 waves more on a SIMD (the third at 78: 29.3 us); a row's own
// numbers are kept in scalar registers for that (29.2 us without). Without the
// row in registers the first two took 130 and 305 us.
template <int VECS, int WAVES>
constexpr int kResident = WAVES == 7 ? 6 : VECS == 7 ? 8 : 1;  // waves on a SIMD, at least
template <int TYPE, int GRAD, int VECS, int WAVES>
__global__ __launch_bounds__(64 * WAVES + 64, (kResident<VECS, WAVES>)) void distill_rows(DistillArgs a, uint32_t row0) {
    constexpr int kP = kPer<TYPE>, kThreads = 64 * WAVES;
    extern __shared__ uint32_t marks[];  // a bit for each class of the entries
    __shared__ float part[WAVES];
    __shared__ double sums[WAVES];
    __shared__ float of_entries;  // their largest logit
    __shared__ EntryTable entries;
    __shared__ Entries found;
    const uint64_t m = (uint64_t)row0 + blockIdx.x;
    const uint32_t t = threadIdx.x, lane = t % 64, wave = __builtin_amdgcn_readfirstlane(t / 64);
    const uint32_t pieces = (a.V + kP - 1) / kP;
    const uint8_t *row = (const uint8_t *)a.logits + m * a.ld * (TYPE == ENTQ_F32 ? 4 : 2);
    uint8_t *grad = (uint8_t *)a.dlogits + m * a.ldd * (GRAD == ENTQ_F32 ? 4 : 2);
    const float weight = a.weight ? a.weight[m] : 1.0f;
    auto put = [&](uint32_t p, const float(&g)[kP]) {
        if constexpr (TYPE == GRAD) {
            // (not read again here: 111.8 us where ordinary stores take 115.5,
            // 4096 x 32000 bf16)
            const v4i v = pack<TYPE>(g);
            if ((p + 1) * kP <= a.V)
                __builtin_nontemporal_store(v, (any_v4i *)(grad + p * 16));
            else
                store_piece<TYPE>(grad, p, a.V, v);
        } else {  // 16-bit gradients of fp32 logits
            uint16_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = bits16(g[i], GRAD == ENTQ_F16);
            uint16_t *to = (uint16_t *)grad + p * 4;
            if (p * 4 + 4 <= a.V) {
                ((any8 *)to)->v = v2i{(int)(b[0] | (uint32_t)b[1] << 16), (int)(b[2] | (uint32_t)b[3] << 16)};
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 3; ++i)
                    if (p * 4 + i < a.V) to[i] = b[i];
            }
        }
    };
    if (weight == 0.0f) {  // whatever the row holds
        if (a.loss && t == 0) a.loss[m] = 0.0f;
        if (a.dlogits && t < kThreads) {
            const float none[kP] = {};
            for (uint32_t p = t; p < pieces; p += kThreads) put(p, none);
        }
        return;
    }
    float top = -INFINITY, from, all_from, c;
    bool far;
    const bool tail = a.lse != nullptr;
    auto piece = [&](uint32_t p) {
        v4i v = load_piece<TYPE>(row, p, a.V);
        if ((p + 1) * kP > a.V) {
#pragma unroll
            for (int i = 0; i < kP; ++i)
                if (p * kP + i >= a.V) remove<TYPE>(v, i);
        }
        return v;
    };
    // the entries' classes leave the row, with a tail
    auto outside = [&](v4i &v, uint32_t p) {
        const uint32_t at = p * kP, out = at < a.V ? (marks[at / 32] >> (at % 32)) & ((1u << kP) - 1) : 0;
        if (out) {
#pragma unroll
            for (int i = 0; i < kP; ++i)
                if (out >> i & 1) remove<TYPE>(v, i);
        }
    };
    // A row whose largest logit is some 2^24 T or more in size (what a mask of the
    // type's lowest value leaves of a row, say) is replaced by its differences from
    // it: exact where they count.
    auto nearer = [&](v4i &v) {
        float d[kP];
#pragma unroll
        for (int i = 0; i < kP; ++i) d[i] = act_of<TYPE>(v, i) - from;
        v = pack<TYPE>(d);
    };
    auto masked = [&](uint32_t p) {
        v4i v = piece(p);
        if (tail) outside(v, p);
        return v;
    };
    auto again = [&](uint32_t p) {
        v4i v = masked(p);
        if (far) nearer(v);
        return v;
    };
    // The largest logit is there: `from` that of the classes in the sum,
    // `all_from` of all.
    auto refer = [&] {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) top = fmaxf(top, part[w]);
        const float most = fmaxf(top, of_entries);
        from = scalar(top == -INFINITY ? 0.0f : top);
        all_from = scalar(most == -INFINITY ? 0.0f : most);
        far = fabs((double)from * a.scale64) >= 0x1p24;
        c = scalar(far ? 0.0f : (float)(-(double)from * a.scale));
    };
    // What is added to log2 of the row's waves' sum: from all_from, and c's rounding
    // out of all exponents.
    auto shift = [&] {
        return ((double)from - all_from) * a.scale64 - (far ? 0.0 : (double)c + (double)from * (double)a.scale);
    };
    auto raise = [&](v4i v) {
#pragma unroll
        for (int i = 0; i < kP; ++i) top = fmaxf(top, act_of<TYPE>(v, i));
    };
    float own = 0.0f;
    auto add = [&](v4i v) {
#pragma unroll
        for (int i = 0; i < kP; ++i) own += __builtin_amdgcn_exp2f(__builtin_fmaf(act_of<TYPE>(v, i), a.scale, c));
    };
    v4i held[VECS ? VECS : 1];
    // (between two passes: values unpacked in one are not kept for the next,
    // which would take twice the registers of the pieces)
    auto forget = [&] {
#pragma unroll
        for (int i = 0; i < (VECS ? VECS : 1); ++i) asm("" : "+v"(held[i]));
    };
    if (wave < WAVES) {
        if (VECS) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) held[i] = piece(i * kThreads + t);
        }
        for (uint32_t i = t; i < (a.V + 31) / 32; i += kThreads) marks[i] = 0;
        __syncthreads();
        __syncthreads();
        if (VECS) {
            if (tail) {
#pragma unroll
                for (int i = 0; i < VECS; ++i) outside(held[i], i * kThreads + t);
            }
#pragma unroll
            for (int i = 0; i < VECS; ++i) raise(held[i]);
            forget();
        } else {
            for (uint32_t p = t; p < pieces; p += kThreads) raise(masked(p));
        }
        top = wave_maxf(top);
        if (lane == 0) part[wave] = top;
        __syncthreads();
        refer();
        if (VECS && far) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) nearer(held[i]);
        }
        if (VECS) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) add(held[i]);
            forget();
        } else {
            for (uint32_t p = t; p < pieces; p += kThreads) add(again(p));
        }
        const double all = wave_sum((double)own);
        if (lane == 0) sums[wave] = all;
        __syncthreads();
    } else {
        OwnEntries own;
        load_entries(a, m, lane, own);
        __syncthreads();  // the marks are clear
        Entries f = teacher_side<TYPE>(a, m, row, lane, own, entries, marks, [] { __syncthreads(); });
        float most = -INFINITY;
        ENTQ_OWN_ENTRIES(i, j) {
            if (own.at[i] >= 0) most = fmaxf(most, own.logit[i]);
        }
        most = wave_maxf(most);
        if (lane == 0) of_entries = most;
        __syncthreads();  // the largest logit
        refer();
        student_side(a, lane, all_from, own, entries, f);
        if (tail) f.back = exp2(shift());
        if (lane == 0) found = f;
        __syncthreads();  // the sum
    }
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += sums[w];
    sum = scalar(sum);
    const Entries f = found;
    const double rest = 1.0 - f.mass, pt = !tail || f.distinct == a.V || rest < 0.0 ? 0.0 : rest;
    const double total = f.mass + pt;  // L's coefficient: a NaN of the teacher reaches every class
    // with a tail, the sums outside the entries and of all classes, from all's
    // largest (a sum of 0 is no class's; both 0: all of the row is -infinity, and
    // no softmax)
    const double out = tail && sum != 0.0 ? sum * f.back : 0.0, both = out + f.top;
    const bool broken = f.bad || total != total || (tail && f.any && both == 0.0);
    // What a power in the gradient is multiplied by: total / sum, and with a tail
    // (total qt - pt) / sum, qt = out / both, as one quotient. In 64 bits, since qt -
    // pt may be far below both.
    double factor = 0.0;
    if (a.dlogits) {
        factor = (tail ? total * out - pt * both : total) / (tail ? sum * both : sum);
        if (!f.any || (tail && sum == 0.0)) factor = 0.0;
        if (broken) factor = NAN;
    }
    // log2 of the sums over the classes outside the entries (lo2; of all classes
    // without a tail) and over all (all2)
    double lo2, all2;
    if (wave == WAVES) {
        lo2 = all2 = sum == 0.0 ? -INFINITY : log2(sum) + shift();
        if (tail) all2 = log2(both);
        all2 = scalar(all2);  // (28 bytes of scratch without, where registers are held to 64, and 20 with it)
    }
    if (a.loss && wave == WAVES && lane == 0) {
        double loss = f.any ? f.terms + f.mass * (all2 * kLn2) : 0.0;
        if (f.any && pt > 0.0) loss += pt * (log(pt) + (all2 - lo2) * kLn2);
        a.loss[m] = f.bad ? NAN : (float)(loss * weight);
    }
    if (!a.dlogits) return;
    const double by = scalar((double)weight * (a.dloss ? a.dloss[m] : 1.0f) * a.inv_t);
    if (wave < WAVES) {
        // (2^64 of the powers and both constants' roundings out of them again. A
        // factor that 2^-64 would take out of fp32's normal numbers leaves the powers
        // as they are: what the hardware flushes then is below 2^-126 2^-40.)
        const double one = factor * by;
        const float up = scalar(fabs(one) < 0x1p-40 ? 0.0f : 64.0f);
        const float c64 = scalar(far ? up : (float)(up - (double)from * a.scale));
        const double back = (double)c - (double)c64 + up;
        const float each = scalar(factor == 0.0 ? 0.0f : (float)(one * __builtin_amdgcn_exp2f((float)back) * (up == 0.0f ? 1.0 : 0x1p-64)));
        auto power = [&](v4i v, int i) { return __builtin_amdgcn_exp2f(__builtin_fmaf(act_of<TYPE>(v, i), a.scale, c64)); };
        auto write = [&](uint32_t p, v4i v) {
            float g[kP];
#pragma unroll
            for (int i = 0; i < kP; ++i) g[i] = each == 0.0f ? 0.0f : each * power(v, i);
            put(p, g);
        };
        if (VECS) {
#pragma unroll
            for (int i = 0; i < VECS; ++i)
                if (i * kThreads + t < pieces) write(i * kThreads + t, held[i]);
        } else {
            for (uint32_t p = t; p < pieces; p += kThreads) write(p, again(p));
        }
        __syncthreads();
        return;
    }
    // the entries' classes, each by its first entry, over what the row's waves wrote there
    __syncthreads();
    for (uint32_t j = lane; j < a.K; j += 64) {
        if (entries.where[j] < 0 || entries.later[j]) continue;
        double p = entries.mass[j];
        if (f.twice) {
            for (uint32_t i = j + 1; i < a.K; ++i)
                if (entries.where[i] == entries.where[j]) p += entries.mass[i];
        }
        const float g = broken ? NAN : (float)(by * (total * exp2(entries.z2[j] - all2) - p));
        if (GRAD == ENTQ_F32)
            ((float *)grad)[entries.where[j]] = g;
        else
            ((uint16_t *)grad)[entries.where[j]] = bits16(g, GRAD == ENTQ_F16);
    }
}

template <int TYPE, int GRAD, int VECS, int WAVES>
int launch_rows(const DistillArgs &a, hipStream_t s) {
    constexpr uint32_t kMost = 1u << 20;  // a launch's threads stay below 2^32
    for (uint64_t r = 0; r < a.M; r += kMost)
        distill_rows<TYPE, GRAD, VECS, WAVES><<<(uint32_t)std::min<uint64_t>(kMost, a.M - r), 64 * WAVES + 64,
                                                (a.V + 31) / 32 * 4, s>>>(a, (uint32_t)r);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

// The fewest waves and pieces that hold a row: each of these variants was slower
// than the smaller ones at every size that both take, because unused pieces cost
// what used ones do. 131 million bf16 logits with gradient, us, this choice and the next
// larger one's: 768 pieces 144 and 411, 900 350 and 670, 2000 173 and 277, 4032
// 109 and 143, 5000 127 and 197, 6720 113 and 173, 8000 156 and 188, 8640 157 and
// 189, 10000 178 and (the row read again, VECS 0) 203, 16320 137 and 187; the
// losses alone 768 pieces 96 and 300, 4032 63 and 102, 6720 67 and 111, 8640 97 and
// 136, 16320 85 and 107. Rows of 1024 fp32 logits with a bf16 gradient: 8000 pieces 64
// and 73, 16320 110 and 170. 96 rows: 768 pieces 12.3 and 14.6, 16320 28.3 and
// 36.7. Rows far shorter than their variant pay for it (900 pieces 3.4 times their
// bytes' time, 128 pieces, a workgroup for each 1024 classes, 7 times: 735), and rows
// beyond 16320 pieces for two readings of the loss and three with the gradient
// (16384: 186).
template <int TYPE, int GRAD>
int launch_distill(const DistillArgs &a, hipStream_t s) {
    const uint32_t pieces = (a.V + kPer<TYPE> - 1) / kPer<TYPE>;
    if (pieces <= 768) return launch_rows<TYPE, GRAD, 4, 3>(a, s);
    if (pieces <= 4032) return launch_rows<TYPE, GRAD, 9, 7>(a, s);
    if (pieces <= 6720) return launch_rows<TYPE, GRAD, 7, 15>(a, s);
    if (pieces <= 8640) return launch_rows<TYPE, GRAD, 9, 15>(a, s);
    if (pieces <= 16320) return launch_rows<TYPE, GRAD, 17, 15>(a, s);
    return launch_rows<TYPE, GRAD, 0, 15>(a, s);
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

entq_status run(const entq_distill &d, float *loss, const float *dloss, void *dlogits, int dtype, uint64_t ldd,
                hipStream_t s) {
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
    a.scale64 = 1.44269504088896340736 / d.temperature;
    a.scale = (float)a.scale64;
    if (d.type == ENTQ_BF16) return (entq_status)launch_distill<ENTQ_BF16, ENTQ_BF16>(a, s);
    if (d.type == ENTQ_F16) return (entq_status)launch_distill<ENTQ_F16, ENTQ_F16>(a, s);
    return (entq_status)(dtype == ENTQ_BF16  ? launch_distill<ENTQ_F32, ENTQ_BF16>(a, s)
                         : dtype == ENTQ_F16 ? launch_distill<ENTQ_F32, ENTQ_F16>(a, s)
                                             : launch_distill<ENTQ_F32, ENTQ_F32>(a, s));
}

}  // namespace
}  // namespace entq

extern "C" {

entq_status entq_distill_loss(const entq_distill *d, float *d_loss, void *stream) {
    const entq_status st = entq::check(d);
    if (st != ENTQ_OK) return st;
    if (d->rows && !d_loss) return ENTQ_EINVAL;
    if ((uintptr_t)d_loss % 4) return ENTQ_EALIGN;
    return entq::run(*d, d_loss, nullptr, nullptr, d->type, d->classes, (hipStream_t)stream);
}

entq_status entq_distill_backward(const entq_distill *d, const float *d_dloss, void *d_dlogits, int dlogits_type,
                                  uint64_t lddlogits, float *d_loss, void *stream) {
    const entq_status st = entq::check(d);
    if (st != ENTQ_OK) return st;
    if ((d->rows && !d_dlogits) || lddlogits < d->classes || lddlogits > (1ull << 40)) return ENTQ_EINVAL;
    if (!entq::float_type(dlogits_type) || (dlogits_type != d->type && d->type != ENTQ_F32)) return ENTQ_EINVAL;
    if ((uintptr_t)d_dlogits % entq::bytes_of(dlogits_type) || (uintptr_t)d_dloss % 4 || (uintptr_t)d_loss % 4)
        return ENTQ_EALIGN;
    return entq::run(*d, d_loss, d_dloss, d_dlogits, dlogits_type, lddlogits, (hipStream_t)stream);
}

}  // extern "C"
