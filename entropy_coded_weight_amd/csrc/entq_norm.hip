// entq_norm.hip -- the RMS norms before and after a block with its gate and
// residual scale (entq_norm_block) and their gradients.
#include <algorithm>
#include <cmath>

#include "entq_piece.h"

namespace entq {
namespace {

struct NormArgs {
    const void *x, *branch, *gate;
    const float *post, *pre;
    uint64_t ldx, ldb, ldg;
    uint32_t M, N;
    int gate_kind;
    float alpha, beta, eps;
    double per;             // 1 / N
    // forward
    void *out, *y;
    float *scales;          // of codes in y, or null: y has the type
    uint64_t ldo, ldy;
    // backward
    const void *dout, *dy;
    uint64_t lddo, lddy;
    void *dx, *db, *dgate;  // dgate: of every kind but CHANNEL (which finishes with dpost)
    uint64_t lddx, lddb, lddg;
    float *stats;           // [M][4], of the two launches
    float *part_pre, *part_post;  // [strips][N], or null
    uint32_t strips;
};

template <int TYPE>
__device__ __forceinline__ const uint8_t *row_of(const void *p, uint64_t ld, uint64_t m) {
    return (const uint8_t *)p + m * ld * (TYPE == ENTQ_F32 ? 4 : 2);
}

// The factors of a piece: beta is not in them.
template <int TYPE>
__device__ __forceinline__ void load_gate(const NormArgs &a, uint64_t m, uint32_t p, float token,
                                          float (&g)[kPer<TYPE>]) {
    if (a.gate_kind == ENTQ_GATE_CHANNEL) return load_floats<TYPE>((const float *)a.gate, p, a.N, g);
    if (a.gate_kind == ENTQ_GATE_FULL) {
        const v4i v = load_piece<TYPE>(row_of<TYPE>(a.gate, a.ldg, m), p, a.N);
#pragma unroll
        for (int i = 0; i < kPer<TYPE>; ++i) g[i] = act_of<TYPE>(v, i);
        return;
    }
#pragma unroll
    for (int i = 0; i < kPer<TYPE>; ++i) g[i] = token;
}

__device__ __forceinline__ float token_gate(const NormArgs &a, uint64_t m) {
    return a.gate_kind == ENTQ_GATE_TOKEN ? ((const float *)a.gate)[m * a.ldg] : 1.0f;
}

// A row's sums over its WAVES waves.
template <int WAVES>
__device__ __forceinline__ double row_sum(double v, double *part) {
    v = wave_sum(v);
    if (WAVES == 1) return v;
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) v += part[i];
    return v;
}

// One row for each group of WAVES waves: the branch's norm, the new state, its
// norm. VECS pieces a thread stay in registers; VECS 0: any length, the
// branch and the state read again (the thread's own pieces, out of the L2).
// Row sums are in 64 bits: no sum of squares of fp32 values overflows, and the
// result hardly depends on their order. Bound by memory: 4096 x 8192 bf16 with a
// channel's gate 57.6 us (4.7 TB/s; a copy reaches 5.1), by latency for few
// rows: one of 8192 into codes 5.1 us, 333 of 5121 f16 10.2. (Loading the
// factors with the row, before its first sum: 60.1, and no gain for few rows.)
template <int TYPE, int VECS, int WAVES>
__global__ __launch_bounds__(WAVES < 4 ? 256 : 64 * WAVES) void norm_rows(NormArgs a, uint32_t row0) {
    constexpr int kP = kPer<TYPE>, kThreads = 64 * WAVES, kRows = WAVES < 4 ? 4 / WAVES : 1;
    __shared__ double part[2][WAVES < 4 ? 1 : WAVES];
    __shared__ uint32_t top[WAVES < 4 ? 1 : WAVES];
    const uint64_t m = (uint64_t)row0 + blockIdx.x * kRows + (WAVES < 4 ? threadIdx.x / kThreads : 0);
    if (m >= a.M) return;  // (a whole wave, where rows are waves)
    const uint32_t t = WAVES < 4 ? threadIdx.x % kThreads : threadIdx.x;
    const uint32_t pieces = (a.N + kP - 1) / kP;
    const uint8_t *x = row_of<TYPE>(a.x, a.ldx, m);
    const float token = token_gate(a, m);
    v4i state[VECS ? VECS : 1];
    double ss = 0.0;
    uint32_t big = 0;
    const bool codes = a.scales != nullptr;
    auto took = [&](uint32_t p, v4i v) {  // a piece of the state: its part of the row's sums
        float w[kP];
        if (codes) load_floats<TYPE>(a.pre, p, a.N, w);
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            const float s = act_of<TYPE>(v, i);
            ss += (double)s * (double)s;
            if (codes) big = max(big, __float_as_uint(s * w[i]) & 0x7FFFFFFFu);
        }
    };
    if (a.branch) {
        const uint8_t *b = row_of<TYPE>(a.branch, a.ldb, m);
        uint8_t *out = const_cast<uint8_t *>(row_of<TYPE>(a.out, a.ldo, m));
        v4i held[VECS ? VECS : 1];
        if (VECS) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                held[i] = load_piece<TYPE>(b, i * kThreads + t, a.N);
                state[i] = load_piece<TYPE>(x, i * kThreads + t, a.N);
            }
        }
        float rho = 1.0f;
        if (a.post) {
            double sb = 0.0;
            auto add = [&](v4i v) {
#pragma unroll
                for (int i = 0; i < kP; ++i) {
                    const double f = act_of<TYPE>(v, i);
                    sb += f * f;
                }
            };
            if (VECS) {
#pragma unroll
                for (int i = 0; i < VECS; ++i) add(held[i]);
            } else {
                for (uint32_t p = t; p < pieces; p += kThreads) add(load_piece<TYPE>(b, p, a.N));
            }
            rho = rsqrt64(row_sum<WAVES>(sb, part[0]) * a.per + (double)a.eps);
        }
        auto join = [&](uint32_t p, v4i xv, v4i bv) {
            float g[kP], w[kP], s[kP];
            load_gate<TYPE>(a, m, p, token, g);
            if (a.post) load_floats<TYPE>(a.post, p, a.N, w);
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                float v = act_of<TYPE>(bv, i);
                if (a.post) v = v * rho * w[i];
                s[i] = a.alpha * act_of<TYPE>(xv, i) + a.beta * g[i] * v;
            }
            const v4i r = pack<TYPE>(s);
            store_piece<TYPE>(out, p, a.N, r);
            return r;
        };
        if (VECS) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                const uint32_t p = i * kThreads + t;
                if (p < pieces) state[i] = join(p, state[i], held[i]);
            }
        } else {
            for (uint32_t p = t; p < pieces; p += kThreads) {
                const v4i r = join(p, load_piece<TYPE>(x, p, a.N), load_piece<TYPE>(b, p, a.N));
                if (a.y) took(p, r);
            }
            x = out;
        }
    } else if (VECS) {
#pragma unroll
        for (int i = 0; i < VECS; ++i) state[i] = load_piece<TYPE>(x, i * kThreads + t, a.N);
    } else {
        for (uint32_t p = t; p < pieces; p += kThreads) took(p, load_piece<TYPE>(x, p, a.N));
    }
    if (!a.y) return;
    if (VECS) {
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const uint32_t p = i * kThreads + t;
            if (p < pieces) took(p, state[i]);
        }
    }
    if (codes) {
        big = greatest(big);
        if (WAVES > 1 && threadIdx.x % 64 == 0) top[threadIdx.x / 64] = big;
    }
    const float rho = rsqrt64(row_sum<WAVES>(ss, part[1]) * a.per + (double)a.eps);
    if (codes) {
        if (WAVES > 1) {
#pragma unroll
            for (int i = 0; i < WAVES; ++i) big = max(big, top[i]);
        }
        const Quantizer z(big);
        if (t == 0) a.scales[m] = z.scale * rho;
        uint8_t *y = (uint8_t *)a.y + m * a.ldy;
        auto put = [&](uint32_t p, v4i v) {
            float w[kP];
            load_floats<TYPE>(a.pre, p, a.N, w);
            uint32_t q[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < kP; ++i) q[i / 4] |= z.code(act_of<TYPE>(v, i) * w[i]) << (8 * (i % 4));
            const uint32_t c = p * kP;
            if (c + kP <= a.N) {
                if constexpr (kP == 8)
                    ((any8 *)(y + c))->v = v2i{(int)q[0], (int)q[1]};
                else
                    ((any4 *)(y + c))->v = (int)q[0];
            } else {
#pragma unroll
                for (int i = 0; i < kP - 1; ++i)
                    if (c + i < a.N) y[c + i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
            }
        };
        if (VECS) {
#pragma unroll
            for (int i = 0; i < VECS; ++i)
                if (i * kThreads + t < pieces) put(i * kThreads + t, state[i]);
        } else {
            for (uint32_t p = t; p < pieces; p += kThreads) put(p, load_piece<TYPE>(x, p, a.N));
        }
        return;
    }
    uint8_t *y = const_cast<uint8_t *>(row_of<TYPE>(a.y, a.ldy, m));
    auto put = [&](uint32_t p, v4i v) {
        float w[kP], f[kP];
        load_floats<TYPE>(a.pre, p, a.N, w);
#pragma unroll
        for (int i = 0; i < kP; ++i) f[i] = act_of<TYPE>(v, i) * rho * w[i];
        store_piece<TYPE>(y, p, a.N, pack<TYPE>(f));
    };
    if (VECS) {
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            if (i * kThreads + t < pieces) put(i * kThreads + t, state[i]);
    } else {
        for (uint32_t p = t; p < pieces; p += kThreads) put(p, load_piece<TYPE>(x, p, a.N));
    }
}

template <int TYPE, int VECS, int WAVES>
int launch_norm(const NormArgs &a, hipStream_t s) {
    constexpr uint32_t kRows = WAVES < 4 ? 4 / WAVES : 1, kThreads = WAVES < 4 ? 256 : 64 * WAVES;
    constexpr uint32_t kMost = 1u << 20;  // a launch's threads stay below 2^32
    for (uint64_t r = 0; r < a.M; r += (uint64_t)kMost * kRows) {
        const uint64_t groups = (a.M - r + kRows - 1) / kRows;
        norm_rows<TYPE, VECS, WAVES><<<(uint32_t)std::min<uint64_t>(kMost, groups), kThreads, 0, s>>>(a, (uint32_t)r);
    }
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

// As few waves as hold a row with one or two pieces a thread: more of them only
// wait for each other, fewer leave too few on a CU. 4096 rows of bf16, us with
// the next smaller row's choice or the next larger one's for this: 2048 values
// 15.1 (two pieces in 8 waves 18.1), 4096 31.8 and 8192 57.6 (four in 16: 40.1
// and 62.1), 16384 112.6 (146.8).
template <int TYPE>
int launch_norm_typed(const NormArgs &a, hipStream_t s) {
    const uint32_t pieces = (a.N + kPer<TYPE> - 1) / kPer<TYPE>;
    if (pieces <= 64) return launch_norm<TYPE, 1, 1>(a, s);
    if (pieces <= 256) return launch_norm<TYPE, 1, 4>(a, s);
    if (pieces <= 1024) return launch_norm<TYPE, 2, 8>(a, s);
    if (pieces <= 2048) return launch_norm<TYPE, 2, 16>(a, s);
    if (pieces <= 4096) return launch_norm<TYPE, 4, 16>(a, s);
    return launch_norm<TYPE, 0, 16>(a, s);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
//
// With rho1 = rho(s), rho2 = rho(branch), unit = branch rho2 (branch itself
// without a norm behind it), v = unit post:
//   D  = dout + rho1 (pre dy - s rho1 c1),   c1 = rho1 mean(s pre dy)
//   dx = alpha D
//   dv = beta gate D
//   dbranch = rho2 (post dv - unit c2),   c2 = rho2 mean(branch post dv)
//   dgate = beta D v summed over what the gate was spread over
//   dpre = sum over tokens of dy s rho1, dpost of dv unit
// mean(branch post dv) is linear in D, so that every sum along a row comes out
// of one pass: over s^2, branch^2, s pre dy, and branch post gate times each of
// dout, pre dy and s. Both column sums of D unit (dpost, and dgate of a
// channel) are one sum up to factors that do not depend on the token.

// Which of a row's sums.
enum { kSS, kBB, kSY, kBD, kBY, kBS, kRowSums };

// What the row's sums give; dgate: of a gate for each token.
struct RowStats {
    float rho1, c1, rho2, c2, dgate;
};
__device__ __forceinline__ RowStats row_stats(const NormArgs &a, const double (&sum)[kRowSums], float token) {
    RowStats r{0.0f, 0.0f, 1.0f, 0.0f, 0.0f};
    double d = sum[kBD];
    if (a.dy) {
        r.rho1 = rsqrt64(sum[kSS] * a.per + (double)a.eps);
        const double c1 = r.rho1 * (sum[kSY] * a.per);
        r.c1 = (float)c1;
        d += r.rho1 * (sum[kBY] - c1 * (r.rho1 * sum[kBS]));
    }
    if (a.post) {
        r.rho2 = rsqrt64(sum[kBB] * a.per + (double)a.eps);
        // (a token's gate is not in the sums)
        r.c2 = (float)(r.rho2 * (a.beta * d * a.per) * token);
    }
    r.dgate = (float)(a.beta * (double)r.rho2 * d);
    return r;
}

// What the columns of a piece have of their own. Absent factors are 1.
template <int TYPE>
struct Columns {
    float pre[kPer<TYPE>], post[kPer<TYPE>], gate[kPer<TYPE>];
};
template <int TYPE>
__device__ __forceinline__ void load_columns(const NormArgs &a, uint32_t p, Columns<TYPE> &c) {
#pragma unroll
    for (int i = 0; i < kPer<TYPE>; ++i) c.pre[i] = c.post[i] = c.gate[i] = 1.0f;
    // (each with an offset of its own: none is left for the compiler to share
    // between branches of which a call takes some)
    auto read = [&](const float *w, float (&f)[kPer<TYPE>]) {
        uint32_t q = p;
        asm("" : "+v"(q));
        load_floats<TYPE>(w, q, a.N, f);
    };
    if (a.pre) read(a.pre, c.pre);
    if (a.post) read(a.post, c.post);
    if (a.gate_kind == ENTQ_GATE_CHANNEL) read((const float *)a.gate, c.gate);
}

// A piece of each of a row's matrices, zeros for those that are absent or not
// needed (FULL: the gate is a matrix).
struct RowPiece {
    v4i s, b, dout, dy, gate;
};
template <int TYPE, bool FULL>
__device__ __forceinline__ RowPiece load_row(const NormArgs &a, uint64_t m, uint32_t p) {
    RowPiece r{};
    const uint8_t *s = row_of<TYPE>(a.x, a.ldx, m), *b = row_of<TYPE>(a.branch, a.ldb, m),
                  *dout = row_of<TYPE>(a.dout, a.lddo, m), *dy = row_of<TYPE>(a.dy, a.lddy, m),
                  *gate = row_of<TYPE>(a.gate, a.ldg, m);
    const bool unit = a.branch && (a.post || a.gate_kind != ENTQ_GATE_NONE);
    if (whole_piece<TYPE>(p, a.N)) {
        if (a.dout) r.dout = load_whole(dout, p);
        if (a.dy) {
            r.s = load_whole(s, p);
            r.dy = load_whole(dy, p);
        }
        if (unit) r.b = load_whole(b, p);
        if (FULL) r.gate = load_whole(gate, p);
    } else {
        if (a.dout) r.dout = load_rest<TYPE>(dout, p, a.N);
        if (a.dy) {
            r.s = load_rest<TYPE>(s, p, a.N);
            r.dy = load_rest<TYPE>(dy, p, a.N);
        }
        if (unit) r.b = load_rest<TYPE>(b, p, a.N);
        if (FULL) r.gate = load_rest<TYPE>(gate, p, a.N);
    }
    return r;
}

// A piece's part of the row's sums.
template <int TYPE, bool FULL>
__device__ __forceinline__ void add_sums(const NormArgs &a, const RowPiece &r, const Columns<TYPE> &c,
                                         double (&sum)[kRowSums]) {
    constexpr int kP = kPer<TYPE>;
    double y[kP], s[kP];
    if (a.dy) {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            s[i] = act_of<TYPE>(r.s, i);
            y[i] = act_of<TYPE>(r.dy, i) * c.pre[i];
            sum[kSS] += s[i] * s[i];
            sum[kSY] += s[i] * y[i];
        }
    }
    if (a.post || a.gate_kind == ENTQ_GATE_TOKEN) {
        double w[kP];
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            const float b = act_of<TYPE>(r.b, i);
            w[i] = b * (c.post[i] * (FULL ? act_of<TYPE>(r.gate, i) : c.gate[i]));
            sum[kBB] += (double)b * (double)b;
            sum[kBD] += w[i] * (double)act_of<TYPE>(r.dout, i);
        }
        if (a.dy) {
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                sum[kBY] += w[i] * y[i];
                sum[kBS] += w[i] * s[i];
            }
        }
    }
}

// A piece's gradients, and its part of the column sums.
template <int TYPE, bool FULL>
__device__ __forceinline__ void gradients(const NormArgs &a, const RowStats &r, uint64_t m, uint32_t p, float token,
                                          const RowPiece &v, const Columns<TYPE> &c, float (&c_pre)[kPer<TYPE>],
                                          float (&c_post)[kPer<TYPE>]) {
    constexpr int kP = kPer<TYPE>;
    float D[kP], f[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) D[i] = act_of<TYPE>(v.dout, i);
    if (a.dy) {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            const float unit = act_of<TYPE>(v.s, i) * r.rho1, dy = act_of<TYPE>(v.dy, i);
            D[i] += r.rho1 * (dy * c.pre[i] - unit * r.c1);
            c_pre[i] += dy * unit;
        }
    }
#pragma unroll
    for (int i = 0; i < kP; ++i) f[i] = a.alpha * D[i];
    const v4i dx = pack<TYPE>(f);
    v4i db = {0, 0, 0, 0}, dgate = {0, 0, 0, 0};
    if (a.branch) {
        float unit[kP];
        const float bt = a.beta * token;
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            unit[i] = act_of<TYPE>(v.b, i) * r.rho2;
            // (its first factor: the gate's part that differs between tokens)
            c_post[i] += (FULL ? act_of<TYPE>(v.gate, i) : token) * D[i] * unit[i];
            f[i] = FULL ? a.beta * act_of<TYPE>(v.gate, i) * D[i] : bt * c.gate[i] * D[i];
        }
        if (a.post) {
#pragma unroll
            for (int i = 0; i < kP; ++i) f[i] = r.rho2 * (c.post[i] * f[i] - unit[i] * r.c2);
        }
        db = pack<TYPE>(f);
        if (FULL) {
#pragma unroll
            for (int i = 0; i < kP; ++i) f[i] = a.beta * D[i] * (unit[i] * c.post[i]);
            dgate = pack<TYPE>(f);
        }
    }
    uint8_t *to_dx = const_cast<uint8_t *>(row_of<TYPE>(a.dx, a.lddx, m)),
            *to_db = const_cast<uint8_t *>(row_of<TYPE>(a.db, a.lddb, m)),
            *to_dgate = const_cast<uint8_t *>(row_of<TYPE>(a.dgate, a.lddg, m));
    if (whole_piece<TYPE>(p, a.N)) {
        if (a.dx) store_whole(to_dx, p, dx);
        if (a.db) store_whole(to_db, p, db);
        if (FULL && a.dgate) store_whole(to_dgate, p, dgate);
    } else {
        if (a.dx) store_rest<TYPE>(to_dx, p, a.N, dx);
        if (a.db) store_rest<TYPE>(to_db, p, a.N, db);
        if (FULL && a.dgate) store_rest<TYPE>(to_dgate, p, a.N, dgate);
    }
}

// The column sums of a piece into row `strip` of the partial sums.
template <int TYPE>
__device__ __forceinline__ void store_columns(const NormArgs &a, uint64_t strip, uint32_t p,
                                              const float (&c_pre)[kPer<TYPE>], const float (&c_post)[kPer<TYPE>]) {
    auto put = [&](float *part, const float(&c)[kPer<TYPE>]) {
        if (!part) return;
#pragma unroll
        for (int i = 0; i < kPer<TYPE>; ++i)
            if (p * kPer<TYPE> + i < a.N) part[strip * a.N + p * kPer<TYPE> + i] = c[i];
    };
    put(a.part_pre, c_pre);
    put(a.part_post, c_post);
}

// Rows that fit the registers, in one pass: a group of WAVES waves takes every
// strips-th row, VECS pieces a thread, and keeps the columns' factors and sums
// over all its rows. The next row's pieces are on their way while this one's
// gradients are computed. One barrier a row, for its sums. (16 waves have half
// the registers: there the factors are read again, and rows come one by one.) Bound by memory: 4096 x
// 8192 bf16 91.2 us with the columns' 4 (4.4 TB/s), by one row's latency for
// few: 96 x 5120 f16 13.2 us and 3.
template <int TYPE, int VECS, int WAVES, bool FULL>
__global__ __launch_bounds__(WAVES < 4 ? 256 : 64 * WAVES) void norm_back_rows(NormArgs a) {
    constexpr int kThreads = 64 * WAVES, kRows = WAVES < 4 ? 4 / WAVES : 1;
    constexpr bool kLean = WAVES == 16;
    __shared__ double part[2][4 * WAVES][8];
    const uint32_t lane = threadIdx.x % 64, t = WAVES < 4 ? threadIdx.x % kThreads : threadIdx.x;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t strip = blockIdx.x * kRows + (WAVES < 4 ? wave / WAVES : 0);
    if (strip >= a.strips) return;  // (a whole wave, where rows are waves)
    const uint32_t pieces = (a.N + kPer<TYPE> - 1) / kPer<TYPE>;
    float c_pre[VECS][kPer<TYPE>] = {}, c_post[VECS][kPer<TYPE>] = {};
    Columns<TYPE> columns[kLean ? 1 : VECS];
    RowPiece v[VECS];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        if (kLean) continue;
        load_columns<TYPE>(a, i * kThreads + t, columns[i]);
        v[i] = load_row<TYPE, FULL>(a, strip, i * kThreads + t);
    }
    uint32_t turn = 0;
    for (uint64_t m = strip; m < a.M; m += a.strips, turn ^= 1) {
        double sum[kRowSums] = {};
        if (kLean) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) v[i] = load_row<TYPE, FULL>(a, m, i * kThreads + t);
        }
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            if (kLean) load_columns<TYPE>(a, i * kThreads + t, columns[0]);
            add_sums<TYPE, FULL>(a, v[i], columns[kLean ? 0 : i], sum);
        }
        RowPiece next[kLean ? 1 : VECS];
        if constexpr (!kLean) {
            const uint64_t after = m + a.strips < a.M ? m + a.strips : m;
#pragma unroll
            for (int i = 0; i < VECS; ++i) next[i] = load_row<TYPE, FULL>(a, after, i * kThreads + t);
        }
        const float token = token_gate(a, m);
#pragma unroll
        for (int i = 0; i < kRowSums; ++i) sum[i] = row16_sum(sum[i]);
        if constexpr (WAVES == 1) {
#pragma unroll
            for (int i = 0; i < kRowSums; ++i) {
                sum[i] += __shfl_xor(sum[i], 16);
                sum[i] += __shfl_xor(sum[i], 32);
            }
        } else {
            if (lane % 16 == 0) {
#pragma unroll
                for (int i = 0; i < kRowSums; ++i) part[turn][wave * 4 + lane / 16][i] = sum[i];
            }
            __syncthreads();
            // lane l: sum l % 8 of every eighth partial sum
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < WAVES / 2; ++i) s += part[turn][i * 8 + lane / 8][lane % 8];
            s += __shfl_xor(s, 8);
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
#pragma unroll
            for (int i = 0; i < kRowSums; ++i) sum[i] = __shfl(s, i);
        }
        const RowStats r = row_stats(a, sum, token);
        if (a.dgate && a.gate_kind == ENTQ_GATE_TOKEN && t == 0) ((float *)a.dgate)[m * a.lddg] = r.dgate;
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const uint32_t p = i * kThreads + t;
            if (kLean) load_columns<TYPE>(a, p, columns[0]);
            if (p < pieces) gradients<TYPE, FULL>(a, r, m, p, token, v[i], columns[kLean ? 0 : i], c_pre[i], c_post[i]);
            if constexpr (!kLean) v[i] = next[i];
        }
    }
#pragma unroll
    for (int i = 0; i < VECS; ++i)
        if (i * kThreads + t < pieces) store_columns<TYPE>(a, strip, i * kThreads + t, c_pre[i], c_post[i]);
}

// Rows of any length, in two launches: the rows' sums, one workgroup a row ...
template <int TYPE, bool FULL>
__global__ __launch_bounds__(512) void norm_back_sums(NormArgs a) {
    constexpr int kThreads = 512, kWaves = kThreads / 64;
    __shared__ double part[kRowSums][kWaves];
    const uint32_t pieces = (a.N + kPer<TYPE> - 1) / kPer<TYPE>;
    for (uint64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        double sum[kRowSums] = {};
        for (uint32_t p = threadIdx.x; p < pieces; p += kThreads) {
            Columns<TYPE> c;
            load_columns<TYPE>(a, p, c);
            add_sums<TYPE, FULL>(a, load_row<TYPE, FULL>(a, m, p), c, sum);
        }
#pragma unroll
        for (int i = 0; i < kRowSums; ++i) {
            sum[i] = wave_sum(sum[i]);
            if (threadIdx.x % 64 == 0) part[i][threadIdx.x / 64] = sum[i];
        }
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int i = 0; i < kRowSums; ++i) {
                sum[i] = 0.0;
                for (int w = 0; w < kWaves; ++w) sum[i] += part[i][w];
            }
            const RowStats r = row_stats(a, sum, token_gate(a, m));
            *(v4f *)(a.stats + m * 4) = v4f{r.rho1, r.c1, r.rho2, r.c2};
            if (a.dgate && a.gate_kind == ENTQ_GATE_TOKEN) ((float *)a.dgate)[m * a.lddg] = r.dgate;
        }
        __syncthreads();
    }
}

// ... and the gradients: a thread keeps the column sums of one piece over a
// strip of the rows.
template <int TYPE, bool FULL>
__global__ __launch_bounds__(256) void norm_back_apply(NormArgs a) {
    constexpr int kP = kPer<TYPE>;
    const uint32_t p = blockIdx.x * 256 + threadIdx.x;
    if (p * kP >= a.N) return;
    float c_pre[kP] = {}, c_post[kP] = {};
    Columns<TYPE> c;
    load_columns<TYPE>(a, p, c);
    for (uint64_t m = blockIdx.y; m < a.M; m += a.strips) {
        const v4f st = *(const v4f *)(a.stats + m * 4);
        gradients<TYPE, FULL>(a, RowStats{st[0], st[1], st[2], st[3], 0.0f}, m, p, token_gate(a, m),
                              load_row<TYPE, FULL>(a, m, p), c, c_pre, c_post);
    }
    store_columns<TYPE>(a, blockIdx.y, p, c_pre, c_post);
}

// The strips' column sums added up, in a fixed order, and what they give.
struct ColumnArgs {
    const float *part_pre, *part_post;
    float *dpre, *dpost, *dgate;      // or null
    const float *gate, *post;         // a channel's, or null
    float beta;
    uint32_t strips, N;
};
constexpr uint32_t kColumnGroups = 32;  // of strips, side by side in a workgroup
__global__ __launch_bounds__(32 * kColumnGroups) void norm_columns(ColumnArgs a) {
    __shared__ double part[kColumnGroups][32];
    const uint32_t c = threadIdx.x % 32, group = threadIdx.x / 32, n = blockIdx.x * 32 + c;
    const bool pre = blockIdx.y == 0;
    if (pre ? !a.dpre : !(a.dpost || a.dgate)) return;
    const float *from = pre ? a.part_pre : a.part_post;
    double s = 0.0;
    if (n < a.N) {
#pragma unroll 8
        for (uint32_t i = group; i < a.strips; i += kColumnGroups) s += from[(uint64_t)i * a.N + n];
    }
    part[group][c] = s;
    __syncthreads();
    if (group || n >= a.N) return;
#pragma unroll
    for (uint32_t i = 1; i < kColumnGroups; ++i) s += part[i][c];
    if (pre) {
        a.dpre[n] = (float)s;
        return;
    }
    const float v = a.beta * (float)s;
    if (a.dpost) a.dpost[n] = a.gate ? v * a.gate[n] : v;
    if (a.dgate) a.dgate[n] = a.post ? v * a.post[n] : v;
}

// ---------------------------------------------------------------------------
// checks and layout
// ---------------------------------------------------------------------------

constexpr uint64_t kMostLd = 1ull << 40;

uint32_t bytes_of(int t) { return t == ENTQ_F32 ? 4 : t == ENTQ_I8 ? 1 : 2; }

// A matrix argument, which may be absent.
entq_status check_matrix(const void *p, int type, uint64_t ld, uint32_t rows, uint32_t cols, bool needed) {
    if (!p) return needed && rows && cols ? ENTQ_EINVAL : ENTQ_OK;
    if (ld < cols || ld > kMostLd) return ENTQ_EINVAL;
    return (uintptr_t)p % bytes_of(type) ? ENTQ_EALIGN : ENTQ_OK;
}

#define ENTQ_TRY(call)                            \
    do {                                          \
        const entq_status st_ = (call);           \
        if (st_ != ENTQ_OK) return st_;           \
    } while (0)

entq_status check_norm(const entq_norm *n) {
    if (!n || n->reserved) return ENTQ_EINVAL;
    if (n->type != ENTQ_BF16 && n->type != ENTQ_F16 && n->type != ENTQ_F32) return ENTQ_EINVAL;
    if (n->cols > ENTQ_INT8_MAX_COLS || n->rows > 0x7FFFFFFFu) return ENTQ_EINVAL;
    if (!(n->eps > 0.0f) || !std::isfinite(n->eps) || !std::isfinite(n->alpha) || !std::isfinite(n->beta))
        return ENTQ_EINVAL;
    if (n->gate < ENTQ_GATE_NONE || n->gate > ENTQ_GATE_FULL) return ENTQ_EINVAL;
    ENTQ_TRY(check_matrix(n->d_x, n->type, n->ldx, n->rows, n->cols, true));
    ENTQ_TRY(check_matrix(n->d_branch, n->type, n->ldbranch, n->rows, n->cols, false));
    const bool some = n->rows && n->cols;
    if (some && !n->d_branch && (n->d_post || n->gate != ENTQ_GATE_NONE)) return ENTQ_EINVAL;
    if ((n->gate == ENTQ_GATE_NONE) != !n->d_gate && (some || n->d_gate)) return ENTQ_EINVAL;
    if (n->gate == ENTQ_GATE_FULL) ENTQ_TRY(check_matrix(n->d_gate, n->type, n->ldgate, n->rows, n->cols, true));
    if (n->gate == ENTQ_GATE_TOKEN) ENTQ_TRY(check_matrix(n->d_gate, ENTQ_F32, n->ldgate, n->rows, 1, true));
    if (n->gate == ENTQ_GATE_CHANNEL && (uintptr_t)n->d_gate % 4) return ENTQ_EALIGN;
    if ((uintptr_t)n->d_post % 4 || (uintptr_t)n->d_pre % 4) return ENTQ_EALIGN;
    return ENTQ_OK;
}

NormArgs args_of(const entq_norm &n) {
    NormArgs a{};
    a.x = n.d_x;
    a.branch = n.d_branch;
    a.gate = n.d_gate;
    a.post = n.d_post;
    a.pre = n.d_pre;
    a.ldx = n.ldx;
    a.ldb = n.ldbranch;
    a.ldg = n.ldgate;
    a.M = n.rows;
    a.N = n.cols;
    a.per = n.cols ? 1.0 / n.cols : 0.0;
    a.gate_kind = n.gate;
    a.alpha = n.alpha;
    a.beta = n.beta;
    a.eps = n.eps;
    return a;
}

__global__ __launch_bounds__(256) void fill(float *p, uint64_t ld, uint32_t n) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i * ld] = 0.0f;
}
void zero(float *p, uint64_t ld, uint32_t n, hipStream_t s) {
    if (p && n) fill<<<(n + 255) / 256, 256, 0, s>>>(p, ld, n);
}

// How the backward pass runs: rows in the registers of `waves` waves, `vecs`
// pieces a thread, or (vecs 0) in two launches; and its strips of rows, each
// with column sums of its own, as many as the chip holds at a time. 4096 rows
// of bf16, us: 512 values 18.4 (512 strips 21.8; four waves a row 26.6), 2048
// 34.5 (256 strips 40.9, 1024 41.7; one piece in 8 waves 48.3), 4096 56.7 (512
// strips 64.0, two pieces in 8 waves 75), 8192 91.2 (in two launches 147). Rows
// of 16 waves keep no next row and no columns' factors: 2048 x 8192 fp32 101
// us (in two launches 136); of 16 bits they spill (210 us for 151).
struct BackPlan {
    uint32_t vecs, waves, strips;
};
BackPlan back_plan(const entq_norm &n) {
    const uint32_t per = n.type == ENTQ_F32 ? 4 : 8, pieces = (n.cols + per - 1) / per;
    const BackPlan p = pieces <= 64     ? BackPlan{1, 1, 1024}
                       : pieces <= 256  ? BackPlan{1, 4, 512}
                       : pieces <= 512  ? BackPlan{1, 8, 256}
                       : pieces <= 1024 ? BackPlan{2, 8, 256}
                       : pieces <= 2048 && per == 4 ? BackPlan{2, 16, 256}
                                        : BackPlan{0, 8, std::max(1u, 1024 / ((n.cols + 2047) / 2048))};
    return {p.vecs, p.waves, std::max(1u, std::min(n.rows, p.strips))};
}

struct Room {
    uint64_t stats, pre, post, all;
};
Room room_of(const entq_norm &n) {
    const auto up = [](uint64_t b) { return (b + 255) / 256 * 256; };
    Room r{};
    r.pre = back_plan(n).vecs ? 0 : up((uint64_t)n.rows * 16);
    const uint64_t one = up((uint64_t)back_plan(n).strips * n.cols * 4);
    r.post = r.pre + one;
    r.all = r.post + one;
    return r;
}

template <int TYPE, bool FULL>
void launch_back(const BackPlan &p, const NormArgs &a, hipStream_t s) {
    if (p.waves == 1) norm_back_rows<TYPE, 1, 1, FULL><<<(a.strips + 3) / 4, 256, 0, s>>>(a);
    if (p.waves == 4) norm_back_rows<TYPE, 1, 4, FULL><<<a.strips, 256, 0, s>>>(a);
    if (p.waves == 8 && p.vecs == 1) norm_back_rows<TYPE, 1, 8, FULL><<<a.strips, 512, 0, s>>>(a);
    if (p.waves == 8 && p.vecs == 2) norm_back_rows<TYPE, 2, 8, FULL><<<a.strips, 512, 0, s>>>(a);
    if constexpr (kPer<TYPE> == 4) {
        if (p.waves == 16) norm_back_rows<TYPE, 2, 16, FULL><<<a.strips, 1024, 0, s>>>(a);
    }
    if (!p.vecs) {
        norm_back_sums<TYPE, FULL><<<std::min(a.M, 1u << 20), 512, 0, s>>>(a);
        const uint32_t pieces = (a.N + kPer<TYPE> - 1) / kPer<TYPE>;
        norm_back_apply<TYPE, FULL><<<dim3((pieces + 255) / 256, a.strips), 256, 0, s>>>(a);
    }
}
template <int TYPE>
int launch_back(const BackPlan &p, const NormArgs &a, hipStream_t s) {
    if (a.gate_kind == ENTQ_GATE_FULL)
        launch_back<TYPE, true>(p, a, s);
    else
        launch_back<TYPE, false>(p, a, s);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

}  // namespace
}  // namespace entq

using namespace entq;

extern "C" {

entq_status entq_norm_block(const entq_norm *n, void *d_out, uint64_t ldout, void *d_y, int y_type, uint64_t ldy,
                            float *d_y_scales, void *stream) {
    ENTQ_TRY(check_norm(n));
    ENTQ_TRY(check_matrix(d_out, n->type, ldout, n->rows, n->cols, n->d_branch != nullptr));
    if (d_out && !n->d_branch) return ENTQ_EINVAL;
    if (!d_y && !n->d_branch && n->rows && n->cols) return ENTQ_EINVAL;  // nothing to do
    if (y_type != n->type && y_type != ENTQ_I8) return ENTQ_EINVAL;
    if (d_y || (y_type == ENTQ_I8 && d_y_scales)) {
        ENTQ_TRY(check_matrix(d_y, y_type, ldy, n->rows, n->cols, true));
        if (n->cols && !n->d_pre) return ENTQ_EINVAL;
        if ((y_type == ENTQ_I8) != (d_y_scales != nullptr) && n->rows) return ENTQ_EINVAL;
        if ((uintptr_t)d_y_scales % 4) return ENTQ_EALIGN;
    } else if (d_y_scales) {
        return ENTQ_EINVAL;
    }
    if (!n->rows) return ENTQ_OK;
    if (!n->cols) {  // (the scale of no codes: 0)
        if (!d_y_scales) return ENTQ_OK;
        zero(d_y_scales, 1, n->rows, (hipStream_t)stream);
        return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
    }
    NormArgs a = args_of(*n);
    a.out = d_out;
    a.ldo = ldout;
    a.y = d_y;
    a.ldy = ldy;
    a.scales = y_type == ENTQ_I8 ? d_y_scales : nullptr;
    const hipStream_t s = (hipStream_t)stream;
    return (entq_status)(n->type == ENTQ_BF16  ? launch_norm_typed<ENTQ_BF16>(a, s)
                         : n->type == ENTQ_F16 ? launch_norm_typed<ENTQ_F16>(a, s)
                                               : launch_norm_typed<ENTQ_F32>(a, s));
}

uint64_t entq_norm_block_backward_workspace_bytes(const entq_norm *n) {
    return check_norm(n) == ENTQ_OK ? room_of(*n).all : 0;
}

entq_status entq_norm_block_backward(const entq_norm *n, const void *d_dout, uint64_t lddout, const void *d_dy,
                                     uint64_t lddy, void *d_dx, uint64_t lddx, void *d_dbranch, uint64_t lddbranch,
                                     void *d_dgate, uint64_t lddgate, float *d_dpre, float *d_dpost,
                                     void *d_workspace, uint64_t workspace_bytes, void *stream) {
    ENTQ_TRY(check_norm(n));
    const bool some = n->rows && n->cols;
    if (some && !d_dout && !d_dy) return ENTQ_EINVAL;
    ENTQ_TRY(check_matrix(d_dout, n->type, lddout, n->rows, n->cols, false));
    ENTQ_TRY(check_matrix(d_dy, n->type, lddy, n->rows, n->cols, false));
    if (some && d_dy && !n->d_pre) return ENTQ_EINVAL;
    ENTQ_TRY(check_matrix(d_dx, n->type, lddx, n->rows, n->cols, false));
    ENTQ_TRY(check_matrix(d_dbranch, n->type, lddbranch, n->rows, n->cols, false));
    if (some && ((d_dbranch && !n->d_branch) || (d_dpre && !d_dy) || (d_dpost && !n->d_post))) return ENTQ_EINVAL;
    if (d_dgate && n->gate == ENTQ_GATE_NONE) return ENTQ_EINVAL;
    if (n->gate == ENTQ_GATE_FULL) ENTQ_TRY(check_matrix(d_dgate, n->type, lddgate, n->rows, n->cols, false));
    if (n->gate == ENTQ_GATE_TOKEN) ENTQ_TRY(check_matrix(d_dgate, ENTQ_F32, lddgate, n->rows, 1, false));
    if (n->gate == ENTQ_GATE_CHANNEL && (uintptr_t)d_dgate % 4) return ENTQ_EALIGN;
    if ((uintptr_t)d_dpre % 4 || (uintptr_t)d_dpost % 4) return ENTQ_EALIGN;
    const Room room = room_of(*n);
    if (room.all) {
        if (!d_workspace || workspace_bytes < room.all) return ENTQ_EWORKSPACE;
        if ((uintptr_t)d_workspace % 256) return ENTQ_EALIGN;
    }
    const hipStream_t s = (hipStream_t)stream;
    float *const channel = n->gate == ENTQ_GATE_CHANNEL ? (float *)d_dgate : nullptr;
    if (!some) {
        zero(d_dpre, 1, n->cols, s);
        zero(d_dpost, 1, n->cols, s);
        zero(channel, 1, n->cols, s);
        if (n->gate == ENTQ_GATE_TOKEN) zero((float *)d_dgate, lddgate, n->rows, s);
        return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
    }
    NormArgs a = args_of(*n);
    a.dout = d_dout;
    a.lddo = lddout;
    a.dy = d_dy;
    a.lddy = lddy;
    a.dx = d_dx;
    a.lddx = lddx;
    a.db = d_dbranch;
    a.lddb = lddbranch;
    a.dgate = channel ? nullptr : d_dgate;
    a.lddg = lddgate;
    a.stats = (float *)d_workspace;
    a.part_pre = d_dpre ? (float *)((uint8_t *)d_workspace + room.pre) : nullptr;
    a.part_post = d_dpost || channel ? (float *)((uint8_t *)d_workspace + room.post) : nullptr;
    const BackPlan plan = back_plan(*n);
    a.strips = plan.strips;
    const int r = n->type == ENTQ_BF16  ? launch_back<ENTQ_BF16>(plan, a, s)
                  : n->type == ENTQ_F16 ? launch_back<ENTQ_F16>(plan, a, s)
                                        : launch_back<ENTQ_F32>(plan, a, s);
    if (r != ENTQ_OK || !(d_dpre || d_dpost || channel)) return (entq_status)r;
    const ColumnArgs c{a.part_pre, a.part_post, d_dpre, d_dpost, channel,
                       n->gate == ENTQ_GATE_CHANNEL ? (const float *)n->d_gate : nullptr, n->d_post, n->beta,
                       a.strips, n->cols};
    norm_columns<<<dim3((n->cols + 31) / 32, 2), 32 * kColumnGroups, 0, s>>>(c);
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

}  // extern "C"
