// entq_int8.hip -- the int8 calls of entq.h: argument checks, workspace
// layout, the quantiser of activation rows and the small kernels around the
// products.
#include <algorithm>

#include "entq_int8.h"

namespace entq {
namespace {

// ---------------------------------------------------------------------------
// aligned copies
// ---------------------------------------------------------------------------

// Up to 3 matrices' rows of K codes at any address into rows of ldc (a
// multiple of 16), zeros after column K.
struct AlignJob {
    const int8_t *src;
    uint64_t ld;
    int8_t *dst;
    uint32_t rows, ldc, first;  // first: its first workgroup
};
struct AlignArgs {
    AlignJob job[3];
    uint32_t K;
};

// Pieces of 16 codes a thread. 1, 2 and 4 (us): the product of 333 x 5121 x
// 4099 29.3, 28.3, 27.6, gated back 515 x 2753 x 1031, whose copies are an
// eighth the size, 42.8, 42.9, 43.9.
constexpr uint32_t kAlignPieces = 2;

__device__ __forceinline__ void align_block(const AlignArgs &a, uint32_t block, uint32_t threads) {
    const AlignJob &j = a.job[block >= a.job[2].first ? 2 : block >= a.job[1].first ? 1 : 0];
    const uint32_t i = (block - j.first) * threads * kAlignPieces + threadIdx.x, pieces = j.ldc / 16;
    v4i v[kAlignPieces];
    int8_t *to[kAlignPieces];
#pragma unroll
    for (uint32_t u = 0; u < kAlignPieces; ++u) {
        const uint32_t p = i + u * threads, r = p / pieces, c = (p - r * pieces) * 16;
        to[u] = r < j.rows ? j.dst + (uint64_t)r * j.ldc + c : nullptr;
        if (to[u]) v[u] = load16_any(j.src + r * j.ld, c, a.K);
    }
#pragma unroll
    for (uint32_t u = 0; u < kAlignPieces; ++u)
        if (to[u]) *(v4i *)to[u] = v[u];
}

__global__ __launch_bounds__(256) void align_rows(AlignArgs a) { align_block(a, blockIdx.x, 256); }

// Collects copies; they run beside the quantiser where there is one, else in
// a launch of their own.
struct Aligner {
    AlignArgs a{};
    uint32_t n = 0;
    void add(const entq_rows &m, int8_t *dst, uint32_t ldc) {
        a.K = m.cols;
        a.job[n++] = {(const int8_t *)m.d_data, m.ld, dst, m.rows, ldc, 0};
    }
    // Their workgroups of that many threads; 0 where one launch cannot hold them.
    uint32_t blocks(uint32_t threads) {
        uint64_t all = 0;
        for (uint32_t i = 0; i < 3; ++i) {
            a.job[i].first = i < n ? (uint32_t)all : 0xFFFFFFFFu;
            const uint64_t per = threads * kAlignPieces;
            if (i < n) all += ((uint64_t)a.job[i].rows * (a.job[i].ldc / 16) + per - 1) / per;
            if (all * per >= 1ull << 32) return 0;
        }
        return (uint32_t)all;
    }
    int launch(hipStream_t s) {
        if (!n) return ENTQ_OK;
        const uint32_t b = blocks(256);
        if (!b) return ENTQ_EINVAL;
        align_rows<<<b, 256, 0, s>>>(a);
        return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
    }
};

// ---------------------------------------------------------------------------
// quantiser
// ---------------------------------------------------------------------------

// One workgroup per row, which is read once: VECS pieces of 16 bytes a thread
// stay in registers between the maximum and the rounding (VECS 0: any length,
// read twice, the second time out of the L2). Pieces may lie at any address.
// Bound by memory: 4096 x 28672 bf16 in 65.6 us, 5.4 TB/s, 4096 x 8192 fp32 in
// 24.7 us, 6.8 TB/s (in part out of the last-level cache); reading each element
// twice as single values took 233 us for the first.
// Columns K..pad-1 are written as 0. The workgroups after the rows make copies.
template <int TYPE, int VECS, int THREADS>
__global__ __launch_bounds__(THREADS) void quantize_rows(const void *x, uint64_t ldx, uint32_t K, int8_t *codes,
                                                         uint64_t ldc, uint32_t pad, float *scales, uint32_t rows,
                                                         AlignArgs copies) {
    if (blockIdx.x >= rows) return align_block(copies, blockIdx.x - rows, THREADS);
    constexpr int kPer = TYPE == ENTQ_F32 ? 4 : 8, kBytes = TYPE == ENTQ_F32 ? 4 : 2;
    __shared__ uint32_t top[THREADS / 64];
    const uint64_t row = blockIdx.x;
    const uint8_t *src = (const uint8_t *)x + row * ldx * kBytes;
    int8_t *dst = codes + row * ldc;
    const uint32_t full = K / kPer;  // whole pieces
    uint32_t big = 0;
    auto take = [&](float v) { big = max(big, __float_as_uint(v) & 0x7FFFFFFFu); };
    auto piece = [&](uint32_t p) { return ((const any16 *)(src + (uint64_t)p * 16))->v; };
    v4i held[VECS ? VECS : 1];
    if (VECS) {
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const uint32_t p = i * THREADS + threadIdx.x;
            held[i] = p < full ? piece(p) : v4i{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < VECS; ++i)
#pragma unroll
            for (int e = 0; e < kPer; ++e) take(act_of<TYPE>(held[i], e));
    } else {
        for (uint32_t p = threadIdx.x; p < full; p += THREADS) {
            const v4i v = piece(p);
#pragma unroll
            for (int e = 0; e < kPer; ++e) take(act_of<TYPE>(v, e));
        }
    }
    const uint32_t rest = full * kPer + threadIdx.x;  // the last columns, one a thread
    float last = 0.0f;
    if (rest < K) take(last = load_act<TYPE>(src, rest));
    big = wave_max(big);
    if (threadIdx.x % 64 == 0) top[threadIdx.x / 64] = big;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) big = max(big, top[i]);
    const Quantizer z(big);
    if (threadIdx.x == 0) scales[row] = z.scale;
    auto put = [&](uint32_t p, v4i v) {
        if constexpr (kPer == 8)
            ((any8 *)(dst + p * 8))->v = v2i{(int)z.code4<TYPE>(v, 0), (int)z.code4<TYPE>(v, 4)};
        else
            ((any4 *)(dst + p * 4))->v = (int)z.code4<TYPE>(v, 0);
    };
    if (VECS) {
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const uint32_t p = i * THREADS + threadIdx.x;
            if (p < full) put(p, held[i]);
        }
    } else {
        for (uint32_t p = threadIdx.x; p < full; p += THREADS) put(p, piece(p));
    }
    if (rest < K) dst[rest] = (int8_t)z.code(last);
    for (uint32_t c = K + threadIdx.x; c < pad; c += THREADS) dst[c] = 0;
}

template <int TYPE>
void quantize_typed(const entq_rows &x, uint32_t rows, uint64_t skip, int8_t *codes, uint64_t ldc, uint32_t pad,
                    float *scales, Aligner &copies, hipStream_t s) {
    const void *p = (const uint8_t *)x.d_data + skip * x.ld * (TYPE == ENTQ_F32 ? 4 : 2);
    int8_t *c = codes + skip * ldc;
    float *sc = scales + skip;
    const uint32_t pieces = x.cols / (TYPE == ENTQ_F32 ? 4 : 8);
    const uint32_t threads = pieces <= 256 ? 256 : pieces <= 1024 ? 512 : 1024;
    const uint32_t more = copies.n ? copies.blocks(threads) : 0;
    const dim3 grid(rows + more);
    if (pieces <= 256)
        quantize_rows<TYPE, 1, 256><<<grid, 256, 0, s>>>(p, x.ld, x.cols, c, ldc, pad, sc, rows, copies.a);
    else if (pieces <= 1024)
        quantize_rows<TYPE, 2, 512><<<grid, 512, 0, s>>>(p, x.ld, x.cols, c, ldc, pad, sc, rows, copies.a);
    else if (pieces <= 4096)
        quantize_rows<TYPE, 4, 1024><<<grid, 1024, 0, s>>>(p, x.ld, x.cols, c, ldc, pad, sc, rows, copies.a);
    else
        quantize_rows<TYPE, 0, 1024><<<grid, 1024, 0, s>>>(p, x.ld, x.cols, c, ldc, pad, sc, rows, copies.a);
    if (more) copies.n = 0;  // done
}

int launch_quantize(const entq_rows &x, int8_t *codes, uint64_t ldc, uint32_t pad, float *scales,
                    Aligner &copies, hipStream_t s) {
    if (x.rows == 0) return ENTQ_OK;
    constexpr uint32_t kRows = 1u << 20;  // a launch's threads stay below 2^32
    for (uint64_t r = 0; r < x.rows; r += kRows) {
        const uint32_t n = (uint32_t)std::min<uint64_t>(kRows, x.rows - r);
        if (x.type == ENTQ_BF16) quantize_typed<ENTQ_BF16>(x, n, r, codes, ldc, pad, scales, copies, s);
        if (x.type == ENTQ_F16) quantize_typed<ENTQ_F16>(x, n, r, codes, ldc, pad, scales, copies, s);
        if (x.type == ENTQ_F32) quantize_typed<ENTQ_F32>(x, n, r, codes, ldc, pad, scales, copies, s);
    }
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

// Whether the products can read the codes where they are.
bool direct(const entq_rows &m) {
    return (uintptr_t)m.d_data % 16 == 0 && m.ld % 16 == 0 && m.cols % 16 == 0 && m.ld < (1u << 23);
}

// ---------------------------------------------------------------------------
// backward helpers
// ---------------------------------------------------------------------------

// The scaled gradients' rows in F16. Bound by memory: gated back 2048 x 28672 x
// 8192 takes 2.48 ms with it, 2.25 ms in bf16, whose products write 16 bits
// themselves; product back 2048 x 8192 x 8192 341 us (bf16 320).
template <bool TWO, int THREADS, int HELD>
__global__ __launch_bounds__(THREADS) void narrow_rows(Int8Args a) {
    __shared__ uint32_t top[16];
    for (uint32_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        narrow_row<TWO, HELD>(a, m, top);
        __syncthreads();
    }
}

template <bool TWO>
void launch_narrow(const Int8Args &a, hipStream_t s) {
    const dim3 grid(std::min(a.M, 65535u));
    const uint64_t quads = a.ldd / 4 * (TWO ? 2 : 1);
    if (quads <= 2048)
        narrow_rows<TWO, 256, 8><<<grid, 256, 0, s>>>(a);
    else
        narrow_rows<TWO, 1024, 8><<<grid, 1024, 0, s>>>(a);
}

__global__ __launch_bounds__(kSumThreads) void sum_parts(SumArgs a) { sum_parts_block(a, blockIdx.x); }

// d = dy sw in bf16, zeros in columns N..ldd-1: what the backward epilogue
// writes, for a call that needs no sums of codes. A thread: 4 channels.
__global__ __launch_bounds__(256) void scale_gradient(Int8Args a) {
    const uint32_t n = 4 * (blockIdx.x * 256 + threadIdx.x);
    if (n >= a.ldd) return;
    float scale[2][4];
    load_scales<kBwd>(a, n, scale);
    for (uint64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
        const uint2 v = load_grad4(a, (uint32_t)m, n);
        const uint16_t b[4] = {(uint16_t)v.x, (uint16_t)(v.x >> 16), (uint16_t)v.y, (uint16_t)(v.y >> 16)};
        uint16_t d[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            d[i] = n + i < a.N ? bits16(from16(b[i], false) * scale[0][i], false) : 0;
        *(uint2 *)(a.d[0] + m * a.ldd + n) = make_uint2(d[0] | (uint32_t)d[1] << 16, d[2] | (uint32_t)d[3] << 16);
    }
}

__global__ __launch_bounds__(256) void fill_zero(uint8_t *p, uint64_t ld, uint64_t bytes) {
    for (uint64_t c = blockIdx.x * 256 + threadIdx.x; c < bytes; c += gridDim.x * 256)
        p[blockIdx.y * ld + c] = 0;
}

// ---------------------------------------------------------------------------
// checks and layout
// ---------------------------------------------------------------------------

// Channels of a backward call: keeps byte offsets inside a tile of scaled
// gradients below 2^32.
constexpr uint32_t kMaxBackChannels = 1u << 22;

uint32_t type_bytes(int t) { return t == ENTQ_F32 ? 4 : t == ENTQ_I8 ? 1 : 2; }

entq_status check_rows(const entq_rows *r, bool acts, bool codes) {
    if (!r || r->reserved) return ENTQ_EINVAL;
    if (r->type < ENTQ_BF16 || r->type > ENTQ_I8) return ENTQ_EINVAL;
    if (r->type == ENTQ_I8 ? !codes : !acts) return ENTQ_EINVAL;
    if (r->cols > ENTQ_INT8_MAX_COLS || r->rows > 0x7FFFFFFFu || r->ld < r->cols) return ENTQ_EINVAL;
    if (r->ld > (1ull << 40)) return ENTQ_EINVAL;
    if (r->rows && r->cols && !r->d_data) return ENTQ_EINVAL;
    if (r->type == ENTQ_I8 && r->rows && !r->d_scales) return ENTQ_EINVAL;
    if (r->type != ENTQ_I8 && r->d_scales) return ENTQ_EINVAL;
    if ((uintptr_t)r->d_data % type_bytes(r->type) || (uintptr_t)r->d_scales % 4) return ENTQ_EALIGN;
    return ENTQ_OK;
}

entq_status check_out(const void *p, int type, uint64_t ld, uint32_t rows, uint32_t cols) {
    if (type != ENTQ_BF16 && type != ENTQ_F16 && type != ENTQ_F32) return ENTQ_EINVAL;
    if (ld < cols || ld > (1ull << 40)) return ENTQ_EINVAL;
    if (rows && cols && !p) return ENTQ_EINVAL;
    if ((uintptr_t)p % type_bytes(type)) return ENTQ_EALIGN;
    return ENTQ_OK;
}

// Takes pieces of the workspace in order; with base null it only counts.
struct Pieces {
    uint8_t *base;
    uint64_t used = 0;
    explicit Pieces(void *b) : base((uint8_t *)b) {}
    template <class T>
    T *take(uint64_t n) {
        const uint64_t at = used;
        used += (n * sizeof(T) + 255) / 256 * 256;
        return base ? (T *)(base + at) : nullptr;
    }
};

struct Call {
    Int8Mode mode;
    const entq_rows *x, *w[2], *dy;
    int n_w;
    entq_status bad;
};

Call describe(Int8Mode mode, const entq_rows *x, const entq_rows *w0, const entq_rows *w1, const entq_rows *dy) {
    Call c{mode, x, {w0, w1}, dy, mode == kGated || mode == kGatedBwd ? 2 : 1, ENTQ_OK};
    const bool back = mode == kBwd || mode == kGatedBwd;
    if ((c.bad = check_rows(x, !back, true)) != ENTQ_OK) return c;
    for (int i = 0; i < c.n_w; ++i) {
        if ((c.bad = check_rows(c.w[i], false, true)) != ENTQ_OK) return c;
        if (c.w[i]->cols != x->cols || c.w[i]->rows != w0->rows) {
            c.bad = ENTQ_EINVAL;
            return c;
        }
    }
    if (back) {
        // (the gradient's columns are channels: not bounded by the sums' limit)
        if (!dy || dy->reserved || (dy->type != ENTQ_BF16 && dy->type != ENTQ_F16) || dy->d_scales ||
            dy->rows != x->rows || dy->cols != w0->rows || dy->ld < dy->cols || dy->ld > (1ull << 40) ||
            (dy->rows && dy->cols && !dy->d_data))
            c.bad = ENTQ_EINVAL;
        else if (w0->rows > kMaxBackChannels)
            c.bad = ENTQ_EINVAL;
        else if ((uintptr_t)dy->d_data % 2)
            c.bad = ENTQ_EALIGN;
    }
    return c;
}

// What a call keeps in the workspace.
struct Layout {
    int8_t *codes;      // quantised activations or an aligned copy of codes, or null
    float *scales;
    uint64_t ldc;
    int8_t *w[2];       // aligned copies of weights, or null
    uint32_t ldw;
    int32_t *sums;      // the splits' integer sums, or null
    uint16_t *d[2];     // scaled gradients
    float *wide[2];     // in fp32, or null
    float *back;        // F16: one for each token
    uint64_t ldd;
    float *part[2];
    Int8Plan plan;
    GradPlan grad;
    float *parts;       // partial sums of dX, or null
    uint64_t bytes;
};

Layout lay_out(const Call &c, void *ws) {
    Layout l{};
    Pieces p(ws);
    const uint64_t M = c.x->rows, N = c.w[0]->rows;
    l.ldc = (c.x->cols + 127ull) / 128 * 128;
    l.ldd = (N + 63) / 64 * 64;
    l.ldw = (c.x->cols + 15) / 16 * 16;
    l.plan = int8_plan(c.mode, c.x->type, (uint32_t)M, (uint32_t)N, l.ldw);
    if (c.x->type != ENTQ_I8 && !l.plan.quantizes) {
        l.codes = p.take<int8_t>(M * l.ldc);
        l.scales = p.take<float>(M);
    } else if (c.x->type == ENTQ_I8 && !l.plan.few && !direct(*c.x)) {
        l.codes = p.take<int8_t>(M * l.ldc);
    }
    const bool copies = !l.plan.few || c.mode == kBwd || c.mode == kGatedBwd;
    if (l.plan.splits > 1) l.sums = p.take<int32_t>(l.plan.splits * c.n_w * M * ((N + 3) / 4 * 4));
    for (int i = 0; i < c.n_w; ++i)
        if (copies && !direct(*c.w[i])) l.w[i] = p.take<int8_t>(N * l.ldw);
    if (c.mode == kBwd || c.mode == kGatedBwd) {
        for (int i = 0; i < c.n_w; ++i) {
            l.d[i] = p.take<uint16_t>(M * l.ldd);
            if (c.mode == kGatedBwd && c.dy->type == ENTQ_F16) l.wide[i] = p.take<float>(M * l.ldd);
            l.part[i] = p.take<float>((uint64_t)l.plan.part_rows * N);
        }
        if (c.dy->type == ENTQ_F16) l.back = p.take<float>(M);
        l.grad = grad_plan((uint32_t)M, (uint32_t)N, l.ldw, c.n_w);
        if (l.grad.splits > 1) l.parts = p.take<float>((uint64_t)l.grad.splits * M * l.ldw);
    }
    l.bytes = p.used;
    return l;
}

uint64_t workspace_bytes_of(const Call &c) { return c.bad == ENTQ_OK ? lay_out(c, nullptr).bytes : 0; }

entq_status zero_rows(void *p, int type, uint64_t ld, uint32_t rows, uint32_t cols, hipStream_t s) {
    if (!p || !rows || !cols) return ENTQ_OK;
    const uint64_t b = type_bytes(type), bytes = cols * b;
    for (uint32_t r = 0; r < rows; r += 65535) {
        const uint32_t n = std::min(rows - r, 65535u);
        const dim3 grid((uint32_t)std::min<uint64_t>(rows > 64 ? 64 : 4096, bytes / 256 + 1), n);
        fill_zero<<<grid, 256, 0, s>>>((uint8_t *)p + r * ld * b, ld * b, bytes);
    }
    return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
}

// The products' operands: quantised or copied into the workspace where they
// have to be.
entq_status operands(const Call &c, const Layout &l, Int8Args &a, hipStream_t s) {
    a = Int8Args{};
    a.M = c.x->rows;
    a.N = c.w[0]->rows;
    a.K = l.plan.few ? c.x->cols : l.ldw;
    a.splits = l.plan.splits;
    a.sums = l.sums;
    a.x = (const int8_t *)c.x->d_data;
    a.sx = c.x->d_scales;
    a.ldx = c.x->ld;
    a.x_type = l.plan.quantizes ? c.x->type : (int)ENTQ_I8;
    Aligner copies;
    if (l.codes) {
        a.x = l.codes;
        a.ldx = l.ldc;
        if (c.x->type == ENTQ_I8) copies.add(*c.x, l.codes, (uint32_t)l.ldc);
    }
    for (int i = 0; i < c.n_w; ++i) {
        a.w[i] = (const int8_t *)c.w[i]->d_data;
        a.ldw[i] = c.w[i]->ld;
        a.sw[i] = c.w[i]->d_scales;
        if (l.w[i]) {
            copies.add(*c.w[i], l.w[i], l.ldw);
            a.w[i] = l.w[i];
            a.ldw[i] = l.ldw;
        }
    }
    int r = ENTQ_OK;
    if (c.x->type != ENTQ_I8 && !l.plan.quantizes) {
        r = launch_quantize(*c.x, l.codes, l.ldc, (uint32_t)l.ldc, l.scales, copies, s);
        a.sx = l.scales;
    }
    return (entq_status)(r != ENTQ_OK ? r : copies.launch(s));
}

entq_status check_workspace(const void *ws, uint64_t bytes, uint64_t need) {
    if (!need) return ENTQ_OK;
    if (!ws || bytes < need) return ENTQ_EWORKSPACE;
    return (uintptr_t)ws % 256 ? ENTQ_EALIGN : ENTQ_OK;
}

entq_status forward(const Call &c, int act, void *y, int type, uint64_t ldy, void *ws, uint64_t ws_bytes,
                    hipStream_t s) {
    if (c.bad != ENTQ_OK) return c.bad;
    entq_status st = check_out(y, type, ldy, c.x->rows, c.w[0]->rows);
    if (st != ENTQ_OK) return st;
    if ((st = check_workspace(ws, ws_bytes, workspace_bytes_of(c))) != ENTQ_OK) return st;
    if (c.x->rows == 0 || c.w[0]->rows == 0) return ENTQ_OK;
    if (c.x->cols == 0) return zero_rows(y, type, ldy, c.x->rows, c.w[0]->rows, s);
    const Layout l = lay_out(c, ws);
    Int8Args a;
    if ((st = operands(c, l, a, s)) != ENTQ_OK) return st;
    a.act = act;
    a.y = y;
    a.type = type;
    a.ldy = ldy;
    return (entq_status)launch_int8_product(c.mode, l.plan, a, s);
}

entq_status backward(const Call &c, int act, void *dx, uint64_t lddx, float *ds0, float *ds1, void *ws,
                     uint64_t ws_bytes, hipStream_t s) {
    if (c.bad != ENTQ_OK) return c.bad;
    const uint32_t M = c.x->rows, N = c.w[0]->rows, K = c.x->cols;
    if (dx) {
        const entq_status st = check_out(dx, c.dy->type, lddx, M, K);
        if (st != ENTQ_OK) return st;
    }
    if ((uintptr_t)ds0 % 4 || (uintptr_t)ds1 % 4) return ENTQ_EALIGN;
    entq_status st = check_workspace(ws, ws_bytes, workspace_bytes_of(c));
    if (st != ENTQ_OK) return st;
    if (M == 0 || N == 0 || K == 0) {
        if (zero_rows(dx, c.dy->type, lddx, M, K, s) != ENTQ_OK) return ENTQ_EHIP;
        if (zero_rows(ds0, ENTQ_F32, N, 1, N, s) != ENTQ_OK) return ENTQ_EHIP;
        return zero_rows(ds1, ENTQ_F32, N, 1, N, s);
    }
    if (!dx && !ds0 && !ds1) return ENTQ_OK;
    const Layout l = lay_out(c, ws);
    Int8Args a;
    if ((st = operands(c, l, a, s)) != ENTQ_OK) return st;
    const bool f16 = c.dy->type == ENTQ_F16;
    a.act = act;
    a.y = const_cast<void *>(c.dy->d_data);
    a.type = c.dy->type;
    a.ldy = c.dy->ld;
    a.ldd = l.ldd;
    // (one block of tokens: its sums are the results)
    const bool direct_sums = l.plan.part_rows == 1;
    float *const ds[2] = {ds0, ds1};
    SumArgs sums{};
    sums.n = N;
    for (int i = 0; i < c.n_w; ++i) {
        a.d[i] = dx ? l.d[i] : nullptr;
        a.wide[i] = dx ? l.wide[i] : nullptr;
        a.part[i] = !ds[i] ? nullptr : direct_sums ? ds[i] : l.part[i];
        sums.part[i] = l.part[i];
        sums.out[i] = ds[i];
    }
    if ((ds0 || ds1) && !direct_sums) sums.rows = l.plan.part_rows;
    int r = ENTQ_OK;
    const bool narrow = f16 && dx;
    a.back = l.back;
    a.narrows = narrow && c.mode == kBwd && ds0 && l.plan.splits > 1;
    if (narrow && c.mode == kBwd && !a.narrows) launch_narrow<false>(a, s);
    if (c.mode == kBwd && !ds0) {
        if (!f16) scale_gradient<<<dim3((uint32_t)(l.ldd / 4 + 255) / 256, std::min(M, 65535u)), 256, 0, s>>>(a);
    } else {
        r = launch_int8_product(c.mode, l.plan, a, s);
    }
    if (narrow && c.mode == kGatedBwd && r == ENTQ_OK) launch_narrow<true>(a, s);
    if (r != ENTQ_OK || hipGetLastError() != hipSuccess) return r != ENTQ_OK ? (entq_status)r : ENTQ_EHIP;
    if (!dx) {
        if (sums.rows) sum_parts<<<sum_blocks(sums), kSumThreads, 0, s>>>(sums);
        return hipGetLastError() == hipSuccess ? ENTQ_OK : ENTQ_EHIP;
    }
    GradArgs g{};
    for (int i = 0; i < c.n_w; ++i) {
        g.d[i] = l.d[i];
        g.w[i] = a.w[i];
        g.ldw[i] = a.ldw[i];
    }
    g.ldd = l.ldd;
    g.M = M;
    g.N = N;
    g.K = l.ldw;
    g.cols = K;
    g.splits = l.grad.splits;
    g.parts = l.parts;
    g.n_w = c.n_w;
    g.f16 = f16;
    g.dx = dx;
    g.lddx = lddx;
    g.back = a.back;
    g.sums = sums;
    return (entq_status)launch_grad_product(l.grad, g, s);
}

bool bad_act(int act) { return act < ENTQ_ACT_SILU || act > ENTQ_ACT_RELU; }

}  // namespace
}  // namespace entq

using entq::describe;

extern "C" {

entq_status entq_quantize_rows(const entq_rows *x, int8_t *d_codes, uint64_t ldc, float *d_scales,
                               void *stream) {
    const entq_status st = entq::check_rows(x, true, false);
    if (st != ENTQ_OK) return st;
    if (ldc < x->cols || ldc > (1ull << 40)) return ENTQ_EINVAL;
    if (x->rows && ((x->cols && !d_codes) || !d_scales)) return ENTQ_EINVAL;
    if ((uintptr_t)d_scales % 4) return ENTQ_EALIGN;
    entq::Aligner none;
    return (entq_status)entq::launch_quantize(*x, d_codes, ldc, x->cols, d_scales, none, (hipStream_t)stream);
}

uint64_t entq_int8_gemm_workspace_bytes(const entq_rows *x, const entq_rows *w) {
    return entq::workspace_bytes_of(describe(entq::kFwd, x, w, nullptr, nullptr));
}

entq_status entq_int8_gemm(const entq_rows *x, const entq_rows *w, void *d_y, int y_type, uint64_t ldy,
                           void *d_workspace, uint64_t workspace_bytes, void *stream) {
    return entq::forward(describe(entq::kFwd, x, w, nullptr, nullptr), 0, d_y, y_type, ldy, d_workspace,
                         workspace_bytes, (hipStream_t)stream);
}

uint64_t entq_int8_gated_workspace_bytes(const entq_rows *x, const entq_rows *gate, const entq_rows *up) {
    return entq::workspace_bytes_of(describe(entq::kGated, x, gate, up, nullptr));
}

entq_status entq_int8_gated(const entq_rows *x, const entq_rows *gate, const entq_rows *up, int activation,
                            void *d_h, int h_type, uint64_t ldh, void *d_workspace, uint64_t workspace_bytes,
                            void *stream) {
    if (entq::bad_act(activation)) return ENTQ_EINVAL;
    return entq::forward(describe(entq::kGated, x, gate, up, nullptr), activation, d_h, h_type, ldh, d_workspace,
                         workspace_bytes, (hipStream_t)stream);
}

uint64_t entq_int8_gemm_backward_workspace_bytes(const entq_rows *dy, const entq_rows *x, const entq_rows *w) {
    return entq::workspace_bytes_of(describe(entq::kBwd, x, w, nullptr, dy));
}

entq_status entq_int8_gemm_backward(const entq_rows *dy, const entq_rows *x, const entq_rows *w, void *d_dx,
                                    uint64_t lddx, float *d_dw_scales, void *d_workspace,
                                    uint64_t workspace_bytes, void *stream) {
    return entq::backward(describe(entq::kBwd, x, w, nullptr, dy), 0, d_dx, lddx, d_dw_scales, nullptr,
                          d_workspace, workspace_bytes, (hipStream_t)stream);
}

uint64_t entq_int8_gated_backward_workspace_bytes(const entq_rows *dh, const entq_rows *x, const entq_rows *gate,
                                                  const entq_rows *up) {
    return entq::workspace_bytes_of(describe(entq::kGatedBwd, x, gate, up, dh));
}

entq_status entq_int8_gated_backward(const entq_rows *dh, const entq_rows *x, const entq_rows *gate,
                                     const entq_rows *up, int activation, void *d_dx, uint64_t lddx,
                                     float *d_dgate_scales, float *d_dup_scales, void *d_workspace,
                                     uint64_t workspace_bytes, void *stream) {
    if (entq::bad_act(activation)) return ENTQ_EINVAL;
    return entq::backward(describe(entq::kGatedBwd, x, gate, up, dh), activation, d_dx, lddx, d_dgate_scales,
                          d_dup_scales, d_workspace, workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"
