/* A linear layer with bias, activation and residual, and its gradient
 * (msim_linear and msim_linear_backward of include/msim.h, which has the
 * definitions).
 */

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "msim_gemm.h"

namespace {

/* ------------------------------------------------------------------------ */
/* few rows                                                                  */
/* ------------------------------------------------------------------------ */

/* A linear layer of up to 16 MT rows: 16 outs a workgroup, whose wavefronts
 * share k.  The weights are read once, from where they lie on any element.  A small
 * one is as long as a launch; 16 x 4,096 -> 4,096 bf16 takes 9.5 us, 3.5 TB/s. */
struct FewP {
    const void *x, *w;
    uint64_t x_ld, w_ld;
    uint32_t K;
    Epilogue e;
};

template <int MODE, int MT, int WAVES> __global__ void __launch_bounds__(64 * WAVES) msim_linear_few(FewP p)
{
    typedef typename Type<MODE>::D D;
    typedef typename D::raw raw;
    __shared__ __attribute__((aligned(16))) char lds[WAVES * STREAM_LDS<MT, 1>];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = lane & 15;
    const uint32_t n0 = blockIdx.x * 16;
    Rows<D> w[1], x[MT];
    w[0].set([&](uint32_t r) { return (const raw *)p.w + min(n0 + r, p.e.N - 1) * p.w_ld; });
    for (int i = 0; i < MT; i++) x[i].set([&](uint32_t r) { return (const raw *)p.x + min(i * 16 + r, p.e.M - 1) * p.x_ld; });
    f32x4 acc[MT][1];
    for (int i = 0; i < MT; i++) acc[i][0] = f32x4{0, 0, 0, 0};
    stream<D, MT, 1, WAVES>(w, x, p.K, wave, lds + wave * STREAM_LDS<MT, 1>, acc);
    join<MT, 1, WAVES>(lds, wave, acc);
    _Pragma("unroll") for (int i = 0; i < MT; i++) {
        const uint32_t m = i * 16 + l, n = n0 + (lane >> 4) * 4, have = n < p.e.N ? min(4u, p.e.N - n) : 0;
        if (i % WAVES != (int)wave || m >= p.e.M) continue;
        float v[4];
        for (uint32_t k = 0; k < 4; k++) {
            v[k] = acc[i][0][k] + (p.e.bias && k < have ? p.e.bias[n + k] : 0.0f);
            if (p.e.pre && k < have) ((raw *)p.e.pre)[m * p.e.pre_ld + n + k] = D::put(v[k]);
        }
        if (MODE == M_F32 || p.e.out32) act_of<4, true>(v, p.e.act);
        else act_of<4, false>(v, p.e.act);
        for (uint32_t k = 0; k < have; k++) {
            const uint64_t at = m * p.e.res_ld + n + k;
            if (p.e.res) v[k] += p.e.out32 ? ((const float *)p.e.res)[at] : D::get(((const raw *)p.e.res)[at]);
            if (p.e.out32) ((float *)p.e.out)[m * p.e.out_ld + n + k] = v[k];
            else ((raw *)p.e.out)[m * p.e.out_ld + n + k] = D::put(v[k]);
        }
    }
}

/* ------------------------------------------------------------------------ */
/* operands that do not lie as the product reads them                        */
/* ------------------------------------------------------------------------ */

/* rows x cols of a strided matrix to rows of `wide` columns, zeros behind the last; TWO: as sums of two bf16 */
struct PackP {
    const void *from;
    uint64_t ld;
    void *to;
    uint32_t rows, cols, wide, blocks;
};

template <typename D, bool TWO> __device__ __forceinline__ void pack_rows(const PackP &p, uint32_t block)
{
    constexpr uint32_t PER = TWO ? 8 : 16 / sizeof(typename D::raw);
    const uint32_t turns = p.wide / PER;
    const uint64_t n = (uint64_t)p.rows * turns;
    _Pragma("unroll 2") for (uint64_t id = block * 256ull + threadIdx.x; id < n; id += p.blocks * 256ull) {
        const uint64_t r = id / turns;
        const uint32_t c = (uint32_t)(id - r * turns) * PER;
        if constexpr (TWO) {
            float v[8];
            load8<D>(v, p.from, r * p.ld + c, c < p.cols ? min(8u, p.cols - c) : 0);
            store_two(v, p.to, split_at(p.wide, (uint32_t)r, c));
        } else
            *(u32x4 *)((typename D::raw *)p.to + r * p.wide + c) = piece<D>((const typename D::raw *)p.from + r * p.ld, c, p.cols);
    }
}

/* What is further than MAX from 0 taken as that far, infinities too; a NaN stays one. */
template <int MAX> __device__ __forceinline__ float within(float z) { return z < -MAX ? -MAX : z > MAX ? MAX : z; }

/* v[i] = the activation's slope at v[i].  Far from 0 it is 0 or 1 in 32 bits, but a product of 0 and what overflows is
 * NaN (gelu_tanh from -1.2e13 on, all at infinities): taken where both factors are still finite and the one that is 0
 * or 1 is so, e^-142 and e^-200 being 0 and their reciprocals infinite. */
template <int N, bool FULL> __device__ __forceinline__ void slope_of(float *v, uint32_t act)
{
    switch (act) {
    case MSIM_ACT_RELU: return each<N>(v, [](float z) { return z > 0 ? 1.0f : z != z ? z : 0.0f; });
    case MSIM_ACT_SILU:
        return each<N>(v, [](float y) {
            const float z = within<200>(y), s = logistic<FULL>(z);
            return s * (1.0f + z * (1.0f - s));
        });
    case MSIM_ACT_GELU:
        return each<N>(v, [](float y) {
            const float z = within<20>(y);
            return normal_below<FULL>(z) + z * 0.39894228f * expf(-0.5f * z * z);
        });
    case MSIM_ACT_GELU_TANH:
        return each<N>(v, [](float y) {
            const float z = within<12>(y), s = logistic<FULL>(z * (TANH_A + TANH_B * z * z));
            return s * (1.0f + (1.0f - s) * z * (TANH_A + 3.0f * TANH_B * z * z));
        });
    }
}

/* 131,072 x 256 without an activation, for the bias alone, 36 us, 1.9 TB/s; 2,047 x 513 f32 6 us.
 *
 * The gradient in front of the activation, d = grad act'(pre), as the products
 * read it, and the sums of its columns over each workgroup's rows.  A workgroup
 * has `part` rows and 8 * lanes columns.  d is rounded to the operands' type,
 * as a matrix instruction reads it, half a step of that type; the sums are of what is
 * not rounded.  TWO: a grad of 32 bits beside f16, whose range it may leave on both sides
 * (a mean's over 10^5 rows has elements below 6e-8): d, x and weight as sums of two
 * bf16, 16 bits in the range of 32, and three products (8,192 x 1,024 -> 4,096 400 us, and
 * 177 of single f16; 2,047 x 1,000 -> 513 35 and 31). */

struct GradP {
    const void *grad, *pre;
    uint64_t grad_ld, pre_ld;
    void *d;                     /* NULL: grad itself is read by the products */
    float *sums;                 /* [blocks of rows][outs] (dbias itself, of one block), or NULL */
    uint32_t rows, outs, wide;   /* wide: columns of d */
    uint32_t act, grad32, lglanes, part, blocks;
};

/* eight elements as they lie, the first n of them there, others zero */
template <typename D> __device__ __forceinline__ auto raw8(const void *at, uint64_t i, uint32_t n)
{
    typedef typename D::raw raw;
    typedef raw vec __attribute__((ext_vector_type(8)));
    typedef raw loose __attribute__((ext_vector_type(8), aligned(sizeof(raw))));
    const raw *q = (const raw *)at + i;
    if (n == 8) return (vec)*(const loose *)q;
    vec v = 0;
    for (uint32_t k = 0; k < 8; k++)
        if (k < n) v[k] = q[k];
    return v;
}

/* The sums of a thread's eight columns (k of them there) over its rows, m and every `step`-th up to end, two of
 * which are read before the first is used; G: the type of grad. */
template <typename D, typename G, bool TWO> __device__ __forceinline__ void grad_columns(const GradP &p, uint32_t m, uint32_t step, uint32_t end, uint32_t n, uint32_t k, float *sum)
{
    constexpr uint32_t U = 2;
    for (; m < end; m += U * step) {
        decltype(raw8<G>(nullptr, 0, 0)) g[U];
        decltype(raw8<D>(nullptr, 0, 0)) z[U];
        _Pragma("unroll") for (uint32_t u = 0; u < U; u++) {
            const uint32_t row = m + u * step, there = row < end ? k : 0;
            g[u] = raw8<G>(p.grad, row * p.grad_ld + n, there);
            if (p.act) z[u] = raw8<D>(p.pre, row * p.pre_ld + n, there);
        }
        _Pragma("unroll") for (uint32_t u = 0; u < U; u++) {
            const uint32_t row = m + u * step;
            if (row >= end) break;
            float v[8], slope[8];
            for (uint32_t i = 0; i < 8; i++) v[i] = G::get(g[u][i]);
            if (p.act) {
                for (uint32_t i = 0; i < 8; i++) slope[i] = D::get(z[u][i]);
                slope_of<8, std::is_same<D, F32>::value>(slope, p.act);
                for (uint32_t i = 0; i < 8; i++) v[i] = i < k ? v[i] * slope[i] : 0.0f;
            }
            for (int i = 0; i < 8; i++) sum[i] += v[i];
            if (p.d) {
                if constexpr (TWO) store_two(v, p.d, split_at(p.wide, row, n));
                else store8<D>(v, p.d, (uint64_t)row * p.wide + n, 8);
            }
        }
    }
}

template <typename D, bool TWO> __device__ __forceinline__ void grad_rows(const GradP &p, uint32_t block, float *part)
{
    const uint32_t lanes = 1u << p.lglanes, cols = 8 * lanes;
    const uint32_t across = (p.wide + cols - 1) / cols, by = block / across, bx = block - by * across;
    const uint32_t n = bx * cols + (threadIdx.x & (lanes - 1)) * 8, k = n < p.outs ? min(8u, p.outs - n) : 0;
    const uint32_t first = by * p.part + (threadIdx.x >> p.lglanes), step = 256u >> p.lglanes, end = min(p.rows, (by + 1) * p.part);
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n < p.wide) {
        if (TWO || p.grad32) grad_columns<D, F32, TWO>(p, first, step, end, n, k, sum);
        else grad_columns<D, D, false>(p, first, step, end, n, k, sum);
    }
    if (!p.sums) return;
    /* lanes of the same columns together, then the four wavefronts */
    for (int i = 0; i < 8; i++)
        for (uint32_t d = lanes; d < 64; d *= 2) sum[i] += __shfl_xor(sum[i], d);
    if ((threadIdx.x & 63) < lanes)
        for (int i = 0; i < 8; i++) part[(threadIdx.x >> 6) * cols + (threadIdx.x & 63) * 8 + i] = sum[i];
    __syncthreads();
    const uint32_t c = threadIdx.x;
    if (c < cols && bx * cols + c < p.outs)
        p.sums[(uint64_t)by * p.outs + bx * cols + c] = part[c] + part[cols + c] + part[2 * cols + c] + part[3 * cols + c];
}

/* What the products of a call need first: x and weight packed, and the gradient. */
template <typename D, bool TWO> __global__ void __launch_bounds__(256) msim_linear_prepare(PackP x, PackP w, GradP g)
{
    __shared__ float part[4 * 256];
    if (blockIdx.x < x.blocks) pack_rows<D, TWO>(x, blockIdx.x);
    else if (blockIdx.x < x.blocks + w.blocks) pack_rows<D, TWO>(w, blockIdx.x - x.blocks);
    else grad_rows<D, TWO>(g, blockIdx.x - x.blocks - w.blocks, part);
}

/* ------------------------------------------------------------------------ */
/* host: products                                                            */
/* ------------------------------------------------------------------------ */

uint32_t size_of(uint32_t dtype) { return dtype == MSIM_F32 ? 4 : 2; }
constexpr uint64_t MAX_LD = 8000000;       /* bytes: the offsets of a tile's 256 rows stay below 2^31 */

/* Whether the products read rows of `cols` elements as they lie: 16 bytes at a time,
 * which end with the row and lie on 4. */
bool ready(const void *at, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t size)
{
    return (uintptr_t)at % 4 == 0 && cols * size % 16 == 0 && (rows <= 1 || (ld * size % 4 == 0 && ld * size <= MAX_LD));
}

/* A rows x cols matrix as an operand: as it lies, or packed at ws, as sums of two bf16 (two). */
struct Matrix {
    const void *at;
    uint64_t rows, cols, ld;
    uint32_t size;
    bool packed, two;
    uint64_t wide() const { return two ? up(cols, 32) : packed ? up(cols, 16 / size) : cols; }
    uint64_t row() const { return wide() * (two ? 4 : size); }
    uint64_t bytes() const { return packed ? up(rows * row(), 256) : 0; }
    Operand operand(const char *ws) const
    {
        if (packed) return {ws, rows * row(), row(), 0};
        return {(const char *)at, rows ? ((rows - 1) * ld + cols) * size : 0, (rows > 1 ? ld : cols) * size, 0};
    }
};

Matrix matrix_of(const void *at, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t size, bool two = false)
{
    return {at, rows, cols, ld, size, two || !ready(at, rows, cols, ld, size), two};
}

PackP pack_of(const Matrix &m, char *ws)
{
    if (!m.packed || !m.rows) return {};
    const uint64_t n = m.rows * m.wide() / (m.two ? 8 : 16 / m.size);
    return {m.at, m.ld, ws, (uint32_t)m.rows, (uint32_t)m.cols, (uint32_t)m.wide(), (uint32_t)std::min<uint64_t>((n + 511) / 512, 1u << 14)};
}

template <typename D, bool TWO = false> hipError_t prepare(const PackP &x, const PackP &w, const GradP &g, hipStream_t st)
{
    const uint32_t grid = x.blocks + w.blocks + g.blocks;
    return grid ? launch(msim_linear_prepare<D, TWO>, grid, 256, 0, st, x, w, g) : hipSuccess;
}

const char *check_linear(const msim_linear_spec *s, int *code)
{
    *code = MSIM_E_ARG;
    if (!s) return "linear: null spec";
    if (s->version != MSIM_ABI_VERSION) return "linear: spec version mismatch";
    if (s->dtype > MSIM_BF16) return "linear: unknown dtype";
    if (s->out_dtype != s->dtype && s->out_dtype != MSIM_F32) return "linear: out_dtype must be dtype or MSIM_F32";
    if (s->act > MSIM_ACT_SILU) return "linear: unknown activation";
    if (!s->cols || !s->outs) return "linear: cols and outs must be at least 1";
    *code = MSIM_E_LIMIT;
    if (s->rows >> 31) return "linear: 2^31 rows or more";
    if (s->cols > MSIM_MAX_LINEAR || s->outs > MSIM_MAX_LINEAR) return "linear: cols or outs above MSIM_MAX_LINEAR";
    if (s->rows * s->cols >> 40 || s->rows * s->outs >> 40) return "linear: 2^40 elements or more";
    for (uint64_t ld : {s->x_stride, s->weight_stride, s->out_stride, s->residual_stride, s->pre_stride, s->dx_stride, s->dweight_stride})
        if (ld >> 40) return "linear: a stride of 2^40 or more";
    *code = MSIM_E_ARG;
    if (s->x_stride < s->cols && s->rows > 1) return "linear: x_stride below cols";
    if (s->weight_stride < s->cols && s->outs > 1) return "linear: weight_stride below cols";
    if (s->out_stride < s->outs && s->rows > 1) return "linear: out_stride below outs";
    return nullptr;
}

/* Few rows are streamed while that is faster than tiles, in the stream of calls: up to
 * 16 of them 16 x 4,096 -> 4,096 bf16 9.5 us (14.0 in tiles, which is two launches),
 * -> 16,384 33.7 (22.0), 16 x 20,000 -> 256 16.4 (14.1); up to 64 64 x 2,048 -> 4,096 10.5
 * (11.0), 64 x 2,001 -> 2,001 f16 10.3 (17.8), 32 x 4,096 -> 4,096 19.1 (14.0), 64 x 2,048
 * -> 512 f32 15.9 (14.5).  A workgroup's 16 wavefronts take 4 KiB of k at a time, so long
 * rows want several workgroups: tiles of parts of k. */
bool few_rows(const msim_linear_spec *s)
{
    const uint64_t size = size_of(s->dtype);
    if (s->outs > MSIM_LINEAR_FEW_OUTS) return false;
    if (s->rows <= MSIM_LINEAR_FEW) return s->cols * size <= 16384;
    return s->rows <= 64 && s->cols <= (size == 4 ? 1024 : 4096) && s->cols * size * s->outs <= 1u << 24;
}

struct Forward {
    Matrix x, w;
    Plan plan;
    uint64_t bytes;
    bool few;
};

Forward forward_of(const msim_linear_spec *s, const void *x, const void *weight)
{
    Forward f = {};
    const uint32_t size = size_of(s->dtype);
    f.few = few_rows(s);
    f.x = matrix_of(x, s->rows, s->cols, s->x_stride, size);
    f.w = matrix_of(weight, s->outs, s->cols, s->weight_stride, size);
    if (f.few) return f;
    f.plan = plan_of(s->dtype, {s->rows, s->outs, f.x.wide(), 1});
    f.bytes = f.x.bytes() + f.w.bytes() + f.plan.part_bytes;
    return f;
}

template <int MODE>
int run_forward(const msim_linear_spec *s, const Forward &f, const Epilogue &e, char *ws, hipStream_t st)
{
    if (f.few) {
        const FewP q = {f.x.at, f.w.at, f.x.ld, f.w.ld, s->cols, e};
        const uint32_t grid = (s->outs + 15) / 16;
        const hipError_t r = s->rows > 32 ? launch(msim_linear_few<MODE, 4, 8>, grid, 512, 0, st, q)
            : s->rows > 16 ? launch(msim_linear_few<MODE, 2, 16>, grid, 1024, 0, st, q) : launch(msim_linear_few<MODE, 1, 16>, grid, 1024, 0, st, q);
        return launched(r, "linear launch");
    }
    GemmP p = {};
    char *wx = ws, *ww = wx + f.x.bytes();
    p.a = f.x.operand(wx);
    p.b = f.w.operand(ww);
    p.M = (uint32_t)s->rows;
    p.N = s->outs;
    p.K = (uint32_t)f.x.wide();
    p.batch = 1;
    p.part = (float *)(ww + f.w.bytes());
    p.e = e;
    hipError_t r = prepare<typename Type<MODE>::D>(pack_of(f.x, wx), pack_of(f.w, ww), GradP{}, st);
    if (r == hipSuccess) r = launch_gemm<MODE, false>(p, f.plan, st);
    return launched(r, "linear launch");
}

/* The backward pass: d (the gradient in front of the activation), its columns' sums, and two products. */
struct Backward {
    Matrix x, w;
    bool own;                    /* d is made: an activation, another type, or a grad that does not lie as it is read */
    bool two;                    /* operands as sums of two bf16: f16 and a grad of 32 bits */
    uint64_t wide, row;          /* columns of d, bytes of a row */
    uint64_t d_bytes, sum_bytes;
    uint32_t blocks, part;       /* of rows, for the sums, and rows of one */
    Plan px, pw;
    uint64_t bytes;
};

Backward backward_of(const msim_linear_spec *s, const void *x, const void *weight, const void *grad, bool dx, bool dw, bool db)
{
    Backward b = {};
    const uint32_t size = size_of(s->dtype);
    dx &= s->rows != 0;
    const bool need = dx || dw;
    b.two = need && s->dtype == MSIM_F16 && s->out_dtype == MSIM_F32;
    if (dw) b.x = matrix_of(x, s->rows, s->cols, s->x_stride, size, b.two);
    if (dx) b.w = matrix_of(weight, s->outs, s->cols, s->weight_stride, size, b.two);
    b.own = need && (s->act || s->out_dtype != s->dtype || !ready(grad, s->rows, s->outs, s->out_stride, size));
    b.wide = b.own ? up(s->outs, b.two ? 32 : 8) : s->outs;
    b.row = b.wide * (b.two ? 4 : size);
    /* a thread has 8 columns: two rows of them at least where there are several workgroups of rows, of which there are about
     * 1,024 at most */
    uint32_t lanes = 1;
    while (lanes < 32 && 8 * lanes < s->outs) lanes *= 2;
    b.part = s->rows <= 256 ? 256 : (uint32_t)std::max<uint64_t>(512 / lanes, (s->rows + 1023) / 1024);
    b.blocks = (uint32_t)((s->rows + b.part - 1) / b.part);
    b.d_bytes = b.own ? up(s->rows * b.row, 256) : 0;
    b.sum_bytes = db ? up((uint64_t)b.blocks * s->outs * 4, 256) : 0;
    const Product x1 = {s->rows, s->cols, b.wide, 1}, w1 = {s->outs, s->cols, s->rows, 1};
    const uint32_t mode = b.two ? (uint32_t)M_TWO : s->dtype;
    if (dx && dw) plan_pair(mode, x1, w1, &b.px, &b.pw);
    else if (dx) b.px = plan_of(mode, x1);
    else if (dw) b.pw = plan_of(mode, w1);
    b.bytes = b.x.bytes() + b.w.bytes() + b.d_bytes + b.sum_bytes + b.px.part_bytes + b.pw.part_bytes;
    return b;
}

template <int MODE>
int run_backward(const msim_linear_spec *s, const Backward &b, const void *grad, const void *pre, void *dx, void *dweight,
                 float *dbias, char *ws, hipStream_t st)
{
    typedef typename Type<MODE>::D D;
    const uint32_t size = size_of(s->dtype);
    char *wx = ws, *ww = wx + b.x.bytes(), *wd = ww + b.w.bytes(), *wsum = wd + b.d_bytes, *wpart = wsum + b.sum_bytes;
    GradP g = {};
    if ((b.own || dbias) && s->rows) {
        g = {grad, pre, s->out_stride, s->pre_stride, b.own ? wd : nullptr, !dbias ? nullptr : b.blocks == 1 ? dbias : (float *)wsum,
             (uint32_t)s->rows, s->outs, b.own ? (uint32_t)b.wide : (uint32_t)up(s->outs, 8), s->act, s->out_dtype == MSIM_F32, 0, b.part, 0};
        /* of rows for one workgroup 64 at a time, four a thread (69 x 142 f16 with gelu 22 -> 9 us) */
        while (g.lglanes < (b.blocks == 1 ? 2 : 5) && (8u << g.lglanes) < g.wide) g.lglanes++;
        g.blocks = b.blocks * ((g.wide + (8u << g.lglanes) - 1) / (8u << g.lglanes));
    }
    hipError_t r = prepare<D, MODE == M_TWO>(dweight ? pack_of(b.x, wx) : PackP{}, dx ? pack_of(b.w, ww) : PackP{}, g, st);
    const Columns c = dbias && b.blocks != 1 ? Columns{(const float *)wsum, b.blocks, s->outs, dbias} : Columns{};
    const Operand d = b.own ? Operand{wd, s->rows * b.row, b.row, 0}
                            : Matrix{grad, s->rows, s->outs, s->out_stride, size, false, false}.operand(nullptr);
    GemmP px = {}, pw = {};
    if (dx) {
        px.a = d;
        px.b = b.w.operand(ww);
        px.M = px.e.M = (uint32_t)s->rows;
        px.N = px.e.N = s->cols;
        px.K = (uint32_t)b.wide;
        px.batch = 1;
        px.part = (float *)wpart;
        px.e.out = dx;
        px.e.out_ld = s->dx_stride;
    }
    if (dweight) {
        pw.a = d;
        pw.b = b.x.operand(wx);
        pw.M = pw.e.M = s->outs;
        pw.N = pw.e.N = s->cols;
        pw.K = (uint32_t)s->rows;
        pw.batch = 1;
        pw.part = (float *)(wpart + b.px.part_bytes);
        pw.e.out = dweight;
        pw.e.out_ld = s->dweight_stride;
    }
    if (r == hipSuccess) r = launch_pair<MODE>(px, b.px, pw, b.pw, c, st);
    return launched(r, "linear backward launch");
}

}   // namespace

extern "C" int msim_linear_workspace(const msim_linear_spec *s, const void *x, const void *weight, uint64_t *bytes)
{
    int code;
    if (const char *why = check_linear(s, &code)) return fail(code, why);
    if (!bytes) return fail(MSIM_E_ARG, "linear: null bytes");
    *bytes = s->rows ? forward_of(s, x, weight).bytes : 0;
    return MSIM_OK;
}

extern "C" int msim_linear(const msim_linear_spec *s, const void *x, const void *weight, const float *bias,
                           const void *residual, void *out, void *pre, void *workspace, uint64_t workspace_bytes,
                           void *hip_stream)
{
    int code;
    if (const char *why = check_linear(s, &code)) return fail(code, why);
    if (s->rows == 0) return MSIM_OK;
    if (!x || !weight || !out) return fail(MSIM_E_ARG, "linear: null x, weight or out");
    if (residual && s->rows > 1 && s->residual_stride < s->outs) return fail(MSIM_E_ARG, "linear: residual_stride below outs");
    if (pre && s->rows > 1 && s->pre_stride < s->outs) return fail(MSIM_E_ARG, "linear: pre_stride below outs");
    if (residual == out && s->rows > 1 && s->residual_stride != s->out_stride)
        return fail(MSIM_E_ARG, "linear: residual is out, with two strides");
    const Forward f = forward_of(s, x, weight);
    if (int rc = check_workspace(workspace, workspace_bytes, f.bytes, "linear: workspace missing, too small or not on 256 bytes")) return rc;
    Epilogue e = {};
    e.M = (uint32_t)s->rows;
    e.N = s->outs;
    e.out = out;
    e.out_ld = s->out_stride;
    e.bias = bias;
    e.res = residual;
    e.res_ld = s->residual_stride;
    e.pre = pre;
    e.pre_ld = s->pre_stride;
    e.act = s->act;
    e.out32 = s->out_dtype == MSIM_F32 && s->dtype != MSIM_F32;
    char *ws = (char *)workspace;
    hipStream_t st = (hipStream_t)hip_stream;
    return s->dtype == MSIM_F32 ? run_forward<M_F32>(s, f, e, ws, st)
        : s->dtype == MSIM_F16 ? run_forward<M_F16>(s, f, e, ws, st) : run_forward<M_BF16>(s, f, e, ws, st);
}

extern "C" int msim_linear_backward_workspace(const msim_linear_spec *s, const void *x, const void *weight, const void *grad,
                                              uint32_t dx, uint32_t dweight, uint32_t dbias, uint64_t *bytes)
{
    int code;
    if (const char *why = check_linear(s, &code)) return fail(code, why);
    if (!bytes) return fail(MSIM_E_ARG, "linear: null bytes");
    *bytes = backward_of(s, x, weight, grad, dx, dweight, dbias).bytes;
    return MSIM_OK;
}

extern "C" int msim_linear_backward(const msim_linear_spec *s, const void *x, const void *weight, const void *pre,
                                    const void *grad, void *dx, void *dweight, float *dbias, void *workspace,
                                    uint64_t workspace_bytes, void *hip_stream)
{
    int code;
    if (const char *why = check_linear(s, &code)) return fail(code, why);
    if (s->rows && (!grad || (dx && !weight) || (dweight && !x))) return fail(MSIM_E_ARG, "linear: null grad, weight or x");
    if (s->act && s->rows && !pre) return fail(MSIM_E_ARG, "linear: the gradient of an activation needs pre");
    if (s->act && s->rows > 1 && s->pre_stride < s->outs) return fail(MSIM_E_ARG, "linear: pre_stride below outs");
    if (!s->rows) dx = nullptr;            /* nothing of it: weight, which may be NULL then, is not read */
    if (dx && s->rows > 1 && s->dx_stride < s->cols) return fail(MSIM_E_ARG, "linear: dx_stride below cols");
    if (dweight && s->outs > 1 && s->dweight_stride < s->cols) return fail(MSIM_E_ARG, "linear: dweight_stride below cols");
    const Backward b = backward_of(s, x, weight, grad, dx, dweight, dbias);
    if (int rc = check_workspace(workspace, workspace_bytes, b.bytes, "linear: workspace missing, too small or not on 256 bytes")) return rc;
    char *ws = (char *)workspace;
    hipStream_t st = (hipStream_t)hip_stream;
    return s->dtype == MSIM_F32 ? run_backward<M_F32>(s, b, grad, pre, dx, dweight, dbias, ws, st)
        : b.two ? run_backward<M_TWO>(s, b, grad, pre, dx, dweight, dbias, ws, st)
        : s->dtype == MSIM_F16 ? run_backward<M_F16>(s, b, grad, pre, dx, dweight, dbias, ws, st)
                               : run_backward<M_BF16>(s, b, grad, pre, dx, dweight, dbias, ws, st);
}
