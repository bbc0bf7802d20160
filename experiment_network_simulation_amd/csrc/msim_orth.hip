/* The orthogonal update of a weight matrix by Newton-Schulz products
 * (msim_orthogonalize of include/msim.h, which has the definition).
 *
 * X, P = X X^T and B = b P + c P P are held as sums of two f16, 22 bits, and a
 * product is three of f16: their rate leaves it three times as fast as one of 32
 * bits, and its error near that.  Only one side of P and B, which are
 * symmetric, is computed.
 */

#include <algorithm>
#include <cmath>

#include "msim_gemm.h"

namespace {

/* X is held times this: its singular values stay near 1, so high parts are well
 * inside f16 and low parts above its subnormal numbers where they matter. */
constexpr float ORTH_SCALE = 2048.0f;
constexpr uint32_t NORM_PARTS = 256;
/* a product of several steps' factors, which reaches a^3, is held times this less */
constexpr float PASS_DOWN = 16.0f;

/* Sums of squares in 64 bits: NORM_PARTS workgroups a matrix, or as many as have an element (4 of 2,048 x 7,168 bf16
 * 27 us, 4.3 TB/s).  part: [matrix][workgroups]. */
template <typename D> uint32_t norm_parts(uint64_t size)
{
    constexpr uint64_t EACH = 256 * 16 / sizeof(typename D::raw);
    return (uint32_t)std::min<uint64_t>(NORM_PARTS, (size + EACH - 1) / EACH);
}
template <typename D> __global__ void __launch_bounds__(256) msim_orth_norm(const void *from, uint64_t size, double *part, uint32_t parts, uint32_t first)
{
    constexpr uint32_t PER = 16 / sizeof(typename D::raw);
    typedef typename D::raw vec __attribute__((ext_vector_type(PER)));
    __shared__ double sums[4];
    const uint32_t block = first + blockIdx.x, batch = block / parts, k = block - batch * parts;
    const typename D::raw *x = (const typename D::raw *)from + batch * size;
    double s = 0;
    _Pragma("unroll 2") for (uint64_t i = (k * 256 + threadIdx.x) * PER; i < size; i += (uint64_t)parts * 256 * PER) {
        const vec v = __builtin_bit_cast(vec, i + PER <= size ? piece<D>(x + i) : piece<D>(x + i, 0, (uint32_t)(size - i)));
        for (uint32_t j = 0; j < PER; j++) {
            const double d = D::get(v[j]);
            s += d * d;
        }
    }
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) part[block] = sums[0] + sums[1] + sums[2] + sums[3];
}

/* what X is the update times: one wavefront asks, all its lanes know.  A norm that is not finite makes it NaN. */
__device__ __forceinline__ double scale_of(const double *part, uint32_t batch, uint32_t parts, double eps)
{
    const uint32_t lane = threadIdx.x & 63;
    part += (uint64_t)batch * parts;
    double s = 0;
    for (uint32_t k = 0; k < NORM_PARTS; k += 64) s += lane + k < parts ? part[lane + k] : 0.0;
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    return s < INFINITY ? ORTH_SCALE / (sqrt(s) + eps) : NAN;
}

struct OrthP {
    const void *in;
    void *out;
    char *x;                     /* split, m rows of ld columns */
    const double *part;
    uint64_t rows, cols, ld, batch;        /* batch: bytes between matrices of x */
    double eps;
    uint32_t parts, first;
};

/* Tiles of 32 x 64 between the caller's matrices and X (flip: its transpose, through
 * LDS).  BEGIN: X = scale in / (norm + eps); otherwise out = X / scale.  A launch
 * each; what bounds them is the way from the norm's parts to the result, so the
 * elements are asked for before those. */
template <typename D, bool BEGIN, bool FLIP> __global__ void __launch_bounds__(256) msim_orth_move(OrthP p)
{
    typedef typename D::raw raw;
    __shared__ float tile[32][65];
    __shared__ double factor;
    const uint64_t m = FLIP ? p.cols : p.rows, n = FLIP ? p.rows : p.cols;
    const uint64_t tn = (p.ld + 63) / 64, tm = (m + 31) / 32;
    const uint64_t block = p.first + blockIdx.x;
    const uint32_t batch = (uint32_t)(block / (tm * tn)), at = (uint32_t)(block - batch * tm * tn);
    const uint64_t m0 = at / tn * 32, n0 = at % tn * 64;
    char *x = p.x + batch * p.batch;
    const uint64_t base = batch * p.rows * p.cols;
    /* eight columns of a row of X; there are `there` of them in the caller's */
    const uint32_t r = threadIdx.x / 8, c = threadIdx.x % 8 * 8;
    const uint64_t row = m0 + r, col = n0 + c;
    const bool mine = row < m && col < p.ld;
    const uint32_t there = mine && col < n ? (uint32_t)min((uint64_t)8, n - col) : 0;
    float v[8];
    if constexpr (BEGIN) {
        raw u[8];
        if constexpr (FLIP) {
            for (uint32_t i = 0; i < 8; i++) {
                const uint64_t mm = m0 + threadIdx.x % 32, nn = n0 + i * 8 + threadIdx.x / 32;
                u[i] = mm < m && nn < n ? ((const raw *)p.in)[base + nn * p.cols + mm] : raw(0);
            }
        } else {
            load8<D>(v, p.in, base + row * p.cols + col, there);
        }
        if (threadIdx.x < 64) {
            const double f = scale_of(p.part, batch, p.parts, p.eps);
            if (threadIdx.x == 0) factor = f;
        }
        if constexpr (FLIP)
            for (uint32_t i = 0; i < 8; i++) tile[threadIdx.x % 32][i * 8 + threadIdx.x / 32] = D::get(u[i]);
        __syncthreads();
        if (!mine) return;
        for (int i = 0; i < 8; i++) v[i] = (float)(factor * (double)(FLIP ? tile[r][c + i] : v[i]));
        store_split(v, x, split_at(p.ld, (uint32_t)row, (uint32_t)col));
    } else {
        if (mine) {
            load_split(v, x, split_at(p.ld, (uint32_t)row, (uint32_t)col));
            for (int i = 0; i < 8; i++) v[i] *= 1.0f / ORTH_SCALE;
        }
        if constexpr (!FLIP) {
            store8<D>(v, p.out, base + row * p.cols + col, there);
        } else {
            if (mine)
                for (int i = 0; i < 8; i++) tile[r][c + i] = v[i];
            __syncthreads();
            for (uint32_t i = 0; i < 8; i++) {
                const uint64_t mm = m0 + threadIdx.x % 32, nn = n0 + i * 8 + threadIdx.x / 32;
                if (mm < m && nn < n) ((raw *)p.out)[base + nn * p.cols + mm] = D::put(tile[threadIdx.x % 32][i * 8 + threadIdx.x / 32]);
            }
        }
    }
}

/* ------------------------------------------------------------------------ */
/* matrices of up to 64 rows (of X): a launch a step                         */
/* ------------------------------------------------------------------------ */

/* A workgroup has a slab of X's columns in LDS.  A step takes the slabs' sums of
 * products together to P, makes B = b P + c P P by itself, X = a X + B X of its
 * slab, and the slab's part of the next P.  Bound by latency: a launch, the parts
 * through memory, and four products one after another (64 x 1,000 bf16 48 us, in
 * separate products 110). */
constexpr uint32_t SLAB_ROWS = 64, SLAB_COLS = 256, SLABS = 32;       /* at most */
constexpr uint32_t SLAB_THREADS = 512;

struct SlabP {
    const void *in;
    void *out;
    const double *norm;
    char *x;                     /* slabs as they lie in LDS, kept from step to step */
    const float *part;           /* [count][slabs][ROWS][ROWS] of the step before */
    float *next;
    uint64_t size, sm, sn;       /* of in and out: elements of a matrix, between rows and columns of X */
    double eps;
    uint32_t m, n, slabs, wide;  /* wide: columns of a slab, a multiple of 32 */
    uint32_t first, last, parts;           /* parts: of the norm */
    float a, b, c;
};

/* ROWS (32 or 64) rows by 32 columns of a split matrix in LDS: rows of 128 bytes,
 * high parts and low ones, in pieces of 16 that are exchanged by the row; further
 * columns follow. */
template <uint32_t ROWS> struct Slab {
    static constexpr uint32_t BYTES = ROWS * 128;    /* of 32 columns */
    typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
    typedef int16_t i16x4 __attribute__((ext_vector_type(4)));

    /* where the parts of columns c, c + 1, ... of a row begin */
    static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t c, uint32_t low)
    {
        return c / 32 * BYTES + row * 128 + ((c % 32 / 8 + low * 4) ^ (row >> 1 & 7)) * 16 + c % 8 * 2;
    }
    /* four columns */
    static __device__ __forceinline__ void put(char *lds, uint32_t row, uint32_t c, const float *v)
    {
        u16x4 h, l;
        for (int i = 0; i < 4; i++) {
            uint16_t a, b;
            split_of(v[i], a, b);
            h[i] = a;
            l[i] = b;
        }
        *(u16x4 *)(lds + at(row, c, 0)) = h;
        *(u16x4 *)(lds + at(row, c, 1)) = l;
    }
    static __device__ __forceinline__ void get(const char *lds, uint32_t row, uint32_t c, float *v)
    {
        const u16x4 h = *(const u16x4 *)(lds + at(row, c, 0)), l = *(const u16x4 *)(lds + at(row, c, 1));
        for (int i = 0; i < 4; i++) v[i] = F16::get(h[i]) + F16::get(l[i]);
    }
    /* fragments: 32 rows from `row` on, 16 columns from c on */
    static __device__ __forceinline__ f16x8 rows(const char *lds, uint32_t row, uint32_t c, uint32_t low)
    {
        const uint32_t lane = threadIdx.x & 63;
        return *(const f16x8 *)(lds + at(row + (lane & 31), c + (lane >> 5) * 8, low));
    }
    /* 16 rows from `row` on, 32 columns from c on, transposed */
    static __device__ __forceinline__ f16x8 columns(const char *lds, uint32_t row, uint32_t c, uint32_t low)
    {
        const uint32_t lane = threadIdx.x & 63, r = row + (lane >> 5) * 8 + (lane >> 2 & 3), k = c + (lane >> 4 & 1) * 16 + (lane & 3) * 4;
        typedef __attribute__((address_space(3))) i16x4 *ptr;
        const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds + at(r, k, low)));
        const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds + at(r + 4, k, low)));
        return __builtin_bit_cast(f16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

typedef float f32x16 __attribute__((ext_vector_type(16)));

/* all four products: the low parts' own, which tiles leave out, halves the error of a small matrix and costs no time here */
__device__ __forceinline__ f32x16 mma_split(f16x8 ah, f16x8 al, f16x8 bh, f16x8 bl, f32x16 c)
{
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(al, bl, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(al, bh, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah, bl, c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(ah, bh, c, 0, 0, 0);
}

/* rows i .. times rows j .. over columns k0 .. k1 - 1: lane l has row i + l % 32 and columns j + 8 g + 4 (l / 32) + 0 .. 3 */
template <uint32_t ROWS> __device__ __forceinline__ f32x16 slab_square(const char *lds, uint32_t i, uint32_t j, uint32_t k0, uint32_t k1)
{
    typedef Slab<ROWS> S;
    f32x16 c = 0.0f;
    for (uint32_t k = k0; k < k1; k += 16) c = mma_split(S::rows(lds, j, k, 0), S::rows(lds, j, k, 1), S::rows(lds, i, k, 0), S::rows(lds, i, k, 1), c);
    return c;
}

template <typename D, uint32_t ROWS> __global__ void __launch_bounds__(SLAB_THREADS) msim_orth_slab(SlabP p)
{
    typedef typename D::raw raw;
    typedef Slab<ROWS> S;
    constexpr uint32_t BLOCKS = ROWS / 32 * (ROWS / 32), WAVES = SLAB_THREADS / 64, RUNS = WAVES / BLOCKS;
    constexpr uint32_t SQUARE = ROWS * ROWS, PER = SQUARE / SLAB_THREADS;          /* elements of P, and of them a thread's */
    __shared__ __attribute__((aligned(256))) char xs[SLAB_COLS / 32 * S::BYTES], ps[ROWS / 32 * S::BYTES], bs[ROWS / 32 * S::BYTES];
    __shared__ f32x4 sums[(WAVES - BLOCKS) * 4 * 64];
    __shared__ double factor;
    const uint32_t batch = blockIdx.x / p.slabs, slab = blockIdx.x - batch * p.slabs, n0 = slab * p.wide, tid = threadIdx.x;
    const uint32_t lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane & 31, half = lane >> 5;
    const uint32_t block = wave % BLOCKS, i = block % (ROWS / 32) * 32, j = block / (ROWS / 32) * 32;    /* of a ROWS x ROWS product */
    char *const kept = p.x + (uint64_t)blockIdx.x * (p.wide / 32 * S::BYTES);
    const uint32_t units = ROWS * p.wide / 4, pieces = p.wide / 32 * (S::BYTES / 16);
    /* four columns of a row; neighbouring lanes take neighbouring elements of the caller's matrix */
    const auto unit = [&](uint32_t e, uint32_t &row, uint32_t &c) {
        if (p.sn == 1) row = e / (p.wide / 4), c = e % (p.wide / 4) * 4;
        else row = e % ROWS, c = e / ROWS * 4;
    };
    if (p.first) {
        if (tid < 64) {
            const double f = scale_of(p.norm, batch, p.parts, p.eps);
            if (tid == 0) factor = f;
        }
        __syncthreads();
        const double f = factor;
        const raw *in = (const raw *)p.in + batch * p.size;
        _Pragma("unroll 2") for (uint32_t e = tid; e < units; e += SLAB_THREADS) {
            uint32_t row, c;
            unit(e, row, c);
            float v[4];
            for (uint32_t k = 0; k < 4; k++)
                v[k] = row < p.m && n0 + c + k < p.n ? (float)(f * (double)D::get(in[row * p.sm + (n0 + c + k) * p.sn])) : 0.0f;
            S::put(xs, row, c, v);
        }
    } else {
        typedef float part __attribute__((ext_vector_type(PER < 4 ? PER : 4)));
        constexpr uint32_t N = PER < 4 ? PER : 4, V = PER / N;
        part sum[V] = {};
        const part *q = (const part *)(p.part + (uint64_t)batch * p.slabs * SQUARE) + tid;
        _Pragma("unroll 8") for (uint32_t s = 0; s < p.slabs; s++, q += SQUARE / N)
            for (uint32_t k = 0; k < V; k++) sum[k] += q[k * SLAB_THREADS];
        for (uint32_t e = tid; e < pieces; e += SLAB_THREADS) ((u32x4 *)xs)[e] = ((const u32x4 *)kept)[e];
        for (uint32_t k = 0; k < V; k++) {
            const uint32_t e = (k * SLAB_THREADS + tid) * N, row = e / ROWS, c = e % ROWS;
            for (uint32_t t = 0; t < N; t++) {
                uint16_t h, lo;
                split_of(sum[k][t] * (1.0f / ORTH_SCALE), h, lo);
                *(uint16_t *)(ps + S::at(row, c + t, 0)) = h;
                *(uint16_t *)(ps + S::at(row, c + t, 1)) = lo;
            }
        }
        __syncthreads();
        if (wave < BLOCKS) {
            const f32x16 sq = slab_square<ROWS>(ps, i, j, 0, ROWS);
            for (uint32_t g = 0; g < 4; g++) {
                float v[4];
                S::get(ps, i + l, j + g * 8 + half * 4, v);
                for (int t = 0; t < 4; t++) v[t] = p.b * v[t] + p.c * (1.0f / ORTH_SCALE) * sq[g * 4 + t];
                S::put(bs, i + l, j + g * 8 + half * 4, v);
            }
        }
        __syncthreads();
        for (uint32_t c = wave * 32; c < p.wide; c += WAVES * 32) {
            f32x16 y[ROWS / 32];
            for (uint32_t r = 0; r < ROWS / 32; r++) y[r] = 0.0f;
            for (uint32_t k = 0; k < ROWS; k += 16) {
                const f16x8 xh = S::columns(xs, k, c, 0), xl = S::columns(xs, k, c, 1);
                for (uint32_t r = 0; r < ROWS / 32; r++) y[r] = mma_split(xh, xl, S::rows(bs, r * 32, k, 0), S::rows(bs, r * 32, k, 1), y[r]);
            }
            wave_sync();                   /* the columns are this wavefront's alone, and read */
            for (uint32_t r = 0; r < ROWS / 32; r++)
                for (uint32_t g = 0; g < 4; g++) {
                    float v[4];
                    S::get(xs, r * 32 + l, c + g * 8 + half * 4, v);
                    for (int t = 0; t < 4; t++) v[t] = p.a * v[t] + (1.0f / ORTH_SCALE) * y[r][g * 4 + t];
                    S::put(xs, r * 32 + l, c + g * 8 + half * 4, v);
                }
        }
    }
    __syncthreads();
    if (p.last) {
        raw *out = (raw *)p.out + batch * p.size;
        for (uint32_t e = tid; e < units; e += SLAB_THREADS) {
            uint32_t row, c;
            unit(e, row, c);
            float v[4];
            S::get(xs, row, c, v);
            for (uint32_t k = 0; k < 4; k++)
                if (row < p.m && n0 + c + k < p.n) out[row * p.sm + (n0 + c + k) * p.sn] = D::put(v[k] * (1.0f / ORTH_SCALE));
        }
        return;
    }
    for (uint32_t e = tid; e < pieces; e += SLAB_THREADS) ((u32x4 *)kept)[e] = ((const u32x4 *)xs)[e];
    /* each block of the slab's part of P by RUNS wavefronts, a run of columns each */
    const uint32_t run = wave / BLOCKS, per = (p.wide / 16 + RUNS - 1) / RUNS * 16;
    const f32x16 sq = slab_square<ROWS>(xs, i, j, run * per, min(p.wide, (run + 1) * per));
    f32x4 part[4];
    for (int g = 0; g < 4; g++) part[g] = f32x4{sq[g * 4], sq[g * 4 + 1], sq[g * 4 + 2], sq[g * 4 + 3]};
    if (run)
        for (int g = 0; g < 4; g++) sums[((wave - BLOCKS) * 4 + g) * 64 + lane] = part[g];
    __syncthreads();
    if (run) return;
    float *to = p.next + (uint64_t)blockIdx.x * SQUARE + (i + l) * ROWS + j + half * 4;
    for (uint32_t g = 0; g < 4; g++) {
        for (uint32_t r = 1; r < RUNS; r++) part[g] += sums[(((r - 1) * BLOCKS + block) * 4 + g) * 64 + lane];
        *(f32x4 *)(to + g * 8) = part[g];
    }
}

struct Orth {
    uint64_t m, n, lx, lp;       /* of X: rows, columns, columns as held; of P: as held */
    uint64_t slabs, slab;        /* msim_orth_slab: slabs, or 0, and their columns */
    bool wide;                   /* several steps a pass over X */
    uint32_t squares;            /* of P's size beside P */
    uint64_t norm_bytes, x_bytes, p_bytes, bytes;
    Plan square, poly, update;
};

Orth orth_of(const msim_orthogonalize_spec *s)
{
    Orth o = {};
    o.m = std::min(s->rows, s->cols);
    o.n = std::max(s->rows, s->cols);
    o.lx = up(o.n, 32);
    o.lp = up(o.m, 32);
    o.norm_bytes = up((uint64_t)s->count * NORM_PARTS * 8, 256);
    if (o.m <= SLAB_ROWS && o.n <= SLABS * SLAB_COLS) {
        /* slabs enough to fill the card, of 64 columns at least */
        const uint64_t want = std::min<uint64_t>(SLABS, std::max<uint64_t>(1, 512 / s->count));
        const uint64_t most = std::max((o.n + SLAB_COLS - 1) / SLAB_COLS, std::min((o.n + 63) / 64, want));
        o.slab = up((o.n + most - 1) / most, 32);
        o.slabs = (o.n + o.slab - 1) / o.slab;
        const uint64_t rows = up(o.m, 32);
        o.x_bytes = s->count * o.slabs * o.slab * rows * 4;
        o.p_bytes = s->count * o.slabs * rows * rows * 4;
        o.bytes = o.norm_bytes + o.x_bytes + 2 * o.p_bytes;
        return o;
    }
    o.x_bytes = up(s->count * o.m * o.lx * 4, 256);
    o.p_bytes = up(s->count * o.m * o.lp * 4, 256);
    o.square = plan_of(M_SPLIT, {o.m, o.lp, o.lx, s->count});
    o.poly = plan_of(M_SPLIT, {o.m, o.lp, o.lp, s->count});
    o.update = plan_of(M_SPLIT, {o.m, o.lx, o.lp, s->count});
    /* Of 32 bits every step is taken by itself (pass_of has the errors).  Otherwise what a pass over X costs more than
     * products of m rows has to be worth four launches of those, which are slower by themselves: 1,024 x 4,096 (2.7e9)
     * 405 -> 330 us, 8 x 256 x 2,048 (8.7e8) 202 -> 174, 256 x 5,120 (3.1e8) 162 -> 155, 512 x 2,048 (3.4e8) 181 -> 178;
     * below, 256 x 4,096 (2.4e8) 138 -> 143, 384 x 2,304 (2.6e8) 155 -> 162, 512 x 1,024 (6.7e7) 159 -> 174, 1,536 x
     * 2,304 681 -> 765; but 768 x 2,048 (5.3e8) 221 -> 226.  64 x 20,000 148 -> 125. */
    o.wide = s->dtype != MSIM_F32 && s->steps > 1 &&
             (o.n >= 64 * o.m || (2 * o.n > 3 * o.m && (double)s->count * o.m * o.m * (o.n - 1.5 * o.m) >= 3e8));
    o.squares = o.wide ? 5 : 1;
    o.bytes = o.norm_bytes + 2 * o.x_bytes + (1 + o.squares) * o.p_bytes +
              std::max(o.square.part_bytes, std::max(o.poly.part_bytes, o.update.part_bytes));
    return o;
}

/* What a step can meet, from singular values of 0 .. top: the largest it leaves, and the largest |B| and |a + B|. */
struct Range { double left, poly, factor; };

Range range_of(const msim_orthogonalize_spec *s, double top)
{
    const double a = s->a, b = s->b, c = s->c, d = 9 * b * b - 20 * a * c, r = d > 0 ? std::sqrt(d) : 0;
    /* of q, a singular value's square: the ends, and where a derivative is 0 */
    const double at[] = {0, top * top, -b / (2 * c), -a / (3 * b), (-3 * b + r) / (10 * c), (-3 * b - r) / (10 * c)};
    Range x = {0, 0, 0};
    for (double q : at) {
        if (!(q >= 0 && q <= top * top)) continue;
        const double poly = q * (b + c * q);
        x.left = std::max(x.left, std::sqrt(q) * std::fabs(a + poly));
        x.poly = std::max(x.poly, std::fabs(poly));
        x.factor = std::max(x.factor, std::fabs(a + poly));
    }
    return x;
}

/* Singular values and |B| of all steps, from any update's, 0 .. 1: both have to fit f16 times ORTH_SCALE. */
const char *check_steps(const msim_orthogonalize_spec *s)
{
    static const char *const why = "orthogonalize: steps with these coefficients leave the range of the products";
    double top = 1.0;
    if (!std::isfinite(s->a) || !std::isfinite(s->b) || !std::isfinite(s->c)) return "orthogonalize: coefficients out of range";
    for (uint32_t k = 0; k < s->steps; k++) {
        const Range x = range_of(s, top);
        if (!(x.poly <= 24.0 && top * top <= 24.0)) return why;
        top = x.left * 1.001;
        if (!(top <= 24.0)) return why;
    }
    return nullptr;
}

/* How many steps, from step k on, are taken in one pass over X: without it, P of the
 * next step is (a + B) P (a + B), and X gets the product Q of all a + B.  That is 3
 * m^2 n a pass and 4 m^3 a step more (symmetric ones counted by their half),
 * instead of 3 m^2 n + m^3 a step.  Errors of 22 bits grow with P's small values
 * until P is made of X again, so these are up to three steps from the start and two
 * later.  Measured against 64 bits, relative to the norm: after two steps 3e-7 to
 * 6e-7, single ones 0.9e-7 to 4e-7 and products of 32 bits 0.6e-7 to 5e-7; after five
 * 1.4e-6 to 6.3e-6, 1.2e-6 to 2.8e-6 and 1.4e-6 to 6e-6 (70 x 4,481 to 1,024 x 4,096, noise, a
 * momentum, singular values over three orders).  A hundredth of what a result of 16 bits
 * is rounded by, but not for one of 32 bits. */
uint32_t pass_of(const msim_orthogonalize_spec *s, bool wide, uint32_t k)
{
    const uint32_t most = std::min(s->steps - k, !wide ? 1u : k == 0 ? 3u : 2u);
    double top = 1.0, q = 1.0;
    for (uint32_t i = 0; i < k; i++) top = range_of(s, top).left * 1.001;
    uint32_t n = 0;
    for (; n < most; n++) {
        const Range x = range_of(s, top);
        q *= x.factor;
        if (!(x.factor <= 24.0 && q <= 24.0 * PASS_DOWN)) break;      /* as check_steps */
        top = x.left * 1.001;
    }
    return std::max(n, 1u);
}

const char *check_orth(const msim_orthogonalize_spec *s, int *code)
{
    *code = MSIM_E_ARG;
    if (!s) return "orthogonalize: null spec";
    if (s->version != MSIM_ABI_VERSION) return "orthogonalize: spec version mismatch";
    if (s->dtype > MSIM_BF16) return "orthogonalize: unknown dtype";
    if (!s->rows || !s->cols) return "orthogonalize: rows and cols must be at least 1";
    if (s->reserved) return "orthogonalize: reserved must be 0";
    if (!(s->eps >= 0) || !std::isfinite(s->eps)) return "orthogonalize: eps must be finite and not negative";
    *code = MSIM_E_LIMIT;
    if (s->rows > MSIM_MAX_LINEAR || s->cols > MSIM_MAX_LINEAR) return "orthogonalize: rows or cols above MSIM_MAX_LINEAR";
    if (s->count > 65536 || (uint64_t)s->count * s->rows * s->cols >> 36) return "orthogonalize: more than 65,536 matrices or 2^36 elements";
    if (s->steps > 64) return "orthogonalize: more than 64 steps";
    *code = MSIM_E_ARG;
    return check_steps(s);
}

template <typename D> hipError_t launch_norm(const msim_orthogonalize_spec *s, const void *in, void *to, hipStream_t st)
{
    const uint64_t size = s->rows * s->cols;
    const uint32_t parts = norm_parts<D>(size);
    return in_turns((uint64_t)s->count * parts, 256, [&](uint32_t first, uint32_t grid) {
        return launch(msim_orth_norm<D>, grid, 256, 0, st, in, size, (double *)to, parts, first);
    });
}

template <typename D, bool BEGIN> hipError_t launch_move(const msim_orthogonalize_spec *s, const Orth &o, OrthP q, hipStream_t st)
{
    return in_turns((o.lx + 63) / 64 * ((o.m + 31) / 32) * s->count, 256, [&](uint32_t first, uint32_t grid) {
        q.first = first;
        return launch(s->rows > s->cols ? msim_orth_move<D, BEGIN, true> : msim_orth_move<D, BEGIN, false>, grid, 256, 0, st, q);
    });
}

template <typename D>
hipError_t run_slabs(const msim_orthogonalize_spec *s, const Orth &o, const void *in, void *out, char *ws, hipStream_t st)
{
    char *x = ws + o.norm_bytes, *part = x + o.x_bytes, *next = part + o.p_bytes;
    const bool flip = s->rows > s->cols;
    SlabP p = {in, out, (const double *)ws, x, (const float *)part, (float *)next, s->rows * s->cols, flip ? 1 : s->cols, flip ? s->cols : 1,
               s->eps, (uint32_t)o.m, (uint32_t)o.n, (uint32_t)o.slabs, (uint32_t)o.slab, 1, s->steps == 0, norm_parts<D>(s->rows * s->cols), s->a, s->b, s->c};
    hipError_t e = launch_norm<D>(s, in, ws, st);
    for (uint32_t k = 0; k <= s->steps && e == hipSuccess; k++) {
        p.first = k == 0;
        p.last = k == s->steps;
        e = launch(o.m <= 32 ? msim_orth_slab<D, 32> : msim_orth_slab<D, 64>, s->count * p.slabs, SLAB_THREADS, 0, st, p);
        const float *was = p.part;
        p.part = p.next;
        p.next = (float *)was;
    }
    return e;
}

template <typename D>
hipError_t run_orth(const msim_orthogonalize_spec *s, const Orth &o, const void *in, void *out, char *ws, hipStream_t st)
{
    if (o.slabs) return run_slabs<D>(s, o, in, out, ws, st);
    char *norms = ws, *x = norms + o.norm_bytes, *y = x + o.x_bytes, *sq = y + o.x_bytes, *m2[5], *part = sq + o.p_bytes;
    for (uint32_t i = 0; i < o.squares; i++, part += o.p_bytes) m2[i] = part;
    OrthP q = {in, out, x, (const double *)norms, s->rows, s->cols, o.lx, o.m * o.lx * 4, s->eps, norm_parts<D>(s->rows * s->cols), 0};
    hipError_t e = launch_norm<D>(s, in, norms, st);
    if (e == hipSuccess) e = launch_move<D, true>(s, o, q, st);
    /* to = alpha src + beta a b + diag I, symmetric; b of X or of a matrix of m columns */
    const auto square = [&](char *to, const char *fa, const char *fb, uint64_t ld, const Plan &plan, const char *src, float alpha, float beta, float diag) {
        GemmP p = {};
        p.batch = s->count;
        p.part = (float *)part;
        p.M = p.N = p.e.M = p.e.N = (uint32_t)o.m;
        p.mirror = 1;
        p.a = {fa, o.m * ld * 4, ld * 4, o.m * ld * 4};
        p.b = {fb, o.m * ld * 4, ld * 4, o.m * ld * 4};
        p.K = (uint32_t)ld;
        p.e.out = to;
        p.e.out_ld = o.lp;
        p.e.out_batch = o.m * o.lp * 4;
        p.e.src = src;
        p.e.alpha = alpha;
        p.e.beta = beta;
        p.e.diag = diag;
        if (e == hipSuccess) e = launch_gemm<M_SPLIT, false>(p, plan, st);
    };
    constexpr float ONE = 1.0f / ORTH_SCALE;
    for (uint32_t k = 0; k < s->steps && e == hipSuccess;) {
        const uint32_t n = pass_of(s, o.wide, k);
        k += n;
        square(sq, x, x, o.lx, o.square, nullptr, 0, ONE, 0);
        char *w = m2[0], *factor = w;
        for (uint32_t i = 0; i < n; i++) {
            /* B, or a + B where there are several steps */
            square(w, sq, sq, o.lp, o.poly, sq, s->b, s->c * ONE, n > 1 ? s->a * ORTH_SCALE : 0);
            if (i) {
                char *to = m2[2 + (i & 1)];
                square(to, w, factor, o.lp, o.poly, nullptr, 0, i == 1 ? ONE / PASS_DOWN : ONE, 0);
                factor = to;
            }
            if (i + 1 < n) {
                square(m2[4], w, sq, o.lp, o.poly, nullptr, 0, ONE, 0);
                square(sq, m2[4], w, o.lp, o.poly, nullptr, 0, ONE, 0);
                w = i ? m2[0] : m2[1];
            }
        }
        if (e != hipSuccess) break;
        GemmP p = {};
        p.batch = s->count;
        p.part = (float *)part;
        p.M = p.e.M = (uint32_t)o.m;
        p.N = p.e.N = (uint32_t)o.n;
        p.a = {factor, o.m * o.lp * 4, o.lp * 4, o.m * o.lp * 4};
        p.b = {x, o.m * o.lx * 4, o.lx * 4, o.m * o.lx * 4};
        p.K = (uint32_t)o.lp;
        p.e.out = y;
        p.e.out_ld = o.lx;
        p.e.out_batch = o.m * o.lx * 4;
        p.e.src = n == 1 ? x : nullptr;
        p.e.alpha = s->a;
        p.e.beta = n == 1 ? ONE : ONE * PASS_DOWN;
        e = launch_gemm<M_SPLIT, true>(p, o.update, st);
        std::swap(x, y);
    }
    q.x = x;
    return e == hipSuccess ? launch_move<D, false>(s, o, q, st) : e;
}

}   // namespace

extern "C" int msim_orthogonalize_workspace(const msim_orthogonalize_spec *s, uint64_t *bytes)
{
    int code;
    if (const char *why = check_orth(s, &code)) return fail(code, why);
    if (!bytes) return fail(MSIM_E_ARG, "orthogonalize: null bytes");
    *bytes = s->count ? orth_of(s).bytes : 0;
    return MSIM_OK;
}

extern "C" int msim_orthogonalize(const msim_orthogonalize_spec *s, const void *update, void *out, void *workspace,
                                  uint64_t workspace_bytes, void *hip_stream)
{
    int code;
    if (const char *why = check_orth(s, &code)) return fail(code, why);
    if (s->count == 0) return MSIM_OK;
    if (!update || !out) return fail(MSIM_E_ARG, "orthogonalize: null update or out");
    const Orth o = orth_of(s);
    if (int rc = check_workspace(workspace, workspace_bytes, o.bytes, "orthogonalize: workspace missing, too small or not on 256 bytes")) return rc;
    hipStream_t st = (hipStream_t)hip_stream;
    const hipError_t e = s->dtype == MSIM_F32 ? run_orth<F32>(s, o, update, out, (char *)workspace, st)
        : s->dtype == MSIM_F16 ? run_orth<F16>(s, o, update, out, (char *)workspace, st)
                               : run_orth<BF16>(s, o, update, out, (char *)workspace, st);
    return launched(e, "orthogonalize launch");
}
