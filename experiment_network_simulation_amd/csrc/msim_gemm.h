/* Large matrix products, C[m][n] = sum over k of A[m][k] B[n][k], from operands that
 * are contiguous along k or along m (n); what becomes of the sums is their
 * epilogue.  Sums are 32-bit, their order depends on the sizes alone.
 *
 * msim_gemm_kernel.h has the kernel, and each element type a file that makes its
 * kernels (msim_gemm_*.hip), so that they compile side by side.
 */
#ifndef MSIM_GEMM_H
#define MSIM_GEMM_H

#include "msim_stream.h"

namespace msim {

/* element types of a product: the three of the library, and a number as the sum
 * of two f16 (M_SPLIT) or two bf16 (M_TWO, results in f16), of which 32 columns lie as 32 high parts and 32 low ones */
enum { M_F32 = MSIM_F32, M_F16 = MSIM_F16, M_BF16 = MSIM_BF16, M_SPLIT = 3, M_TWO = 4 };

struct Operand {
    const char *at;
    uint64_t extent;             /* bytes that may be read from `at` on */
    uint64_t ld, batch;          /* bytes between rows, between matrices */
};

struct Epilogue {
    uint32_t M, N;
    void *out;                   /* 32 bits (out32) or the operands' type, as res */
    uint64_t out_ld;             /* elements, as the others */
    const float *bias;
    const void *res;
    uint64_t res_ld;
    void *pre;                   /* of the operands' type */
    uint64_t pre_ld;
    uint32_t act, out32;
    /* orthogonal update: out = alpha src + beta sum + diag I, split matrices of out_ld columns (a multiple of 32) */
    const void *src;
    uint64_t out_batch;          /* bytes between matrices of out and src */
    float alpha, beta, diag;
};

struct GemmP {
    Operand a, b;
    uint32_t M, N, K, batch;
    uint32_t tm, tn, nk, parts, per;       /* tiles of m, n and k; parts of k, tiles of k a part */
    uint32_t mirror;                       /* C is symmetric: tiles below the diagonal are written on both sides */
    uint32_t plain;              /* sums leave as they are, 1: in 32 bits (parts, or out), 2: rounded to 16 */
    float *part;                 /* parts > 1: sums of the parts, [batch][parts][M][part_ld] */
    uint64_t part_ld;
    Epilogue e;
};

/* Sums of columns to be joined beside the parts of a backward pass's products: [blocks][outs] */
struct Columns { const float *sums; uint32_t blocks, outs; float *out; };

/* A kernel: tiles of bt x bt, stages in LDS, threads. */
struct Kind { uint32_t bt, depth, threads; };
constexpr Kind KINDS[] = {{256, 2, 512}, {128, 2, 256}, {64, 4, 256}};
constexpr uint32_t N_KINDS = sizeof(KINDS) / sizeof(Kind);

/* How a product is cut: the kernel, and parts of k. */
struct Plan { uint32_t kind, parts, per, nk; uint64_t part_bytes; };

/* The plan of a product, and those of two in one launch, each on half of the card (their operations are as many). */
struct Product { uint64_t M, N, K, batch; };
__attribute__((visibility("hidden"))) Plan plan_of(uint32_t mode, const Product &q);
__attribute__((visibility("hidden"))) void plan_pair(uint32_t mode, const Product &a, const Product &b, Plan *pa, Plan *pb);

/* Enqueues a product of A contiguous along k and B along k (BMC: along n); p.part
 * has room for the plan's parts.  launch_pair: of a backward pass, x of A along k
 * and B along n, w of both along m and n, in one launch and with plans of one
 * kind; either may be left out (batch 0).  The columns, if any, are joined behind them. */
template <int MODE, bool BMC> __attribute__((visibility("hidden"))) hipError_t launch_gemm(GemmP p, const Plan &c, hipStream_t st);
template <int MODE> __attribute__((visibility("hidden"))) hipError_t launch_pair(GemmP x, const Plan &cx, GemmP w, const Plan &cw, const Columns &c, hipStream_t st);

inline uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

} // namespace msim

namespace {

using namespace msim;

template <int MODE> struct Type { typedef F16 D; };
template <> struct Type<M_F32> { typedef F32 D; };
template <> struct Type<M_BF16> { typedef BF16 D; };


/* eight elements, n of them there; on any element, which costs an access or two more than on 16 bytes */
template <typename D> __device__ __forceinline__ void load8(float *v, const void *p, uint64_t at, uint32_t n)
{
    typedef typename D::raw raw;
    constexpr uint32_t PER = 16 / sizeof(raw);
    typedef raw part __attribute__((ext_vector_type(PER)));
    const raw *q = (const raw *)p + at;
    if (n == 8) {
        _Pragma("unroll") for (uint32_t i = 0; i < 8; i += PER) {
            const part w = __builtin_bit_cast(part, piece<D>(q + i));
            for (uint32_t j = 0; j < PER; j++) v[i + j] = D::get(w[j]);
        }
    } else {
        _Pragma("unroll") for (uint32_t i = 0; i < 8; i++) v[i] = i < n ? D::get(q[i]) : 0.0f;
    }
}
template <typename D> __device__ __forceinline__ void store8(const float *v, void *p, uint64_t at, uint32_t n)
{
    typedef typename D::raw raw;
    constexpr uint32_t PER = 16 / sizeof(raw);
    typedef raw part __attribute__((ext_vector_type(PER)));
    typedef raw loose __attribute__((ext_vector_type(PER), aligned(sizeof(raw))));
    raw *q = (raw *)p + at;
    if (n == 8) {
        _Pragma("unroll") for (uint32_t i = 0; i < 8; i += PER) {
            part w;
            for (uint32_t j = 0; j < PER; j++) w[j] = D::put(v[i + j]);
            *(loose *)(q + i) = w;
        }
    } else {
        _Pragma("unroll") for (uint32_t i = 0; i < 8; i++)
            if (i < n) q[i] = D::put(v[i]);
    }
}

/* A number as the sum of two f16: 22 bits of it, for what is not below 2^-14. */
__device__ __forceinline__ void split_of(float v, uint16_t &hi, uint16_t &lo)
{
    const _Float16 h = (_Float16)v;
    hi = __builtin_bit_cast(uint16_t, h);
    lo = __builtin_bit_cast(uint16_t, (_Float16)(v - (float)h));
}

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

/* eight columns from n (a multiple of 8) on of row m of a split matrix: where the high parts begin */
__device__ __forceinline__ uint64_t split_at(uint64_t ld, uint32_t m, uint32_t n)
{
    return ((uint64_t)m * ld + (n & ~31u)) * 2 + (n & 31);
}
__device__ __forceinline__ void load_split(float *v, const void *p, uint64_t at)
{
    const u16x8 h = *(const u16x8 *)((const uint16_t *)p + at), l = *(const u16x8 *)((const uint16_t *)p + at + 32);
    for (int i = 0; i < 8; i++) v[i] = F16::get(h[i]) + F16::get(l[i]);
}
__device__ __forceinline__ void store_split(const float *v, void *p, uint64_t at)
{
    u16x8 h, l;
    for (int i = 0; i < 8; i++) {
        uint16_t a, b;
        split_of(v[i], a, b);
        h[i] = a;
        l[i] = b;
    }
    *(u16x8 *)((uint16_t *)p + at) = h;
    *(u16x8 *)((uint16_t *)p + at + 32) = l;
}

/* A number as the sum of two bf16: 16 bits of it, in the range of 32 bits; the 11 of an f16 whole.  What is not finite is so in
 * both products with the other number's parts, which makes it NaN. */
__device__ __forceinline__ void store_two(const float *v, void *p, uint64_t at)
{
    u16x8 h, l;
    for (int i = 0; i < 8; i++) {
        const uint32_t bits = __builtin_bit_cast(uint32_t, v[i]);
        uint16_t a = BF16::put(v[i]);
        if ((a & 0x7FFF) == 0x7F80) a = bits >> 16;        /* the largest numbers: the high part by truncation */
        h[i] = a;
        l[i] = (a & 0x7F80) == 0x7F80 ? uint16_t(0) : BF16::put(v[i] - BF16::get(a));
    }
    *(u16x8 *)((uint16_t *)p + at) = h;
    *(u16x8 *)((uint16_t *)p + at + 32) = l;
}

} // namespace

#endif
