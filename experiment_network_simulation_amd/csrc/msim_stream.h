/* Products of a weight matrix with a few vectors: the weights are read once, from
 * memory to registers, and nothing of them passes through LDS.
 *
 * A wavefront has 16 rows of weights (NT times) and 16 vectors (MT times).  Lane l
 * reads 16 bytes of row (or vector) l % 16 at every fourth 16 bytes of k, which is
 * a matrix instruction's operand as it lies; the order of k is the same for both.
 * Wavefronts of a workgroup take runs of 256 bytes of k in turn, so that every
 * cache line is read by one of them, and join their sums in LDS.
 */
#ifndef MSIM_STREAM_H
#define MSIM_STREAM_H

#include "msim_device.h"

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

/* sums of products of 16 bytes of k: c[row][vector] */
template <typename D> __device__ __forceinline__ f32x4 mma16(u32x4 w, u32x4 x, f32x4 c);
template <> __device__ __forceinline__ f32x4 mma16<BF16>(u32x4 w, u32x4 x, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x4 mma16<F16>(u32x4 w, u32x4 x, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x4 mma16<F32>(u32x4 w, u32x4 x, f32x4 c)
{
    const f32x4 a = __builtin_bit_cast(f32x4, w), b = __builtin_bit_cast(f32x4, x);
    for (int e = 0; e < 4; e++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

/* 16 bytes of a row, which lies on any element */
template <typename D> __device__ __forceinline__ u32x4 piece(const typename D::raw *at)
{
    typedef typename D::raw raw;
    constexpr uint32_t PER = 16 / sizeof(raw);
    typedef raw vec __attribute__((ext_vector_type(PER)));
    typedef raw loose __attribute__((ext_vector_type(PER), aligned(sizeof(raw))));
    return __builtin_bit_cast(u32x4, (vec)*(const loose *)at);
}

/* 16 bytes from element k on of a row of K; zeros behind its end */
template <typename D> __device__ __forceinline__ u32x4 piece(const typename D::raw *row, uint32_t k, uint32_t K)
{
    typedef typename D::raw raw;
    constexpr uint32_t PER = 16 / sizeof(raw);
    typedef raw vec __attribute__((ext_vector_type(PER)));
    if (k + PER <= K) return piece<D>(row + k);
    vec v;
    for (uint32_t i = 0; i < PER; i++) v[i] = k + i < K ? row[k + i] : raw(0);
    return __builtin_bit_cast(u32x4, v);
}

/* elements of k that a wavefront takes at a time */
template <typename D> constexpr uint32_t RUN = 256 / sizeof(typename D::raw);

/* acc[i][j] += over N runs of k, at k, k + step, ..., all within K: weight rows
 * w[j], vectors x[i], both those of lane % 16.  ALL: all loads are asked for before the
 * first is used, which the compiler would not do by itself (32 tokens of 7,168
 * columns, 8 of 128 experts 1,430 -> 1,286 us); where there are so many of them that
 * their registers cost wavefronts, it is left to it. */
template <typename D, int MT, int NT, int N, bool ALL>
__device__ __forceinline__ void stream_whole(const typename D::raw *const *w, const typename D::raw *const *x, uint32_t k, uint32_t step,
                                             f32x4 (&acc)[MT][NT])
{
    constexpr uint32_t PER = 16 / sizeof(typename D::raw), U = 4;
    const uint32_t q = (threadIdx.x & 63) >> 4;
    u32x4 a[N * U][NT], b[N * U][MT];
    _Pragma("unroll") for (uint32_t u = 0; u < N * U; u++) {
        const uint32_t at = k + u / U * step + (u % U * 4 + q) * PER;
        _Pragma("unroll") for (int j = 0; j < NT; j++) a[u][j] = piece<D>(w[j] + at);
        _Pragma("unroll") for (int i = 0; i < MT; i++) b[u][i] = piece<D>(x[i] + at);
    }
    if constexpr (ALL) __builtin_amdgcn_sched_barrier(0);
    _Pragma("unroll") for (uint32_t u = 0; u < N * U; u++)
        _Pragma("unroll") for (int i = 0; i < MT; i++)
            _Pragma("unroll") for (int j = 0; j < NT; j++) acc[i][j] = mma16<D>(a[u][j], b[u][i], acc[i][j]);
}

/* one run, or what there is of it */
template <typename D, int MT, int NT, bool ALL = true>
__device__ __forceinline__ void stream_run(const typename D::raw *const *w, const typename D::raw *const *x, uint32_t k, uint32_t K,
                                           f32x4 (&acc)[MT][NT])
{
    constexpr uint32_t PER = 16 / sizeof(typename D::raw);
    const uint32_t q = (threadIdx.x & 63) >> 4;
    if (k + RUN<D> <= K) return stream_whole<D, MT, NT, 1, ALL>(w, x, k, 0, acc);
    for (; k < K; k += 4 * PER) {
        u32x4 a[NT], b[MT];
        _Pragma("unroll") for (int j = 0; j < NT; j++) a[j] = piece<D>(w[j], k + q * PER, K);
        _Pragma("unroll") for (int i = 0; i < MT; i++) b[i] = piece<D>(x[i], k + q * PER, K);
        _Pragma("unroll") for (int i = 0; i < MT; i++)
            _Pragma("unroll") for (int j = 0; j < NT; j++) acc[i][j] = mma16<D>(a[j], b[i], acc[i][j]);
    }
}

/* the wavefront's share of k, every waves-th run: of few vectors two at a time, whose loads fit its registers */
template <typename D, int MT, int NT, bool ALL = true>
__device__ __forceinline__ void stream(const typename D::raw *const *w, const typename D::raw *const *x, uint32_t K,
                                       uint32_t wave, uint32_t waves, f32x4 (&acc)[MT][NT])
{
    uint32_t k = wave * RUN<D>;
    const uint32_t step = waves * RUN<D>;
    if constexpr (MT + NT <= 3)
        for (; k + step + RUN<D> <= K; k += 2 * step) stream_whole<D, MT, NT, 2, ALL>(w, x, k, step, acc);
    for (; k < K; k += step) stream_run<D, MT, NT, ALL>(w, x, k, K, acc);
}

/* The wavefronts' sums together, in order.  lds: waves x MT x NT x 64 pieces.
 * Afterwards wavefront i has acc[i][...] whole, i < MT (in turns of waves). */
template <int MT, int NT, int WAVES> __device__ __forceinline__ void join(f32x4 *lds, uint32_t wave, f32x4 (&acc)[MT][NT])
{
    const uint32_t lane = threadIdx.x & 63;
    _Pragma("unroll") for (int i = 0; i < MT; i++)
        _Pragma("unroll") for (int j = 0; j < NT; j++) lds[((wave * MT + i) * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    _Pragma("unroll") for (int i = 0; i < MT; i++)
        if (i % WAVES == (int)wave)
            _Pragma("unroll") for (int j = 0; j < NT; j++) {
                f32x4 s = lds[(i * NT + j) * 64 + lane];
                for (int v = 1; v < WAVES; v++) s += lds[((v * MT + i) * NT + j) * 64 + lane];
                acc[i][j] = s;
            }
}

/* v[i] = f(v[i]) with the activation's function, chosen once for all N */
template <int N, typename F> __device__ __forceinline__ void each(float *v, F f)
{
    _Pragma("unroll") for (int i = 0; i < N; i++) v[i] = f(v[i]);
}
/* 1 / (1 + e^-z) */
__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.0f + expf(-z)); }

/* The share of a normal distribution below z: 1/2 of erfc of |z| / sqrt(2), by
 * formula 7.1.26 of Abramowitz and Stegun, off by at most 0.8e-7, from the side of
 * the sign.  A third of the library function's instructions: of 8,192 x 8,192 with
 * gelu it takes 40 us off 570. */
__device__ __forceinline__ float normal_below(float z)
{
    const float x = fabsf(z) * 0.70710678f, t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, x, 1.0f));
    const float q = 0.5f * t * expf(-x * x) *
        (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
    return z < 0 ? q : 1.0f - q;
}

constexpr float TANH_A = 1.59576912f, TANH_B = 0.0713548162f;      /* 2 sqrt(2 / pi), times 0.044715 */

template <int N> __device__ __forceinline__ void act_of(float *v, uint32_t act)
{
    switch (act) {
    case MSIM_ACT_RELU: return each<N>(v, [](float z) { return z < 0 ? 0.0f : z; });      /* a NaN stays one */
    case MSIM_ACT_SILU: return each<N>(v, [](float z) { return z * logistic(z); });
    case MSIM_ACT_GELU: return each<N>(v, [](float z) { return z * normal_below(z); });
    case MSIM_ACT_GELU_TANH:               /* (1 + tanh(u)) / 2 = 1 / (1 + e^-2u) */
        return each<N>(v, [](float z) { return z * logistic(z * (TANH_A + TANH_B * z * z)); });
    }
}

} // namespace

#endif
