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

/* acc[i][j] += over this wavefront's share of k: weight rows w[j], vectors x[i], both those of lane % 16 */
template <typename D, int MT, int NT>
__device__ __forceinline__ void stream(const typename D::raw *const *w, const typename D::raw *const *x, uint32_t K,
                                       uint32_t wave, uint32_t waves, f32x4 (&acc)[MT][NT])
{
    constexpr uint32_t PER = 16 / sizeof(typename D::raw), U = 4, RUN = U * 4 * PER;
    const uint32_t q = (threadIdx.x & 63) >> 4;
    const uint32_t whole = K / RUN * RUN;
    uint32_t k = wave * RUN;
    for (; k < whole; k += waves * RUN) {
        u32x4 a[U][NT], b[U][MT];
        _Pragma("unroll") for (uint32_t u = 0; u < U; u++) {
            const uint32_t at = k + u * 4 * PER + q * PER;
            _Pragma("unroll") for (int j = 0; j < NT; j++) a[u][j] = piece<D>(w[j] + at);
            _Pragma("unroll") for (int i = 0; i < MT; i++) b[u][i] = piece<D>(x[i] + at);
        }
        _Pragma("unroll") for (uint32_t u = 0; u < U; u++)
            _Pragma("unroll") for (int i = 0; i < MT; i++)
                _Pragma("unroll") for (int j = 0; j < NT; j++) acc[i][j] = mma16<D>(a[u][j], b[u][i], acc[i][j]);
    }
    if (k == whole)                        /* the wavefront whose turn the rest is */
        for (; k < K; k += 4 * PER) {
            u32x4 a[NT], b[MT];
            _Pragma("unroll") for (int j = 0; j < NT; j++) a[j] = piece<D>(w[j], k + q * PER, K);
            _Pragma("unroll") for (int i = 0; i < MT; i++) b[i] = piece<D>(x[i], k + q * PER, K);
            _Pragma("unroll") for (int i = 0; i < MT; i++)
                _Pragma("unroll") for (int j = 0; j < NT; j++) acc[i][j] = mma16<D>(a[j], b[i], acc[i][j]);
        }
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
template <int N> __device__ __forceinline__ void act_of(float *v, uint32_t act)
{
    switch (act) {
    case MSIM_ACT_RELU: return each<N>(v, [](float z) { return z < 0 ? 0.0f : z; });      /* a NaN stays one */
    case MSIM_ACT_SILU: return each<N>(v, [](float z) { return z / (1.0f + expf(-z)); });
    case MSIM_ACT_GELU: return each<N>(v, [](float z) { return 0.5f * z * (1.0f + erff(z * 0.70710678f)); });
    case MSIM_ACT_GELU_TANH:
        return each<N>(v, [](float z) { return 0.5f * z * (1.0f + tanhf(0.79788456f * (z + 0.044715f * z * z * z))); });
    }
}

} // namespace

#endif
