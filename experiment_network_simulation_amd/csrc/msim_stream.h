/* Products of a weight matrix with a few vectors: the weights are read once, from
 * memory to registers.
 *
 * A wavefront has 16 rows of weights (NT times) and 16 vectors (MT times), and takes
 * 256 bytes of k at a time.  A matrix instruction wants 16 bytes of row l % 16 in
 * lane l, but loads of neighbouring lanes in different rows are a cache access for
 * each lane (53 counted for a load of 64 lanes, which bounded these products: 512 x
 * 2,048, 6 of 64 experts bf16 525 us, and 424 like this); so 16 lanes read a row's 256
 * bytes, and four such loads are exchanged among the lanes through LDS.  The order of k is the same for weights and vectors.  Wavefronts of
 * a workgroup take runs of k in turn and join their sums in LDS.
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

/* Of a block of 16 rows, those that a lane reads: row 4 u + lane / 16. */
template <typename D> struct Rows {
    const typename D::raw *at[4];
    /* row(r): where row r of the block begins */
    template <typename F> __device__ __forceinline__ void set(F row)
    {
        for (uint32_t u = 0; u < 4; u++) at[u] = row(4 * u + ((threadIdx.x & 63) >> 4));
    }
    __device__ __forceinline__ const typename D::raw *operator[](uint32_t u) const { return at[u]; }
};

/* Rows 8 to 15 of the block lie `low` elements behind rows 0 to 7: half as many addresses. */
template <typename D> struct RowsOfTwo {
    const typename D::raw *at[2];
    uint64_t low;
    template <typename F> __device__ __forceinline__ void set(uint64_t behind, F row)
    {
        low = behind;
        for (uint32_t u = 0; u < 2; u++) at[u] = row(4 * u + ((threadIdx.x & 63) >> 4));
    }
    __device__ __forceinline__ const typename D::raw *operator[](uint32_t u) const { return at[u & 1] + (u & 2 ? low : 0); }
};

/* LDS of a wavefront: what its lanes exchange, and then its sums for join() */
template <int MT, int NT> constexpr uint32_t STREAM_LDS = (MT * NT < 4 ? 4 : MT * NT) * 1024;

/* v[u] is piece lane % 16 of row 4 u + lane / 16; then piece 4 u + lane / 16 of row
 * lane % 16.  In LDS the pieces of a row are exchanged by the row, so that 16 lanes
 * cover all banks both ways. */
__device__ __forceinline__ void exchange(char *lds, u32x4 (&v)[4])
{
    const uint32_t lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    for (uint32_t u = 0; u < 4; u++) *(u32x4 *)(lds + u * 1024 + g * 256 + ((l ^ g) ^ u * 4) * 16) = v[u];
    wave_sync();
    for (uint32_t u = 0; u < 4; u++) v[u] = *(const u32x4 *)(lds + l * 256 + ((l ^ g) ^ u * 4) * 16);
    wave_sync();
}

/* What 16 bytes that were read `early` elements too early have from their place on, and zeros. */
template <typename D> __device__ __forceinline__ u32x4 behind(u32x4 v, uint32_t early)
{
    const unsigned __int128 q = __builtin_bit_cast(unsigned __int128, v);
    const uint32_t bits = early * sizeof(typename D::raw) * 8;
    return __builtin_bit_cast(u32x4, bits < 128 ? q >> bits : 0);
}

template <uint32_t BITS> struct Bits { typedef uint32_t T; };
template <> struct Bits<16> { typedef uint16_t T; };
/* a row of K elements, less than 16 bytes, and zeros; a loop, for the code of others beside it */
template <typename D> __device__ __forceinline__ u32x4 short_row(const typename D::raw *row, uint32_t K)
{
    constexpr uint32_t BITS = sizeof(typename D::raw) * 8;
    uint64_t half[2] = {0, 0};
    _Pragma("unroll 1") for (uint32_t i = 0; i < K; i++) {
        const uint64_t v = (uint64_t)__builtin_bit_cast(typename Bits<BITS>::T, row[i]) << i * BITS % 64;
        if (i * BITS < 64) half[0] |= v;
        else half[1] |= v;
    }
    return u32x4{(uint32_t)half[0], (uint32_t)(half[0] >> 32), (uint32_t)half[1], (uint32_t)(half[1] >> 32)};
}

enum { WHOLE, END, SHORT };
/* acc[i][j] += over N runs of k, at k, k + step, ...: weights w[j], vectors x[i].
 * WHOLE: all within K.  END: one that is not; 16 bytes that would pass the end of a
 * row are read before it.  SHORT: of rows of less than 16 bytes, by elements.
 *
 * The loads of weights and of the first two blocks of vectors are all asked for before
 * the first is used, which the compiler would not do by itself (32 tokens of 7,168
 * columns, 8 of 128 experts 1,430 -> 1,286 us); those of further vectors when a block before
 * them has been used, in its registers. */
template <typename D, int MT, int NT, int N, int WHERE, typename X>
__device__ __forceinline__ void stream_runs(const Rows<D> *w, const X *x, uint32_t k, uint32_t step, uint32_t K, char *lds, f32x4 (&acc)[MT][NT])
{
    constexpr uint32_t PER = 16 / sizeof(typename D::raw);
    constexpr int AHEAD = MT < 2 ? MT : 2;
    const uint32_t c = k + (threadIdx.x & 15) * PER, at = WHERE == END ? min(c, K - PER) : c, early = c - at;
    const bool cut = K % PER;                  /* a piece has both elements and none */
    u32x4 a[N][NT][4], b[N][AHEAD][4];
    const auto load = [&](const auto &r, int n, u32x4 (&v)[4]) {
        _Pragma("unroll") for (int u = 0; u < 4; u++) {
            if constexpr (WHERE == SHORT) v[u] = short_row<D>(r[u], c ? 0 : K);
            else v[u] = piece<D>(r[u] + at + n * step);
        }
    };
    const auto give = [&](u32x4 (&v)[4]) {
        if constexpr (WHERE == END)
            _Pragma("unroll") for (int u = 0; u < 4; u++) v[u] = cut ? behind<D>(v[u], early) : early ? u32x4{0, 0, 0, 0} : v[u];
        exchange(lds, v);
    };
    _Pragma("unroll") for (int n = 0; n < N; n++) {
        _Pragma("unroll") for (int j = 0; j < NT; j++) load(w[j], n, a[n][j]);
        _Pragma("unroll") for (int i = 0; i < AHEAD; i++) load(x[i], n, b[n][i]);
    }
    __builtin_amdgcn_sched_barrier(0);
    _Pragma("unroll") for (int n = 0; n < N; n++) {
        _Pragma("unroll") for (int j = 0; j < NT; j++) give(a[n][j]);
        _Pragma("unroll") for (int i = 0; i < MT; i++) {
            auto &v = b[n][i % AHEAD];
            give(v);
            _Pragma("unroll") for (int j = 0; j < NT; j++)
                _Pragma("unroll") for (int u = 0; u < 4; u++) acc[i][j] = mma16<D>(a[n][j][u], v[u], acc[i][j]);
            if (i + AHEAD < MT) load(x[i + AHEAD], n, v);
            if (MT > AHEAD) __builtin_amdgcn_sched_barrier(0);
        }
    }
}

/* one run, or what there is of it */
template <typename D, int MT, int NT, typename X>
__device__ __forceinline__ void stream_run(const Rows<D> *w, const X *x, uint32_t k, uint32_t K, char *lds, f32x4 (&acc)[MT][NT])
{
    if (k + RUN<D> <= K) stream_runs<D, MT, NT, 1, WHOLE>(w, x, k, 0, K, lds, acc);
    else if (K * sizeof(typename D::raw) >= 16) stream_runs<D, MT, NT, 1, END>(w, x, k, 0, K, lds, acc);
    else stream_runs<D, MT, NT, 1, SHORT>(w, x, k, 0, K, lds, acc);
}

/* the wavefront's share of k, every WAVES-th run: of few vectors two at a time, where their loads fit its registers */
template <typename D, int MT, int NT, int WAVES, typename X>
__device__ __forceinline__ void stream(const Rows<D> *w, const X *x, uint32_t K, uint32_t wave, char *lds, f32x4 (&acc)[MT][NT])
{
    uint32_t k = wave * RUN<D>;
    const uint32_t step = WAVES * RUN<D>;
    if constexpr (MT + NT <= 3 && WAVES < 16)
        for (; k + step + RUN<D> <= K; k += 2 * step) stream_runs<D, MT, NT, 2, WHOLE>(w, x, k, step, K, lds, acc);
    for (; k < K; k += step) stream_run<D, MT, NT>(w, x, k, K, lds, acc);
}

/* The wavefronts' sums together, in order.  lds: STREAM_LDS<MT, NT> each, of which
 * a wavefront writes its own alone.  Afterwards wavefront i has acc[i][...] whole,
 * i < MT (in turns of waves). */
template <int MT, int NT, int WAVES> __device__ __forceinline__ void join(char *lds, uint32_t wave, f32x4 (&acc)[MT][NT])
{
    const uint32_t lane = threadIdx.x & 63;
    const auto at = [&](uint32_t v, int i, int j) { return (f32x4 *)(lds + v * STREAM_LDS<MT, NT>) + (i * NT + j) * 64 + lane; };
    _Pragma("unroll") for (int i = 0; i < MT; i++)
        _Pragma("unroll") for (int j = 0; j < NT; j++) *at(wave, i, j) = acc[i][j];
    __syncthreads();
    _Pragma("unroll") for (int i = 0; i < MT; i++)
        if (i % WAVES == (int)wave)
            _Pragma("unroll") for (int j = 0; j < NT; j++) {
                f32x4 s = *at(0, i, j);
                for (int v = 1; v < WAVES; v++) s += *at(v, i, j);
                acc[i][j] = s;
            }
}

/* v[i] = f(v[i]) with the activation's function, chosen once for all N */
template <int N, typename F> __device__ __forceinline__ void each(float *v, F f)
{
    _Pragma("unroll") for (int i = 0; i < N; i++) v[i] = f(v[i]);
}
/* Activations and their slopes are FULL where what becomes of them has 32 bits; what is rounded to 16 bits takes shorter
 * ways, off by a hundredth of its own rounding at most. */

/* 1 / (1 + e^-z) */
template <bool FULL> __device__ __forceinline__ float logistic(float z)
{
    const float d = 1.0f + expf(-z);
    return FULL ? 1.0f / d : __builtin_amdgcn_rcpf(d);
}

/* The share of a normal distribution below z: 1/2 of erfc(x), x = |z| / sqrt(2), from the side of the sign.  Otherwise
 * t P(t) e^(-x^2), t = 1 / (1 + 0.51 x), which is smooth down to t = 0: P fits erfc(x) e^(x^2) / 2 t with the least largest
 * relative error for x up to 9.5, 7.4e-7.  In 32 bits off by at most 5e-6 relative and 7e-7 in all, a hundredth of a
 * rounding to 11 bits down to the smallest results (a fit of erfc to 1.5e-7 in all was 5e-4 off at z = -4).  2,048 x
 * 4,096 results of 32 bits 34 us by the library function, 30 like this; 8,192 x 8,192 of 16 bits 501. */
template <bool FULL> __device__ __forceinline__ float normal_below(float z)
{
    if constexpr (FULL) return 0.5f * erfcf(z * -0.70710678f);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.36062446f, fabsf(z), 1.0f));
    const float p = 0.143964782f + t * (0.14199096f + t * (0.140001565f + t * (0.0262380857f + t * (0.181102261f + t * (-0.180954888f + t * 0.0476572923f)))));
    const float q = t * expf(-0.5f * z * z) * p;
    return z < 0 ? q : 1.0f - q;
}

constexpr float TANH_A = 1.59576912f, TANH_B = 0.0713548162f;      /* 2 sqrt(2 / pi), times 0.044715 */

template <int N, bool FULL> __device__ __forceinline__ void act_of(float *v, uint32_t act)
{
    switch (act) {
    case MSIM_ACT_RELU: return each<N>(v, [](float z) { return z < 0 ? 0.0f : z; });      /* a NaN stays one */
    case MSIM_ACT_SILU: return each<N>(v, [](float z) { return z * logistic<FULL>(z); });
    case MSIM_ACT_GELU: return each<N>(v, [](float z) { return z * normal_below<FULL>(z); });
    case MSIM_ACT_GELU_TANH:               /* (1 + tanh(u)) / 2 = 1 / (1 + e^-2u) */
        return each<N>(v, [](float z) { return z * logistic<FULL>(z * (TANH_A + TANH_B * z * z)); });
    }
}

} // namespace

#endif
