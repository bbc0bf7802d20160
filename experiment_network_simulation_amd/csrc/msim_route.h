/* What every kernel that routes shares: exchanges between lanes, orders of keys,
 * weights, and a row routed by one wavefront with keys in 64 bits.
 */
#ifndef MSIM_ROUTE_H
#define MSIM_ROUTE_H

#include "msim_device.h"

namespace {

struct RouteP {
    const void *x;
    const float *bias;
    int32_t *ids;
    float *w;
    int32_t *load;
    uint64_t rows, stride;
    uint32_t E, K, G, TG, gtop, renorm, sigmoid;
    float scale;
    uint32_t size, lglanes, part, vec;     /* msim_route_lists: experts a group, log2 of its lanes, experts a lane,
                                              16-byte loads */
};

/* Exchange with another lane of the same 16: M = 1, 2: lane ^ M; 7, 15: the
 * mirror of 8 and of 16. */
template <int M> __device__ __forceinline__ uint32_t other(uint32_t v)
{
    constexpr int CTRL = M == 1 ? 0xB1 : M == 2 ? 0x4E : M == 7 ? 0x141 : 0x140;
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
}
template <int M> __device__ __forceinline__ float other(float v)
{
    return __builtin_bit_cast(float, other<M>(__builtin_bit_cast(uint32_t, v)));
}
template <int M> __device__ __forceinline__ double other(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)other<M>((uint32_t)(u >> 32)) << 32 | other<M>((uint32_t)u));
}

/* The values that lanes l and l ^ N (16 or 32) hold, in the same order on both:
 * the swap of v with itself. */
template <int N> __device__ __forceinline__ void both(uint32_t v, uint32_t &a, uint32_t &b)
{
    const auto r = N == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                           : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0];
    b = r[1];
}
template <int N, typename F> __device__ __forceinline__ float fold_far(float v, F f)
{
    uint32_t a, b;
    both<N>(__builtin_bit_cast(uint32_t, v), a, b);
    return f(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
template <int N, typename F> __device__ __forceinline__ double fold_far(double v, F f)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t al, ah, bl, bh;
    both<N>((uint32_t)u, al, bl);
    both<N>((uint32_t)(u >> 32), ah, bh);
    return f(__builtin_bit_cast(double, (uint64_t)ah << 32 | al), __builtin_bit_cast(double, (uint64_t)bh << 32 | bl));
}

/* Folds v over blocks of N lanes; every lane has the result. */
template <int N, typename T, typename F> __device__ __forceinline__ T fold(T v, F f)
{
    v = f(v, other<1>(v));
    v = f(v, other<2>(v));
    v = f(v, other<7>(v));
    if constexpr (N > 8) v = f(v, other<15>(v));
    if constexpr (N > 16) v = fold_far<16>(v, f);
    if constexpr (N > 32) v = fold_far<32>(v, f);
    return v;
}
struct Max { __device__ float operator()(float a, float b) const { return fmaxf(a, b); } };
struct Min { __device__ float operator()(float a, float b) const { return fminf(a, b); } };
struct Sum {
    template <typename T> __device__ T operator()(T a, T b) const { return a + b; }
};

/* A key and its expert in one 64-bit number that v_max_f64 orders: the high
 * word is the key as a float, which orders as the high word of a double does
 * (only a float's NaN would be one there), the low word the expert, so coded
 * that of equal keys the lower expert is the larger.  One instruction compares
 * both. */
__device__ __forceinline__ double max64(double a, double b) { return __builtin_fmax(a, b); }
__device__ __forceinline__ double min64(double a, double b) { return __builtin_fmin(a, b); }
struct Max64 { __device__ double operator()(double a, double b) const { return max64(a, b); } };

__device__ __forceinline__ double pack(float key, uint32_t e)
{
    const int32_t hi = __builtin_bit_cast(int32_t, key);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)hi << 32 | ((uint32_t)(hi >> 31) ^ ~e));
}
/* where the order of equal keys is looked at again: the code of positive keys for all */
__device__ __forceinline__ double pack_approx(float key, uint32_t e)
{
    return __builtin_bit_cast(double, (uint64_t)__builtin_bit_cast(uint32_t, key) << 32 | (uint32_t)~e);
}
__device__ __forceinline__ float key_of(double v)
{
    return __builtin_bit_cast(float, (uint32_t)(__builtin_bit_cast(uint64_t, v) >> 32));
}
__device__ __forceinline__ uint32_t expert_of(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return ~((uint32_t)u ^ (uint32_t)((int32_t)(u >> 32) >> 31));
}

__device__ __forceinline__ void order(double &a, double &b)
{
    const double x = max64(a, b);
    b = min64(a, b);
    a = x;
}
/* eight numbers in descending order, 19 comparisons */
__device__ __forceinline__ void sort8(double *a)
{
    order(a[0], a[2]); order(a[1], a[3]); order(a[4], a[6]); order(a[5], a[7]);
    order(a[0], a[4]); order(a[1], a[5]); order(a[2], a[6]); order(a[3], a[7]);
    order(a[0], a[1]); order(a[2], a[3]); order(a[4], a[5]); order(a[6], a[7]);
    order(a[2], a[4]); order(a[3], a[5]);
    order(a[1], a[4]); order(a[3], a[6]);
    order(a[1], a[2]); order(a[3], a[4]); order(a[5], a[6]);
}
/* n numbers, a power of two, that rise and then fall or are such a sequence rotated: in descending order */
template <int N> __device__ __forceinline__ void sort_bitonic(double *a)
{
    for (int d = N / 2; d; d >>= 1)
        for (int i = 0; i < N; i++)
            if (!(i & d)) order(a[i], a[i + d]);
}
/* KL (8 or 16) numbers in descending order */
template <int KL> __device__ __forceinline__ void sort_list(double *a)
{
    sort8(a);
    if constexpr (KL == 16) {
        sort8(a + 8);
        for (int i = 0; i < 8; i++) order(a[i], a[15 - i]);
        sort_bitonic<8>(a);
        sort_bitonic<8>(a + 8);
    }
}
/* a and b in descending order: a becomes the KL largest of both, in order */
template <int KL> __device__ __forceinline__ void keep_list(double *a, const double *b)
{
    for (int i = 0; i < KL; i++) a[i] = max64(a[i], b[KL - 1 - i]);
    sort_bitonic<KL>(a);
}

/* The weight of the slot this lane has (got: it has one), logit xs, over the
 * row's N lanes.  s = e^min(x,0) / (1 + e^-|x|) for a sigmoid, e^(x - top) inv
 * for a softmax; renormalised, the exponentials are taken relative to the
 * largest chosen one, so that no sum vanishes.  All in 32 bits: inv comes from
 * v_exp_f32 of (x - top) times a rounded log2(e), off by 2.4 2^-24 |x - top|
 * relative where expf of the difference is off by 2^-24 |x - top|.  Terms count by
 * their size, so of 1,024 experts inv is off by at most 2^-24 x 17 from there, 2
 * from the function and 36 from the additions. */
template <int N> __device__ __forceinline__ float weight_of(const RouteP &p, float xs, bool got, float top, float inv)
{
    const float t = p.sigmoid ? fminf(xs, 0.0f) : xs;
    const float c = p.renorm ? fold<N>(got ? t : -INFINITY, Max()) : p.sigmoid ? 0.0f : top;
    float q = expf(t - c);
    if (p.sigmoid) q /= 1.0f + expf(-fabsf(xs));
    else if (!p.renorm) q *= inv;
    if (!got) q = 0.0f;
    if (p.renorm) {
        const float sum = fold<N>(q, Sum());
        if (got) q /= sum;
    }
    return p.scale * q;
}

/* A score is n + z, z alone being rounded: a softmax's has n = 0, a sigmoid's z =
 * e / (1 + e), e = e^-|x|, for x < 0, and n = 1 with that negative for x > 0.
 * Sums of two scores and their biases are equal as real numbers where the terms
 * of z are the same or cancel and the rest is equal (s(x) + s(-x) and 1; the same
 * logits and biases in another order); z summed by itself, and n and the biases by
 * themselves, are then equal too, and the tie goes to the lower group.  Scores
 * added one by one gave 1 - 2^-53 or 1 + 2^-52 for 14 % of such pairs.  Takes n
 * off z: n is 1/2 at x = 0. */
__device__ __forceinline__ double exact_part(double &z)
{
    if (fabs(z) == 0.5) {
        z = 0.0;
        return 0.5;
    }
    return __builtin_signbit(z) ? 1.0 : 0.0;
}

/* One row by one wavefront, keys in 64 bits.  Lane l has experts l, l + 64, ...:
 * loads are consecutive, and each of top_k rounds finds the best key left by
 * exchanges between lanes.  lds: experts doubles of this wavefront's own, for
 * the groups.  hist: counts of the chosen experts, or NULL. */
template <typename D, int VPL> __device__ void route_row(const RouteP &p, uint64_t row, double *lds, int32_t *hist)
{
    const uint32_t lane = threadIdx.x & 63;
    const typename D::raw *x = (const typename D::raw *)p.x + row * p.stride;
    float v[VPL];
    double key[VPL];
    bool bad = false;
    float top = -INFINITY;
    for (int i = 0; i < VPL; i++) v[i] = i * WAVE + lane < p.E ? D::get(x[i * WAVE + lane]) : -INFINITY;
    for (int i = 0; i < VPL; i++) {
        bad |= v[i] != v[i] || (!p.sigmoid && v[i] == INFINITY);
        top = fmaxf(top, v[i]);
    }
    const bool is_void = __any(bad), in = __any(top > -INFINITY);
    if (!p.sigmoid) top = fold<WAVE>(top, Max());
    int32_t my_id = -1;
    float xs = -INFINITY;
    double inv = 1.0;
    if (!is_void && in) {
        const bool sums = p.G > 1 && p.gtop > 1;
        double z[VPL];
        if (p.bias || sums || (!p.sigmoid && !p.renorm)) {
            double sum = 0;
            for (int i = 0; i < VPL; i++) {
                z[i] = exp(p.sigmoid ? -fabs((double)v[i]) : (double)v[i] - top);
                sum += z[i];
            }
            if (!p.sigmoid) {
                inv = 1.0 / fold<WAVE>(sum, Sum());
            }
        }
        for (int i = 0; i < VPL; i++) {
            const uint32_t e = i * WAVE + lane;
            double k = v[i];
            if (p.bias || sums) {
                z[i] = p.sigmoid ? z[i] / (1.0 + z[i]) : z[i] * inv;
                if (p.bias) {
                    const float b = e < p.E ? p.bias[e] : 0.0f;
                    k = p.sigmoid && v[i] > 0 ? 1.0 - z[i] : z[i];
                    k = v[i] > -INFINITY && b > -INFINITY ? k + b : -INFINITY;
                }
                if (p.sigmoid && v[i] > 0) z[i] = -z[i];
            }
            key[i] = k;
        }
        if (p.G > 1) {
            /* lane g walks group g: its one or two best members, other lanes' keys among them */
            const uint32_t size = p.E / p.G;
            for (int i = 0; i < VPL; i++)
                if (i * WAVE + lane < p.E) lds[i * WAVE + lane] = key[i];
            wave_sync();
            double worth = -INFINITY, c = -INFINITY;
            uint32_t ea = 0, ec = 0;
            if (lane < p.G) {
                _Pragma("unroll 4") for (uint32_t e = lane * size; e < (lane + 1) * size; e++) {
                    const double k = lds[e];
                    const bool first = k > worth, second = k > c;
                    ec = first ? ea : second ? e : ec;
                    c = fmax(c, fmin(worth, k));
                    ea = first ? e : ea;
                    worth = fmax(worth, k);
                }
            }
            if (sums) {
                wave_sync();
                for (int i = 0; i < VPL; i++)
                    if (i * WAVE + lane < p.E) lds[i * WAVE + lane] = z[i];
                wave_sync();
                if (worth > -INFINITY) {
                    double za = lds[ea], zc = c > -INFINITY ? lds[ec] : 0.0;
                    double rest = p.sigmoid ? exact_part(za) + exact_part(zc) : 0.0;
                    if (p.bias) rest += (double)p.bias[ea] + (c > -INFINITY ? (double)p.bias[ec] : 0.0);
                    worth = za + zc + rest;
                }
            }
            wave_sync();
            uint32_t before = 0;           /* groups better than this lane's */
            for (uint32_t g = 0; g < p.G; g++) {
                const double w = __shfl(worth, (int)g);
                before += w > worth || (w == worth && g < lane);
            }
            const uint64_t stay = __ballot(lane < p.G && before < p.TG);
            for (int i = 0; i < VPL; i++) {
                const uint32_t e = i * WAVE + lane;
                key[i] = e < p.E && (stay >> (e / size) & 1) ? key[i] : -INFINITY;
            }
        }
        _Pragma("unroll 1") for (uint32_t r = 0; r < p.K; r++) {
            double best = -INFINITY;
            int at = INT32_MAX;
            for (int i = 0; i < VPL; i++)
                if (key[i] > best) { best = key[i]; at = i * WAVE + lane; }
            const double m = fold<WAVE>(best, Max64());
            if (m == -INFINITY) break;
            /* of equal keys the lowest index: hardly ever more than one lane has the best */
            uint64_t has = __ballot(best == m);
            int win = INT32_MAX;
            while (has) {
                win = min(win, __builtin_amdgcn_readlane(at, __builtin_ctzll(has)));
                has &= has - 1;
            }
            float won = 0.0f;
            for (int i = 0; i < VPL; i++)
                if (i * WAVE + (int)lane == win) {
                    key[i] = -INFINITY;
                    won = v[i];
                }
            won = __shfl(won, win % WAVE);
            if (lane == r) {
                my_id = win;
                xs = won;
            }
        }
    }
    /* weights: lane j has slot j */
    const float q = weight_of<WAVE>(p, xs, my_id >= 0, top, (float)inv);
    if (lane < p.K) {
        p.ids[row * p.K + lane] = my_id;
        p.w[row * p.K + lane] = is_void ? NAN : q;
        if (hist && my_id >= 0) atomicAdd(&hist[my_id], 1);
    }
}

} // namespace

#endif
