/* Expert-parallel routing: router, its gradient, dropout and the all-to-all
 * traffic that routed tokens cause (msim_route, msim_route_backward,
 * msim_dropout and msim_traffic of include/msim.h, which has the definitions).
 *
 * Nothing here keeps anything between calls or needs a workspace: what one
 * kernel leaves to the next stands in the outputs.  Counts are integers, so the
 * order of their atomic additions changes nothing; sums of floats are made in
 * a fixed order.  Times are of an MI355X that copies 2 GiB at 4.88 TB/s.
 */

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "msim.h"
#include "msim_error.h"

namespace {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int WAVE = 64;
constexpr float LOG2E = 1.44269504f;
constexpr uint32_t THREAD_EXPERTS = 32;    /* experts of msim_route_threads, at most */
constexpr uint32_t FINISH_ROWS = 1024;     /* rows a workgroup of msim_route_finish, at most */
constexpr int32_t UNDECIDED = INT32_MIN;   /* ids of a row that msim_route_lists leaves to the 64-bit path */

/* ------------------------------------------------------------------------ */
/* element types                                                             */
/* ------------------------------------------------------------------------ */

struct F32 {
    typedef float raw;
    static __device__ float get(raw v) { return v; }
    static __device__ raw put(float v) { return v; }
};
struct F16 {
    typedef uint16_t raw;
    static __device__ float get(raw v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ raw put(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};
struct BF16 {
    typedef uint16_t raw;
    static __device__ float get(raw v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
    /* to nearest, ties to even; a NaN stays one */
    static __device__ raw put(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};

/* ------------------------------------------------------------------------ */
/* the generator                                                             */
/* ------------------------------------------------------------------------ */

constexpr uint64_t GAMMA = 0x9E3779B97F4A7C15ull;

/* SplitMix64's output function (Steele, Lea and Flood, OOPSLA 2014).  Output n
 * of a seed is mix64(seed + (n + 1) GAMMA), so any position can be read. */
__device__ __forceinline__ uint64_t mix64(uint64_t z)
{
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

/* base: seed + (offset + 1) GAMMA */
__device__ __forceinline__ uint32_t draw32(uint64_t base, uint64_t i)
{
    const uint64_t z = mix64(base + (i >> 1) * GAMMA);
    return (i & 1) ? (uint32_t)(z >> 32) : (uint32_t)z;
}

/* ------------------------------------------------------------------------ */
/* router                                                                    */
/* ------------------------------------------------------------------------ */

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

/* what the wavefront's lanes wrote to LDS is there for its other lanes */
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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

/* the kernel that chooses clears the counts for the one that counts */
__device__ __forceinline__ void clear_load(const RouteP &p)
{
    if (p.load && blockIdx.x == 0)
        for (uint32_t e = threadIdx.x; e < p.E; e += blockDim.x) p.load[e] = 0;
}

/* A wavefront a row: more than 16 choices, or more than 32 groups.  Bound by the
 * latency of the rounds, each an exchange over all lanes: 131,072 x 256 bf16 take
 * 335 us with 17 choices and 384 with 20, where msim_route_lists takes 62 for 16;
 * 337 with 8 choices in 64 groups (190 in 32, there); 8 rows 11 us.  A lane's
 * registers hold no longer lists, and 64 groups have no lanes of their own for a
 * row's half-wavefront. */
template <typename D, int VPL> __global__ void __launch_bounds__(256) msim_route_rows(RouteP p)
{
    extern __shared__ double keys[];
    clear_load(p);
    const uint64_t step = (uint64_t)gridDim.x * (blockDim.x / WAVE);
    for (uint64_t row = (uint64_t)blockIdx.x * (blockDim.x / WAVE) + threadIdx.x / WAVE; row < p.rows; row += step)
        route_row<D, VPL>(p, row, keys + threadIdx.x / WAVE * p.E, nullptr);
}

/* The end of a routing: counts the ids, and routes the rows that
 * msim_route_lists left undecided.  That path is not in the other kernel: its
 * registers took a third of the wavefronts there, and one wavefront that did
 * such a row late held up all (90 us against 64 for both kernels at 131,072 x
 * 256 bf16).  Counted here, few workgroups add to the same few addresses, at
 * about 13 ns each (4,096 that counted by themselves took 41 us longer than
 * 1,024).  Every workgroup has `part` rows, at most FINISH_ROWS, whose undecided
 * ones its wavefronts share.  Bound by latency: 3.0 us at 10,007 rows, 12.3 at
 * 131,072 of which about 4 are an undecided row's. */
template <typename D, int VPL> __global__ void __launch_bounds__(512) msim_route_finish(RouteP p, uint64_t part)
{
    extern __shared__ double keys[];
    __shared__ int32_t hist[MSIM_MAX_EXPERTS];
    __shared__ uint32_t queue[FINISH_ROWS], queued;
    const uint64_t lo = blockIdx.x * part, hi = min(lo + part, p.rows);
    for (uint32_t e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
    if (threadIdx.x == 0) queued = 0;
    __syncthreads();
    const uint32_t n = (uint32_t)(hi - lo) * p.K;
    for (uint32_t i = threadIdx.x; i < n; i += 8 * blockDim.x) {
        int32_t id[8];                     /* eight loads on their way at once */
        for (int j = 0; j < 8; j++) id[j] = i + j * blockDim.x < n ? p.ids[lo * p.K + i + j * blockDim.x] : -1;
        for (int j = 0; j < 8; j++) {
            if (p.load && id[j] >= 0) atomicAdd(&hist[id[j]], 1);
            const uint32_t at = i + j * blockDim.x;
            if (id[j] == UNDECIDED && at % p.K == 0) queue[atomicAdd(&queued, 1u)] = at / p.K;
        }
    }
    __syncthreads();
    if (queued) {
        const uint32_t wave = threadIdx.x / WAVE;
        for (uint32_t k = wave; k < queued; k += blockDim.x / WAVE)
            route_row<D, VPL>(p, lo + queue[k], keys + wave * p.E, p.load ? hist : nullptr);
        __syncthreads();
    }
    if (p.load)
        for (uint32_t e = threadIdx.x; e < p.E; e += blockDim.x)
            if (hist[e]) atomicAdd(&p.load[e], hist[e]);
}

/* KL (8 or 16) or fewer choices a row, several rows a wavefront.
 *
 * A row has LANES lanes, each with up to VPL consecutive experts; with groups a
 * group has its own lanes, so that its best members meet in few or no exchanges.
 * A lane sorts its experts' keys KL at a time and keeps its KL largest in order;
 * top_k rounds then take the largest head of the row's lists.  Per value that is
 * a score and about eight comparisons (KL = 8), no exchange.
 *
 * Where a lane's experts are not whole 16 bytes, aligned, its 16-byte loads are
 * moved to lie within the row and values that are not the lane's own masked
 * (p.vec = 0; p.vec = 2, for rows shorter than a load: one at a time).
 *
 * Without bias keys are the logits and the choice is exact.  With bias (and for
 * sums of two scores) the keys here are 32-bit approximations with a known
 * error, and a row whose choice depends on a difference within twice that error
 * is left to msim_route_finish, which compares in 64 bits.  Of normal logits with
 * sigmoids and a normal bias that is 1 row in 1,000, with one bias for all or in
 * steps more: at 256 experts and top 8 bf16 9 % and 4 %, for the last chosen and
 * the first left out often have the same logit and bias, and f32 0.2 %.  131,072 x
 * 256 bf16 take 45 us with a normal bias, 66 in steps, 81 with one for all, and 387
 * where logits on a coarse grid leave nearly all rows undecided.  Errors:
 * v_exp_f32 and v_rcp_f32 are off by 2^-23 relative.  A sigmoid is off by less than 2^-22: its exponential's argument by
 * 1.4 2^-24 |x|, and |x| s (1 - s) < 0.23.  A softmax score is off by less than
 * 2^-24 (0.9 + 54 s): the argument by 2.4 2^-24 |x - top|, and |x - top| e^(x -
 * top) < 0.37 in the score and 4.5 of the sum for 1,024 experts; the sum by 36
 * additions (32 terms a lane, five exchanges).  The sum with the bias adds 2^-24
 * |key|.
 *
 * Bound by the issue of vector instructions, 1,087 for eight rows of 256 with
 * groups and bias: 42 us at 131,072 x 256 bf16, where its bytes would take 15.5.
 * Left out in turn, the rounds are 10 us of it, the sorting 8, the sigmoids 6,
 * the groups 4, the weights 3, the loads none.  Tried and no faster: keys as one
 * 32-bit integer with the place in its low bits (fewer instructions, four times
 * the undecided rows), loads a turn ahead, 2,048 or 4,096 workgroups. */
template <typename D, int VPL, int LANES, int KL, bool BIAS>
__global__ void __launch_bounds__(256) msim_route_lists(RouteP p)
{
    constexpr int PER16 = 16 / sizeof(typename D::raw);
    typedef typename D::raw vec __attribute__((ext_vector_type(PER16)));
    typedef vec loose __attribute__((aligned(sizeof(typename D::raw))));
    __shared__ int32_t hist[MSIM_MAX_EXPERTS];
    __shared__ float lds_bias[BIAS ? LANES * (VPL + 4) : 1];
    __shared__ double lds_list[256][KL + 1];                  /* each thread's list, and an end; 8 (KL + 1) bytes apart no
                                                               * two lanes of a half-wavefront meet in a bank */
    constexpr uint32_t ROWS = WAVE / LANES;                   /* rows a wavefront */
    const uint32_t glanes = 1u << p.lglanes;
    const uint32_t lane = threadIdx.x & 63, l = lane % LANES, sub = l & (glanes - 1);
    const uint32_t g = l >> p.lglanes, size = p.size;
    const uint32_t first0 = g * size + sub * p.part;          /* this lane's experts */
    const uint32_t past = g < p.G ? min(first0 + p.part, (g + 1) * size) : first0;
    const uint32_t n0 = past > first0 ? past - first0 : 0;
    /* one workgroup that leaves no row undecided counts by itself */
    const bool count = p.load && gridDim.x == 1 && !(BIAS || p.gtop > 1);
    lds_list[threadIdx.x][KL] = pack(-INFINITY, 0);
    if (count)
        for (uint32_t e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
    else
        clear_load(p);
    if (BIAS && threadIdx.x < LANES)
        for (uint32_t i = 0; i < VPL; i++) {
            const float b = i < n0 ? p.bias[first0 + i] : -INFINITY;
            lds_bias[l * (VPL + 4) + i] = b == b ? b : -INFINITY;
        }
    __syncthreads();
    const uint64_t step = (uint64_t)gridDim.x * (blockDim.x / WAVE) * ROWS;
    const uint64_t row0 = ((uint64_t)blockIdx.x * (blockDim.x / WAVE) + threadIdx.x / WAVE) * ROWS;
    const bool sigmoid = p.sigmoid;
    _Pragma("unroll 1") for (uint64_t rows = row0; rows < p.rows; rows += step) {
        /* computed again each time: kept over the loop, what follows from them takes a register for every expert */
        uint32_t first = first0, n = n0;
        asm("" : "+v"(first), "+v"(n));
        const uint64_t row = min(rows + lane / LANES, p.rows - 1);
        const bool mine = rows + lane / LANES < p.rows;
        const typename D::raw *x = (const typename D::raw *)p.x + row * p.stride;
        vec raw[VPL / PER16];
        const typename D::raw none = D::put(-INFINITY);
        uint32_t from[VPL / PER16];                       /* the expert of each load's first value */
        if (p.vec == 1) {
            for (int c = 0; c < VPL / PER16; c++) {
                from[c] = first + c * PER16;
                raw[c] = none;
                if (n) raw[c] = *(const vec *)(x + from[c]);
            }
        } else if (p.vec == 0) {
            for (int c = 0; c < VPL / PER16; c++) {
                const uint32_t want = first + c * PER16, has = n > c * PER16 ? n - c * PER16 : 0;
                from[c] = min(want, p.E - PER16);
                const vec t = *(const loose *)(x + from[c]);
                for (int i = 0; i < PER16; i++) raw[c][i] = from[c] + i - want < has ? t[i] : none;
            }
        } else {
            for (int c = 0; c < VPL / PER16; c++) from[c] = first + c * PER16;
            for (int i = 0; i < VPL; i++) raw[i / PER16][i % PER16] = (uint32_t)i < n ? x[first + i] : none;
        }
        auto v = [&](int i) { return D::get(raw[i / PER16][i % PER16]); };
        /* is anything not finite?  0 * x is NaN then */
        float odd = 0.0f;
        for (int i = 0; i < VPL; i++) odd = __builtin_fmaf(v(i), 0.0f, odd);
        const bool any_odd = __any(odd != odd);
        bool is_void = false;
        if (any_odd) {
            bool bad = false;
            for (int i = 0; i < VPL; i++) bad |= v(i) != v(i) || (!sigmoid && v(i) == INFINITY);
            is_void = fold<LANES>(bad ? 1.0f : 0.0f, Max()) > 0.0f;
        }
        float top = 0.0f, inv = 1.0f;
        if (!sigmoid && (BIAS || p.G > 1 || !p.renorm)) {
            top = v(0);
            for (int i = 1; i < VPL; i++) top = fmaxf(top, v(i));
            top = fold<LANES>(top, Max());
            if (!(top > -INFINITY && top < INFINITY)) top = 0.0f;     /* nothing in, or void */
            if (BIAS || !p.renorm) {
                float sum = 0.0f;
                for (int i = 0; i < VPL; i++) sum += __builtin_amdgcn_exp2f((v(i) - top) * LOG2E);
                inv = 1.0f / fold<LANES>(sum, Sum());
            }
        }
        double a[KL];
        for (int c = 0; c < VPL; c += KL) {
            double b[KL];
            for (int h = c; h < c + KL; h += 8) {
                float k[8];
                for (int i = 0; i < 8; i++) k[i] = v(h + i);
                if (BIAS) {
                    if (sigmoid)
                        for (int i = 0; i < 8; i++) k[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(k[i] * -LOG2E));
                    else
                        for (int i = 0; i < 8; i++) k[i] = __builtin_amdgcn_exp2f((k[i] - top) * LOG2E) * inv;
                    const float *t = &lds_bias[l * (VPL + 4)];
                    if (p.vec) {
                        for (int i = 0; i < 8; i++) k[i] += (*(const f32x4 *)&t[h + (i & 4)])[i & 3];
                    } else {
                        /* a load moved back begins before the lane's part: an index below zero, but not below lds_bias, for
                         * first is at most VPL experts for each lane before this one */
                        for (int i = 0; i < 8; i++) k[i] += t[(int32_t)(from[(h + i) / PER16] + i % PER16 - first)];
                    }
                    if (any_odd || !p.vec)
                        for (int i = 0; i < 8; i++) k[i] = v(h + i) > -INFINITY ? k[i] : -INFINITY;
                }
                /* + 0: the two zeros are equal (a sum of a score and a bias is never -0); a NaN (of a void row) is
                 * ordered as it falls */
                for (int i = 0; i < 8; i++) {
                    const uint32_t e = from[(h + i) / PER16] + i % PER16;
                    (c ? b : a)[h - c + i] = BIAS ? pack_approx(k[i], e) : pack(k[i] + 0.0f, e);
                }
            }
            sort_list<KL>(c ? b : a);
            if (c) keep_list<KL>(a, b);
        }
        const float slack = sigmoid ? 0x1p-20f : 0x1p-22f + 0x1p-17f * inv;
        bool near = false, left_out = false;
        if (p.G > 1) {
            float t1 = key_of(a[0]), t2 = key_of(a[1]);
            _Pragma("unroll 1") for (uint32_t m = 1; m < glanes; m <<= 1) {
                const float o1 = __shfl_xor(t1, (int)m), o2 = __shfl_xor(t2, (int)m);
                t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
                t1 = fmaxf(t1, o1);
            }
            if (!BIAS && p.gtop > 1) {
                if (sigmoid) {
                    t1 = t1 > -INFINITY ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t1 * -LOG2E)) : t1;
                    t2 = t2 > -INFINITY ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t2 * -LOG2E)) : t2;
                } else {
                    t1 = t1 > -INFINITY ? __builtin_amdgcn_exp2f((t1 - top) * LOG2E) : t1;
                    t2 = t2 > -INFINITY ? __builtin_amdgcn_exp2f((t2 - top) * LOG2E) : t2;
                }
            }
            const float worth = p.gtop > 1 && t2 > -INFINITY ? t1 + t2 : t1;
            uint32_t before = 0;
            _Pragma("unroll 1") for (uint32_t o = glanes; o < LANES; o += glanes) {
                const float w = __shfl_xor(worth, (int)o);
                before += w > worth || (w == worth && (l ^ o) < l);
            }
            const bool stay = before < p.TG;
            if (BIAS || p.gtop > 1) {
                const float in = fold<LANES>(stay ? worth : INFINITY, Min());
                const float out = fold<LANES>(stay ? -INFINITY : worth, Max());
                const float size = fold<LANES>((t1 > -INFINITY ? fabsf(t1) : 0.0f) + (t2 > -INFINITY ? fabsf(t2) : 0.0f), Max());
                near = out > -INFINITY && !(in - out > 2.0f * slack + 0x1p-20f * size);
            }
            left_out = !stay;
        }
        double slot = pack(-INFINITY, 0), last = slot;
        const double *list = lds_list[threadIdx.x];
        for (int i = 0; i < KL; i++) lds_list[threadIdx.x][i] = a[i];
        double head = a[0];
        if (left_out) {
            head = slot;
            list += KL;
        }
        /* with bias one round more, for the difference to the first that is not chosen */
        _Pragma("unroll 1") for (uint32_t r = 0; r < p.K + BIAS; r++) {
            const double m = fold<LANES>(head, Max64());
            if (l == r) slot = m;
            if (BIAS) last = m;
            /* (the end of a list is no key) */
            if (__builtin_bit_cast(uint64_t, m) == __builtin_bit_cast(uint64_t, head) && key_of(m) > -INFINITY) list++;
            head = *list;
        }
        const uint32_t won_all = left_out ? 0 : list - lds_list[threadIdx.x];
        /* a list that is used up hides what comes next to its last */
        if (BIAS && VPL > KL) near |= won_all >= KL;
        const bool got = l < p.K && key_of(slot) > -INFINITY && !is_void;
        const int32_t id = got ? (int32_t)(BIAS ? ~(uint32_t)__builtin_bit_cast(uint64_t, slot) : expert_of(slot)) : -1;
        const float xs = got ? (BIAS ? D::get(x[id]) : key_of(slot)) : -INFINITY;
        if (BIAS) {
            const float k0 = key_of(slot);
            float k1 = __shfl_down(k0, 1);
            if (l == p.K - 1) k1 = key_of(last);
            bool close = got && !(k0 - k1 > slack + 0x1p-22f * fabsf(k0));
            if (__any(close)) {
                /* the same logit and the same bias: the same key, in order already (of positive keys) */
                const float b = got ? p.bias[id] : 0.0f;
                const float xn = __shfl_down(xs, 1), bn = __shfl_down(b, 1);
                if (l < p.K - 1 && xs == xn && b == bn && k0 >= 0.0f) close = false;
            }
            near |= close;
        }
        bool again = false;
        if (BIAS || p.gtop > 1) again = fold<LANES>(near ? 1.0f : 0.0f, Max()) > 0.0f && !is_void;
        const float q = weight_of<LANES>(p, xs, got, top, inv);
        if (mine && l < p.K) {
            p.ids[row * p.K + l] = again ? UNDECIDED : id;
            p.w[row * p.K + l] = is_void ? NAN : q;
            if (count && got) atomicAdd(&hist[id], 1);
        }
    }
    if (count) {
        __syncthreads();
        for (uint32_t e = threadIdx.x; e < p.E; e += blockDim.x) p.load[e] = hist[e];
    }
}

/* Few experts and many rows: a row a thread, which keeps the eight largest keys
 * in order as msim_route_lists does, eight experts at a time, and has all slots
 * of its row; no exchange and no rounds.  With bias top_k < 8, so that the first
 * key that is not chosen is in the list.  Bound by latency until the rows fill
 * the card, then by its instructions: with the counts 1,048,576 x 8 f32 take 27
 * us here (floor 10) and 92 in msim_route_lists, 131,072 x 32 bf16 13 and 19,
 * but 16,384 x 32 8.3 and 7.1, and 1,048,576 x 64 145 and 83, for the rows of a
 * wavefront no longer fit the first-level cache. */
template <typename D, bool BIAS> __global__ void __launch_bounds__(256) msim_route_threads(RouteP p)
{
    constexpr int PER16 = 16 / sizeof(typename D::raw);
    typedef typename D::raw loose __attribute__((ext_vector_type(PER16), aligned(sizeof(typename D::raw))));
    __shared__ float bias[THREAD_EXPERTS];
    clear_load(p);
    if (BIAS) {
        if (threadIdx.x < THREAD_EXPERTS) {
            const float b = threadIdx.x < p.E ? p.bias[threadIdx.x] : -INFINITY;
            bias[threadIdx.x] = b == b ? b : -INFINITY;
        }
        __syncthreads();
    }
    const bool sigmoid = p.sigmoid;
    const uint64_t step = (uint64_t)gridDim.x * blockDim.x;
    for (uint64_t row = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; row < p.rows; row += step) {
        const typename D::raw *x = (const typename D::raw *)p.x + row * p.stride;
        /* eight values from expert c on, -inf where there are no more, and their experts */
        auto eight = [&](uint32_t c, float *v, uint32_t *e) {
            for (int h = 0; h < 8; h += PER16) {
                if (p.vec != 2) {
                    const uint32_t from = min(c + h, p.E - PER16);     /* the load stays within the row */
                    const loose t = *(const loose *)(x + from);
                    for (int i = 0; i < PER16; i++) {
                        e[h + i] = from + i;
                        v[h + i] = from + i >= c + h ? D::get(t[i]) : -INFINITY;
                    }
                } else {
                    for (int i = 0; i < PER16; i++) {
                        e[h + i] = c + h + i;
                        v[h + i] = c + h + i < p.E ? D::get(x[c + h + i]) : -INFINITY;
                    }
                }
            }
        };
        float v[8];
        uint32_t e[8];
        float top = 0.0f, inv = 1.0f;
        if (!sigmoid && (BIAS || !p.renorm)) {
            top = -INFINITY;
            for (uint32_t c = 0; c < p.E; c += 8) {
                eight(c, v, e);
                for (int i = 0; i < 8; i++) top = fmaxf(top, v[i]);
            }
            if (!(top > -INFINITY && top < INFINITY)) top = 0.0f;
            float sum = 0.0f;
            for (uint32_t c = 0; c < p.E; c += 8) {
                eight(c, v, e);
                for (int i = 0; i < 8; i++) sum += __builtin_amdgcn_exp2f((v[i] - top) * LOG2E);
            }
            inv = 1.0f / sum;
        }
        bool bad = false;
        double a[8], b[8];
        for (uint32_t c = 0; c < p.E; c += 8) {
            eight(c, v, e);
            for (int i = 0; i < 8; i++) {
                bad |= sigmoid ? v[i] != v[i] : !(v[i] < INFINITY);
                float k = v[i] + 0.0f;
                if (BIAS) {
                    k = sigmoid ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v[i] * -LOG2E))
                                : __builtin_amdgcn_exp2f((v[i] - top) * LOG2E) * inv;
                    k = v[i] > -INFINITY ? k + bias[e[i]] : -INFINITY;
                }
                b[i] = BIAS ? pack_approx(k, e[i]) : pack(k, e[i]);
            }
            sort8(b);
            if (c == 0)
                for (int i = 0; i < 8; i++) a[i] = b[i];
            else
                keep_list<8>(a, b);
        }
        int32_t id[8];
        float xs[8], most = -INFINITY, sum = 0.0f;
        for (int j = 0; j < 8; j++) {
            const bool got = j < (int)p.K && key_of(a[j]) > -INFINITY && !bad;
            id[j] = got ? (int32_t)(BIAS ? ~(uint32_t)__builtin_bit_cast(uint64_t, a[j]) : expert_of(a[j])) : -1;
            xs[j] = got ? (BIAS ? D::get(x[id[j]]) : key_of(a[j])) : -INFINITY;
            most = fmaxf(most, xs[j]);
        }
        bool again = false;
        if (BIAS) {
            const float slack = sigmoid ? 0x1p-20f : 0x1p-22f + 0x1p-17f * inv;
            for (int j = 0; j < 7; j++) {
                const float k0 = key_of(a[j]), k1 = key_of(a[j + 1]);
                if (id[j] >= 0 && !(k0 - k1 > slack + 0x1p-22f * fabsf(k0)))
                    again |= !(id[j + 1] >= 0 && xs[j] == xs[j + 1] && bias[id[j]] == bias[id[j + 1]] && k0 >= 0.0f);
            }
        }
        /* the weights, as weight_of has them */
        const float c = p.renorm ? (sigmoid ? fminf(most, 0.0f) : most) : sigmoid ? 0.0f : top;
        for (int j = 0; j < 8; j++) {
            float q = 0.0f;
            if (id[j] >= 0) {
                q = expf((sigmoid ? fminf(xs[j], 0.0f) : xs[j]) - c);
                if (sigmoid) q /= 1.0f + expf(-fabsf(xs[j]));
                else if (!p.renorm) q *= inv;
            }
            xs[j] = q;
            sum += q;
        }
        for (int j = 0; j < 8; j++)
            if (j < (int)p.K) {
                float q = xs[j];
                if (p.renorm && id[j] >= 0) q /= sum;
                p.ids[row * p.K + j] = again ? UNDECIDED : id[j];
                p.w[row * p.K + j] = bad ? NAN : p.scale * q;
            }
    }
}

__global__ void msim_route_nothing(RouteP p) { clear_load(p); }

/* ------------------------------------------------------------------------ */
/* the router's gradient                                                     */
/* ------------------------------------------------------------------------ */

struct BackP {
    const void *x;
    const int32_t *ids;
    const float *g;
    void *dx;
    uint64_t rows, stride, dstride;
    uint32_t E, K, renorm, sigmoid;
    float scale;
};

/* The slots of a row on LANES lanes (at least top_k), 64 / LANES rows a
 * wavefront.  Only the chosen logits are read, unless all have a gradient; the
 * gradient's rows, nearly all zeros, are put together in LDS, CHUNK experts at
 * a time, and leave it in 16-byte stores.  What was put there is taken out again
 * afterwards, so the rest stays zero.  Bound by the memory: 25 us at 131,072 x
 * 256 bf16, which writes 67 MB and, a chosen logit bringing its whole cache line,
 * reads about as much (5.4 TB/s).  2,048 workgroups: 1,280 take 29 us, 4,096 27.
 * With all experts (softmax, not renormalised) the row is read three times, its
 * exponentials taken twice: 39 us at 131,072 x 256 bf16 where the memory allows 27,
 * 71 f32.  Scores as weight_of has them, in 32 bits; a lane's part of a
 * denominator is up to 128 additions long. */
template <typename D, int LANES> __global__ void __launch_bounds__(256) msim_route_back(BackP p)
{
    constexpr int PER = 16 / sizeof(typename D::raw), ROWS = WAVE / LANES;
    constexpr uint32_t CHUNK = 256;
    typedef typename D::raw vec __attribute__((ext_vector_type(PER)));
    typedef vec loose __attribute__((aligned(sizeof(typename D::raw))));
    __shared__ float lds[4][ROWS][CHUNK + 4];
    const uint32_t lane = threadIdx.x & 63, l = lane % LANES;
    float (*const buf)[CHUNK + 4] = lds[threadIdx.x / WAVE];
    for (uint32_t i = lane; i < ROWS * (CHUNK + 4); i += WAVE) (&buf[0][0])[i] = 0.0f;
    wave_sync();
    const bool every = !p.sigmoid && !p.renorm;        /* all experts have a gradient */
    const uint64_t step = (uint64_t)gridDim.x * 4 * ROWS;
    for (uint64_t rows = ((uint64_t)blockIdx.x * 4 + threadIdx.x / WAVE) * ROWS; rows < p.rows; rows += step) {
        const uint64_t row = min(rows + lane / LANES, p.rows - 1);
        const bool mine = rows + lane / LANES < p.rows;
        const typename D::raw *x = (const typename D::raw *)p.x + row * p.stride;
        int32_t id = l < p.K ? p.ids[row * p.K + l] : -1;
        float g = l < p.K ? p.g[row * p.K + l] : 0.0f;
        if ((uint32_t)id >= p.E) id = -1;
        const float xs = id >= 0 ? D::get(x[id]) : -INFINITY;
        if (xs == -INFINITY) id = -1;      /* an expert out of the row has no score to change */
        const bool got = id >= 0;
        if (!got) g = 0.0f;
        float top = -INFINITY, inv = 1.0f;
        if (every) {
            const uint32_t whole = p.E - p.E % PER;
            for (uint32_t e = l * PER; e < whole; e += LANES * PER) {
                const vec t = *(const loose *)(x + e);
                for (int i = 0; i < PER; i++) top = fmaxf(top, D::get(t[i]));
            }
            if (whole + l < p.E) top = fmaxf(top, D::get(x[whole + l]));
            top = fold<LANES>(top, Max());
            float sum = 0.0f;
            for (uint32_t e = l * PER; e < whole; e += LANES * PER) {
                const vec t = *(const loose *)(x + e);
                for (int i = 0; i < PER; i++) sum += __builtin_amdgcn_exp2f((D::get(t[i]) - top) * LOG2E);
            }
            if (whole + l < p.E) sum += __builtin_amdgcn_exp2f((D::get(x[whole + l]) - top) * LOG2E);
            inv = 1.0f / fold<LANES>(sum, Sum());
        }
        /* the scores, renormalised or not, as msim_route has them */
        const float t = p.sigmoid ? fminf(xs, 0.0f) : xs;
        const float c = p.renorm ? fold<LANES>(got ? t : -INFINITY, Max()) : p.sigmoid ? 0.0f : top;
        float q = expf(t - c);
        if (p.sigmoid) q /= 1.0f + expf(-fabsf(xs));
        else if (!p.renorm) q *= inv;
        if (!got) q = 0.0f;
        if (p.renorm) {
            const float sum = fold<LANES>(q, Sum());
            if (got) q /= sum;
        }
        const float mean = fold<LANES>(g * q, Sum());
        float d = q * (p.renorm ? g - mean : g);
        if (p.sigmoid) d *= xs > 0.0f ? expf(-xs) / (1.0f + expf(-xs)) : 1.0f / (1.0f + expf(xs));
        d = got ? d * p.scale : 0.0f;
        const float base = -p.scale * mean;            /* times a score: what every expert gets */
        const bool some = fold<LANES>(got ? 1.0f : 0.0f, Max()) > 0.0f;
        /* an expert named twice: its first slot has the sum, in slot order */
        float total = 0.0f;
        bool first = got;
        for (uint32_t j = 0; j < p.K; j++) {
            const int at = (int)(lane - l + j);
            const int32_t oi = __shfl(id, at);
            const float od = __shfl(d, at);
            if (oi == id) {
                total += od;
                if (j < l) first = false;
            }
        }
        typename D::raw *dx = (typename D::raw *)p.dx + row * p.dstride;
        for (uint32_t e0 = 0; e0 < p.E; e0 += CHUNK) {
            const bool in = first && (uint32_t)id - e0 < CHUNK;
            if (in) buf[lane / LANES][id - e0] = total;
            wave_sync();
            const uint32_t end = min(CHUNK, p.E - e0);
            const uint32_t whole = end - end % PER;
            for (uint32_t e = l * PER; e < whole; e += LANES * PER) {
                float v[PER];
                for (int i = 0; i < PER; i += 4) *(f32x4 *)&v[i] = *(const f32x4 *)&buf[lane / LANES][e + i];
                if (every && some) {
                    const vec t = *(const loose *)(x + e0 + e);
                    for (int i = 0; i < PER; i++)
                        v[i] += base * (__builtin_amdgcn_exp2f((D::get(t[i]) - top) * LOG2E) * inv);
                }
                vec o;
                for (int i = 0; i < PER; i++) o[i] = D::put(v[i]);
                if (mine) *(loose *)(dx + e0 + e) = o;
            }
            if (whole + l < end) {
                float v = buf[lane / LANES][whole + l];
                if (every && some) v += base * (__builtin_amdgcn_exp2f((D::get(x[e0 + whole + l]) - top) * LOG2E) * inv);
                if (mine) dx[e0 + whole + l] = D::put(v);
            }
            wave_sync();
            if (in) buf[lane / LANES][id - e0] = 0.0f;
        }
    }
}

/* ------------------------------------------------------------------------ */
/* dropout                                                                   */
/* ------------------------------------------------------------------------ */

struct DropP {
    const void *x;
    void *y;
    uint64_t rows, cols, xs, ys, base, limit;
    float scale;
    uint32_t per_row;
};

/* Elements that lie next to each other, PER of them (16 bytes) a thread and
 * turn: bound by the memory, and nearly by the generator, a 64-bit mix for two
 * elements, so a mix is used whole and its counter moves by an addition.
 * 131,072 x 512 bf16 take 45 - 50 us (5.4 - 6.0 TB/s, the inputs partly from the
 * last-level cache); without the mix it is 5 % less. */
template <typename D> __global__ void __launch_bounds__(256) msim_dropout_flat(DropP p)
{
    constexpr int PER = 16 / sizeof(typename D::raw);
    typedef typename D::raw vec __attribute__((ext_vector_type(PER), aligned(sizeof(typename D::raw))));
    const uint64_t n = p.rows * p.cols, step = (uint64_t)gridDim.x * blockDim.x * PER;
    const uint32_t limit = (uint32_t)p.limit;          /* p < 1 here */
    for (uint64_t i = ((uint64_t)blockIdx.x * blockDim.x + threadIdx.x) * PER; i < n; i += step) {
        const typename D::raw *x = (const typename D::raw *)p.x + i;
        typename D::raw *y = (typename D::raw *)p.y + i;
        uint64_t z = p.base + (i >> 1) * GAMMA;
        bool keep[PER];
        for (int j = 0; j < PER; j += 2, z += GAMMA) {
            const uint64_t d = mix64(z);
            keep[j] = (uint32_t)d >= limit;
            keep[j + 1] = (uint32_t)(d >> 32) >= limit;
        }
        if (i + PER <= n) {
            vec v = *(const vec *)x;
            for (int j = 0; j < PER; j++) v[j] = D::put(keep[j] ? D::get(v[j]) * p.scale : 0.0f);
            *(vec *)y = v;
        } else {
            for (int j = 0; j < PER; j++)
                if (i + j < n) y[j] = D::put(keep[j] ? D::get(x[j]) * p.scale : 0.0f);
        }
    }
}

/* Rows with a stride, or that stay or go whole: 2^lwide threads a row, PER
 * elements (16 bytes, or 2 of rows shorter than that) a thread and turn.  Where a
 * row begins on the second half of a mix, so does every thread's part.  131,072
 * x 512 bf16 out of 520: 51 us (5.3 TB/s); whole rows, of which those that go
 * are not read, 39 us. */
template <typename D, int PER, bool WHOLE> __global__ void __launch_bounds__(256) msim_dropout_rows(DropP p, uint32_t lwide)
{
    typedef typename D::raw vec __attribute__((ext_vector_type(PER), aligned(sizeof(typename D::raw))));
    const uint32_t wide = 1u << lwide, me = threadIdx.x & (wide - 1);
    const uint64_t step = (uint64_t)gridDim.x * (blockDim.x >> lwide);
    for (uint64_t r = (uint64_t)blockIdx.x * (blockDim.x >> lwide) + (threadIdx.x >> lwide); r < p.rows; r += step) {
        const bool stays = !WHOLE || draw32(p.base, r) >= p.limit;
        for (uint64_t c = me * PER; c < p.cols; c += wide * PER) {
            const typename D::raw *x = (const typename D::raw *)p.x + r * p.xs + c;
            typename D::raw *y = (typename D::raw *)p.y + r * p.ys + c;
            bool keep[PER];
            for (int j = 0; j < PER; j++) keep[j] = stays;
            if (!WHOLE) {
                const uint64_t i = r * p.cols + c;
                uint64_t z = p.base + (i >> 1) * GAMMA;
                const bool odd = i & 1;
                uint32_t half[PER + 2];
                for (int j = 0; j < PER; j += 2, z += GAMMA) {
                    const uint64_t d = mix64(z);
                    half[j] = (uint32_t)d;
                    half[j + 1] = (uint32_t)(d >> 32);
                }
                half[PER] = odd ? (uint32_t)mix64(z) : 0;
                for (int j = 0; j < PER; j++) keep[j] = (odd ? half[j + 1] : half[j]) >= p.limit;
            }
            if (c + PER <= p.cols) {
                vec v = {};
                if (stays) v = *(const vec *)x;
                for (int j = 0; j < PER; j++) v[j] = D::put(keep[j] ? D::get(v[j]) * p.scale : 0.0f);
                *(vec *)y = v;
            } else {
                for (int j = 0; j < PER; j++)
                    if (c + j < p.cols) y[j] = D::put(keep[j] ? D::get(x[j]) * p.scale : 0.0f);
            }
        }
    }
}

/* ------------------------------------------------------------------------ */
/* traffic                                                                   */
/* ------------------------------------------------------------------------ */

struct TrafficP {
    const int32_t *ids;
    const int64_t *off;
    const int32_t *home, *place;
    int32_t *out;
    uint64_t rows, n_seg, base, limit;
    uint32_t E, K, H, token_bytes, pkt_bytes, per_row;
    uint32_t vec, small, recip;            /* ids by 16 bytes; bytes below 2^31; floor((2^32 - 1) / pkt_bytes) */
    uint64_t parts;                        /* workgroups a segment */
};

/* the packets of `count` tokens */
__device__ __forceinline__ uint32_t packets_of(const TrafficP &p, uint32_t count)
{
    if (p.small) {
        /* below 2^31 bytes: the quotient by the reciprocal is right or one short */
        const uint32_t b = count * p.token_bytes;
        uint32_t k = __umulhi(b, p.recip), rest = b - k * p.pkt_bytes;
        if (rest >= p.pkt_bytes) { k++; rest -= p.pkt_bytes; }
        return k + (rest != 0);
    }
    const uint64_t b = (uint64_t)count * p.token_bytes;
    return (uint32_t)min(b / p.pkt_bytes + (b % p.pkt_bytes != 0), (uint64_t)0x7FFFFFFF);
}

/* A workgroup a segment: a count per host in LDS, a token a thread, its hosts
 * in registers where each is compared with those before it.  Bound by latency:
 * offsets, ids, hosts and counts follow from one another, so a segment has no
 * more threads than tokens and as many segments as fit run side by side.  64 x
 * 128 hosts, 8 choices: 11 us for 21 MB; 1,024 hosts with 128 tokens: 5.5 for 8.
 * Few long segments are cut into `parts`, whose counts meet in the table, cleared
 * before and turned into packets after: 8 segments of 131,072 tokens and 128
 * hosts 227 -> 16 us, 64 of 16,384 32 -> 16.  All segments in the same number, by
 * their mean length: a long one among many short ones is one workgroup's work (one
 * of 1,048,576 tokens among 1,024 of 128: 3.9 ms, where 1,025 of the same sum take
 * 14 us).  More than 16 choices: 64 registers spill, 166 us for the 64 x 128
 * segments of 128 tokens that take 13 with 8 choices and 24 with 16. */
template <int KMAX> __global__ void __launch_bounds__(1024) msim_traffic_segments(TrafficP p)
{
    extern __shared__ uint32_t count[];
    for (uint64_t w = blockIdx.x; w < p.n_seg * p.parts; w += gridDim.x) {
        const uint64_t s = p.parts == 1 ? w : w / p.parts, part = w - s * p.parts;
        uint64_t lo = min((uint64_t)max(p.off[s], (int64_t)0), p.rows);
        uint64_t hi = min((uint64_t)max(p.off[s + 1], (int64_t)0), p.rows);
        if (p.parts > 1 && hi > lo) {
            const uint64_t each = (hi - lo + p.parts - 1) / p.parts;
            lo = min(lo + part * each, hi);
            hi = min(lo + each, hi);
        }
        const uint32_t home = p.home[s];
        for (uint32_t h = threadIdx.x; h < p.H; h += blockDim.x) count[h] = 0;
        __syncthreads();
        for (uint64_t t = lo + threadIdx.x; t < hi; t += blockDim.x) {
            int32_t h[KMAX];
            if (KMAX >= 4 && p.vec) {
                for (int j = 0; j < KMAX; j += 4) {
                    i32x4 id = {-1, -1, -1, -1};
                    if (j < (int)p.K) id = *(const i32x4 *)(p.ids + t * p.K + j);
                    for (int i = 0; i < 4 && j + i < KMAX; i++) h[j + i] = id[i];
                }
            } else {
                for (int j = 0; j < KMAX; j++) h[j] = j < (int)p.K ? p.ids[t * p.K + j] : -1;
            }
            for (int j = 0; j < KMAX; j++) h[j] = (uint32_t)h[j] < p.E ? p.place[h[j]] : -1;
            if (p.limit) {
                if (p.per_row) {
                    if (draw32(p.base, t) < p.limit)
                        for (int j = 0; j < KMAX; j++) h[j] = -1;
                } else if (p.K % 2 == 0) {
                    uint64_t z = p.base + (t * p.K >> 1) * GAMMA;
                    for (int j = 0; j < KMAX; j += 2, z += GAMMA) {
                        const uint64_t d = mix64(z);
                        if ((uint32_t)d < p.limit) h[j] = -1;
                        if (j + 1 < KMAX && (d >> 32) < p.limit) h[j + 1] = -1;
                    }
                } else {
                    for (int j = 0; j < KMAX; j++)
                        if (draw32(p.base, t * p.K + j) < p.limit) h[j] = -1;
                }
            }
            for (int j = 0; j < KMAX; j++) {
                bool go = (uint32_t)h[j] < p.H;
                for (int i = 0; i < j; i++) go &= h[i] != h[j];
                if (go) atomicAdd(&count[h[j]], 1u);
            }
        }
        __syncthreads();
        for (uint32_t h = threadIdx.x; h < p.H; h += blockDim.x) {
            int32_t *out = p.out + s * p.H + h;
            if (p.parts == 1) *out = h == home ? 0 : (int32_t)packets_of(p, count[h]);
            else if (h != home && count[h]) atomicAdd(out, (int32_t)count[h]);
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(256) msim_traffic_clear(TrafficP p)
{
    const uint64_t n = p.n_seg * p.H, step = (uint64_t)gridDim.x * blockDim.x;
    for (uint64_t i = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) p.out[i] = 0;
}

__global__ void __launch_bounds__(256) msim_traffic_packets(TrafficP p)
{
    const uint64_t n = p.n_seg * p.H, step = (uint64_t)gridDim.x * blockDim.x;
    for (uint64_t i = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step)
        p.out[i] = (int32_t)packets_of(p, (uint32_t)p.out[i]);
}

/* ------------------------------------------------------------------------ */
/* host                                                                      */
/* ------------------------------------------------------------------------ */

int fail(int code, const char *what) { msim_set_error(what); return code; }

/* Enqueues a kernel.  The result is the launch's own: an error that another call
 * left pending on this thread neither fails it nor is taken from its owner. */
template <typename... P, typename... A>
hipError_t launch(void (*kernel)(P...), uint32_t grid, uint32_t block, size_t lds, hipStream_t st, A... args)
{
    return [&](P... p) {
        void *at[] = {&p...};
        return hipLaunchKernel((const void *)kernel, dim3(grid), dim3(block), at, lds, st);
    }(args...);
}

int launched(hipError_t e, const char *what)
{
    if (e == hipSuccess) return MSIM_OK;
    (void)hipGetLastError();               /* it is reported here */
    msim_set_error2(what, hipGetErrorString(e));
    return MSIM_E_HIP;
}

uint64_t splitmix_base(uint64_t seed, uint64_t offset) { return seed + (offset + 1) * GAMMA; }

/* p in [0, 1] as the 32-bit limit below which a draw drops */
bool drop_limit(double p, uint64_t *limit)
{
    if (!(p >= 0.0 && p <= 1.0)) return false;
    *limit = (uint64_t)(p * 4294967296.0 + 0.5);
    return true;
}

const char *check_route(const msim_route_spec *s, bool backward, int *code)
{
    *code = MSIM_E_ARG;
    if (!s) return "route: null spec";
    if (s->version != MSIM_ABI_VERSION) return "route: spec version mismatch";
    if (s->dtype > MSIM_BF16) return "route: unknown dtype";
    if (s->score > MSIM_SCORE_SIGMOID) return "route: unknown score";
    if (s->experts == 0 || s->top_k == 0) return "route: experts and top_k must be at least 1";
    if (s->renorm > 1) return "route: renorm must be 0 or 1";
    if (!std::isfinite(s->scale)) return "route: scale must be finite";
    if (s->rows && s->row_stride < s->experts) return "route: row_stride below experts";
    *code = MSIM_E_LIMIT;
    if (s->experts > MSIM_MAX_EXPERTS) return "route: more than MSIM_MAX_EXPERTS experts";
    if (s->top_k > MSIM_MAX_TOP_K) return "route: top_k above MSIM_MAX_TOP_K";
    if (s->rows >> 31 || s->row_stride >> 40) return "route: 2^31 rows or more, or a row_stride of 2^40 or more";
    *code = MSIM_E_ARG;
    if (backward) return s->top_k > s->experts ? "route: top_k above experts" : nullptr;
    if (s->groups == 0 || s->experts % s->groups) return "route: groups must divide experts";
    if (s->top_groups == 0 || s->top_groups > s->groups) return "route: top_groups must be 1 .. groups";
    if (s->group_top < 1 || s->group_top > 2) return "route: group_top must be 1 or 2";
    if (s->top_k > s->experts / s->groups * s->top_groups) return "route: top_k above the experts of top_groups groups";
    *code = MSIM_E_LIMIT;
    if (s->groups > MSIM_MAX_EXPERT_GROUPS) return "route: more than MSIM_MAX_EXPERT_GROUPS groups";
    return nullptr;
}

uint32_t pow2(uint32_t v)
{
    uint32_t p = 1;
    while (p < v) p *= 2;
    return p;
}

template <typename D> hipError_t launch_finish(const RouteP &p, bool undecided, hipStream_t st)
{
    if (!undecided && !p.load) return hipSuccess;
    /* 256 workgroups, which is few enough to add to the same counts, while they can take the rows */
    const uint64_t part = std::min<uint64_t>(std::max<uint64_t>(256, (p.rows + 255) / 256), FINISH_ROWS);
    const uint32_t grid = (uint32_t)((p.rows + part - 1) / part);
    const uint32_t block = p.E <= 256 ? 512 : 256;            /* LDS: at most 32 KiB of keys */
    const size_t lds = undecided && p.G > 1 ? block / WAVE * p.E * sizeof(double) : 0;
    return launch(p.E <= 256 ? msim_route_finish<D, 4> : msim_route_finish<D, 16>, grid, block, lds, st, p, part);
}

template <typename D, int VPL, int LANES, int KL> hipError_t launch_lists(const RouteP &p, hipStream_t st)
{
    const uint32_t rows = 4 * WAVE / LANES;
    const uint32_t grid = (uint32_t)std::min<uint64_t>((p.rows + rows - 1) / rows, 1024);
    const bool undecided = p.bias || p.gtop > 1;
    const hipError_t e = launch(p.bias ? msim_route_lists<D, VPL, LANES, KL, true> : msim_route_lists<D, VPL, LANES, KL, false>,
                                grid, 256, 0, st, p);
    return e == hipSuccess && (grid > 1 || undecided) ? launch_finish<D>(p, undecided, st) : e;
}

template <typename D> hipError_t launch_route(RouteP p, hipStream_t st)
{
    if (p.rows == 0) return p.load ? launch(msim_route_nothing, 1, 256, 0, st, p) : hipSuccess;
    /* lists: lanes for every group and every choice, at most 32 experts a lane */
    const uint32_t size = p.E / p.G, g2 = pow2(p.G), kl = p.K <= 8 ? 8 : 16;
    uint32_t glanes = std::max(1u, kl / g2);
    while ((size + glanes - 1) / glanes > 32) glanes *= 2;
    const uint32_t lanes = g2 * glanes;
    const size_t sz = sizeof(typename D::raw);
    if (p.G == 1 && p.E <= THREAD_EXPERTS && p.K <= (p.bias ? 7u : 8u) && p.rows >= 2048 * p.E) {
        const uint32_t grid = (uint32_t)std::min<uint64_t>((p.rows + 255) / 256, 4096);
        p.vec = p.E * sz >= 16 ? 0 : 2;
        const hipError_t e = launch(p.bias ? msim_route_threads<D, true> : msim_route_threads<D, false>, grid, 256, 0, st, p);
        return e == hipSuccess ? launch_finish<D>(p, p.bias != nullptr, st) : e;
    }
    if (p.K <= 16 && lanes <= 32) {
        p.size = size;
        p.lglanes = __builtin_ctz(glanes);
        p.part = (size + glanes - 1) / glanes;
        const uint32_t vpl = std::max(lanes == 8 ? 8u : lanes == 16 ? 16u : 32u, pow2(p.part));
        p.vec = p.part == vpl && p.part * glanes == size && (size * sz) % 16 == 0 && (p.stride * sz) % 16 == 0 &&
                (uintptr_t)p.x % 16 == 0 ? 1 : p.E * sz >= 16 ? 0 : 2;
        if (kl == 16 && lanes == 32) return launch_lists<D, 32, 32, 16>(p, st);
        if (kl == 16 && vpl == 32) return launch_lists<D, 32, 16, 16>(p, st);
        if (kl == 16) return launch_lists<D, 16, 16, 16>(p, st);
        if (lanes == 32) return launch_lists<D, 32, 32, 8>(p, st);
        if (lanes == 16 && vpl == 32) return launch_lists<D, 32, 16, 8>(p, st);
        if (lanes == 16) return launch_lists<D, 16, 16, 8>(p, st);
        if (vpl == 32) return launch_lists<D, 32, 8, 8>(p, st);
        if (vpl == 16) return launch_lists<D, 16, 8, 8>(p, st);
        return launch_lists<D, 8, 8, 8>(p, st);
    }
    const uint32_t grid = (uint32_t)std::min<uint64_t>((p.rows + 3) / 4, 2048);
    const size_t lds = p.G > 1 ? 4 * p.E * sizeof(double) : 0;
    const hipError_t e = launch(p.E <= 256 ? msim_route_rows<D, 4> : msim_route_rows<D, 16>, grid, 256, lds, st, p);
    return e == hipSuccess ? launch_finish<D>(p, false, st) : e;
}

template <typename D> hipError_t launch_back(const BackP &p, hipStream_t st)
{
    /* few rows: fewer of them a wavefront, and more wavefronts */
    const uint32_t lanes = p.K <= 8 && p.rows > 16384 ? 8 : p.K <= 16 && p.rows > 4096 ? 16 : 32;
    const uint64_t rows = 4 * WAVE / lanes;
    const uint32_t grid = (uint32_t)std::min<uint64_t>((p.rows + rows - 1) / rows, 2048);
    return launch(lanes == 8 ? msim_route_back<D, 8> : lanes == 16 ? msim_route_back<D, 16> : msim_route_back<D, 32>, grid, 256,
                  0, st, p);
}

template <typename D> hipError_t launch_dropout(const DropP &d, hipStream_t st)
{
    constexpr uint64_t per = 16 / sizeof(typename D::raw);
    const uint64_t n = d.rows * d.cols;
    if (!d.per_row && (d.rows == 1 || (d.xs == d.cols && d.ys == d.cols)) && d.limit >> 32 == 0)
        return launch(msim_dropout_flat<D>, (uint32_t)std::min<uint64_t>((n + 256 * per - 1) / (256 * per), 1u << 16), 256, 0,
                      st, d);
    const uint64_t turns = (d.cols + (d.cols >= per ? per : 2) - 1) / (d.cols >= per ? per : 2);
    const uint32_t lwide = turns >= 256 ? 8 : __builtin_ctz(pow2((uint32_t)turns));
    const uint64_t rows = 256 >> lwide;
    const uint32_t grid = (uint32_t)std::min<uint64_t>((d.rows + rows - 1) / rows, 1u << 16);
    if (d.cols >= per)
        return launch(d.per_row ? msim_dropout_rows<D, per, true> : msim_dropout_rows<D, per, false>, grid, 256, 0, st, d, lwide);
    return launch(d.per_row ? msim_dropout_rows<D, 2, true> : msim_dropout_rows<D, 2, false>, grid, 256, 0, st, d, lwide);
}

} // namespace

extern "C" int msim_route(const msim_route_spec *s, const void *logits, const float *bias, int32_t *ids,
                          float *weights, int32_t *load, void *hip_stream)
{
    int code;
    if (const char *why = check_route(s, false, &code)) return fail(code, why);
    if (s->rows && (!logits || !ids || !weights)) return fail(MSIM_E_ARG, "route: null logits, ids or weights");
    RouteP p = {logits, bias, ids, weights, load, s->rows, s->row_stride, s->experts, s->top_k, s->groups,
                s->top_groups, s->group_top, s->renorm, s->score == MSIM_SCORE_SIGMOID, s->scale, 0, 0, 0, 0};
    if (p.TG == p.G) p.G = p.TG = p.gtop = 1;       /* every group stays */
    hipStream_t st = (hipStream_t)hip_stream;
    const hipError_t e = s->dtype == MSIM_F32 ? launch_route<F32>(p, st)
        : s->dtype == MSIM_F16 ? launch_route<F16>(p, st) : launch_route<BF16>(p, st);
    return launched(e, "route launch");
}

extern "C" int msim_route_backward(const msim_route_spec *s, const void *logits, const int32_t *ids,
                                   const float *grad, void *grad_logits, uint64_t grad_stride, void *hip_stream)
{
    int code;
    if (const char *why = check_route(s, true, &code)) return fail(code, why);
    if (s->rows == 0) return MSIM_OK;
    if (!logits || !ids || !grad || !grad_logits) return fail(MSIM_E_ARG, "route: null logits, ids or gradient");
    if (grad_stride < s->experts) return fail(MSIM_E_ARG, "route: grad_stride below experts");
    if (grad_stride >> 40) return fail(MSIM_E_LIMIT, "route: grad_stride of 2^40 or more");
    const BackP p = {logits, ids, grad, grad_logits, s->rows, s->row_stride, grad_stride, s->experts, s->top_k,
                     s->renorm, s->score == MSIM_SCORE_SIGMOID, s->scale};
    hipStream_t st = (hipStream_t)hip_stream;
    const hipError_t e = s->dtype == MSIM_F32 ? launch_back<F32>(p, st)
        : s->dtype == MSIM_F16 ? launch_back<F16>(p, st) : launch_back<BF16>(p, st);
    return launched(e, "route backward launch");
}

extern "C" int msim_dropout(uint32_t dtype, const void *x, void *y, uint64_t rows, uint64_t cols, uint64_t x_stride,
                            uint64_t y_stride, double p, uint64_t seed, uint64_t offset, uint32_t per_row,
                            void *hip_stream)
{
    DropP d = {x, y, rows, cols, x_stride, y_stride, splitmix_base(seed, offset), 0, 0.0f, per_row};
    if (dtype > MSIM_BF16) return fail(MSIM_E_ARG, "dropout: unknown dtype");
    if (per_row > 1) return fail(MSIM_E_ARG, "dropout: per_row must be 0 or 1");
    if (!drop_limit(p, &d.limit)) return fail(MSIM_E_ARG, "dropout: p must be in [0, 1]");
    if (rows == 0 || cols == 0) return MSIM_OK;
    if (!x || !y) return fail(MSIM_E_ARG, "dropout: null tensor");
    if (x_stride < cols || y_stride < cols) return fail(MSIM_E_ARG, "dropout: stride below cols");
    if (x == y && x_stride != y_stride) return fail(MSIM_E_ARG, "dropout: in place with two strides");
    if (rows >> 40 || cols >> 40 || x_stride >> 40 || y_stride >> 40 || rows > (1ull << 44) / cols)
        return fail(MSIM_E_LIMIT, "dropout: more than 2^44 elements");
    d.scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.0f;
    hipStream_t st = (hipStream_t)hip_stream;
    const hipError_t e = dtype == MSIM_F32 ? launch_dropout<F32>(d, st)
        : dtype == MSIM_F16 ? launch_dropout<F16>(d, st) : launch_dropout<BF16>(d, st);
    return launched(e, "dropout launch");
}

extern "C" int msim_traffic(const msim_traffic_spec *s, const int32_t *ids, const int64_t *token_off,
                            const int32_t *home, const int32_t *place, int32_t *packets, void *hip_stream)
{
    if (!s) return fail(MSIM_E_ARG, "traffic: null spec");
    if (s->version != MSIM_ABI_VERSION) return fail(MSIM_E_ARG, "traffic: spec version mismatch");
    if (!s->experts || !s->top_k || !s->hosts) return fail(MSIM_E_ARG, "traffic: experts, top_k and hosts must be at least 1");
    if (!s->token_bytes || !s->pkt_bytes) return fail(MSIM_E_ARG, "traffic: token_bytes and pkt_bytes must be at least 1");
    if (s->per_row > 1 || s->reserved) return fail(MSIM_E_ARG, "traffic: per_row must be 0 or 1, reserved 0");
    TrafficP p = {ids, token_off, home, place, packets, s->rows, s->n_seg, splitmix_base(s->seed, s->offset), 0,
                  s->experts, s->top_k, s->hosts, s->token_bytes, s->pkt_bytes, s->per_row,
                  s->top_k % 4 == 0 && (uintptr_t)ids % 16 == 0, 0, 0xFFFFFFFFu / std::max(s->pkt_bytes, 1u), 1};
    if (!drop_limit(s->drop, &p.limit)) return fail(MSIM_E_ARG, "traffic: drop must be in [0, 1]");
    if (s->experts > (1u << 24)) return fail(MSIM_E_LIMIT, "traffic: more than 2^24 experts");
    if (s->top_k > MSIM_MAX_TOP_K) return fail(MSIM_E_LIMIT, "traffic: top_k above MSIM_MAX_TOP_K");
    if (s->hosts > MSIM_MAX_TRAFFIC_HOSTS) return fail(MSIM_E_LIMIT, "traffic: more than MSIM_MAX_TRAFFIC_HOSTS hosts");
    if (s->rows >> 32) return fail(MSIM_E_LIMIT, "traffic: 2^32 rows or more");
    if (s->n_seg >> 32) return fail(MSIM_E_LIMIT, "traffic: 2^32 segments or more");
    if (s->n_seg == 0) return MSIM_OK;
    if (!token_off || !home || !place || !packets || (s->rows && !ids)) return fail(MSIM_E_ARG, "traffic: null array");
    p.small = s->rows * s->token_bytes < (1ull << 31);
    /* As many threads as a segment has tokens (about) or quarters of its hosts, while all segments' together fill
     * the card: 1,024 segments of 128 tokens and 1,024 hosts take 5.4 us with 256 threads, 7.6 with 64; 8,192 of 64
     * and 128 hosts 11.1 with 64, 16.5 with 256. */
    const uint64_t want = std::max<uint64_t>((s->rows + s->n_seg - 1) / s->n_seg, s->hosts / 4);
    const uint64_t most = std::max<uint64_t>(64, 524288 / s->n_seg);
    uint32_t block = 64;
    while (block < 1024 && block < want && 2 * block <= most) block *= 2;
    /* A workgroup for every 4,096 tokens of a segment of mean length (rows behind the last segment counted in), up
     * to 1,024 in all: token_off is on the device, so the host knows no other length. */
    p.parts = std::max<uint64_t>(1, std::min((s->rows / s->n_seg) / 4096, 1024 / s->n_seg));
    const uint32_t grid = (uint32_t)std::min<uint64_t>(s->n_seg * p.parts, 1u << 20);
    const uint32_t every = (uint32_t)std::min<uint64_t>((s->n_seg * s->hosts + 255) / 256, 4096);
    const size_t lds = 4 * s->hosts;
    hipStream_t st = (hipStream_t)hip_stream;
    void (*const segments)(TrafficP) = p.K <= 2 ? msim_traffic_segments<2> : p.K <= 4 ? msim_traffic_segments<4>
        : p.K <= 8 ? msim_traffic_segments<8> : p.K <= 16 ? msim_traffic_segments<16> : msim_traffic_segments<32>;
    hipError_t e = p.parts > 1 ? launch(msim_traffic_clear, every, 256, 0, st, p) : hipSuccess;
    if (e == hipSuccess) e = launch(segments, grid, block, lds, st, p);
    if (e == hipSuccess && p.parts > 1) e = launch(msim_traffic_packets, every, 256, 0, st, p);
    return launched(e, "traffic launch");
}
