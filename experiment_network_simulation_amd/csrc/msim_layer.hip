/* A whole mixture-of-experts layer for a few tokens (msim_layer of include/msim.h,
 * which has the definition): gate logits, msim_route, the experts' two products,
 * and the weighted sum of what the chosen experts answer.
 *
 * What bounds it is reading the chosen experts' weights once; each of the two
 * products has a workgroup for an expert that some token chose and a few of its
 * rows of weights, and that workgroup has all of the expert's tokens.
 */

#include <algorithm>
#include <type_traits>

#include "msim_route.h"
#include "msim_stream.h"

namespace {

constexpr uint32_t MAX_ROWS = MSIM_MAX_LAYER_ROWS;

struct LayerP {
    const void *x, *gate, *w_in, *w_out, *res;
    const uint8_t *mask;
    void *out;
    float *logits;
    const int32_t *ids;
    const float *weights;
    int32_t *load;               /* tokens of each expert */
    void *h;                     /* [rows * top_k][h_ld], of the layer's type; of f16 low parts follow, h_low elements on */
    float *part;                 /* [rows * top_k][part_ld] */
    uint64_t x_ld, out_ld, res_ld, h_ld, h_low, part_ld;
    uint32_t rows, E, K, C, F, act, gated;
    /* Of a product.  slots: assignments, of which the first that names an expert has it, if they are fewer than
     * experts; otherwise experts.  tiles of weight rows. */
    uint32_t slots, tiles;
};

/* Logits in 64 bits, rounded to 32: of 16-bit inputs every product is exact, and
 * the choice of experts follows from the inputs, not from an order of additions.
 * One expert and TT tokens a workgroup.  Rows that are masked out route nowhere.
 * Bound by conversions to 64 bits and their products: 512 x 2,048 and 64 experts 22
 * us; of one token 3, a launch. */
template <typename D, int TT> __global__ void __launch_bounds__(256) msim_layer_gate(LayerP p)
{
    typedef typename D::raw raw;
    constexpr uint32_t PER = 16 / sizeof(raw);
    typedef raw vec __attribute__((ext_vector_type(PER)));
    __shared__ double part[4][TT];
    const uint32_t e = blockIdx.x % p.E, t0 = blockIdx.x / p.E * TT;
    const raw *g = (const raw *)p.gate + (uint64_t)e * p.C;
    double sum[TT];
    for (int t = 0; t < TT; t++) sum[t] = 0;
    for (uint32_t c = threadIdx.x * PER; c < p.C; c += 256 * PER) {
        const vec w = __builtin_bit_cast(vec, piece<D>(g, c, p.C));
        vec x[TT];
        for (int t = 0; t < TT; t++)
            x[t] = __builtin_bit_cast(vec, piece<D>((const raw *)p.x + min(t0 + t, p.rows - 1) * p.x_ld, c, p.C));
        for (uint32_t i = 0; i < PER; i++) {
            const double v = D::get(w[i]);
            for (int t = 0; t < TT; t++) sum[t] = __builtin_fma(v, (double)D::get(x[t][i]), sum[t]);
        }
    }
    for (int t = 0; t < TT; t++) {
        for (int d = 1; d < 64; d *= 2) sum[t] += __shfl_xor(sum[t], d);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][t] = sum[t];
    }
    __syncthreads();
    const uint32_t t = t0 + threadIdx.x;
    if (threadIdx.x < TT && t < p.rows) {
        const double s = part[0][threadIdx.x] + part[1][threadIdx.x] + part[2][threadIdx.x] + part[3][threadIdx.x];
        p.logits[(uint64_t)t * p.E + e] = p.mask && !p.mask[t] ? -INFINITY : (float)s;
    }
}

/* The list of an expert's assignments (row * K + choice), in order, and their number.
 * Each thread looks at as many ids next to each other as it takes. */
template <int WAVES> __device__ __forceinline__ uint32_t tokens_of(const LayerP &p, const int32_t *ids, int32_t expert, uint32_t *list, uint32_t *counts)
{
    const uint32_t n = p.rows * p.K, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t per = (n + 64 * WAVES - 1) / (64 * WAVES), first = threadIdx.x * per, last = min(n, first + per);
    uint32_t mine = 0;
    for (uint32_t j = first; j < last; j++) mine += ids[j] == expert;
    uint32_t upto = mine;
    for (uint32_t d = 1; d < 64; d *= 2) {
        const uint32_t before = __shfl_up(upto, d);
        if (lane >= d) upto += before;
    }
    if (lane == 63) counts[wave] = upto;
    __syncthreads();
    uint32_t at = upto - mine, have = 0;
    for (uint32_t w = 0; w < WAVES; w++) {
        if (w < wave) at += counts[w];
        have += counts[w];
    }
    if (mine)
        for (uint32_t j = first; j < last; j++)
            if (ids[j] == expert && at < MAX_ROWS) list[at++] = j;
    __syncthreads();
    return min(have, MAX_ROWS);
}

/* Hidden units are rounded to the layer's type, as matrix instructions read them, half a step of it.  In f16 a product of two
 * halves is soon above 65,504, so there they are held in two parts, HIGH times the first and the second: 22 bits, and
 * up to 2.7e8.  16 vectors of a matrix instruction of the second product are both parts of 8 tokens: no more time
 * up to 8 tokens an expert, and then (100 x 1,000, 3 of 24 experts 33.5 -> 38.6 us, 512 x 2,048, 6 of 64 315 -> 396)
 * what bf16 is spared, whose range is that of 32 bits. */
template <typename D> constexpr bool PARTS = std::is_same<D, F16>::value;
constexpr float HIGH = 4096.0f;
template <typename D> constexpr uint32_t TOKENS = PARTS<D> ? 8 : 16;      /* of 16 vectors */

/* 16 vectors of the second product: row(t) is where token t's first part begins, t < TOKENS */
template <typename D> struct Hidden : std::conditional<PARTS<D>, RowsOfTwo<D>, Rows<D>>::type {
    template <typename F> __device__ __forceinline__ void of(const LayerP &p, F row)
    {
        if constexpr (PARTS<D>) this->set(p.h_low, row);
        else this->set(row);
    }
};

/* Four hidden units from f on (16 more of them 16 further, without a gate) of what
 * goes into a token's row h of the second product.  h has room to a multiple of 8. */
template <typename D> __device__ __forceinline__ void hidden_of(const LayerP &p, const f32x4 *sums, uint32_t f, typename D::raw *h)
{
    for (uint32_t j = 0; j < (p.gated ? 1 : 2); j++, f += 16) {
        if (f >= p.F) continue;
        float v[4];
        for (int k = 0; k < 4; k++) v[k] = j ? sums[1][k] : sums[0][k];
        act_of<4, std::is_same<D, F32>::value>(v, p.act);
        for (int k = 0; k < 4; k++) {
            const float x = p.gated ? v[k] * sums[1][k] : v[k];
            const typename D::raw high = D::put(PARTS<D> ? x * (1.0f / HIGH) : x);
            h[f + k] = high;
            if constexpr (PARTS<D>) {
                const float y = D::get(high) * HIGH;
                h[p.h_low + f + k] = fabsf(y) < INFINITY ? D::put(x - y) : typename D::raw(0);
            }
        }
    }
}

/* h = act(gate rows x) (up rows x), or act(rows x): 16 hidden units (32 without a
 * gate) of one expert for up to 16 MT of its tokens */
template <typename D, int MT, int WAVES>
__device__ __forceinline__ void up_tokens(const LayerP &p, int32_t expert, uint32_t tile, const uint32_t *list, uint32_t n, char *lds)
{
    typedef typename D::raw raw;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & 15;
    const uint32_t f0 = tile * (p.gated ? 16 : 32);
    Rows<D> w[2], x[MT];
    const raw *base = (const raw *)p.w_in + (uint64_t)expert * (p.gated ? 2 : 1) * p.F * p.C;
    w[0].set([&](uint32_t r) { return base + (uint64_t)min(f0 + r, p.F - 1) * p.C; });
    w[1].set([&](uint32_t r) { return base + (uint64_t)(p.gated ? p.F + min(f0 + r, p.F - 1) : min(f0 + 16 + r, p.F - 1)) * p.C; });
    for (int i = 0; i < MT; i++) x[i].set([&](uint32_t r) { return (const raw *)p.x + list[min(i * 16 + r, n - 1)] / p.K * p.x_ld; });
    f32x4 acc[MT][2];
    for (int i = 0; i < MT; i++) acc[i][0] = acc[i][1] = f32x4{0, 0, 0, 0};
    stream<D, MT, 2, WAVES>(w, x, p.C, wave, lds + wave * STREAM_LDS<MT, 2>, acc);
    join<MT, 2, WAVES>(lds, wave, acc);
    _Pragma("unroll") for (int i = 0; i < MT; i++) {
        if (i % WAVES != (int)wave || i * 16 + l >= n) continue;
        hidden_of<D>(p, acc[i], f0 + (lane >> 4) * 4, (raw *)p.h + (uint64_t)list[i * 16 + l] * p.h_ld);
    }
}

/* what both parts of a hidden row gave, in the lanes of the first: lane ^ 8 has the second */
template <typename D> __device__ __forceinline__ f32x4 whole(f32x4 v)
{
    if constexpr (PARTS<D>)
        for (int k = 0; k < 4; k++) v[k] = HIGH * v[k] + __shfl_xor(v[k], 8);
    return v;
}

/* 32 columns of what one expert answers to up to TOKENS MT of its tokens, in 32 bits */
template <typename D, int MT, int WAVES>
__device__ __forceinline__ void down_tokens(const LayerP &p, int32_t expert, uint32_t tile, const uint32_t *list, uint32_t n, char *lds)
{
    typedef typename D::raw raw;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & 15;
    const uint32_t c0 = tile * 32;
    Rows<D> w[2];
    Hidden<D> x[MT];
    const raw *base = (const raw *)p.w_out + (uint64_t)expert * p.C * p.F;
    for (int j = 0; j < 2; j++) w[j].set([&](uint32_t r) { return base + (uint64_t)min(c0 + j * 16 + r, p.C - 1) * p.F; });
    constexpr uint32_t T = TOKENS<D>;
    for (int i = 0; i < MT; i++) x[i].of(p, [&](uint32_t t) { return (const raw *)p.h + (uint64_t)list[min(i * T + t, n - 1)] * p.h_ld; });
    f32x4 acc[MT][2];
    for (int i = 0; i < MT; i++) acc[i][0] = acc[i][1] = f32x4{0, 0, 0, 0};
    stream<D, MT, 2, WAVES>(w, x, p.F, wave, lds + wave * STREAM_LDS<MT, 2>, acc);
    join<MT, 2, WAVES>(lds, wave, acc);
    _Pragma("unroll") for (int i = 0; i < MT; i++) {
        if (i % WAVES != (int)wave) continue;
        const f32x4 y[2] = {whole<D>(acc[i][0]), whole<D>(acc[i][1])};
        if (l >= T || i * T + l >= n) continue;
        float *to = p.part + (uint64_t)list[i * T + l] * p.part_ld;
        for (int j = 0; j < 2; j++) {
            const uint32_t c = c0 + j * 16 + (lane >> 4) * 4;
            if (c < p.C) *(f32x4 *)(to + c) = y[j];            /* rows of part have room to a multiple of 4 */
        }
    }
}

/* The first product of up to FEW_ROWS tokens, which routes, too: every workgroup all
 * rows, a wavefront each, by route_row, which takes 1 to 2 us where msim_route
 * would be a launch or two more (one token of 2,048, 2 of 64 experts bf16, the whole
 * layer 28.9 us so, 23.7 like this). */
constexpr uint32_t FEW_ROWS = 16;
constexpr int FEW_WAVES = 16;

template <typename D, int VPL> __global__ void __launch_bounds__(64 * FEW_WAVES) msim_layer_up_few(LayerP p, RouteP r, int32_t *ids, float *weights)
{
    extern __shared__ double keys[];
    __shared__ int32_t chosen[FEW_ROWS * MSIM_MAX_TOP_K];
    __shared__ float shares[FEW_ROWS * MSIM_MAX_TOP_K];
    __shared__ uint32_t list[MAX_ROWS], counts[FEW_WAVES];
    __shared__ __attribute__((aligned(16))) char sums[FEW_WAVES * STREAM_LDS<1, 2>];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = p.rows * p.K;
    r.ids = chosen;
    r.w = shares;
    if (wave < p.rows) route_row<F32, VPL>(r, wave, keys + wave * p.E, nullptr);
    __syncthreads();
    if (blockIdx.x == 0) {
        for (uint32_t j = threadIdx.x; j < n; j += blockDim.x) {
            ids[j] = chosen[j];
            weights[j] = shares[j];
        }
        for (uint32_t e = threadIdx.x; e < p.E; e += blockDim.x) {
            int32_t c = 0;
            for (uint32_t j = 0; j < n; j++) c += chosen[j] == (int32_t)e;
            p.load[e] = c;
        }
    }
    const uint32_t slot = blockIdx.x / p.tiles;
    const int32_t expert = p.slots < p.E ? chosen[slot] : (int32_t)slot;
    if (expert < 0) return;
    const uint32_t have = tokens_of<FEW_WAVES>(p, chosen, expert, list, counts);
    if (have && (p.slots == p.E || list[0] == slot)) up_tokens<D, 1, FEW_WAVES>(p, expert, blockIdx.x % p.tiles, list, have, sums);
}

/* The second product and the sum of few tokens: 32 columns of one token's result a
 * workgroup, whose wavefronts share all runs of k of all its choices.  An expert
 * that two tokens chose is read twice.  4.4 us for one token of 2,048, two experts
 * of 1,024 units: a launch and the chain from a choice to its weights. */
template <typename D> __global__ void __launch_bounds__(64 * FEW_WAVES) msim_layer_down_few(LayerP p)
{
    typedef typename D::raw raw;
    __shared__ __attribute__((aligned(16))) char sums[FEW_WAVES * STREAM_LDS<1, 2>];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane & 15;
    const uint32_t t = blockIdx.x / p.tiles, c0 = blockIdx.x % p.tiles * 32, runs = (p.F + RUN<D> - 1) / RUN<D>;
    /* lane k has choice k; the residual is asked for now */
    const bool mine = lane < p.K;
    const int32_t id = mine ? p.ids[t * p.K + lane] : -1;
    const float share = mine ? p.weights[t * p.K + lane] : 0.0f;
    const uint32_t c = c0 + (lane >> 4) * 4;
    float res[8];
    for (uint32_t i = 0; i < 8; i++) {
        const uint32_t at = c + i / 4 * 16 + i % 4;
        res[i] = wave == 0 && l == 0 && p.res && at < p.C ? D::get(((const raw *)p.res)[t * p.res_ld + at]) : 0.0f;
    }
    f32x4 y[1][2] = {};
    for (uint32_t i = wave; i < p.K * runs; i += FEW_WAVES) {
        const uint32_t k = i / runs;
        const int32_t expert = __builtin_amdgcn_readlane(id, k);
        if (expert < 0) continue;
        const raw *base = (const raw *)p.w_out + (uint64_t)expert * p.C * p.F;
        Rows<D> w[2];
        Hidden<D> x[1];
        for (int j = 0; j < 2; j++) w[j].set([&](uint32_t r) { return base + (uint64_t)min(c0 + j * 16 + r, p.C - 1) * p.F; });
        x[0].of(p, [&](uint32_t) { return (const raw *)p.h + (uint64_t)(t * p.K + k) * p.h_ld; });
        f32x4 acc[1][2] = {};
        stream_run<D, 1, 2>(w, x, i % runs * RUN<D>, p.F, sums + wave * STREAM_LDS<1, 2>, acc);
        const float s = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int32_t, share), k));
        for (int m = 0; m < 2; m++) y[0][m] += s * acc[0][m];
    }
    join<1, 2, FEW_WAVES>(sums, wave, y);
    for (int m = 0; m < 2; m++) y[0][m] = whole<D>(y[0][m]);
    const bool is_void = __any(share != share);        /* by the router */
    if (wave != 0 || l != 0) return;
    for (uint32_t i = 0; i < 8; i++) {
        const uint32_t at = c + i / 4 * 16 + i % 4;
        const float v = is_void ? NAN : y[0][i / 4][i % 4];
        if (at < p.C) ((raw *)p.out)[t * p.out_ld + at] = D::put(v + res[i]);
    }
}

/* Which expert has run `run`, and which of its own that is: an expert has a run for every
 * `tokens` that chose it, or part of them.  -1 behind the last.  Each wavefront by itself. */
__device__ __forceinline__ int32_t expert_of(const LayerP &p, uint32_t run, uint32_t tokens, uint32_t &own)
{
    const uint32_t lane = threadIdx.x & 63, per = (p.E + 63) / 64, first = lane * per, last = min(p.E, first + per);
    uint32_t mine = 0;
    for (uint32_t e = first; e < last; e++) mine += (p.load[e] + tokens - 1) / tokens;
    uint32_t upto = mine;
    for (uint32_t d = 1; d < 64; d *= 2) {
        const uint32_t before = __shfl_up(upto, d);
        if (lane >= d) upto += before;
    }
    const uint64_t behind = __ballot(upto > run);
    if (!behind) return -1;
    const uint32_t at = __builtin_ctzll(behind);
    own = run - __builtin_amdgcn_readlane(upto - mine, at);
    for (uint32_t e = at * per; e < p.E; e++) {
        const uint32_t n = (p.load[e] + tokens - 1) / tokens;
        if (own < n) return e;
        own -= n;
    }
    return -1;
}

/* MT: tokens of a run, in 16; fewer take leaner code.  WAVES: k is shared among them.  Bound by reading the
 * weights: 32 x 7,168, 8 of 128 experts bf16 takes 7.7 GB in 790 + 396 us, 6.4 TB/s. */
template <typename D, int MT, int WAVES, bool DOWN> __global__ void __launch_bounds__(64 * WAVES, MT * (DOWN && PARTS<D> ? 2 : 1) <= 2 ? 3 : 2) msim_layer_product(LayerP p)
{
    constexpr int MORE = DOWN && PARTS<D> ? 2 : 1;       /* vectors a token */
    __shared__ uint32_t list[MAX_ROWS], counts[WAVES];
    __shared__ __attribute__((aligned(16))) char sums[WAVES * STREAM_LDS<MORE * MT, 2>];
    const uint32_t run = blockIdx.x / p.tiles, tile = blockIdx.x - run * p.tiles;
    uint32_t own = 0;
    const int32_t expert = p.rows > 16 * MT ? expert_of(p, run, 16 * MT, own) : p.slots < p.E ? p.ids[run] : p.load[run] ? (int32_t)run : -1;
    if (expert < 0) return;
    const uint32_t all = tokens_of<WAVES>(p, p.ids, expert, list, counts), first = own * 16 * MT;
    if (first >= all || (p.rows <= 16 * MT && p.slots < p.E && list[0] != run)) return;
    const uint32_t n = min(all - first, 16u * MT);
    const auto part = [&](auto mt) {
        if constexpr (DOWN) down_tokens<D, mt.value, WAVES>(p, expert, tile, list + first, n, sums);
        else up_tokens<D, mt.value, WAVES>(p, expert, tile, list + first, n, sums);
    };
    if (MORE == 2 && n <= 8) part(std::integral_constant<int, 1>());
    else if (n <= 16) part(std::integral_constant<int, MORE>());
    else if (MT > 2 && n <= 32) part(std::integral_constant<int, MORE * 2>());
    else part(std::integral_constant<int, MORE * MT>());
}

/* The weighted sum over a token's choices, in their order, and the residual.  A
 * row that the router voids (weights NaN) answers NaN.  3 us for 100 x 1,000, 9
 * for 512 x 2,048 and 6 choices, 2.9 TB/s of what a cache holds. */
template <typename D> __global__ void __launch_bounds__(256) msim_layer_sum(LayerP p)
{
    typedef typename D::raw raw;
    const uint32_t turns = (p.C + 3) / 4;
    const uint64_t id = blockIdx.x * 256ull + threadIdx.x;
    const uint32_t t = (uint32_t)(id / turns), c = (uint32_t)(id - (uint64_t)t * turns) * 4;
    if (t >= p.rows) return;
    f32x4 y = {0, 0, 0, 0};
    for (uint32_t k = 0; k < p.K; k++) {
        const uint32_t j = t * p.K + k;
        const float w = p.weights[j];
        if (p.ids[j] >= 0) y += w * *(const f32x4 *)(p.part + (uint64_t)j * p.part_ld + c);
        else if (w != w) y += w;
    }
    for (uint32_t i = 0; i < 4 && c + i < p.C; i++) {
        const float r = p.res ? D::get(((const raw *)p.res)[t * p.res_ld + c + i]) : 0.0f;
        ((raw *)p.out)[t * p.out_ld + c + i] = D::put(y[i] + r);
    }
}

/* ------------------------------------------------------------------------ */
/* host                                                                      */
/* ------------------------------------------------------------------------ */

uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

struct Layout { uint64_t logits, h, part, load, bytes, h_ld, part_ld; };

Layout layout_of(const msim_layer_spec *s)
{
    const uint64_t n = s->route.rows * s->route.top_k;
    Layout l;
    l.h_ld = up(s->hidden, 8);
    l.part_ld = up(s->cols, 4);
    l.logits = up(s->route.rows * s->route.experts * 4, 256);
    l.h = up(n * l.h_ld * (s->dtype == MSIM_BF16 ? 2 : 4), 256);         /* of f16 two parts */
    l.part = up(n * l.part_ld * 4, 256);
    l.load = up(s->route.experts * 4ull, 256);
    l.bytes = l.logits + l.h + l.part + l.load;
    return l;
}

const char *check_layer(const msim_layer_spec *s, int *code)
{
    *code = MSIM_E_ARG;
    if (!s) return "layer: null spec";
    if (s->version != MSIM_ABI_VERSION) return "layer: spec version mismatch";
    if (s->dtype > MSIM_BF16) return "layer: unknown dtype";
    if (s->act > MSIM_ACT_SILU) return "layer: unknown activation";
    if (s->gated > 1) return "layer: gated must be 0 or 1";
    if (!s->cols || !s->hidden) return "layer: cols and hidden must be at least 1";
    if (s->route.dtype != MSIM_F32 || s->route.row_stride != s->route.experts)
        return "layer: the router's logits are 32-bit and contiguous";
    if (s->route.rows > 1 && (s->x_stride < s->cols || s->out_stride < s->cols)) return "layer: x_stride or out_stride below cols";
    if (const char *why = msim_check_route(&s->route, false, code)) return why;
    *code = MSIM_E_LIMIT;
    if (s->route.rows > MAX_ROWS) return "layer: more than MSIM_MAX_LAYER_ROWS rows";
    if (s->cols > MSIM_MAX_LINEAR || s->hidden > MSIM_MAX_LINEAR) return "layer: cols or hidden above MSIM_MAX_LINEAR";
    if ((uint64_t)s->route.experts * std::max(s->cols, s->hidden) >> 24) return "layer: experts * cols or experts * hidden of 2^24 or more";
    if (s->x_stride >> 40 || s->out_stride >> 40 || s->residual_stride >> 40) return "layer: a stride of 2^40 or more";
    return nullptr;
}

template <typename D, bool DOWN> hipError_t launch_product(LayerP p, uint64_t tiles, hipStream_t st)
{
    /* runs of up to 64 tokens read an expert's weights once more seldom, those of 32 leave room for half as many wavefronts
     * again: 200 x 2,048, 6 of 64 experts bf16 (19 tokens each) 289 us in runs of 64, 271 of 32, with 512 rows (48) 424 and
     * 442; 400 x 7,168, 8 of 128 (25) 2,490 and 2,580 */
    constexpr bool MORE = DOWN && PARTS<D>;
    uint32_t mt = p.rows <= 16 ? 1 : p.rows <= 32 || p.rows * p.K <= 24 * p.E ? 2 : 4;
    /* two vectors a token: as many tokens a run as without, half of them (100 x 1,000, 3 of 24 experts f16 38.6 us in runs
     * of 16, 40.7 of 32; 200 x 7,168, 8 of 128 (13) 2,155 and 2,220, 250 (16) 2,455 and 2,442; 8 blocks of vectors spill) */
    if (MORE && mt > 1) mt = p.rows * p.K <= 16 * p.E ? 1 : 2;
    p.tiles = (uint32_t)tiles;
    /* a run for each expert that may be chosen, and one more for every 16 mt assignments */
    const uint32_t grid = (p.slots + (p.rows <= 16 * mt ? 0 : p.rows * p.K / (16 * mt))) * p.tiles;
    /* few workgroups and long rows: more wavefronts in each (32 x 2,048, 768 hidden units, 2 of 16 experts bf16 52.8 ->
     * 47.2 us; rows of up to 8 runs 24 x 1,000, 520, 3 of 24 f16 34.7, with more 39.5) */
    if (grid < 1024 && ((DOWN ? p.F : p.C) + RUN<D> - 1) / RUN<D> > 8) {
        if (mt == 1) return launch(msim_layer_product<D, 1, 16, DOWN>, grid, 1024, 0, st, p);
        if (mt == 2) return launch(msim_layer_product<D, 2, 8, DOWN>, grid, 512, 0, st, p);
        if constexpr (!MORE) return launch(msim_layer_product<D, 4, 8, DOWN>, grid, 512, 0, st, p);
    }
    if (mt == 1) return launch(msim_layer_product<D, 1, 4, DOWN>, grid, 256, 0, st, p);
    if (mt == 2) return launch(msim_layer_product<D, 2, 4, DOWN>, grid, 256, 0, st, p);
    if constexpr (!MORE) return launch(msim_layer_product<D, 4, 4, DOWN>, grid, 256, 0, st, p);
    return hipErrorInvalidValue;
}

template <typename D> int run_layer(const msim_layer_spec *s, LayerP p, const float *bias, int32_t *ids, float *weights, hipStream_t st)
{
    hipError_t e = p.rows == 1 ? launch(msim_layer_gate<D, 1>, p.E, 256, 0, st, p)
                               : launch(msim_layer_gate<D, 4>, p.E * ((p.rows + 3) / 4), 256, 0, st, p);
    if (e != hipSuccess) return launched(e, "layer launch");
    const uint64_t in = (p.F + (p.gated ? 15 : 31)) / (p.gated ? 16 : 32), out = (p.C + 31) / 32;
    p.slots = std::min(p.rows * p.K, p.E);
    const size_t keys = s->route.groups > 1 ? p.rows * p.E * sizeof(double) : 0;
    /* every workgroup routes: one round of them, two a compute unit */
    if (p.rows <= FEW_ROWS && p.slots * in <= 512 && keys <= 32768) {
        const msim_route_spec &r = s->route;
        RouteP q = {p.logits, bias, nullptr, nullptr, nullptr, r.rows, r.experts, r.experts, r.top_k, r.groups, r.top_groups,
                    r.group_top, r.renorm, r.score == MSIM_SCORE_SIGMOID, r.scale, 0, 0, 0, 0};
        if (q.TG == q.G) q.G = q.TG = q.gtop = 1;       /* every group stays */
        p.tiles = (uint32_t)in;
        e = launch(p.E <= 256 ? msim_layer_up_few<D, 4> : msim_layer_up_few<D, 16>, p.slots * p.tiles, 64 * FEW_WAVES, keys, st, p, q, ids, weights);
        if (e != hipSuccess) return launched(e, "layer launch");
    } else {
        if (int rc = msim_route(&s->route, p.logits, bias, ids, weights, p.load, st)) return rc;
        e = launch_product<D, false>(p, in, st);
        if (e != hipSuccess) return launched(e, "layer launch");
    }
    /* one token, or experts that are read again from a cache, and few runs of k, in less time than a launch takes */
    const uint64_t runs = (p.F + RUN<D> - 1) / RUN<D> * p.K;
    if (p.rows == 1 || (p.rows <= FEW_ROWS && (uint64_t)p.rows * p.K * p.C * p.F * sizeof(typename D::raw) <= 64u << 20 && runs <= 4 * FEW_WAVES)) {
        p.tiles = (uint32_t)out;
        return launched(launch(msim_layer_down_few<D>, p.rows * p.tiles, 64 * FEW_WAVES, 0, st, p), "layer launch");
    }
    e = launch_product<D, true>(p, out, st);
    if (e == hipSuccess) e = launch(msim_layer_sum<D>, (uint32_t)(((uint64_t)p.rows * ((p.C + 3) / 4) + 255) / 256), 256, 0, st, p);
    return launched(e, "layer launch");
}

} // namespace

extern "C" int msim_layer_workspace(const msim_layer_spec *s, uint64_t *bytes)
{
    int code;
    if (const char *why = check_layer(s, &code)) return fail(code, why);
    if (!bytes) return fail(MSIM_E_ARG, "layer: null bytes");
    *bytes = s->route.rows ? layout_of(s).bytes : 0;
    return MSIM_OK;
}

extern "C" int msim_layer(const msim_layer_spec *s, const void *x, const void *gate, const float *bias, const void *w_in,
                          const void *w_out, const uint8_t *mask, const void *residual, void *out, int32_t *ids,
                          float *weights, int32_t *load, void *workspace, uint64_t workspace_bytes, void *hip_stream)
{
    int code;
    if (const char *why = check_layer(s, &code)) return fail(code, why);
    if (s->route.rows == 0) return msim_route(&s->route, nullptr, bias, ids, weights, load, hip_stream);
    if (!x || !gate || !w_in || !w_out || !out || !ids || !weights) return fail(MSIM_E_ARG, "layer: null array");
    if (residual && s->route.rows > 1 && s->residual_stride < s->cols) return fail(MSIM_E_ARG, "layer: residual_stride below cols");
    if (residual == out && s->route.rows > 1 && s->residual_stride != s->out_stride)
        return fail(MSIM_E_ARG, "layer: residual is out, with two strides");
    const Layout l = layout_of(s);
    if (!workspace || workspace_bytes < l.bytes || (uintptr_t)workspace % 256)
        return fail(MSIM_E_WORKSPACE, "layer: workspace missing, too small or not on 256 bytes");
    char *ws = (char *)workspace;
    const LayerP p = {x, gate, w_in, w_out, residual, mask, out, (float *)ws, ids, weights, load ? load : (int32_t *)(ws + l.logits + l.h + l.part), ws + l.logits,
                      (float *)(ws + l.logits + l.h), s->x_stride, s->out_stride, s->residual_stride, l.h_ld, s->route.rows * s->route.top_k * l.h_ld, l.part_ld,
                      (uint32_t)s->route.rows, s->route.experts, s->route.top_k, s->cols, s->hidden, s->act, s->gated, 0, 0};
    hipStream_t st = (hipStream_t)hip_stream;
    return s->dtype == MSIM_F32 ? run_layer<F32>(s, p, bias, ids, weights, st)
        : s->dtype == MSIM_F16 ? run_layer<F16>(s, p, bias, ids, weights, st)
                               : run_layer<BF16>(s, p, bias, ids, weights, st);
}
