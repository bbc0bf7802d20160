/* Expert-parallel routing: router, its gradient, assignment dropout and the
 * all-to-all traffic that routed tokens cause (the msim_route, msim_dropout and
 * msim_traffic families of include/msim.h).
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

constexpr int WAVE = 64;

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
};

template <typename T> __device__ __forceinline__ T wave_max(T v)
{
    for (int m = 32; m; m >>= 1) v = max(v, __shfl_xor(v, m));
    return v;
}
template <typename T> __device__ __forceinline__ T wave_sum(T v)
{
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

__device__ __forceinline__ double score64(double x, bool sigmoid, double top, double inv)
{
    if (sigmoid) {
        const double e = exp(-fabs(x));
        return (x >= 0 ? 1.0 : e) / (1.0 + e);
    }
    return exp(x - top) * inv;
}

/* One row by one wavefront, keys in 64 bits.  Lane l holds experts l, l + 64,
 * ...: loads are consecutive, and each of top_k rounds finds the best key left
 * by exchanges of (key, index) between lanes. */
template <typename D, int VPL>
__device__ void route_row(const RouteP &p, uint64_t row, int32_t *hist)
{
    const int lane = threadIdx.x & 63;
    const typename D::raw *x = (const typename D::raw *)p.x + row * p.stride;
    float v[VPL];
    double key[VPL];
    bool bad = false;
    float top = -INFINITY;
    for (int i = 0; i < VPL; i++) {
        const uint32_t e = i * WAVE + lane;
        v[i] = e < p.E ? D::get(x[e]) : -INFINITY;
        bad |= v[i] != v[i] || (!p.sigmoid && v[i] == INFINITY);
        top = fmaxf(top, v[i]);
    }
    const bool is_void = __any(bad);
    top = wave_max(top);
    int32_t my_id = -1;
    if (!is_void && top > -INFINITY) {
        double inv = 1.0;
        if (!p.sigmoid) {
            double sum = 0;
            for (int i = 0; i < VPL; i++) sum += v[i] > -INFINITY ? exp((double)v[i] - top) : 0.0;
            inv = 1.0 / wave_sum(sum);
        }
        for (int i = 0; i < VPL; i++) {
            const uint32_t e = i * WAVE + lane;
            key[i] = v[i];
            if (p.bias && e < p.E && v[i] > -INFINITY) {
                const double b = p.bias[e];
                key[i] = b > -INFINITY ? score64(v[i], p.sigmoid, top, inv) + b : -INFINITY;
            }
        }
        if (p.G > 1) {
            /* lane g walks group g: its one or two best members */
            const uint32_t size = p.E / p.G;
            double total = -INFINITY;
            if (lane < (int)p.G) {
                double a = -INFINITY, c = -INFINITY;
                for (uint32_t k = 0; k < size; k++) {
                    const uint32_t e = lane * size + k;
                    const float t = D::get(x[e]);
                    double q = t;
                    if (t > -INFINITY && (p.bias || p.gtop > 1)) {
                        q = score64(t, p.sigmoid, top, inv);
                        if (p.bias) q = p.bias[e] > -INFINITY ? q + p.bias[e] : -INFINITY;
                    }
                    if (q > a) { c = a; a = q; }
                    else if (q > c) c = q;
                }
                total = p.gtop > 1 && c > -INFINITY ? a + c : a;
            }
            uint32_t before = 0;           /* groups better than this lane's */
            for (uint32_t g = 0; g < p.G; g++) {
                const double t = __shfl(total, (int)g);
                before += t > total || (t == total && g < (uint32_t)lane);
            }
            const uint64_t stay = __ballot(lane < (int)p.G && before < p.TG);
            for (int i = 0; i < VPL; i++) {
                const uint32_t e = i * WAVE + lane;
                if (e < p.E && !((stay >> (e / size)) & 1)) key[i] = -INFINITY;
            }
        }
        for (uint32_t r = 0; r < p.K; r++) {
            double best = -INFINITY;
            int at = -1;
            for (int i = 0; i < VPL; i++)
                if (key[i] > best) { best = key[i]; at = i * WAVE + lane; }
            for (int m = 32; m; m >>= 1) {
                const double ob = __shfl_xor(best, m);
                const int oa = __shfl_xor(at, m);
                if (oa >= 0 && (at < 0 || ob > best || (ob == best && oa < at))) { best = ob; at = oa; }
            }
            if (at < 0) break;
            for (int i = 0; i < VPL; i++)
                if (i * WAVE + lane == at) key[i] = -INFINITY;
            if (lane == (int)r) my_id = at;
        }
    }
    /* weights: lane j has slot j */
    const float xs = my_id >= 0 ? D::get(x[my_id]) : -INFINITY;
    float q;
    if (p.sigmoid) {
        /* s = e^min(x,0) / (1 + e^-|x|); renormalised, the first factor is
         * taken relative to the largest chosen one, so that no sum vanishes */
        const float lo = fminf(xs, 0.0f);
        const float c = p.renorm ? wave_max(lo) : 0.0f;
        q = my_id >= 0 ? expf(lo - c) / (1.0f + expf(-fabsf(xs))) : 0.0f;
    } else {
        const float c = p.renorm ? wave_max(xs) : top;
        q = my_id >= 0 ? expf(xs - c) : 0.0f;
        if (!p.renorm) {
            float sum = 0;
            for (int i = 0; i < VPL; i++) sum += v[i] > -INFINITY ? expf(v[i] - top) : 0.0f;
            q /= wave_sum(sum);
        }
    }
    if (p.renorm) {
        const float sum = wave_sum(q);
        q = my_id >= 0 ? q / sum : 0.0f;
    }
    if (my_id < 0) q = 0.0f;
    if (lane < (int)p.K) {
        p.ids[row * p.K + lane] = my_id;
        p.w[row * p.K + lane] = is_void ? NAN : p.scale * q;
        if (p.load && my_id >= 0) atomicAdd(&hist[my_id], 1);
    }
}

template <typename D, int VPL> __global__ void __launch_bounds__(256) msim_route_rows(RouteP p)
{
    __shared__ int32_t hist[MSIM_MAX_EXPERTS];
    if (p.load) {
        for (uint32_t e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
        __syncthreads();
    }
    const uint64_t step = (uint64_t)gridDim.x * (blockDim.x / WAVE);
    for (uint64_t row = (uint64_t)blockIdx.x * (blockDim.x / WAVE) + threadIdx.x / WAVE; row < p.rows; row += step)
        route_row<D, VPL>(p, row, hist);
    if (p.load) {
        __syncthreads();
        for (uint32_t e = threadIdx.x; e < p.E; e += blockDim.x) {
            if (gridDim.x == 1) p.load[e] = hist[e];
            else if (hist[e]) atomicAdd(&p.load[e], hist[e]);
        }
    }
}

__global__ void msim_fill_words(int32_t *out, uint32_t n)
{
    const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) out[i] = 0;
}

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

template <typename D> __global__ void __launch_bounds__(256) msim_route_back(BackP p)
{
    const int lane = threadIdx.x & 63;
    const uint64_t step = (uint64_t)gridDim.x * (blockDim.x / WAVE);
    for (uint64_t row = (uint64_t)blockIdx.x * (blockDim.x / WAVE) + threadIdx.x / WAVE; row < p.rows; row += step) {
        const typename D::raw *x = (const typename D::raw *)p.x + row * p.stride;
        typename D::raw *dx = (typename D::raw *)p.dx + row * p.dstride;
        /* lane j has slot j */
        int32_t id = lane < (int)p.K ? p.ids[row * p.K + lane] : -1;
        if ((uint32_t)id >= p.E) id = -1;
        float xs = id >= 0 ? D::get(x[id]) : -INFINITY;
        if (xs == -INFINITY) id = -1;      /* an expert out of the row has no score to change */
        const float g = id >= 0 ? p.g[row * p.K + lane] : 0.0f;
        const bool any = __any(id >= 0);
        const bool every = !p.sigmoid && !p.renorm;    /* all experts have a gradient */
        float top = -INFINITY, z = 1.0f, q, d;
        if (every) {
            for (uint32_t e = lane; e < p.E; e += WAVE) top = fmaxf(top, D::get(x[e]));
            top = wave_max(top);
            float sum = 0;
            for (uint32_t e = lane; e < p.E; e += WAVE) sum += expf(D::get(x[e]) - top);
            z = wave_sum(sum);
            q = id >= 0 ? expf(xs - top) / z : 0.0f;
        } else if (p.sigmoid) {
            const float lo = fminf(xs, 0.0f);
            const float c = p.renorm ? wave_max(id >= 0 ? lo : -INFINITY) : 0.0f;
            q = id >= 0 ? expf(lo - c) / (1.0f + expf(-fabsf(xs))) : 0.0f;
        } else {
            const float c = wave_max(xs);
            q = id >= 0 ? expf(xs - c) : 0.0f;
        }
        if (p.renorm) {
            const float sum = wave_sum(q);
            q = id >= 0 ? q / sum : 0.0f;
        }
        const float mean = wave_sum(g * q);
        d = q * (p.renorm || every ? g - mean : g);
        if (every) d = q * g;
        if (p.sigmoid) d *= xs > 0 ? expf(-xs) / (1.0f + expf(-xs)) : 1.0f / (1.0f + expf(xs));
        d = id >= 0 ? d * p.scale : 0.0f;
        /* an expert's gradient is the sum over the slots that name it, in slot order */
        for (uint32_t e0 = 0; e0 < p.E; e0 += WAVE) {
            const uint32_t e = e0 + lane;
            float v = every && any && e < p.E ? -p.scale * mean * (expf(D::get(x[e]) - top) / z) : 0.0f;
            for (uint32_t j = 0; j < p.K; j++) {
                const int oi = __shfl(id, (int)j);
                const float od = __shfl(d, (int)j);
                if (oi == (int)e) v += od;
            }
            if (e < p.E) dx[e] = D::put(v);
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

template <typename D> __global__ void __launch_bounds__(256) msim_dropout_any(DropP p)
{
    const uint64_t n = p.rows * p.cols, step = (uint64_t)gridDim.x * blockDim.x;
    for (uint64_t i = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
        const uint64_t r = i / p.cols, c = i - r * p.cols;
        const float v = D::get(((const typename D::raw *)p.x)[r * p.xs + c]);
        const bool keep = draw32(p.base, p.per_row ? r : i) >= p.limit;
        ((typename D::raw *)p.y)[r * p.ys + c] = D::put(keep ? v * p.scale : 0.0f);
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
};

/* One workgroup a segment: a count per host in LDS, each token by one thread. */
__global__ void __launch_bounds__(256) msim_traffic_segments(TrafficP p)
{
    extern __shared__ uint32_t count[];
    for (uint64_t s = blockIdx.x; s < p.n_seg; s += gridDim.x) {
        for (uint32_t h = threadIdx.x; h < p.H; h += blockDim.x) count[h] = 0;
        __syncthreads();
        const uint64_t lo = min((uint64_t)max(p.off[s], (int64_t)0), p.rows);
        const uint64_t hi = min((uint64_t)max(p.off[s + 1], (int64_t)0), p.rows);
        for (uint64_t t = lo + threadIdx.x; t < hi; t += blockDim.x) {
            int32_t seen[MSIM_MAX_TOP_K];
            for (uint32_t j = 0; j < p.K; j++) {
                const int32_t id = p.ids[t * p.K + j];
                int32_t h = (uint32_t)id < p.E ? p.place[id] : -1;
                if (p.limit && draw32(p.base, p.per_row ? t : t * p.K + j) < p.limit) h = -1;
                if ((uint32_t)h >= p.H) h = -1;
                bool again = false;
                for (uint32_t i = 0; i < j; i++) again |= seen[i] == h;
                seen[j] = h;
                if (h >= 0 && !again) atomicAdd(&count[h], 1u);
            }
        }
        __syncthreads();
        const int32_t home = p.home[s];
        for (uint32_t h = threadIdx.x; h < p.H; h += blockDim.x) {
            const uint64_t b = (uint64_t)count[h] * p.token_bytes;
            const uint64_t k = b / p.pkt_bytes + (b % p.pkt_bytes != 0);
            p.out[s * p.H + h] = (int32_t)h == home ? 0 : (int32_t)min(k, (uint64_t)0x7FFFFFFF);
        }
        __syncthreads();
    }
}

/* ------------------------------------------------------------------------ */
/* host                                                                      */
/* ------------------------------------------------------------------------ */

int fail(int code, const char *what) { msim_set_error(what); return code; }

int launched(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return MSIM_OK;
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
    if (s->rows >> 40 || s->row_stride >> 40) return "route: rows or row_stride of 2^40 or more";
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

template <typename D> void launch_route(const RouteP &p, hipStream_t st)
{
    const uint32_t grid = (uint32_t)std::min<uint64_t>((p.rows + 3) / 4, 2048);
    if (p.load && grid != 1) msim_fill_words<<<(p.E + 255) / 256, 256, 0, st>>>(p.load, p.E);
    if (!grid) return;
    if (p.E <= 64) msim_route_rows<D, 1><<<grid, 256, 0, st>>>(p);
    else if (p.E <= 128) msim_route_rows<D, 2><<<grid, 256, 0, st>>>(p);
    else if (p.E <= 256) msim_route_rows<D, 4><<<grid, 256, 0, st>>>(p);
    else if (p.E <= 512) msim_route_rows<D, 8><<<grid, 256, 0, st>>>(p);
    else msim_route_rows<D, 16><<<grid, 256, 0, st>>>(p);
}

} // namespace

extern "C" int msim_route(const msim_route_spec *s, const void *logits, const float *bias, int32_t *ids,
                          float *weights, int32_t *load, void *hip_stream)
{
    int code;
    if (const char *why = check_route(s, false, &code)) return fail(code, why);
    if (s->rows && (!logits || !ids || !weights)) return fail(MSIM_E_ARG, "route: null logits, ids or weights");
    RouteP p = {logits, bias, ids, weights, load, s->rows, s->row_stride, s->experts, s->top_k, s->groups,
                s->top_groups, s->group_top, s->renorm, s->score == MSIM_SCORE_SIGMOID, s->scale};
    if (p.TG == p.G) p.G = p.TG = 1;       /* every group stays */
    hipStream_t st = (hipStream_t)hip_stream;
    if (s->dtype == MSIM_F32) launch_route<F32>(p, st);
    else if (s->dtype == MSIM_F16) launch_route<F16>(p, st);
    else launch_route<BF16>(p, st);
    return launched("route launch");
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
    const uint32_t grid = (uint32_t)std::min<uint64_t>((p.rows + 3) / 4, 4096);
    if (s->dtype == MSIM_F32) msim_route_back<F32><<<grid, 256, 0, st>>>(p);
    else if (s->dtype == MSIM_F16) msim_route_back<F16><<<grid, 256, 0, st>>>(p);
    else msim_route_back<BF16><<<grid, 256, 0, st>>>(p);
    return launched("route backward launch");
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
    const uint32_t grid = (uint32_t)std::min<uint64_t>((rows * cols + 255) / 256, 1u << 16);
    if (dtype == MSIM_F32) msim_dropout_any<F32><<<grid, 256, 0, st>>>(d);
    else if (dtype == MSIM_F16) msim_dropout_any<F16><<<grid, 256, 0, st>>>(d);
    else msim_dropout_any<BF16><<<grid, 256, 0, st>>>(d);
    return launched("dropout launch");
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
                  s->experts, s->top_k, s->hosts, s->token_bytes, s->pkt_bytes, s->per_row};
    if (!drop_limit(s->drop, &p.limit)) return fail(MSIM_E_ARG, "traffic: drop must be in [0, 1]");
    if (s->experts > (1u << 24)) return fail(MSIM_E_LIMIT, "traffic: more than 2^24 experts");
    if (s->top_k > MSIM_MAX_TOP_K) return fail(MSIM_E_LIMIT, "traffic: top_k above MSIM_MAX_TOP_K");
    if (s->hosts > MSIM_MAX_TRAFFIC_HOSTS) return fail(MSIM_E_LIMIT, "traffic: more than MSIM_MAX_TRAFFIC_HOSTS hosts");
    if (s->rows >> 32) return fail(MSIM_E_LIMIT, "traffic: 2^32 rows or more");
    if (s->n_seg >> 32) return fail(MSIM_E_LIMIT, "traffic: 2^32 segments or more");
    if (s->n_seg == 0) return MSIM_OK;
    if (!token_off || !home || !place || !packets || (s->rows && !ids)) return fail(MSIM_E_ARG, "traffic: null array");
    const uint32_t grid = (uint32_t)std::min<uint64_t>(s->n_seg, 1u << 16);
    msim_traffic_segments<<<grid, 256, 4 * s->hosts, (hipStream_t)hip_stream>>>(p);
    return launched("traffic launch");
}
