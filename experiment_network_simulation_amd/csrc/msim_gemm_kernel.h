/* The kernel of msim_gemm.h. */
#ifndef MSIM_GEMM_KERNEL_H
#define MSIM_GEMM_KERNEL_H

#include <algorithm>

#include "msim_gemm.h"

namespace {

typedef int16_t i16x4 __attribute__((ext_vector_type(4)));

/* numbers as sums of two */
template <int MODE> constexpr bool HALVES = MODE == M_SPLIT || MODE == M_TWO;

constexpr uint32_t OUTSIDE = 0x80000000u;  /* an offset past every buffer: the load gives zeros */

/* BT rows (m or n) by 128 bytes of k (64 columns of 16 bits, 32 of 32 bits or of
 * two halves) in LDS.
 *
 * Contiguous along k: LDS rows are the operand's, 128 bytes each, a cache line (64
 * bytes at a time took a third more time where memory counts).  A wavefront's
 * fragments are 16 bytes of each of 32 rows; the 16-byte pieces of a row are
 * exchanged by (row / 2) mod 8, so that 16 rows cover all banks.
 * Contiguous along m (MC): LDS rows are those of k, BT columns each.  16-bit
 * fragments are read with a transposition, 32 bytes of 4 rows by 16 lanes; pieces
 * of 64 bytes are exchanged by the row, so that those 4 rows lie in different
 * banks.  32-bit fragments are one element of two rows, 4 apart; pieces of 128
 * bytes are exchanged between those.
 *
 * Tiles go from memory to LDS without registers; the exchange is made in the
 * addresses that the lanes read.  Rows and columns outside the operand are read
 * as zeros, through an offset outside the buffer. */
template <int MODE, bool MC, int BT, int THREADS> struct Tile {
    static constexpr int ES = MODE == M_F16 || MODE == M_BF16 ? 2 : 4;   /* bytes of a column */
    static constexpr int BK = 128 / ES;                                   /* columns of k */
    static constexpr int W = MC ? BT * ES : 128, R = MC ? BK : BT;        /* bytes of an LDS row, rows */
    static constexpr int BYTES = R * W, LOADS = BYTES / 16 / THREADS;
    static_assert(R * W == BT * 128 && LOADS * 16 * THREADS == BYTES, "whole loads");

    const char *at;
    uint64_t extent, step;
    uint32_t off[LOADS];
    uint32_t k_end;              /* MC: rows of k; otherwise bytes of a row */

    /* the source of LDS byte b of row r, and the other way round */
    static __device__ __forceinline__ uint32_t exchange(uint32_t r, uint32_t b)
    {
        if constexpr (!MC) return b ^ (r >> 1 & 7) << 4;
        else if constexpr (MODE == M_F32) return b ^ (r >> 2 & 1) << 7;
        else return W >= 256 ? b ^ (r & 3) << 6 : b ^ (r >> 1 & 1) << 6;
    }

    __device__ __forceinline__ void init(const Operand &o, uint32_t batch, uint32_t row0, uint32_t rows, uint32_t K)
    {
        const uint64_t first = MC ? (uint64_t)row0 * ES : row0 * o.ld;
        at = o.at + batch * o.batch + first;
        extent = o.extent > first ? o.extent - first : 0;
        step = MC ? BK * o.ld : 128;
        k_end = MC ? K : K * ES;
        _Pragma("unroll") for (int i = 0; i < LOADS; i++) {
            const uint32_t c = i * THREADS + threadIdx.x, r = c / (W / 16), b = exchange(r, c % (W / 16) * 16);
            /* of halves 32 columns lie together, high parts and low ones */
            const uint32_t col = HALVES<MODE> ? b / 128 * 32 : b / ES;
            const bool in = MC ? row0 + col < rows : row0 + r < rows;
            off[i] = in ? (uint32_t)(r * o.ld) + b : OUTSIDE;
        }
    }

    /* tile kt of k, zeros if it is not `there`; every lane of the workgroup takes part */
    __device__ __forceinline__ void load(uint32_t kt, bool there, char *lds) const
    {
        const uint64_t done = kt * step, left = there && extent > done ? extent - done : 0;
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
            (void *)(at + done), 0, (int)(left < 0x7FFFFFFF ? left : 0x7FFFFFFF), 0x00020000);
        const uint32_t k0 = kt * (MC ? BK : 128);
        const bool whole = !there || k0 + (MC ? BK : 128) <= k_end;
        _Pragma("unroll") for (int i = 0; i < LOADS; i++) {
            uint32_t o = off[i];
            if (!whole) {
                const uint32_t c = i * THREADS + threadIdx.x, r = c / (W / 16);
                const uint32_t k = k0 + (MC ? r : exchange(r, c % (W / 16) * 16));
                o = k < k_end ? o : OUTSIDE;
            }
            const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)(lds + (i * THREADS + wave * WAVE) * 16),
                                                     16, o, 0, 0, 0);
        }
    }
};

/* Fragments of 32 rows by 16 bytes of k (in each half of the wavefront) out of a Tile. */
template <int MODE, bool MC, int BT> struct Reader {
    typedef Tile<MODE, MC, BT, 64> T;
    uint32_t base, x;

    __device__ __forceinline__ void init(uint32_t row0)
    {
        const uint32_t lane = threadIdx.x & 63, l = lane & 31, half = lane >> 5;
        if constexpr (!MC) {
            base = (row0 + l) * 128;
            x = T::exchange(l, half << 4);
        } else if constexpr (MODE == M_F32) {
            base = half * 4 * T::W + l * 4;
            x = T::exchange(half * 4, row0 * 4);
        } else {
            const uint32_t r = half * 8 + (lane >> 2 & 3);
            base = r * T::W + (lane & 3) * 8;
            x = T::exchange(r, row0 * T::ES + (l >> 4) * 32);
        }
    }

    /* Block i of 32 rows, step s of k (32 bytes; of halves 32 of high parts
     * and 32 of low ones).  The rows of k that a lane reads have the same exchange;
     * row0 is a multiple of the wavefront's rows, so blocks are other bits of x. */
    __device__ __forceinline__ u32x4 get(const char *lds, int i, int s, int low) const
    {
        if constexpr (!MC) {
            return *(const u32x4 *)(lds + base + i * (32 * 128) + (x ^ (s * 32 + low * 64)));
        } else if constexpr (MODE == M_F32) {
            u32x4 v;
            for (int e = 0; e < 4; e++) v[e] = *(const uint32_t *)(lds + base + (s * 8 + e) * T::W + (x ^ (i * 128)));
            return v;
        } else {
            const uint32_t b = base + s * 16 * T::W + (x ^ (HALVES<MODE> ? i * 128 + low * 64 : i * 64));
            typedef __attribute__((address_space(3))) i16x4 *ptr;
            const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds + b));
            const i16x4 c = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds + b + 4 * T::W));
            return __builtin_bit_cast(u32x4, __builtin_shufflevector(a, c, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int MODE> __device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c)
{
    if constexpr (MODE == M_F32) {
        const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
        for (int e = 0; e < 4; e++) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[e], y[e], c, 0, 0, 0);
        return c;
    } else if constexpr (MODE == M_BF16 || MODE == M_TWO)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

/* ------------------------------------------------------------------------ */
/* what becomes of a sum                                                     */
/* ------------------------------------------------------------------------ */

/* What the epilogue reads of memory for eight columns, as it lies: the residual, or the split matrix. */
template <int MODE> struct Early { struct T { u32x4 a, b; }; };

template <int MODE> __device__ __forceinline__ void early_of(const Epilogue &e, uint32_t batch, uint32_t m, uint32_t n, typename Early<MODE>::T &x)
{
    if constexpr (MODE == M_SPLIT) {
        if (!e.src || m >= e.M || n >= e.out_ld) return;
        const uint16_t *q = (const uint16_t *)((const char *)e.src + batch * e.out_batch) + split_at(e.out_ld, m, n);
        x.a = *(const u32x4 *)q;
        x.b = *(const u32x4 *)(q + 32);
    } else {
        if (!e.res || m >= e.M || n + 8 > e.N) return;
        if (MODE == M_F32 || e.out32) {
            const float *q = (const float *)e.res + m * e.res_ld + n;
            x.a = piece<F32>(q);
            x.b = piece<F32>(q + 4);
        } else {
            x.a = piece<F16>((const uint16_t *)e.res + m * e.res_ld + n);
        }
    }
}

/* The sums v of row m, columns n .. n + 7 (n a multiple of 8), the bias added: the activation, */
template <int MODE> __device__ __forceinline__ void before(const Epilogue &e, uint32_t m, uint32_t n, float *v)
{
    typedef typename Type<MODE>::D D;
    if (m >= e.M || n >= e.N) return;
    const uint32_t k = min(8u, e.N - n);
    if (e.pre) store8<D>(v, e.pre, m * e.pre_ld + n, k);
    if (MODE == M_F32 || e.out32) act_of<8, true>(v, e.act);
    else act_of<8, false>(v, e.act);
}

/* and residual and result, or the next split matrix */
template <int MODE>
__device__ __forceinline__ void after(const Epilogue &e, uint32_t batch, uint32_t m, uint32_t n, float *v, const typename Early<MODE>::T &x)
{
    if (m >= e.M) return;
    if constexpr (MODE == M_SPLIT) {
        if (n >= e.out_ld) return;         /* columns behind N: sums of zeros, which keep them zero */
        if (e.src) {
            const u16x8 h = __builtin_bit_cast(u16x8, x.a), l = __builtin_bit_cast(u16x8, x.b);
            for (int i = 0; i < 8; i++) v[i] = e.alpha * (F16::get(h[i]) + F16::get(l[i])) + e.beta * v[i];
        } else {
            for (int i = 0; i < 8; i++) v[i] *= e.beta;
        }
        for (int i = 0; i < 8; i++) v[i] += m == n + i ? e.diag : 0.0f;
        store_split(v, (char *)e.out + batch * e.out_batch, split_at(e.out_ld, m, n));
    } else {
        typedef typename Type<MODE>::D D;
        if (n >= e.N) return;
        const uint32_t k = min(8u, e.N - n);
        if (e.res) {
            float r[8];
            if (k == 8 && (MODE == M_F32 || e.out32)) {
                const f32x4 a = __builtin_bit_cast(f32x4, x.a), b = __builtin_bit_cast(f32x4, x.b);
                for (int i = 0; i < 8; i++) r[i] = i < 4 ? a[i] : b[i - 4];
            } else if (k == 8) {
                const u16x8 a = __builtin_bit_cast(u16x8, x.a);
                for (int i = 0; i < 8; i++) r[i] = Type<MODE == M_F32 ? M_F16 : MODE>::D::get(a[i]);
            } else if (e.out32) {
                load8<F32>(r, e.res, m * e.res_ld + n, k);
            } else {
                load8<D>(r, e.res, m * e.res_ld + n, k);
            }
            for (int i = 0; i < 8; i++) v[i] += r[i];
        }
        if (e.out32) store8<F32>(v, e.out, m * e.out_ld + n, k);
        else store8<D>(v, e.out, m * e.out_ld + n, k);
    }
}

/* ------------------------------------------------------------------------ */
/* the product                                                               */
/* ------------------------------------------------------------------------ */

/* BT x BT of C a workgroup, which is number `block` of `total`; DEPTH stages in LDS,
 * in arrays of their own, so that the compiler knows which of them a load to LDS
 * writes.
 *
 * Large products are bound by the matrix instructions' turns with LDS reads and the
 * barrier of a stage: 8,192 x 4,096 -> 8,192 bf16 470 us, 1,170 TFLOP/s, the matrix pipes
 * busy for 58 % of it (three f16 products of split matrices alike: 1,130 to 1,200);
 * 131,072 x 7,168 -> 256 by memory, 490 us, 3.9 TB/s, for two stages are all that 160 KB
 * hold.  Small ones are as long as a launch and the chain of loads, 5 us. */
template <int MODE, bool AMC, bool BMC, int BT, int DEPTH, int THREADS>
__device__ __forceinline__ void product(const GemmP &p, uint32_t total, uint32_t block, char *lds0, char *lds1, char *lds2, char *lds3)
{
    constexpr int WAVES = THREADS / WAVE, WM = 2, WN = WAVES / WM;      /* wavefronts along m and n */
    constexpr int RM = BT / WM, RN = BT / WN, IM = RM / 32, IN = RN / 32;
    constexpr int STEPS = HALVES<MODE> ? 2 : 4;
    typedef Tile<MODE, AMC, BT, THREADS> TA;
    typedef Tile<MODE, BMC, BT, THREADS> TB;
    constexpr int STAGE = TA::BYTES + TB::BYTES;

    /* Workgroups go to the 8 dies in turn: each die takes consecutive tiles, and
     * those walk along m within bands of 8 tiles of n, so that what a die reads
     * together stays in its cache. */
    const uint32_t q = total >> 3, r = total & 7, die = block & 7;
    uint32_t id = die * q + min(die, r) + (block >> 3);
    const uint32_t tiles = p.tm * p.tn;
    const uint32_t group = id / tiles;
    id -= group * tiles;
    const uint32_t batch = group / p.parts, part = group - batch * p.parts;
    const uint32_t band = id / (8 * p.tm), width = min(8u, p.tn - band * 8), in = id - band * 8 * p.tm;
    const uint32_t bm = in / width, bn = band * 8 + in - bm * width;
    if (p.mirror && bm < bn) return;
    const uint32_t m0 = bm * BT, n0 = bn * BT;

    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const uint32_t wm = wave % WM, wn = wave / WM;
    TA ta;
    TB tb;
    ta.init(p.a, batch, m0, p.M, p.K);
    tb.init(p.b, batch, n0, p.N, p.K);
    Reader<MODE, AMC, BT> ra;
    Reader<MODE, BMC, BT> rb;
    ra.init(wm * RM);
    rb.init(wn * RN);
    f32x16 acc[IM][IN];
    _Pragma("unroll") for (int i = 0; i < IM; i++)
        _Pragma("unroll") for (int j = 0; j < IN; j++) acc[i][j] = 0.0f;

    const uint32_t first = part * p.per, last = min(first + p.per, p.nk);
    const auto load = [&](uint32_t kt, char *to) {
        ta.load(kt, kt < last, to);
        tb.load(kt, kt < last, to + TA::BYTES);
    };
    /* Fragments of a step; those of the next one are read while the matrix
     * instructions of this one run, across stages too. */
    struct Step { u32x4 a[IM], b[IN], al[HALVES<MODE> ? IM : 1], bl[HALVES<MODE> ? IN : 1]; };
    const auto read = [&](const char *from, int k, Step &f) {
        _Pragma("unroll") for (int j = 0; j < IN; j++) f.b[j] = rb.get(from + TA::BYTES, j, k, 0);
        _Pragma("unroll") for (int i = 0; i < IM; i++) f.a[i] = ra.get(from, i, k, 0);
        if constexpr (HALVES<MODE>) {
            _Pragma("unroll") for (int j = 0; j < IN; j++) f.bl[j] = rb.get(from + TA::BYTES, j, k, 1);
            _Pragma("unroll") for (int i = 0; i < IM; i++) f.al[i] = ra.get(from, i, k, 1);
        }
    };
    const auto multiply = [&](const Step &f) {
        _Pragma("unroll") for (int i = 0; i < IM; i++)
            _Pragma("unroll") for (int j = 0; j < IN; j++) acc[i][j] = mma<MODE>(f.b[j], f.a[i], acc[i][j]);
        if constexpr (HALVES<MODE>) {
            _Pragma("unroll") for (int i = 0; i < IM; i++)
                _Pragma("unroll") for (int j = 0; j < IN; j++) acc[i][j] = mma<MODE>(f.bl[j], f.a[i], acc[i][j]);
            _Pragma("unroll") for (int i = 0; i < IM; i++)
                _Pragma("unroll") for (int j = 0; j < IN; j++) acc[i][j] = mma<MODE>(f.b[j], f.al[i], acc[i][j]);
        }
    };
    constexpr int LOADS = TA::LOADS + TB::LOADS;
    /* All wavefronts have read `cur` whole and its next stage is there: of this
     * wavefront's loads only those of the other DEPTH - 2 stages are outstanding
     * (loads behind the last stage are made too, of nothing, so that their number is
     * always the same), and all wavefronts say so at the barrier. */
    constexpr int MORE = (DEPTH - 2) * LOADS;
    static_assert(MORE + LOADS < 64, "the counter of outstanding loads");
    Step f[2];
    const auto turn = [&](uint32_t kt, char *cur, const char *next) {
        _Pragma("unroll") for (int s = 0; s < STEPS; s++) {
            if (s + 1 < STEPS) {
                read(cur, s + 1, f[(s + 1) & 1]);
            } else {
                __builtin_amdgcn_s_waitcnt((MORE & 15) | (MORE >> 4) << 14 | 0x70);      /* and what it read of LDS */
                __builtin_amdgcn_s_barrier();
                load(kt + DEPTH, cur);
                read(next, 0, f[(s + 1) & 1]);
            }
            multiply(f[s & 1]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (first < last) {
        char *const lds[4] = {lds0, lds1, lds2, lds3};
        _Pragma("unroll") for (int d = 0; d < DEPTH; d++) load(first + d, lds[d]);
        __builtin_amdgcn_s_waitcnt(((MORE + LOADS) & 15) | ((MORE + LOADS) >> 4) << 14 | 0xF70);
        __builtin_amdgcn_s_barrier();
        read(lds0, 0, f[0]);
        for (uint32_t kt = first; kt < last; kt += DEPTH)          /* stages behind the last are zeros */
            _Pragma("unroll") for (int d = 0; d < DEPTH; d++) turn(kt + d, lds[d], lds[(d + 1) % DEPTH]);
        __builtin_amdgcn_s_waitcnt(0x0F70);          /* nothing is on its way to LDS any more */
    }

    /* Through LDS to rows: a lane has, of row l of a block of 32, four columns next
     * to each other; it gets pieces of one row, next to those of the lanes beside
     * it, so that lines are written whole. */
    __syncthreads();
    const uint32_t l = lane & 31, ni = n0 + wn * RN;
    const auto room = [&](uint32_t i) -> char * { return i == 0 ? lds0 : i == 1 ? lds1 : i == 2 ? lds2 : lds3; };
    if constexpr (MODE != M_F32 && MODE != M_SPLIT)
        if (p.plain == 2) {
            /* nothing but a rounding: all rows of the wavefront at once, 16 bits each */
            typedef typename Type<MODE>::D D;
            typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
            typedef u32x4 loose16 __attribute__((aligned(2)));
            constexpr int C = RN / 8, BLOCK = RM * RN * 2, FIT = STAGE / BLOCK;
            static_assert(WAVES <= DEPTH * FIT, "room for the rows of every wavefront");
            char *const stage = room(wave / FIT) + wave % FIT * BLOCK;
            _Pragma("unroll") for (int i = 0; i < IM; i++)
                _Pragma("unroll") for (int j = 0; j < IN; j++)
                    _Pragma("unroll") for (int g = 0; g < 4; g++) {
                        const auto &t = acc[i][j];
                        const u16x4 v = {D::put(t[g * 4]), D::put(t[g * 4 + 1]), D::put(t[g * 4 + 2]), D::put(t[g * 4 + 3])};
                        *(u16x4 *)(stage + (i * 32 + l) * RN * 2 + ((j * 4 + g) ^ (l & (C - 1))) * 16 + (lane >> 5) * 8) = v;
                    }
            wave_sync();
            const uint32_t c = lane % C;
            uint16_t *to = (uint16_t *)p.e.out + (m0 + wm * RM + lane / C) * p.e.out_ld + ni + c * 8;
            const uint32_t rows = ni + c * 8 < p.N ? p.M - min(p.M, m0 + wm * RM + lane / C) : 0;
            _Pragma("unroll 8") for (uint32_t r = 0; r < RM; r += 64 / C) {
                const u32x4 v = *(const u32x4 *)(stage + (r + lane / C) * RN * 2 + (c ^ ((r + lane / C) & (C - 1))) * 16);
                if (r < rows) *(loose16 *)(to + r * p.e.out_ld) = v;
            }
            return;
        }
    constexpr int HR = RM < 64 ? RM : 64, C = RN / 4, BLOCK = HR * RN * 4;      /* rows at a time; 16-byte pieces of a row */
    constexpr int FIT = STAGE / BLOCK, TURNS = HR * RN / 512;
    static_assert(WAVES <= DEPTH * FIT, "room for a block of every wavefront");
    float *const stage = (float *)(room(wave / FIT) + wave % FIT * BLOCK);
    /* the lane's eight columns, and its row among those of a turn */
    const uint32_t c8 = lane % (RN / 8), n8 = ni + c8 * 8, r8 = lane / (RN / 8);
    const auto at = [&](uint32_t row, uint32_t half) { return (f32x4 *)(stage + row * RN + ((c8 * 2 + half) ^ (row & 15 & (C - 1))) * 4); };
    float bias[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (p.e.bias && p.parts == 1 && n8 < p.N) load8<F32>(bias, p.e.bias, n8, min(8u, p.N - n8));
    _Pragma("unroll") for (int h = 0; h < RM / HR; h++) {
        const uint32_t mi = m0 + wm * RM + h * HR;
        /* what is read of memory is asked for first */
        typename Early<MODE>::T early[TURNS];
        if (!p.plain)
            _Pragma("unroll") for (int t = 0; t < TURNS; t++) early_of<MODE>(p.e, batch, mi + t * (512 / RN) + r8, n8, early[t]);
        _Pragma("unroll") for (int i = 0; i < HR / 32; i++)
            _Pragma("unroll") for (int j = 0; j < IN; j++)
                _Pragma("unroll") for (int g = 0; g < 4; g++) {             /* columns 8 g + 4 (lane / 32) of a block */
                    const auto &t = acc[h * (HR / 32) + i][j];
                    const f32x4 v = {t[g * 4], t[g * 4 + 1], t[g * 4 + 2], t[g * 4 + 3]};
                    *(f32x4 *)(stage + (i * 32 + l) * RN + ((j * 8 + g * 2 + (lane >> 5)) ^ (l & 15 & (C - 1))) * 4) = v;
                }
        wave_sync();
        if (p.plain) {
            /* 32 bits as they are: parts of a sum, or results */
            typedef f32x4 loose32 __attribute__((aligned(4)));
            const uint32_t c = lane % C, wide = p.parts > 1 ? (uint32_t)p.part_ld : p.N, r0 = lane / C;
            const uint64_t ld = p.parts > 1 ? p.part_ld : p.e.out_ld;
            float *to = (p.parts > 1 ? p.part + (uint64_t)group * p.M * ld : (float *)p.e.out) + (mi + r0) * ld + ni + c * 4;
            const uint32_t rows = ni + c * 4 < wide ? p.M - min(p.M, mi + r0) : 0;
            _Pragma("unroll 8") for (uint32_t r = 0; r < HR; r += 64 / C) {
                const f32x4 v = *(const f32x4 *)(stage + (r + r0) * RN + (c ^ ((r + r0) & 15 & (C - 1))) * 4);
                if (r < rows) *(loose32 *)(to + r * ld) = v;
            }
        } else {
            /* bias and activation, whose code is there once; then, in LDS until what is read of memory has
             * come, the residual */
            if constexpr (MODE != M_SPLIT) {
                _Pragma("unroll 1") for (uint32_t row = r8; row < HR; row += 512 / RN) {
                    const f32x4 x = *at(row, 0), y = *at(row, 1);
                    float v[8];
                    for (int i = 0; i < 8; i++) v[i] = (i < 4 ? x[i] : y[i - 4]) + bias[i];
                    before<MODE>(p.e, mi + row, n8, v);
                    if (p.e.res) {
                        *at(row, 0) = f32x4{v[0], v[1], v[2], v[3]};
                        *at(row, 1) = f32x4{v[4], v[5], v[6], v[7]};
                    } else {
                        after<MODE>(p.e, batch, mi + row, n8, v, early[0]);
                    }
                }
            }
            if (MODE == M_SPLIT || p.e.res)
                _Pragma("unroll") for (int t = 0; t < TURNS; t++) {
                    const uint32_t row = t * (512 / RN) + r8;
                    const f32x4 x = *at(row, 0), y = *at(row, 1);
                    float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
                    after<MODE>(p.e, batch, mi + row, n8, v, early[t]);
                }
        }
        if constexpr (MODE == M_SPLIT) {
            if (p.mirror && bm != bn) {
                _Pragma("unroll 1") for (uint32_t id = lane; id < HR / 8 * RN; id += 64) {
                    const uint32_t col = id % RN, up8 = id / RN * 8;
                    float v[8];
                    for (uint32_t k = 0; k < 8; k++)
                        v[k] = stage[(up8 + k) * RN + ((col / 4) ^ ((up8 + k) & 15 & (C - 1))) * 4 + col % 4];
                    typename Early<MODE>::T e;
                    early_of<MODE>(p.e, batch, ni + col, mi + up8, e);
                    after<MODE>(p.e, batch, ni + col, mi + up8, v, e);
                }
            }
        }
        wave_sync();
    }
}

template <int BT, int DEPTH> struct Room {
    static constexpr int STAGE = 2 * BT * 128;
    static constexpr int SPARE = DEPTH > 2 ? STAGE : 16;
};
#define MSIM_ROOM(BT, DEPTH)                                                                        \
    typedef Room<BT, DEPTH> R_;                                                                     \
    __shared__ __attribute__((aligned(256))) char lds0[R_::STAGE], lds1[R_::STAGE], lds2[R_::SPARE], lds3[R_::SPARE]

template <int MODE, bool BMC, int BT, int DEPTH, int THREADS> __global__ void __launch_bounds__(THREADS, 2) msim_gemm(GemmP p, uint32_t total, uint32_t first)
{
    MSIM_ROOM(BT, DEPTH);
    product<MODE, false, BMC, BT, DEPTH, THREADS>(p, total, first + blockIdx.x, lds0, lds1, lds2, lds3);
}

/* The two products of a backward pass in one launch: n of the first, and from the
 * next multiple of 8 on, so that dies are numbered alike, those of the second. */
template <int MODE, int BT, int DEPTH, int THREADS>
__global__ void __launch_bounds__(THREADS, 2) msim_gemm_pair(GemmP x, GemmP w, uint32_t n, uint32_t nw, uint32_t first)
{
    MSIM_ROOM(BT, DEPTH);
    const uint32_t n8 = (n + 7) & ~7u, block = first + blockIdx.x;
    if (block < n) product<MODE, false, true, BT, DEPTH, THREADS>(x, n, block, lds0, lds1, lds2, lds3);
    else if (block >= n8) product<MODE, true, true, BT, DEPTH, THREADS>(w, nw, block - n8, lds0, lds1, lds2, lds3);
}

/* The parts' sums together, in order, and what becomes of them: of one product, or of two.  Eight columns a thread;
 * 3 to 9 us, the latency of a launch and of the parts, which come from a cache. */
template <int MODE> __device__ __forceinline__ void join_parts(const GemmP &p, uint64_t id)
{
    const uint32_t wide = (uint32_t)(p.part_ld / 8);
    const uint64_t size = (uint64_t)p.M * p.part_ld, row = id / wide;
    const uint32_t c = (uint32_t)(id - row * wide) * 8, batch = (uint32_t)(row / p.M), m = (uint32_t)(row - (uint64_t)batch * p.M);
    typename Early<MODE>::T early;
    early_of<MODE>(p.e, batch, m, c, early);
    const float *q = p.part + (uint64_t)batch * p.parts * size + (uint64_t)m * p.part_ld + c;
    f32x4 x = *(const f32x4 *)q, y = *(const f32x4 *)(q + 4);
    _Pragma("unroll 8") for (uint32_t k = 1; k < p.parts; k++) {
        q += size;
        x += *(const f32x4 *)q;
        y += *(const f32x4 *)(q + 4);
    }
    float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    if constexpr (MODE != M_SPLIT) {
        float bias[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (p.e.bias && c < p.N) load8<F32>(bias, p.e.bias, c, min(8u, p.N - c));
        for (int i = 0; i < 8; i++) v[i] += bias[i];
        before<MODE>(p.e, m, c, v);
    }
    after<MODE>(p.e, batch, m, c, v, early);
}

/* eight columns of a workgroup's, 32 runs of blocks, in 64 bits */
__device__ __forceinline__ void join_columns(const Columns &p, uint32_t block, double *part)
{
    const uint32_t c = block * 8 + (threadIdx.x & 7);
    double s = 0;
    if (c < p.outs)
        _Pragma("unroll 8") for (uint32_t b = threadIdx.x >> 3; b < p.blocks; b += 32) s += p.sums[(uint64_t)b * p.outs + c];
    part[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x >= 8 || c >= p.outs) return;
    for (int i = 1; i < 32; i++) s += part[i * 8 + threadIdx.x];
    p.out[c] = (float)s;
}

/* the first workgroups have the columns */
template <int MODE> __global__ void __launch_bounds__(256) msim_gemm_join(GemmP a, uint64_t na, GemmP b, uint64_t nb, Columns c)
{
    __shared__ double part[256];
    const uint32_t first = (c.outs + 7) / 8;
    if (blockIdx.x < first) return join_columns(c, blockIdx.x, part);
    for (uint64_t id = (blockIdx.x - first) * 256ull + threadIdx.x; id < na + nb; id += (gridDim.x - first) * 256ull) {
        if (id < na) join_parts<MODE>(a, id);
        else join_parts<MODE>(b, id - na);
    }
}

} // namespace

namespace msim {

/* what the plan and the epilogue make of a product; its workgroups */
template <int MODE> uint64_t ready(GemmP &p, const Plan &c)
{
    const uint32_t bt = KINDS[c.kind].bt;
    p.tm = (p.M + bt - 1) / bt;
    p.tn = (p.N + bt - 1) / bt;
    p.nk = c.nk;
    p.parts = c.parts;
    p.per = c.per;
    p.part_ld = up(p.N, MODE == M_SPLIT ? 32 : 8);
    if (p.parts > 1) p.mirror = 0;
    const Epilogue &e = p.e;
    const bool only = MODE != M_SPLIT && !e.bias && !e.res && !e.pre && !e.act && p.N % 8 == 0;
    p.plain = p.parts > 1 || (only && (MODE == M_F32 || e.out32)) ? 1 : only ? 2 : 0;
    return (uint64_t)p.tm * p.tn * p.parts * p.batch;
}

template <int MODE> hipError_t launch_join(const GemmP &a, const GemmP &b, const Columns &c, hipStream_t st)
{
    const uint64_t na = a.parts > 1 ? (uint64_t)a.batch * a.M * (a.part_ld / 8) : 0, nb = b.parts > 1 ? (uint64_t)b.batch * b.M * (b.part_ld / 8) : 0;
    if (na + nb + c.outs == 0) return hipSuccess;
    return launch(msim_gemm_join<MODE>, (c.outs + 7) / 8 + (uint32_t)std::min<uint64_t>((na + nb + 255) / 256, 1u << 16), 256, 0, st, a, na, b, nb, c);
}

template <int MODE, bool BMC, uint32_t I = 0> hipError_t launch_kind(uint32_t kind, uint64_t total, const GemmP &p, hipStream_t st)
{
    if constexpr (I < N_KINDS) {
        constexpr Kind k = KINDS[I];
        if (kind != I) return launch_kind<MODE, BMC, I + 1>(kind, total, p, st);
        if constexpr (!(MODE == M_F32 && k.bt == 256))
            return in_turns(total, k.threads, [&](uint32_t first, uint32_t grid) {
                return launch(msim_gemm<MODE, BMC, k.bt, k.depth, k.threads>, grid, k.threads, 0, st, p, (uint32_t)total, first);
            });
    }
    return hipErrorInvalidValue;
}

template <int MODE, bool BMC> hipError_t launch_gemm(GemmP p, const Plan &c, hipStream_t st)
{
    const uint64_t total = ready<MODE>(p, c);
    if (!total) return hipSuccess;
    const hipError_t r = launch_kind<MODE, BMC>(c.kind, total, p, st);
    return r == hipSuccess ? launch_join<MODE>(p, GemmP{}, Columns{}, st) : r;
}

template <int MODE, uint32_t I = 0> hipError_t launch_pair_kind(uint32_t kind, uint64_t nx, uint64_t nw, const GemmP &x, const GemmP &w, hipStream_t st)
{
    if constexpr (I < N_KINDS) {
        constexpr Kind k = KINDS[I];
        if (kind != I) return launch_pair_kind<MODE, I + 1>(kind, nx, nw, x, w, st);
        if constexpr (!(MODE == M_F32 && k.bt == 256))
            return in_turns(up(nx, 8) + nw, k.threads, [&](uint32_t first, uint32_t grid) {
                return launch(msim_gemm_pair<MODE, k.bt, k.depth, k.threads>, grid, k.threads, 0, st, x, w, (uint32_t)nx, (uint32_t)nw, first);
            });
    }
    return hipErrorInvalidValue;
}

template <int MODE> hipError_t launch_pair(GemmP x, const Plan &cx, GemmP w, const Plan &cw, const Columns &c, hipStream_t st)
{
    const uint64_t nx = x.batch ? ready<MODE>(x, cx) : 0, nw = w.batch ? ready<MODE>(w, cw) : 0;
    const hipError_t r = nx + nw == 0 ? hipSuccess : launch_pair_kind<MODE>(x.batch ? cx.kind : cw.kind, nx, nw, x, w, st);
    return r == hipSuccess ? launch_join<MODE>(x, w, c, st) : r;
}

} // namespace msim

#endif
