/* How the matrix products of msim_gemm.h are cut, by an estimate of their time. */

#include <algorithm>
#include <cmath>

#include "msim_gemm.h"

namespace {

/* The cheapest by an estimate in us.  Workgroups of a kind are on the card `slots`
 * at a time; one takes `more`, and for a stage `low` where it has a compute unit to
 * itself, `high` where the card is full (measured with sizes of 1,024 and 8,192);
 * parts of k add the time of their sums through memory. */
constexpr struct { double slots, more, low[3], high[3]; } TIMES[] = {         /* 16 bits, 32 bits, split */
    {256, 9, {1.15, 8.0, 1.7}, {1.6, 8.0, 2.2}}, {512, 4, {0.53, 2.0, 0.6}, {1.0, 3.6, 1.3}}, {512, 2, {0.25, 0.63, 0.3}, {0.41, 1.2, 0.5}},
};

uint64_t tiles_of(const Product &q, uint32_t kind)
{
    const uint32_t bt = KINDS[kind].bt;
    return ((q.M + bt - 1) / bt) * ((q.N + bt - 1) / bt) * q.batch;
}

/* The best parts for a kernel, and the estimate.  `share` of the card is this
 * product's; it is crowded where another one fills the rest. */
double plan_kind(uint32_t mode, const Product &q, uint32_t kind, double share, bool crowded, Plan *best)
{
    const auto &c = TIMES[kind];
    const uint32_t bk = mode == M_F16 || mode == M_BF16 ? 64 : 32, t = bk == 64 ? 0 : mode == M_F32 ? 1 : 2;
    const uint64_t nk = (q.K + bk - 1) / bk, n = std::max<uint64_t>(nk, 1), tiles = tiles_of(q, kind);
    const double slots = c.slots * share;
    double least = INFINITY;
    for (uint64_t parts : {1, 2, 3, 4, 6, 8, 9, 12, 16, 24, 32, 48, 64}) {
        if (parts > n) break;
        const uint64_t per = (n + parts - 1) / parts;
        if ((n + per - 1) / per != parts) continue;
        const double groups = (double)(tiles * parts), rounds = std::floor(groups / slots), rest = groups - rounds * slots;
        double cost = rounds * (c.more + c.high[t] * per);
        if (rest > 0) cost += c.more + (rest <= slots / 2 && !crowded ? c.low[t] : c.high[t]) * per;
        if (parts > 1) cost += 4.0 + (double)q.batch * q.M * q.N * parts * 8.0 / 4e6;
        if (cost < least) {
            least = cost;
            *best = {kind, (uint32_t)parts, (uint32_t)per, (uint32_t)nk,
                     parts > 1 ? up(q.batch * parts * q.M * up(q.N, mode == M_SPLIT ? 32 : 8) * 4, 256) : 0};
        }
    }
    return least;
}

/* the kernels that a type has: 32-bit products are so slow that tiles of 128 feed them as well as larger ones */
bool has_kind(uint32_t mode, uint32_t kind) { return mode != M_F32 || KINDS[kind].bt < 256; }

} // namespace

namespace msim {

Plan plan_of(uint32_t mode, const Product &q)
{
    Plan best = {}, p;
    double least = INFINITY;
    for (uint32_t i = 0; i < N_KINDS; i++) {
        if (!has_kind(mode, i)) continue;
        const double cost = plan_kind(mode, q, i, 1.0, false, &p);
        if (cost < least) least = cost, best = p;
    }
    return best;
}

void plan_pair(uint32_t mode, const Product &a, const Product &b, Plan *pa, Plan *pb)
{
    Plan x, y;
    double least = INFINITY;
    for (uint32_t i = 0; i < N_KINDS; i++) {
        if (!has_kind(mode, i)) continue;
        double cost = std::max(plan_kind(mode, a, i, 0.5, false, &x), plan_kind(mode, b, i, 0.5, false, &y));
        if (tiles_of(a, i) * x.parts + tiles_of(b, i) * y.parts > 256)
            cost = std::max(plan_kind(mode, a, i, 0.5, true, &x), plan_kind(mode, b, i, 0.5, true, &y));
        if (cost < least) least = cost, *pa = x, *pb = y;
    }
}

} // namespace msim
