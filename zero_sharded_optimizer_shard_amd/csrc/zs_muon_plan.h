// Which kernels a Newton-Schulz call launches: the stacks of a call, the tiles
// of their products by estimated time, and the steps that are taken two
// together.  Host arithmetic on sizes alone (the constants were measured on
// MI355X); the kernels are in zs_muon.hip.
#pragma once

#include <cmath>
#include <cstdint>

#include "zs_muon.h"

namespace zs {
namespace muon {

constexpr int kMaxMats = ZS_MAX_GROUP;
constexpr int kPad = 64;                // sides are stored rounded up to this

constexpr int32_t padded(int32_t n)
{
    return (n + kPad - 1) / kPad * kPad;
}

// One stack of matrices in the workspace.
struct Mat {
    char* ws;
    int32_t R, C;           // rows, cols
    int32_t batch;
    int32_t nparts;         // partial sums of squares per matrix
    uint32_t tiles;         // workgroups of the present launch
};

struct Group {
    int32_t count;
    uint32_t start[kMaxMats];           // first workgroup of each stack; past
                                        // the last one 2^32 - 1
    Mat m[kMaxMats];
};

// What a product's epilogue makes of D, and which operands it has:
//   kGram     A = X X^T
//   kPoly     C = a + b A + c A A
//   kProd     the product of two of the squares, which commute
//   kUpdate   X <- C X; the last one goes to the caller instead: kOutBf16,
//             kOutF32, or kStep, which steps the weights by it
enum Epi { kGram, kPoly, kProd, kUpdate, kOutBf16, kOutF32, kStep };

constexpr bool symmetric(int epi) { return epi <= kProd; }

// Tiles of one matrix's D.
template <int BT>
constexpr uint32_t tri_tiles(int32_t mp)
{
    const uint32_t t = (mp + BT - 1) / BT;
    return t * (t + 1) / 2;
}

// Which of the small kernels takes a matrix: 1 .. kSmalls, 0 for none.  Full
// precision's pairs leave LDS for the first two.
constexpr int kSmalls = 4;
inline int small_kind(int32_t R, int32_t C, bool full)
{
    const int32_t rp = padded(R), cp = padded(C);
    const int32_t m = rp < cp ? rp : cp, n = rp < cp ? cp : rp;
    if (m == 64 && n <= 64) return 1;
    if (m == 64 && n <= 256) return 2;
    if (full) return 0;
    if (m == 64 && n <= 512) return 3;
    return m == 128 && n == 128 ? 4 : 0;
}

// The order in which the members enter the group: by the larger side, then
// the smaller, so that the tiles with the longest sums start first.
template <class Sides>
void sort_members(int32_t* order, int32_t count, Sides sides)
{
    for (int32_t i = 0; i < count; ++i) {
        int64_t r, c;
        sides(i, r, c);
        int32_t k = i;
        for (; k > 0; --k) {
            int64_t qr, qc;
            sides(order[k - 1], qr, qc);
            const int64_t hi = r > c ? r : c, lo = r > c ? c : r;
            const int64_t qh = qr > qc ? qr : qc, ql = qr > qc ? qc : qr;
            if (qh > hi || (qh == hi && ql >= lo)) break;
            order[k] = order[k - 1];
        }
        order[k] = i;
    }
}

// Workgroup prefix sums: fn(mat) workgroups per matrix of the stack, each
// stack's from a multiple of `align` on.
template <class Fn>
uint32_t set_starts(Group& g, Fn fn, uint32_t align = 1)
{
    uint32_t n = 0;
    for (int i = 0; i < g.count; ++i) {
        g.start[i] = n;
        g.m[i].tiles = (uint32_t)g.m[i].batch * (uint32_t)fn(g.m[i]);
        n += (g.m[i].tiles + align - 1) / align * align;
    }
    for (int i = g.count; i < kMaxMats; ++i)
        g.start[i] = UINT32_MAX;
    return n;
}

// Tiles of one matrix's D in a product.
template <int BT, int EPI>
uint32_t d_tiles(const Mat& m)
{
    const int32_t rp = padded(m.R), cp = padded(m.C);
    if (symmetric(EPI))
        return tri_tiles<BT>(rp < cp ? rp : cp);
    return ((rp + BT - 1) / BT) * ((cp + BT - 1) / BT);
}

// Time of a launch in tiles of one size, in us: `stage` per 64 k and `fixed`
// per tile with `resident` tiles on each of the 256 CUs, or `alone` per 64 k
// while there is at most one.  The stacks' tiles go to the free places in
// order, longest first (the group is sorted so).
template <int BT, int EPI>
double estimate(const Group& g, double stage, double alone, double fixed,
                int resident)
{
    struct Places {
        double free;
        int64_t n;
    } at[64];
    int64_t n = 0;
    for (int p = 0; p < g.count; ++p)
        n += (int64_t)g.m[p].batch * d_tiles<BT, EPI>(g.m[p]);
    const double per = n <= 256 ? alone : stage;
    int used = 1;
    at[0] = {0, 256 * (int64_t)resident};
    double end = 0;
    for (int p = 0; p < g.count; ++p) {
        const Mat& m = g.m[p];
        const int32_t rp = padded(m.R), cp = padded(m.C);
        const int nk = ((EPI == kGram) == (rp < cp) ? cp : rp) / 64;
        const double t = nk * per + fixed;
        int64_t left = (int64_t)m.batch * d_tiles<BT, EPI>(m);
        // whole rounds of everything, then the rest
        const int64_t rounds = left / (256 * resident);
        for (int k = 0; k < used; ++k)
            at[k].free += (double)rounds * t;
        left -= rounds * 256 * resident;
        while (left > 0) {
            int k = 0;
            for (int q = 1; q < used; ++q)
                if (at[q].free < at[k].free) k = q;
            if (at[k].n > left && used < 64) {
                at[used++] = {at[k].free, at[k].n - left};
                at[k].n = left;
            }
            left -= at[k].n;
            at[k].free += t;
        }
    }
    for (int k = 0; k < used; ++k)
        end = at[k].free > end ? at[k].free : end;
    return end;
}

// The tile for a product on these stacks, by estimated time.
struct Choice {
    int tile;
    double us;
};

template <int EPI, bool FULL>
Choice choose_tile(const Group& g)
{
    const double c = FULL ? 2.7 : 1;    // three products for one
    // beside the products: a launch, the first loads, and the epilogue, which
    // moves four bytes an element in a square, ten in an update, and in the
    // step fourteen to sixteen with the tiles of a round all at once
    const int k = symmetric(EPI) ? 0 : EPI == kStep ? 2 : 1;
    constexpr double fixed[3][4] = {
        {5, 7, 9, 10}, {7, 13, 20, 22}, {8, 20, 35, 55}};
    Choice best = {64,
                   estimate<64, EPI>(g, 0.36 * c, 0.18 * c, fixed[k][0], 2)};
    auto offer = [&](int t, double us) {
        if (us < best.us) best = {t, us};
    };
    offer(128, estimate<128, EPI>(g, 0.98 * c, 0.6 * c, fixed[k][1], 2));
    offer(192, estimate<192, EPI>(g, 1.12 * c, 0.95 * c, fixed[k][2], 1));
    offer(256, estimate<256, EPI>(g, 1.5 * c, 1.4 * c, fixed[k][3], 1));
    return best;
}

// Bits that a step takes from the exponent e of a matrix held as 2^e X, so that
// 2^e X stays below one: it multiplies a singular value s by at most
// |a| + |b| s^2 + |c| s^4, and from e = 2 on s is below 1/4.  (Where e is 1 X
// is within two of its usual range, whatever the step takes.)  The usual
// coefficients take 2 and multiply by 3.4; 3 a step would leave the low parts
// of ten steps without their bits.
inline int shift_of(const float (&coef)[3])
{
    const double g = std::fabs((double)coef[0]) +
                     std::fabs((double)coef[1]) / 16 +
                     std::fabs((double)coef[2]) / 256;
    int t = 0;
    while (t < 128 && std::ldexp(1.0, t) < g)
        ++t;
    return t;
}

// Two steps taken together on the m x m side.  In units of m^3 flops with
// r = n/m, a symmetric product being 1:
//   one by one   A = X X^T (r), C = a + b A + c A A (1), X <- C X (2 r),
//                twice: 6 r + 2
//   together     A (r), C (1), T = C A (1), A' = T C (1), C' from A' (1),
//                E = C' C (1), X <- E X (2 r): 3 r + 5
// for A' = C A C is the next step's A: polynomials of one matrix commute.
// The small directions of A' carry the rounding of the large ones, a^2 times,
// but only into C', where they count for a^2 b 2^-12; X itself stays exact.  A
// third step in the same way would multiply that by a^2 = 12 again (a matrix
// of 1024 x 3584 with singular values 1/k: 2.2e-4 one by one, 1e-3 in twos,
// 5e-3 in threes), so it is at most two.  In fast precision twos are the first
// two steps alone, where no direction is near one yet (256 x 3000, eight
// directions 100 times the others, five steps: 1.7e-4 one by one, 2.2e-4 so,
// 8.7e-4 with the last two together as well; singular values 1/k: 3.2e-4,
// 3.5e-4, 1.2e-3): the rounding of a gram is seen and corrected by the next
// one, which a later two leaves out.  In full precision all are twos; of an odd
// number the second turn is the single one.
//
// Whether step k goes together with the next, where twos are taken at all.  E
// is about a a' where A is small and has to stay in fp16's range.
inline bool together(const zs_newton_schulz& ns, int k)
{
    const bool may = ns.precision == ZS_NS_FULL
                         ? !(ns.steps % 2 && k == 2)
                         : k == 0;
    return may && k + 1 < ns.steps &&
           std::fabs(ns.coef[k][0] * ns.coef[k + 1][0]) < 24;
}

// Whether twos take less time, by the estimates of the launches.
inline bool in_pairs(const zs_newton_schulz& ns, double gram, double square,
                     double update)
{
    double pairs = 0;
    for (int k = 0; k < ns.steps;) {
        const bool two = together(ns, k);
        pairs += gram + (two ? 5.2 : 1) * square + update;
        k += two ? 2 : 1;
    }
    return pairs < 0.97 * ns.steps * (gram + square + update);
}

// The tiles of a group's products; LAST: the epilogue of the last update.
struct Tiles {
    Choice gram, square, update, last;
};

template <int LAST, bool FULL>
Tiles choose_tiles(const Group& g)
{
    return {choose_tile<kGram, FULL>(g), choose_tile<kPoly, FULL>(g),
            choose_tile<kUpdate, FULL>(g), choose_tile<LAST, FULL>(g)};
}

// In fast precision twos are not for matrices of few rows: a strong
// direction's part of A off the diagonal is then spread over few elements,
// and its rounding does not average out.  Roundings modelled in 64 bits, n =
// 1200 and one direction f times the others, one by one and in twos:
//   rows      8               64              96              128
//   f =   6   4.3e-4, 7.2e-3  2.9e-4, 5.6e-4  3.2e-4, 4.6e-4  3.4e-4, 4.0e-4
//   f =  30   5.9e-4, 1.1e-3  2.1e-4, 5.6e-4  2.4e-4, 5.3e-4  2.6e-4, 4.7e-4
//   f = 100   1.7e-3, 2.3e-3  2.3e-4, 5.3e-4  1.7e-4, 4.2e-4  1.9e-4, 3.8e-4
// From 128 rows on twos are at most about twice as far off.  Below, one by one
// costs 8 to 21 % (24 x 64 x 3000 154 -> 167 us, 60 x 120 x 8000 996 -> 1203).
// A single row has nothing off the diagonal.
inline bool thin(const Mat& m)
{
    const int32_t side = m.R < m.C ? m.R : m.C;
    return side > 1 && side < 128;
}

// Members that take their steps in launches of their own, whether some of
// them in twos, and by which tiles.
struct Part {
    int32_t count;
    int32_t at[kMaxMats];               // which of the group's
    Tiles tiles;
    bool pairs;
};

template <int LAST, bool FULL>
void plan_part(const Group& g, const zs_newton_schulz& ns, Part& p)
{
    Group sub;
    sub.count = p.count;
    for (int k = 0; k < p.count; ++k)
        sub.m[k] = g.m[p.at[k]];
    p.tiles = choose_tiles<LAST, FULL>(sub);
    p.pairs = in_pairs(ns, p.tiles.gram.us, p.tiles.square.us,
                       p.tiles.update.us);
}

// A group's steps: everything at once, or where twos are taken in fast
// precision the thin matrices by themselves and then the others.
template <int LAST, bool FULL>
int plan_steps(const Group& g, const zs_newton_schulz& ns, Part (&parts)[2])
{
    parts[0].count = g.count;
    int n = 0;
    for (int i = 0; i < g.count; ++i) {
        parts[0].at[i] = i;
        n += thin(g.m[i]);
    }
    plan_part<LAST, FULL>(g, ns, parts[0]);
    if (FULL || !parts[0].pairs || n == 0) return 1;
    if (n == g.count) {
        parts[0].pairs = false;
        return 1;
    }
    parts[0].count = parts[1].count = 0;
    for (int i = 0; i < g.count; ++i) {
        Part& p = parts[thin(g.m[i]) ? 0 : 1];
        p.at[p.count++] = i;
    }
    for (Part& p : parts)
        plan_part<LAST, FULL>(g, ns, p);
    parts[0].pairs = false;
    return 2;
}

}  // namespace muon
}  // namespace zs
