// The launches that a Newton-Schulz call's plan (csrc/zs_muon_plan.h) asks
// for, for tests of which kernels a call runs.  Host arithmetic only.

#include "zs_muon_plan.h"

using namespace zs::muon;

namespace {

struct Out {
    int32_t* rec;                       // [n][3]: product, tile, part
    int n, room;
    void add(int epi, int tile, int part)
    {
        if (n < room) {
            rec[3 * n] = epi;
            rec[3 * n + 1] = tile;
            rec[3 * n + 2] = part;
        }
        ++n;
    }
};

template <int LAST, bool FULL>
void launches(const Group& g, const zs_newton_schulz& ns, Out& out)
{
    Part parts[2];
    const int n = plan_steps<LAST, FULL>(g, ns, parts);
    for (int p = 0; p < n; ++p) {
        const Tiles& t = parts[p].tiles;
        for (int k = 0; k < ns.steps;) {
            const bool two = parts[p].pairs && together(ns, k);
            out.add(kGram, t.gram.tile, p);
            for (int q = 0; q < (two ? 2 : 1); ++q)
                out.add(kPoly, t.square.tile, p);
            for (int q = 0; two && q < 3; ++q)
                out.add(kProd, t.square.tile, p);
            k += two ? 2 : 1;
            if (k < ns.steps)
                out.add(kUpdate, t.update.tile, p);
            else
                out.add(LAST, t.last.tile, p);
        }
    }
}

template <bool FULL>
void launches(int last, const Group& g, const zs_newton_schulz& ns, Out& out)
{
    if (last == kOutBf16)
        launches<kOutBf16, FULL>(g, ns, out);
    else if (last == kOutF32)
        launches<kOutF32, FULL>(g, ns, out);
    else
        launches<kStep, FULL>(g, ns, out);
}

}  // namespace

// sizes: [count][3] batch, rows, cols.  Returns the number of products
// launched (small matrices have none), -1 where room is short.
extern "C" int muon_plan(int32_t count, const int64_t* sizes, int32_t last,
                         const zs_newton_schulz* ns, int32_t* rec,
                         int32_t room)
{
    const bool full = ns->precision == ZS_NS_FULL;
    int32_t order[kMaxMats];
    sort_members(order, count, [&](int32_t i, int64_t& r, int64_t& c) {
        r = sizes[3 * i + 1];
        c = sizes[3 * i + 2];
    });
    Group g = {};
    for (int i = 0; i < count; ++i) {
        const int64_t* const s = sizes + 3 * order[i];
        if (small_kind((int32_t)s[1], (int32_t)s[2], full)) continue;
        Mat& m = g.m[g.count++];
        m.batch = (int32_t)s[0];
        m.R = (int32_t)s[1];
        m.C = (int32_t)s[2];
    }
    Out out = {rec, 0, room};
    if (g.count && full)
        launches<true>(last, g, *ns, out);
    else if (g.count)
        launches<false>(last, g, *ns, out);
    return out.n > room ? -1 : out.n;
}
