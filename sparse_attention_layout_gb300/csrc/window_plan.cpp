// How a dense launch's steps are split over its CTAs: the line of window.cuh,
// cut into equal runs on the host.  A call's sizes and the handle's rule decide
// it, so a handle keeps the splits of the last sizes it met (a training step
// asks for the same three every time).
#include <list>
#include <mutex>
#include <new>
#include <vector>

#include "window.h"

namespace bsp {
namespace win {

namespace {

constexpr size_t kKeep = 48;
// steps below which a CTA is not worth starting while tiles are long
constexpr int kMinShare = 2;

struct Key {
    int side, rep, TQ, kshift, Sq, Sk, ctas;
    bool operator==(const Key& o) const {
        return side == o.side && rep == o.rep && TQ == o.TQ && kshift == o.kshift && Sq == o.Sq && Sk == o.Sk &&
               ctas == o.ctas;
    }
};

// Boundaries lie at equal steps, but never inside a tile of at most 4 steps or
// a 32nd of a share: cutting one saves less than its join costs (us, whole and
// cut: 256 rows of 4 heads, window 64: 11.4 and 13.6; 4 x 16 heads of 8192 rows,
// window 128, with gradient: 475 and 494; the gradient of 1037 rows of 12 heads
// 39.6 and 43.2, with tiles of 8 steps whole 47.6; up to an eighth of a share,
// full attention over 8192 keys took 244 for 224).  False: more steps than an int
// counts.
bool split(const std::vector<int>& steps, int rep, int ctas, Table* tab, CtaStart* out) {
    int64_t one = 0;
    for (int s : steps) one += s;  // every tile has a step
    if (one > INT32_MAX / rep) return false;
    const int ntiles = (int)steps.size(), items = ntiles * rep, tot = (int)one * rep;
    const Shares sh(tot, imax(1, imin(ctas, imax(items, tot / kMinShare))));
    *tab = Table(items, ctas);
    std::vector<int> at(ctas + 1, tot);
    int c = 0, pos = 0;
    for (int col = 0; col < ctas && c < sh.n; ++col)
        for (int row = 0; row < tab->height(col) && c < sh.n; ++row) {
            const int v = steps[tab->number(col, row) % ntiles];
            const bool keep_whole = v <= 4 || v <= sh.base / 32;
            while (c < sh.n && sh.at(c) < pos + v) {
                const int off = keep_whole ? 0 : sh.at(c) - pos;
                out[c] = CtaStart{col, row, off, 0};
                at[c++] = pos + off;
            }
            pos += v;
        }
    for (int i = 0; i < ctas; ++i) {
        if (i >= c) out[i] = CtaStart{0, 0, 0, 0};
        out[i].count = at[i + 1] - at[i];
    }
    return true;
}

}  // namespace

struct Plans {
    std::mutex mu;
    struct Entry {
        Key key;
        Table tab;
        bool cut;
        std::vector<CtaStart> s;
    };
    std::list<Entry> kept;
};

Plans* plans_create() { return new (std::nothrow) Plans; }
void plans_destroy(Plans* p) { delete p; }

namespace {

template <typename F>
int find(const Call& c, const Key& key, int ntiles, F steps_of, Table* tab, CtaStart* out,
         bool* cut) {
    try {
        Plans& P = *c.w->plans;
        std::lock_guard<std::mutex> lock(P.mu);
        for (const auto& e : P.kept)
            if (e.key == key) {
                *tab = e.tab;
                *cut = e.cut;
                for (int i = 0; i < key.ctas; ++i) out[i] = e.s[i];
                return BSP_OK;
            }
        std::vector<int> steps(ntiles);
        for (int t = 0; t < ntiles; ++t) steps[t] = steps_of(t);
        if (!split(steps, key.rep, key.ctas, tab, out)) return BSP_ERR_UNSUPPORTED;
        *cut = false;
        for (int i = 0; i < key.ctas; ++i) *cut |= out[i].off > 0;
        if (P.kept.size() >= kKeep) P.kept.pop_front();
        P.kept.push_back({key, *tab, *cut, std::vector<CtaStart>(out, out + key.ctas)});
        return BSP_OK;
    } catch (...) {
        return BSP_ERR_OOM;
    }
}

}  // namespace

int query_plan(const Call& c, int ctas, Table* tab, CtaStart* starts, bool* cut) {
    const Prob& p = c.p;
    const Seg g{0, p.Sq, p.Sk, (p.Sq + p.TQ - 1) / p.TQ};
    return find(c, Key{0, p.rep, p.TQ, p.kshift, p.Sq, p.Sk, ctas}, g.ntiles, [&](int t) { return p.steps(g, t); }, tab,
                starts, cut);
}

int key_plan(const Call& c, const KProb& k, int ctas, Table* tab, CtaStart* starts, bool* cut) {
    const int ntiles = (int)(((int64_t)k.Sk + (1 << k.kshift) - 1) >> k.kshift);
    return find(c, Key{1, k.rep, k.TQ, k.kshift, k.Sq, k.Sk, ctas}, ntiles,
                [&](int t) { return k.steps(Seg{}, t); }, tab, starts, cut);
}

}  // namespace win
}  // namespace bsp
