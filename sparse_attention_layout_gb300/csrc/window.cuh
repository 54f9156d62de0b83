// Work geometry of the windowed attention operators (dense and paged): which
// key tiles a tile of query rows sees, and the even split of all the
// (query tile, key tile) steps of a launch over its CTAs.
//
// Visibility: key j is visible to the query at position p when j <= p and
// (p - j < window or j < sinks).
//
// A query tile holds TQ consecutive tokens of one sequence times the G query
// heads that share one KV head, token after token (row r: token r / G, head
// r % G), so that one pass over the keys serves the whole group and the rows
// of a single new token are the tile's first G.
//
// Split: the steps of all tiles form one line, of which each CTA takes an equal
// run (of a dense batch, up to the next short tile's edge).  A tile that a
// boundary cuts leaves partial results, which a second kernel joins in the order
// of the pieces, so results do not depend on timing.  Tiles are numbered
// (segment, repetition, tile); a segment is a shape of tiles: the whole of a
// dense batch, repeated for each (batch entry, KV head), which the host splits,
// or one sequence of a ragged one, whose lengths only the device knows, repeated
// for each KV head.  The line holds them column by column of a table with one
// column per CTA, filled row by row: CTAs then work on neighbouring tiles at the
// same time and share their keys in L2 (with each CTA on a run of consecutive
// tiles instead, the band of 8192 keys and 16 heads read 954 MB from HBM instead
// of the 402 MB that it holds).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/bsp.h"

#if defined(__CUDACC__)
#define BSP_HD __host__ __device__ __forceinline__
#else
#define BSP_HD inline
#endif

namespace bsp {
namespace win {

// positions, lengths and windows stay within this (a window at least as large
// as every position has no effect), so sums of two of them fit an int
constexpr int kMaxLen = 1 << 30;
constexpr int kMaxGroup = 64;      // query heads per KV head
constexpr int kMaxSeqs = 16384;    // sequences of one ragged call (their tile counts sit in shared memory)

// Attempts of a bounded wait of the tensor-core kernels.  A failed one takes 1.4
// us (measured: 20 in 27.6 us), and tens of cycles at the least: 2^21 are 3 s, and
// 40 ms at the least, for waits that last about a step of another role.  An
// epilogue waits for its whole tile, some microseconds for each of its steps: 128
// attempts more for each, enough even at the least.
constexpr int kLeastAttempts = 1 << 21;
inline int wait_attempts(int64_t steps) {
    const int64_t n = kLeastAttempts + 128 * steps;
    return n > INT32_MAX ? INT32_MAX : (int)n;
}

// element (i, j, k, d) at ptr + i * s[0] + j * s[1] + k * s[2] + d
struct View {
    void* ptr;
    int64_t s[3];
};

// Key tiles of a query tile whose rows stand at positions a .. b: the tiles
// that hold sinks and lie wholly before the window's, then the window's.
// A tile of rows that see nothing (b < 0) gets one step with every key
// hidden, so that every tile writes its output.
struct Span {
    int n;    // steps
    int n_s;  // of them over sink tiles 0 .. n_s - 1
    int lo;   // first tile of the window's range
    BSP_HD int tile(int i) const { return i < n_s ? i : lo + (i - n_s); }
};

BSP_HD int imax(int a, int b) { return a > b ? a : b; }
BSP_HD int imin(int a, int b) { return a < b ? a : b; }

// lowest visible key position (sinks aside) of rows at positions a .., a the first
BSP_HD int window_low(int a, int window) { return imax(0, imax(a, 0) - window + 1); }

BSP_HD Span span_of(int a, int b, int window, int sinks, int kshift) {
    Span s;
    if (b < 0) {
        s.n = 1;
        s.n_s = 0;
        s.lo = 0;
        return s;
    }
    s.lo = window_low(a, window) >> kshift;
    s.n_s = imin((int)(((int64_t)sinks + (1 << kshift) - 1) >> kshift), s.lo);
    s.n = s.n_s + (b >> kshift) - s.lo + 1;
    return s;
}

struct Seg {
    int t0;     // first token's row in the ragged tensors (dense: 0)
    int qlen;   // query tokens
    int kvlen;  // key positions
    int ntiles;
};

// A query tile: tokens tok0 .. tok0 + nt - 1 of its segment at positions a .. b.
struct QTile {
    int tok0, nt, a, b;
};

// The forward and dQ kernels' problem: tiles are query tiles, steps key tiles.
struct Prob {
    int paged;
    int nseg, rep;  // dense: 1 and Z * Hkv; paged: sequences and Hkv
    int G, TQ, kshift;
    int Hq, Hkv;
    int Sq, Sk;     // dense
    int T, max_pages, n_pages, page_shift;
    int window, sinks;
    const int* q_start;
    const int* kv_len;
    const int* table;
    int* status;
    int attempts;   // of the wait for a tile (tensor-core kernels)

    BSP_HD bool bad_seg(int q0, int q1, int kv) const {
        return q0 < 0 || q1 < q0 || q1 > T || kv < 0 || kv > (max_pages << page_shift);
    }
#if defined(__CUDACC__)
    __device__ __forceinline__ Seg seg(int s) const {
        if (!paged) return Seg{0, Sq, Sk, (Sq + TQ - 1) / TQ};
        const int q0 = q_start[s], q1 = q_start[s + 1], kv = kv_len[s];
        if (bad_seg(q0, q1, kv)) return Seg{0, 0, 0, 0};
        return Seg{q0, q1 - q0, kv, (q1 - q0 + TQ - 1) / TQ};
    }
    // Offsets that descend let sequences overlap, and their steps then add up to
    // more than the host has allowed for: such a call has no tiles at all.
    __device__ __forceinline__ bool descends(int s) const { return q_start[s + 1] < q_start[s]; }
#endif
    BSP_HD QTile qtile(const Seg& g, int t) const {
        QTile q;
        q.tok0 = t * TQ;
        q.nt = imin(TQ, g.qlen - q.tok0);
        q.a = g.kvlen - g.qlen + q.tok0;
        q.b = q.a + q.nt - 1;
        return q;
    }
    BSP_HD Span span(const QTile& q) const { return span_of(q.a, q.b, window, sinks, kshift); }
    BSP_HD int steps(const Seg& g, int t) const { return span(qtile(g, t)).n; }
    BSP_HD int describe(const Seg& g, int t, QTile& q, Span& sp) const {
        q = qtile(g, t);
        sp = span(q);
        return sp.n;
    }
};

// The dK / dV kernel's problem (dense only): tiles are key tiles, steps the
// query tiles with a row that sees one of its keys.
struct KProb {
    int nseg, rep;
    int G, TQ, kshift;
    int Hq, Hkv, Sq, Sk;
    int window, sinks;

#if defined(__CUDACC__)
    __device__ __forceinline__ Seg seg(int) const {
        return Seg{0, Sq, Sk, (int)(((int64_t)Sk + (1 << kshift) - 1) >> kshift)};
    }
#endif
    // first query tile and count (0 rows that see the tile: one hidden step)
    BSP_HD void qrange(int t, int* first, int* n) const {
        const int off = Sk - Sq, kb = t << kshift, ke = imin(kb + (1 << kshift), Sk) - 1;
        const int t_lo = imax(0, kb - off);
        int64_t t_hi = Sq - 1;
        if (kb >= sinks) {
            const int64_t w = (int64_t)ke + window - 1 - off;
            t_hi = w < t_hi ? w : t_hi;
        }
        if (t_hi < t_lo) {
            *first = 0;
            *n = 1;
            return;
        }
        *first = t_lo / TQ;
        *n = (int)(t_hi / TQ) - *first + 1;
    }
    BSP_HD int steps(const Seg&, int t) const {
        int f, n;
        qrange(t, &f, &n);
        return n;
    }
    // the first query tile as the span's lo
    BSP_HD int describe(const Seg&, int t, QTile&, Span& sp) const {
        qrange(t, &sp.lo, &sp.n);
        return sp.n;
    }
};

// CTA c's share of `tot` steps: [at(c), at(c + 1)), the first `rem` CTAs with
// one more than the `base` of the others.
struct Shares {
    int n, base, rem;
    BSP_HD Shares(int tot, int ctas) : n(ctas), base((uint32_t)tot / (uint32_t)ctas), rem((uint32_t)tot % (uint32_t)ctas) {}
    Shares() = default;
    BSP_HD int at(int c) const { return base * c + imin(c, rem); }
    BSP_HD int of(int c) const { return c < n ? base + (c < rem) : 0; }
};

// The table of `items` tiles in `cols` columns: every column has q rows, and r
// of them, evenly spread, one more (with the first r columns the longer ones
// instead, the shares' starts drifted over whole columns, neighbouring CTAs lost
// step, and chunks of prompts read their 170 MB of keys 11 times from HBM).
struct Table {
    int cols, q, r, items;
    BSP_HD Table(int n, int columns)
        : cols(columns), q((uint32_t)n / (uint32_t)columns), r((uint32_t)n % (uint32_t)columns), items(n) {}
    Table() = default;
    BSP_HD int longer(int col) const { return (uint32_t)(col * r) / (uint32_t)cols; }  // longer columns before col
    BSP_HD int before(int col) const { return col * q + longer(col); }
    BSP_HD int height(int col) const { return before(col + 1) - before(col); }
    BSP_HD int number(int col, int row) const { return row * cols + (row < q ? col : longer(col)); }
    // column and row of place l on the line
    BSP_HD void place(int l, int* col, int* row) const {
        int c = imin((int)(((float)l + 1.0f) * cols / items), cols - 1);
        while (before(c) > l) --c;  // the float quotient is off by one or so
        while (before(c + 1) <= l) ++c;
        *col = c;
        *row = l - before(c);
    }
};

// Where a CTA's share begins: step `off` of the tile at (col, row), `count`
// steps in all.
struct CtaStart {
    int col, row, off, count;
};

// A dense launch's split, which the host knows: one start per CTA, handed over
// as a kernel parameter (finding them in the kernel took a call of one tile
// 4.6 of its 12 us).
template <int N>
struct Plan {
    static constexpr int kCtas = N;  // the most CTAs of a launch
    Table tab;
    CtaStart s[N];
};
using TcPlan = Plan<160>;    // one CTA per SM
using SimtPlan = Plan<320>;  // two

// A tile that begins in CTA c and goes on in later ones: `pieces` of it (0:
// none), the first in slot 2 c + 1, the others in slots 2 (c + 1), 2 (c + 2) ...
struct Cut {
    int pieces;
    int seg, rep, tile;
};

#if defined(__CUDACC__)

// How a launch is split: a dense batch, by the host; a ragged batch, on the
// device; a ragged batch of single tokens, whose tiles share no keys, in the
// order of their numbers: finding the shares then is one scan, and the walk a
// count.
enum Mode { kDense, kRagged, kPlain };

// A ragged launch's split.
struct Start {
    Table tab;
    Shares shares;
    CtaStart cta;
    int seg, rep, tile;  // kPlain: the first tile
};

// exclusive prefix over the block's threads; *total = the block's sum
template <int NT>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* red, uint32_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    uint32_t w = lane < NT / 32 ? red[lane] : 0;
#pragma unroll
    for (int o = 1; o < NT / 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, NT / 32 - 1);
    const uint32_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return (warp ? before : 0) + x - v;
}

// as many CTAs as there are tiles, or more if each still gets min_share steps
__device__ __forceinline__ Shares shares_of(int tot, int items, int min_share) {
    return Shares(tot, imax(1, imin(gridDim.x, imax(items, tot / min_share))));
}

// The plain split of at most NT segments; called by every thread of the block.
template <int NT>
__device__ __forceinline__ void locate_plain(const Prob& p, int min_share, uint32_t* red, Start* out) {
    const int s = threadIdx.x;
    const Seg g = s < p.nseg ? p.seg(s) : Seg{0, 0, 0, 0};
    int w = 0;
#pragma unroll 1
    for (int t = 0; t < g.ntiles; ++t) w += p.steps(g, t);
    if (__syncthreads_or(s < p.nseg && p.descends(s))) w = 0;
    uint32_t tot;
    const int ex = (int)block_scan<NT>(w * p.rep, red, &tot);
    // (items counted as if every segment had one tile: close enough)
    const Shares sh = shares_of(tot, p.nseg * p.rep, min_share);
    const int at = sh.at(blockIdx.x), count = sh.of(blockIdx.x);
    if (threadIdx.x == 0) {
        out->shares = sh;
        out->cta.count = count;
    }
    if (count > 0 && at >= ex && at < ex + w * p.rep) {
        out->seg = s;
        out->rep = (uint32_t)(at - ex) / (uint32_t)w;
        int off = (uint32_t)(at - ex) % (uint32_t)w, t = 0;
#pragma unroll 1
        for (int v; off >= (v = p.steps(g, t)); ++t) off -= v;
        out->tile = t;
        out->cta.off = off;
    }
    __syncthreads();
}

// Finds this CTA's share of a ragged launch; called by every thread of the
// block.  seg_end: scratch of nseg ints in shared memory, the tiles of the
// segments up to each; red: 32 words.  min_share: CTAs are used only while each
// gets this many steps.  Each thread adds up a run of the line, one scan gives
// the runs' starts, and the thread whose run holds the share's first step finds
// it.  Out of line: the kernels' loops then stay within the instruction cache.
template <int NT>
__device__ __noinline__ void locate(const Prob& p, int min_share, int* seg_end, uint32_t* red, Start* out) {
    const int tid = threadIdx.x;
    int tiles = 0;  // one repetition of every segment
    bool bad = false;
#pragma unroll 1
    for (int s0 = 0; s0 < p.nseg; s0 += NT) {
        const int s = s0 + tid;
        const uint32_t v = s < p.nseg ? p.seg(s).ntiles : 0;
        bad |= s < p.nseg && p.descends(s);
        uint32_t total;
        const uint32_t ex = block_scan<NT>(v, red, &total);
        if (s < p.nseg) seg_end[s] = tiles + (int)(ex + v);
        tiles += (int)total;
    }
    if (__syncthreads_or(bad)) tiles = 0;
    const int items = tiles * p.rep;
    const Table tab(items, gridDim.x);
    const int run = (items + NT - 1) / NT;
    const int l0 = imin(tid * run, items), l1 = imin(l0 + run, items);
    int at = -1, sum = 0;
    // twice: the sum, then (by the thread that holds it) the first step's tile
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        int pos = sum;  // second pass: steps before this run
        sum = 0;
        int col = 0, row = 0, height = 0;
#pragma unroll 1
        for (int l = l0; l < l1; ++l) {
            if (l == l0) {
                tab.place(l, &col, &row);
                height = tab.height(col);
            } else {
                ++row;
                while (row >= height) {  // a column may be empty
                    ++col;
                    row = 0;
                    height = tab.height(col);
                }
            }
            // the segment that holds tile number a
            const int a = tab.number(col, row);
            int lo = 0, hi = p.nseg - 1;
#pragma unroll 1
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (seg_end[mid] * p.rep > a) hi = mid;
                else lo = mid + 1;
            }
            const Seg g = p.seg(lo);
            const int v = p.steps(g, (uint32_t)(a - (seg_end[lo] - g.ntiles) * p.rep) % (uint32_t)g.ntiles);
            if (pass == 1) {
                if (at < pos + v) {
                    out->cta.col = col;
                    out->cta.row = row;
                    out->cta.off = at - pos;
                    break;
                }
                pos += v;
            }
            sum += v;
        }
        if (pass == 0) {
            uint32_t tot;
            const uint32_t ex = block_scan<NT>(sum, red, &tot);
            const Shares sh = shares_of(tot, items, min_share);
            const int count = sh.of(blockIdx.x);
            if (tid == 0) {
                out->tab = tab;
                out->shares = sh;
                out->cta.count = count;
            }
            at = sh.at(blockIdx.x);
            if (count == 0 || at < (int)ex || at >= (int)ex + sum) break;
            sum = (int)ex;
        }
    }
    __syncthreads();
}

// A tile of a CTA's share: steps s0 .. s0 + ns - 1 of its n.
struct Item {
    int seg, rep, tile;
    int s0, ns, n;
    Seg g;
    QTile q;  // of a Prob
    Span sp;
    __device__ __forceinline__ bool whole() const { return ns == n; }
    // where a piece's partial result goes
    __device__ __forceinline__ int slot() const { return 2 * blockIdx.x + (s0 == 0); }
};

// Walks the tiles of a CTA's share; of a ragged batch, all lanes of a warp
// together.
template <typename P, int MODE>
struct Walk {
    const P& p;
    Table tab;
    int left;
    int col, row, height, tail;  // tail: place in the last row
    int off;
    int seg, seg0;  // a segment and the number of its first tile
    Seg g;
    int rep = 0, tile = 0;  // kPlain: the tile that comes next
    __device__ __forceinline__ Walk(const P& prob, const Start& st)
        : p(prob), tab(st.tab), left(st.cta.count), off(st.cta.off), seg(0), seg0(0) {
        if (left <= 0) return;
        if (MODE == kPlain) {
            seg = st.seg, rep = st.rep, tile = st.tile;
            g = p.seg(seg);
        } else {
            enter(st.cta.col, st.cta.row);
        }
    }
    __device__ __forceinline__ Walk(const P& prob, const Table& t, const CtaStart& st)
        : p(prob), tab(t), left(st.count), off(st.off), seg(0), seg0(0) {
        enter(st.col, st.row);
        g = p.seg(0);
    }
    __device__ __forceinline__ void enter(int c, int r) {
        col = c;
        row = r;
        height = tab.height(c);
        tail = tab.longer(c);
    }
    __device__ __forceinline__ bool next(Item& it) {
        if (left <= 0) return false;
        if constexpr (MODE == kPlain) {
            it.seg = seg, it.rep = rep, it.tile = tile, it.g = g;
            take(it);
            if (left > 0 && ++tile >= g.ntiles) {
                tile = 0;
                if (++rep >= p.rep) {
                    rep = 0;
                    do {
                        if (++seg >= p.nseg) {  // only when q_start or kv_len changed under the call
                            left = 0;
                            break;
                        }
                        g = p.seg(seg);
                    } while (g.ntiles == 0);
                }
            }
            return true;
        } else {
            return next_in_table(it);
        }
    }
    __device__ __forceinline__ bool next_in_table(Item& it) {
        while (row >= height) {  // a column may be empty
            enter(col + 1, 0);
            seg = 0;
            seg0 = 0;
        }
        const int a = row * tab.cols + (row < tab.q ? col : tail);
        ++row;
        if constexpr (MODE == kRagged) {
            // 32 segments at a time: the one that holds tile number a
            const int lane = threadIdx.x & 31;
#pragma unroll 1
            while (true) {
                const int s = seg + lane;
                const Seg h = s < p.nseg ? p.seg(s) : Seg{0, 0, 0, 0};
                int end = h.ntiles * p.rep;
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, end, o);
                    if (lane >= o) end += y;
                }
                end += seg0;
                const unsigned m = __ballot_sync(0xffffffffu, end > a);
                if (m == 0) {
                    if (seg + 32 >= p.nseg) {  // only when q_start or kv_len changed under the call
                        left = 0;
                        return false;
                    }
                    seg += 32;
                    seg0 = __shfl_sync(0xffffffffu, end, 31);
                    continue;
                }
                const int src = __ffs(m) - 1;
                seg += src;
                seg0 = __shfl_sync(0xffffffffu, end - h.ntiles * p.rep, src);
                g.t0 = __shfl_sync(0xffffffffu, h.t0, src);
                g.qlen = __shfl_sync(0xffffffffu, h.qlen, src);
                g.kvlen = __shfl_sync(0xffffffffu, h.kvlen, src);
                g.ntiles = __shfl_sync(0xffffffffu, h.ntiles, src);
                break;
            }
        }
        it.seg = seg;
        it.rep = (uint32_t)(a - seg0) / (uint32_t)g.ntiles;
        it.tile = (uint32_t)(a - seg0) % (uint32_t)g.ntiles;
        it.g = g;
        take(it);
        return true;
    }
    // the steps of the tile that fall into the share
    __device__ __forceinline__ void take(Item& it) {
        it.n = p.describe(it.g, it.tile, it.q, it.sp);
        it.s0 = off;
        it.ns = imin(it.n - off, left);
        left -= it.ns;
        off = 0;
    }
};

// The record of a tile that begins in this CTA and goes on for `left` steps
// after its share; count(c): steps of CTA c.
template <typename F>
__device__ __forceinline__ void write_cut(Cut* cuts, int seg, int rep, int tile, int left, F count) {
    int pieces = 1;
#pragma unroll 1
    for (int c = blockIdx.x + 1; left > 0 && c < gridDim.x; ++c, ++pieces) left -= count(c);
    cuts[blockIdx.x] = Cut{pieces, seg, rep, tile};
}

#endif  // __CUDACC__

}  // namespace win
}  // namespace bsp
