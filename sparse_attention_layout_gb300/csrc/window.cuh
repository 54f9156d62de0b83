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
// Split: the steps of all tiles, in the order (segment, repetition, tile,
// step), form one line; CTA c of n takes [c tot / n, (c + 1) tot / n).  A
// tile that a boundary cuts leaves partial results, which a second kernel
// joins in the order of the pieces, so results do not depend on timing.  One
// segment is a shape of tiles: the whole of a dense batch (repeated for each
// (batch entry, KV head)), or one sequence of a ragged one (repeated for each
// KV head), whose lengths only the device knows.
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
constexpr int kMaxSeqs = 16384;    // sequences of one ragged call (their step counts sit in shared memory)

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
};

// Share of CTA c among n: [share_at(c), share_at(c + 1)).
BSP_HD int64_t share_at(int64_t tot, int n, int c) { return c >= n ? tot : tot / n * c + tot % n * c / n; }

// Where a CTA's share begins, how long it is.
struct Start {
    int64_t tot;
    int n;         // CTAs that share the steps (the others do nothing)
    int64_t count; // steps of this CTA
    int seg, rep, tile, off;
};

// A tile that begins in CTA c and goes on in later ones: `pieces` of it (0:
// none), the first in slot 2 c + 1, the next in slot 2 c' of each further CTA
// c' with a share.
struct Cut {
    int pieces;
    int seg, rep, tile;
    int64_t tot;
    int n, pad;
};

#if defined(__CUDACC__)

template <int NT>
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* red) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    int64_t t = 0;
    for (int i = 0; i < NT / 32; ++i) t += red[i];
    return t;
}

// exclusive prefix over the block's threads; *total = the block's sum
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* red, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int64_t before = 0, t = 0;
    for (int i = 0; i < NT / 32; ++i) {
        if (i < warp) before += red[i];
        t += red[i];
    }
    *total = t;
    return before + x - v;
}

// Finds this CTA's share; called by every thread of the block.  seg_steps:
// scratch of nseg ints in shared memory (unused when nseg == 1); red: 32
// int64.  min_share: CTAs are used only while each gets this many steps.
template <int NT, typename P>
__device__ __forceinline__ void locate(const P& p, int n_cta, int min_share, int* seg_steps, int64_t* red, Start* out) {
    const int tid = threadIdx.x;
    int64_t sum = 0;  // steps of all segments, one repetition
    int64_t one = 0;  // dense: the only segment's
    if (p.nseg == 1) {
        const Seg g = p.seg(0);
        for (int t = tid; t < g.ntiles; t += NT) sum += p.steps(g, t);
        one = sum = block_sum<NT>(sum, red);
    } else {
        const int lane = tid & 31;
        for (int s0 = tid - lane; s0 < p.nseg; s0 += NT) {
            const int s = s0 + lane;
            const Seg g = s < p.nseg ? p.seg(s) : Seg{0, 0, 0, 0};
            int w = 0;
            const bool many = g.ntiles > 8;
            if (!many)
                for (int t = 0; t < g.ntiles; ++t) w += p.steps(g, t);
            unsigned left = __ballot_sync(0xffffffffu, many);
            while (left) {  // long chunks: the warp counts one together
                const int src = __ffs(left) - 1;
                left &= left - 1;
                Seg h;
                h.t0 = __shfl_sync(0xffffffffu, g.t0, src);
                h.qlen = __shfl_sync(0xffffffffu, g.qlen, src);
                h.kvlen = __shfl_sync(0xffffffffu, g.kvlen, src);
                h.ntiles = __shfl_sync(0xffffffffu, g.ntiles, src);
                int c = 0;
                for (int t = lane; t < h.ntiles; t += 32) c += p.steps(h, t);
                for (int o = 16; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
                if (lane == src) w = c;
            }
            if (s < p.nseg) seg_steps[s] = w;
            sum += w;
        }
        sum = block_sum<NT>(sum, red);
    }
    Start st;
    st.tot = sum * p.rep;
    const int64_t most = (st.tot + min_share - 1) / min_share;
    st.n = most < 1 ? 1 : (most < n_cta ? (int)most : n_cta);
    const int c = blockIdx.x;
    int64_t at = share_at(st.tot, st.n, c);
    st.count = share_at(st.tot, st.n, c + 1) - at;
    st.seg = st.rep = st.tile = st.off = 0;
    if (st.count > 0) {
        int64_t w = one;
        if (p.nseg > 1) {
            __syncthreads();
            int64_t before = 0;
            for (int s0 = 0; s0 < p.nseg; s0 += NT) {
                const int s = s0 + tid;
                const int64_t v = s < p.nseg ? (int64_t)seg_steps[s] * p.rep : 0;
                int64_t total;
                const int64_t ex = before + block_scan<NT>(v, red, &total);
                if (v > 0 && ex <= at && at < ex + v) {
                    out->seg = s;
                    out->count = at - ex;  // step within the segment, all repetitions
                }
                before += total;
                if (at < before) break;
            }
            __syncthreads();
            st.seg = out->seg;
            at = out->count;
            w = seg_steps[st.seg];
            __syncthreads();
        }
        st.rep = (int)(at / w);
        at -= (int64_t)st.rep * w;
        const Seg g = p.seg(st.seg);
        int64_t before = 0;
        for (int t0 = 0; t0 < g.ntiles; t0 += NT) {
            const int t = t0 + tid;
            const int64_t v = t < g.ntiles ? p.steps(g, t) : 0;
            int64_t total;
            const int64_t ex = before + block_scan<NT>(v, red, &total);
            if (v > 0 && ex <= at && at < ex + v) {
                out->tile = t;
                out->off = (int)(at - ex);
            }
            before += total;
            if (at < before) break;
        }
        __syncthreads();
        st.tile = out->tile;
        st.off = out->off;
    }
    __syncthreads();
    if (tid == 0) *out = st;
    __syncthreads();
}

// Walks the tiles of a CTA's share.
struct Item {
    int seg, rep, tile;
    int s0, ns, n;  // steps s0 .. s0 + ns - 1 of the tile's n
    Seg g;
    __device__ __forceinline__ bool whole() const { return ns == n; }
    // where a piece's partial result goes
    __device__ __forceinline__ int slot() const { return 2 * blockIdx.x + (s0 == 0); }
};

template <typename P>
struct Walk {
    const P& p;
    int64_t left;
    int seg, rep, tile, off;
    Seg g;
    __device__ __forceinline__ Walk(const P& prob, const Start& st)
        : p(prob), left(st.count), seg(st.seg), rep(st.rep), tile(st.tile), off(st.off) {
        if (left > 0) g = p.seg(seg);
    }
    __device__ __forceinline__ bool next(Item& it) {
        if (left <= 0) return false;
        while (tile >= g.ntiles) {  // next repetition, or next segment with tiles
            tile = 0;
            if (g.ntiles == 0 || ++rep >= p.rep) {
                rep = 0;
                if (++seg >= p.nseg) {
                    left = 0;
                    return false;
                }
                g = p.seg(seg);
            }
        }
        it.seg = seg;
        it.rep = rep;
        it.tile = tile;
        it.g = g;
        it.n = p.steps(g, tile);
        it.s0 = off;
        it.ns = it.n - off;
        if (it.ns > left) it.ns = (int)left;
        left -= it.ns;
        off = 0;
        ++tile;
        return true;
    }
};

// The record of a tile that begins in this CTA and is cut at its end.
__device__ __forceinline__ void write_cut(Cut* cuts, const Item& it, const Start& st) {
    int left = it.n - it.ns, pieces = 1;
    for (int c = blockIdx.x + 1; left > 0 && c < st.n; ++c) {
        const int64_t sh = share_at(st.tot, st.n, c + 1) - share_at(st.tot, st.n, c);
        if (sh <= 0) continue;
        left -= (int)(sh < left ? sh : left);
        ++pieces;
    }
    Cut c{pieces, it.seg, it.rep, it.tile, st.tot, st.n, 0};
    cuts[blockIdx.x] = c;
}

#endif  // __CUDACC__

}  // namespace win
}  // namespace bsp
