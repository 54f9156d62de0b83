// Shared by the tensor-core kernels of the windowed attention.
#pragma once

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "tc_common.cuh"
#include "window.h"

namespace bsp {
namespace win {

using namespace tc;

constexpr int kThreads = 512;
// Registers per thread: producers and issuers give some of the launch's 128 to
// the two softmax warpgroups, the epilogue keeps its own; 80 + 128 + 152 + 152 =
// 4 * 128.
constexpr uint32_t kRegsLaunch = 128, kRegsCtl = 80, kRegsSoftmax = 152;
static_assert(kRegsCtl + kRegsLaunch + 2 * kRegsSoftmax <= 4 * kRegsLaunch, "register split exceeds the launch allocation");

// The code that the roles run between them has to fit the SM's instruction
// cache: at 120 KB of kernel its refills kept the cache behind it 88 % busy and
// doubled the time of short windows.  So the waits are short (a count of
// attempts in place of mbar_wait's clock, the code of a failure left to the end
// of the kernel), loops are rolled where that costs nothing, and what runs once
// is out of line.
//
// Shared abort flag: 0, or the BSP_ERR_* code that stopped the kernel.
struct Stop {
    volatile int* flag;
    __device__ __forceinline__ void fail(int code) const { *flag = code; }
};
// Attempts: a constant where a wait lasts about a step of another role (held in a
// register or read from the parameters there, the forward took 2 % longer), the
// call's own for an epilogue's wait for its tile, the only one that lasts as long
// as the tile's steps.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const Stop& ab, int attempts = kLeastAttempts) {
    for (int n = attempts; !mbar_try_wait(bar, parity);) {
        if (*ab.flag) return false;
        if (--n == 0) ab.fail(BSP_ERR_TIMEOUT);
    }
    return true;
}
// After an abort, by one thread: wait, bounded, for the phase of `bar` with the
// given parity, whatever the flag says: copies and products in flight end by
// themselves.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
    for (int n = kLeastAttempts; !mbar_try_wait(bar, parity) && --n;) {}
}
// The arrivals of commits that no role waits for any more follow the drained
// ones at once; the CTA's shared memory outlasts them.
__device__ __forceinline__ void drain_end() { __nanosleep(10000); }
// The same for a ring of nst stages whose phases 0 .. next - 1 were begun.
__device__ __forceinline__ void drain_ring(uint64_t* bars, uint32_t nst, uint32_t next) {
#pragma unroll 1
    for (uint32_t s = 0; s < nst && s < next; ++s)
        drain_wait(&bars[s], (s + ((next - 1 - s) / nst) * nst) / nst & 1);
}

// Visible keys of a tile's rows: j <= hi and (j >= lo or j < sinks).
struct Keys {
    int lo, hi, sinks;
    __device__ __forceinline__ bool any(int a, int b) const { return (a <= hi) & ((b >= lo) | (a < sinks)); }
    // bit i: some of the 16 keys from kb + 16 i is visible (i < 8)
    __device__ __forceinline__ uint32_t pieces(int kb) const {
        const int end = imin(hi + 1 - kb, 128);  // > 0 bounds the visible part of the tile
        const uint32_t upto = (1u << (imax(end + 15, 0) >> 4)) - 1;
        const uint32_t from = ~0u << (imin(imax(lo - kb, 0), 128) >> 4);
        const uint32_t sink = (1u << (imin(imax(sinks - kb + 15, 0), 128 + 15) >> 4)) - 1;
        return upto & (from | sink) & 0xffu;
    }
};
// What the roles of a kernel need to know of a tile, handed out through a ring
// in shared memory by the warp that walks the CTA's share: the walk's state and
// its divisions then burden no other role's registers (with every role on a
// walk of its own the softmax spilled, and a step of full attention took 1.33
// us).  ns == 0 ends the share.
struct __align__(16) Work {
    int ns, s0, n;       // steps s0 .. s0 + ns - 1 of the tile's n
    int tile;
    int a, nt;           // position of its first token, tokens
    int n_s, lo;         // sink steps, first window tile (dkv: first query tile in lo)
    int row0, z, hk, seg;
    int rep;
    int zlo, zhi;        // keys that some query of the segment sees, sinks aside
    int pad;
    __device__ __forceinline__ bool whole() const { return ns == n; }
    __device__ __forceinline__ int slot() const { return 2 * blockIdx.x + (s0 == 0); }
    __device__ __forceinline__ int key_tile(int i) const { return s0 + i < n_s ? s0 + i : lo + (s0 + i - n_s); }
};

constexpr int kRing = 4;
constexpr int kReaders = 15;  // three single-thread or producer roles, 4 epilogue warps, 8 softmax warps

struct Ring {
    uint64_t full[kRing], empty[kRing];
    Work w[kRing];
    __device__ __forceinline__ void init() {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kReaders);
        }
    }
    // by a whole warp, in order i = 0, 1, ...
    __device__ __forceinline__ bool put(uint32_t i, const Work& x, int lane, const Stop& ab) {
        const uint32_t s = i % kRing;
        const bool ok = wait(&empty[s], ((i / kRing) & 1) ^ 1, ab);
        if (!__all_sync(0xffffffffu, ok)) return false;
        if (lane == 0) {
            w[s] = x;
            mbar_arrive(&full[s]);
        }
        return true;
    }
    // by one thread, or by all lanes of a warp (`one`: the lane that answers)
    __device__ __forceinline__ bool take(uint32_t i, Work& x, bool one, bool warp, const Stop& ab) {
        const uint32_t s = i % kRing;
        bool ok = wait(&full[s], (i / kRing) & 1, ab);
        if (warp) ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        x = w[s];
        if (warp) __syncwarp();
        if (one) mbar_arrive(&empty[s]);
        return x.ns > 0;
    }
};

// Rows r0 .. r1 - 1 of a tile in shared memory (KP panels of 128 rows of 128
// bytes) set to 0 by a warp.
template <int KP>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0, int r1, int lane) {
#pragma unroll 1
    for (int i = r0 * 8 + lane; i < r1 * 8; i += 32)
#pragma unroll
        for (int c = 0; c < KP; ++c) *reinterpret_cast<uint4*>(tile + c * 16384 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
}
// The rows of the key tile that begins at key kb that no query of a dense call
// sees (the keys between the sinks and the first query's window), as a range.
struct Unseen {
    int r0, r1;
    __device__ __forceinline__ Unseen(int kb, int sinks, int zlo) : r0(imax(sinks - kb, 0)), r1(imin(zlo - kb, 128)) {}
    __device__ __forceinline__ bool any() const { return r0 < r1; }
};

__device__ __forceinline__ Keys tile_keys(const Prob& p, const Work& w) {
    return Keys{window_low(w.a, p.window), w.a + w.nt - 1, p.sinks};
}
__device__ __forceinline__ Keys tile_keys(const TreeProb& p, const Work& w) {
    return Keys{window_low(w.a, p.window), w.zhi, p.sinks};
}

__device__ __forceinline__ Work make_work(const Prob& p, const Item& it) {
    const QTile& q = it.q;
    const Span& sp = it.sp;
    Work w;
    w.ns = it.ns, w.s0 = it.s0, w.n = it.n, w.tile = it.tile;
    w.a = q.a, w.nt = q.nt, w.n_s = sp.n_s, w.lo = sp.lo;
    w.row0 = it.g.t0 + q.tok0;
    w.z = p.paged ? 0 : it.rep / p.Hkv;
    w.hk = p.paged ? it.rep : it.rep % p.Hkv;
    w.seg = it.seg, w.rep = it.rep;
    w.zlo = window_low(it.g.kvlen - it.g.qlen, p.window);
    w.zhi = it.g.kvlen - 1;
    w.pad = 0;
    return w;
}

// bits [0, c) of 64
__device__ __forceinline__ unsigned long long below(int c) { return c >= 64 ? ~0ull : (1ull << c) - 1; }

// x[j] = -inf where bit j is clear
__device__ __forceinline__ void hide(float (&x)[64], unsigned long long vis) {
    const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> 32);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        x[j] = (v0 >> j) & 1 ? x[j] : -INFINITY;
        x[j + 32] = (v1 >> j) & 1 ? x[j + 32] : -INFINITY;
    }
}

// What a warp's rows, at positions first .. last, see of the 64 keys from kb:
// all of them, none, or (neither) the bits that row_keys gives each row.
// Comparisons of per-tile values: a vote over the rows' own bits, or branches
// here, put 400 cycles between a warp's steps (of 2300).
struct Seen {
    int first, last;  // positions of the warp's first and last live row
    __device__ __forceinline__ bool all(const Prob& p, int kb) const {
        return (first >= kb + 63) & ((last - p.window < kb) | (p.sinks >= kb + 64));
    }
    __device__ __forceinline__ bool none(const Prob& p, int kb) const {
        return (last < kb) | ((first - p.window >= kb + 63) & (p.sinks <= kb));
    }
};
// Visible keys of one row at position pos among the 64 that start at kb.
__device__ __forceinline__ unsigned long long row_keys(int pos, int low, int sinks, int kb) {
    const int hi = imin(imax(pos - kb + 1, 0), 64), lo = imin(imax(low - kb, 0), 64);
    const int sk = imin(imax(sinks - kb, 0), 64);
    return below(hi) & (~below(lo) | below(sk));
}

// 64 accumulator columns of a thread's row, scaled and rounded
template <typename T>
__device__ __forceinline__ void read_panel(uint32_t tacc, float scale, uint32_t (&pk)[32]) {
    uint32_t r[64];
    tmem_ld64_sync(tacc, tacc + 32, r);
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        const float2 v = __fmul2_rn(make_float2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])),
                                    make_float2(scale, scale));
        pk[k] = Pack2<T>::pack(v.x, v.y);
    }
}

// 64 columns of a warp's 32 rows (thread = row, two values per register) to
// memory through the warp's 4 KB staging panel (16-byte piece j of row r at
// j ^ (r % 8), so neither side meets a bank twice): 8 lanes then write 128
// contiguous bytes of a row.  dst(r): where row r's 64 columns begin, or null.
__device__ __forceinline__ void stage_panel(uint8_t* stage, const uint32_t (&pk)[32], int lane) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
            make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
    __syncwarp();
}
template <typename T, typename F>
__device__ __forceinline__ void store_panel(const uint8_t* stage, int lane, int cols, F dst) {
    const int j = lane & 7;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3);
        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((j ^ (r & 7)) << 4));
        T* p = dst(r);
        if (p && j * 8 < cols) *reinterpret_cast<uint4*>(p + j * 8) = v;
    }
}
// KP panels, one loop for all; `mask`: all ones, or 0 for a row of zeros
template <typename T, int KP, typename F>
__device__ __forceinline__ void store_panels(uint8_t* stage, const uint32_t (&pk)[KP][32], uint32_t mask, int lane, int D,
                                             F dst) {
#pragma unroll 1
    for (int c = 0; c < KP; ++c) {
        uint32_t x[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = (c == 0 ? pk[0][k] : pk[KP - 1][k]) & mask;
        stage_panel(stage, x, lane);
        store_panel<T>(stage, lane, D - c * 64, [&](int i) -> T* {
            T* p = dst(i);
            return p ? p + c * 64 : nullptr;
        });
    }
}

// Tensor maps of a call: rows of the query heads that share a KV head (box of
// G heads x tq tokens), and of keys (box of `rows` rows or slots).
inline int query_map(CUtensorMap* m, const View& v, const Call& c, int is_bf16, int64_t tokens, int tq) {
    const uint64_t n[3] = {(uint64_t)c.p.Hq, (uint64_t)tokens, (uint64_t)c.Z};
    const uint64_t s[3] = {(uint64_t)v.s[1], (uint64_t)v.s[2], (uint64_t)v.s[0]};
    return make_tmap_4d(m, v.ptr, is_bf16, c.D, n, s, c.p.G, tq);
}
inline int key_map(CUtensorMap* m, const View& v, const Call& c, int is_bf16, int rows) {
    const Prob& p = c.p;
    const uint64_t n[3] = {p.paged ? 1ull << p.page_shift : (uint64_t)imax(p.Sk, 1), (uint64_t)p.Hkv,
                           p.paged ? (uint64_t)p.n_pages : (uint64_t)c.Z};
    const uint64_t s[3] = {(uint64_t)v.s[2], (uint64_t)v.s[1], (uint64_t)v.s[0]};
    return make_tmap_4d(m, v.ptr, is_bf16, c.D, n, s, rows, 1);
}

// Launch preparation: the shared memory limit, and the register count that the
// split at kernel start divides: with any other the split would wait forever, so
// a library built that way gets an error.  Both belong to the kernel on a device,
// so one launch per device asks.
template <typename K>
int prepare_kernel(K kern, int smem, std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BSP_ERR_CUDA;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return BSP_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return BSP_ERR_CUDA;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return BSP_ERR_CUDA;
    if ((uint32_t)fa.numRegs != kRegsLaunch) return BSP_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_release);
    return BSP_OK;
}

}  // namespace win
}  // namespace bsp
