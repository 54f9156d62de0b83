// Small kernels around the windowed attention: joining the pieces of cut
// tiles, the rows' dO . O, and the append of new tokens' keys and values to
// the pages.
#include <type_traits>

#include "common.cuh"
#include "window.h"

namespace bsp {
namespace win {
namespace {

constexpr int kJoinT = 128;
constexpr int kJoinCols = 16;                    // columns of a block
constexpr int kJoinParts = kSlotD / kJoinCols;  // blocks per cut tile

// The slots of a cut tile's pieces, in order: every CTA among those that share
// the steps has one of at least one step.
__device__ __forceinline__ int piece_slot(int i) { return i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i); }

struct JoinArgs {
    const Cut* cuts;
    const float* slots;
    Prob p;
    View out, out2;
    float* lse;
    int64_t lz, lh, lt;
    int D, R;
    float scale;
};

// 16 columns of a row of a piece (MANY: of a tile of many rows)
template <bool MANY>
__device__ __forceinline__ void load_piece(const float* slot, int rows, int row, int col, bool on, float (&v)[kJoinCols]) {
    const float* at = slot + (MANY ? 4 * row + col * rows : kSlotD * row + col);
    const int step = MANY ? 4 * rows : 4;
#pragma unroll
    for (int k = 0; k < kJoinCols; k += 4) {
        const float4 x = on ? *reinterpret_cast<const float4*>(at + k / 4 * step) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[k] = x.x, v[k + 1] = x.y, v[k + 2] = x.z, v[k + 3] = x.w;
    }
}
template <typename T>
__device__ __forceinline__ void store_cols(T* dst, float (&v)[kJoinCols], float f) {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int k = 0; k < kJoinCols; k += N) {
        float x[N];
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = v[k + j] * f;
        Vec16<T>::store(dst + k, x);
    }
}

// The pieces of row r that a thread group adds up: group, group + np, ...
template <bool DQ, bool MANY>
__device__ __forceinline__ void add_pieces(const JoinArgs& a, int pieces, int group, int np, int r, int rows, int c0,
                                           float& m, float& l, float (&o)[kJoinCols]) {
    m = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinCols; ++k) o[k] = 0.f;
#pragma unroll 1
    for (int i0 = group; i0 < pieces; i0 += 4 * np) {
        float mi[4], li[4], v[4][kJoinCols];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * np;
            const bool on = r < rows && i < pieces;
            const float* slot = a.slots + piece_slot(on ? i : 0) * slot_floats(a.R);
            if (!DQ) {
                mi[j] = on ? slot[a.R * kSlotD + r] : -INFINITY;
                li[j] = on ? slot[a.R * kSlotD + a.R + r] : 0.f;
            }
            load_piece<MANY>(slot, rows, r, c0, on, v[j]);
        }
        if (DQ) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < kJoinCols; ++k) o[k] += v[j][k];
            continue;
        }
        const float mn = fmaxf(fmaxf(fmaxf(mi[0], mi[1]), fmaxf(mi[2], mi[3])), m);
        const float keep = m == -INFINITY ? 0.f : exp2f(m - mn);
        l *= keep;
#pragma unroll
        for (int k = 0; k < kJoinCols; ++k) o[k] *= keep;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float w = mi[j] == -INFINITY ? 0.f : exp2f(mi[j] - mn);
            l += w * li[j];
#pragma unroll
            for (int k = 0; k < kJoinCols; ++k)
                if (w != 0.f) o[k] = fmaf(w, v[j][k], o[k]);  // a piece that saw nothing may hold anything
        }
        m = mn;
    }
}

// Rows of cut query tiles.  Forward: the pieces' outputs are relative to each
// piece's own maximum m_i (in log2 units): with m = max m_i,
// o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.  dQ: their sum, scaled.
// The order of the sums is fixed, whoever wrote the pieces first.
//
// A thread holds 16 columns of a row and has four pieces on their way at once:
// bound by the latency of one read (a warp per row, piece after piece, four
// rows in turn took 11.4 us behind a launch with cut tiles of 128 rows; this 6.7).
// A tile of few rows (a new token's heads over a long history) has many pieces: groups
// of threads then take every np-th piece and add up in shared memory.
template <typename T, bool DQ>
__global__ void __launch_bounds__(kJoinT) join_kernel(const JoinArgs a) {
    cudaGridDependencySynchronize();
    const Cut cut = a.cuts[blockIdx.x];
    const int c0 = blockIdx.y * kJoinCols;
    if (cut.pieces == 0 || c0 >= a.D) return;
    const Prob& p = a.p;
    const Seg g = p.seg(cut.seg);
    const QTile q = p.qtile(g, cut.tile);
    const int z = p.paged ? 0 : cut.rep / p.Hkv, hk = p.paged ? cut.rep : cut.rep % p.Hkv;
    const int rows = imin(q.nt * p.G, kJoinT), tid = threadIdx.x;
    // a thread group is 2^wide >= rows threads
    const int wide = cut.pieces <= 4 ? 7 : rows <= 1 ? 0 : 32 - __clz(rows - 1);
    const int np = kJoinT >> wide, parts = imin(np, cut.pieces);
    const int r = tid & ((1 << wide) - 1), group = tid >> wide;
    float m = -INFINITY, l = 0.f, o[kJoinCols];
    // (with strides that are known only at run time, 31 tokens' join took 6.9 us, not 5)
    if (rows >= kManyRows) add_pieces<DQ, true>(a, cut.pieces, group, np, r, rows, c0, m, l, o);
    else add_pieces<DQ, false>(a, cut.pieces, group, np, r, rows, c0, m, l, o);
    auto place = [&](int row, int64_t* h, int64_t* t) {
        *h = (int64_t)hk * p.G + row % p.G;
        *t = (int64_t)g.t0 + q.tok0 + row / p.G;
    };
    auto out = [&](int64_t h, int64_t t) { return static_cast<T*>(a.out.ptr) + z * a.out.s[0] + h * a.out.s[1] + t * a.out.s[2] + c0; };
    auto put_lse = [&](int64_t h, int64_t t, float mx, float sum) {
        if (!DQ && a.lse && c0 == 0)
            a.lse[z * a.lz + h * a.lh + t * a.lt] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
    };
    int64_t h, t;
    if (np == 1) {
        if (r >= rows) return;
        place(r, &h, &t);
        store_cols(out(h, t), o, DQ ? a.scale : (l != 0.f ? 1.0f / l : 0.f));  // l may be no number
        put_lse(h, t, m, l);
        return;
    }
    __shared__ float part_m[kJoinT], part_l[kJoinT], part_o[kJoinCols][kJoinT + 1];
    part_m[tid] = m, part_l[tid] = l;
#pragma unroll
    for (int k = 0; k < kJoinCols; ++k) part_o[k][tid] = o[k];
    __syncthreads();
    for (int x = tid; x < rows * kJoinCols; x += kJoinT) {
        const int row = x / kJoinCols, k = x % kJoinCols;
        float mx = -INFINITY, sum = 0.f, y = 0.f;
        if (!DQ)
#pragma unroll 8
            for (int i = 0; i < parts; ++i) mx = fmaxf(mx, part_m[(i << wide) + row]);
#pragma unroll 8
        for (int i = 0; i < parts; ++i) {
            const int at = (i << wide) + row;
            const float w = DQ ? 1.f : (part_m[at] == -INFINITY ? 0.f : exp2f(part_m[at] - mx));
            sum += w * part_l[at];
            y += w * part_o[k][at];
        }
        place(row, &h, &t);
        out(h, t)[k] = from_f32<T>(y * (DQ ? a.scale : (sum != 0.f ? 1.0f / sum : 0.f)));
        if (k == 0) put_lse(h, t, mx, sum);
    }
}

// Keys of cut key tiles: dK (scaled) and dV as the sums of their pieces.  A
// thread holds 16 columns of a key's dK or dV.
template <typename T>
__global__ void __launch_bounds__(kJoinT) join_kv_kernel(const JoinArgs a, const KProb kp) {
    cudaGridDependencySynchronize();
    const Cut cut = a.cuts[blockIdx.x];
    const bool is_v = blockIdx.y >= kJoinParts;
    const int c0 = (blockIdx.y % kJoinParts) * kJoinCols;
    if (cut.pieces == 0 || c0 >= a.D) return;
    const int z = cut.rep / kp.Hkv, hk = cut.rep % kp.Hkv, r = threadIdx.x;
    const int kb = cut.tile << kp.kshift;
    if (r >= imin(a.R, kp.Sk - kb)) return;
    float o[kJoinCols];
#pragma unroll
    for (int k = 0; k < kJoinCols; ++k) o[k] = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < cut.pieces; i0 += 4) {
        float v[4][kJoinCols];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool on = i0 + j < cut.pieces;
            const float* slot = a.slots + piece_slot(on ? i0 + j : 0) * kv_slot_floats(a.R);
            load_piece<true>(slot + (is_v ? a.R * kSlotD : 0), a.R, r, c0, on, v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < kJoinCols; ++k) o[k] += v[j][k];
    }
    const View& out = is_v ? a.out2 : a.out;
    store_cols(static_cast<T*>(out.ptr) + z * out.s[0] + hk * out.s[1] + (int64_t)(kb + r) * out.s[2] + c0, o,
               is_v ? 1.0f : a.scale);
}

// Strides of the rows' log-sum-exp (and dO . O): batch entry, head, row.
struct RowStrides {
    int64_t z, h, t;
};

// delta = dO . O of the row, fp32, where the strides say: a group of 8 lanes per
// row, 16 bytes per lane and step.  Reads both tensors once: HBM-bound.
template <typename T>
__global__ void __launch_bounds__(256) delta_kernel(const View O, const View dO, float* delta, const RowStrides at,
                                                    int64_t rows, int Hq, int S, int D) {
    constexpr int N = Vec16<T>::N;
    const int sub = threadIdx.x & 7;
    for (int64_t r = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3); r < rows; r += (int64_t)gridDim.x * 32) {
        const int64_t t = r % S, zh = r / S, h = zh % Hq, z = zh / Hq;
        const T* o = static_cast<const T*>(O.ptr) + z * O.s[0] + h * O.s[1] + t * O.s[2];
        const T* g = static_cast<const T*>(dO.ptr) + z * dO.s[0] + h * dO.s[1] + t * dO.s[2];
        float x = 0.f;
        for (int c = sub * N; c < D; c += 8 * N) {
            float a[N], b[N];
            Vec16<T>::load(o + c, a);
            Vec16<T>::load(g + c, b);
#pragma unroll
            for (int k = 0; k < N; ++k) x = fmaf(a[k], b[k], x);
        }
        const unsigned group = 0xffu << (threadIdx.x & 24);  // the row's 8 lanes
#pragma unroll
        for (int k = 4; k; k >>= 1) x += __shfl_xor_sync(group, x, k);
        if (sub == 0) delta[z * at.z + h * at.h + t * at.t] = x;
    }
}

// Largest of x over the block's threads, in thread 0; scratch: 8 floats.
__device__ __forceinline__ float block_most(float x, float* scratch) {
#pragma unroll
    for (int k = 16; k; k >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    for (int k = 1; k < 8; ++k) x = fmaxf(x, scratch[k]);
    return x;
}

struct StatsArgs {
    View O, dO, V;
    const float* lse;
    RowStrides at;
    float* stats;
    RangePart* range;  // fp16
    int parts;         // fp16: blocks per (batch entry, KV head); else all
    int64_t rows;      // of each, in whole tiles; else all
    int ntiles, G, TQ, Hkv, S, D;
    int Sk, zlo, sinks;  // fp16: V rows below min(sinks, zlo) and from zlo on are seen
};

// dO . O per tile of kStatRows rows (row r: token r / G, head r % G, as the
// tensor-core kernels lay them out), and -lse log2(e), side by side, so that one
// bulk copy brings a tile's statistics.  Rows beyond the sequence get -inf: their
// P is then 0.  fp16 also looks for the longest rows of dO and V of each (batch
// entry, KV head); V rows that no query sees are left out, rows of no finite
// length too, since neither may move the factor of the others.
//
// O comes rounded to the call's type.  Rows that weigh few keys feel that in dO . O:
// errors of dQ and dK are 1.4 to 1.5 of the results' own rounding over windows of
// 32 keys or more (1.4 is dS's one rounding), 1.55 over 16, 1.8 over 4.  From P and
// dP it would take two more products over all key tiles, a third of the gradient.
template <typename T>
__global__ void __launch_bounds__(256) tile_stats_kernel(const __grid_constant__ StatsArgs a) {
    constexpr int N = Vec16<T>::N;
    constexpr bool kF16 = std::is_same<T, __half>::value;
    const int sub = threadIdx.x & 7;
    const unsigned group = 0xffu << (threadIdx.x & 24);  // the row's 8 lanes
    const int rep = kF16 ? blockIdx.x / a.parts : 0, part = kF16 ? blockIdx.x % a.parts : blockIdx.x;
    float o2 = 0.f;
    cudaGridDependencySynchronize();
    for (int64_t j = (int64_t)part * 32 + (threadIdx.x >> 3); j < a.rows; j += (int64_t)a.parts * 32) {
        const int64_t i = rep * a.rows + j;
        const int r = (int)(i % kStatRows);
        const int64_t tile = i / kStatRows, zh = tile / a.ntiles;
        const int z = (int)(zh / a.Hkv), t = (int)(tile % a.ntiles) * a.TQ + r / a.G;
        const int64_t h = zh % a.Hkv * a.G + r % a.G;
        const bool live = r < a.TQ * a.G && t < a.S;
        float x = 0.f, y = 0.f;
        if (live) {
            const T* o = static_cast<const T*>(a.O.ptr) + z * a.O.s[0] + h * a.O.s[1] + t * a.O.s[2];
            const T* g = static_cast<const T*>(a.dO.ptr) + z * a.dO.s[0] + h * a.dO.s[1] + t * a.dO.s[2];
            for (int c = sub * N; c < a.D; c += 8 * N) {
                float u[N], v[N];
                Vec16<T>::load(o + c, u);
                Vec16<T>::load(g + c, v);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    x = fmaf(u[k], v[k], x);
                    if (kF16) y = fmaf(v[k], v[k], y);
                }
            }
        }
#pragma unroll
        for (int k = 4; k; k >>= 1) {
            x += __shfl_xor_sync(group, x, k);
            if (kF16) y += __shfl_xor_sync(group, y, k);
        }
        if (y < INFINITY) o2 = fmaxf(o2, y);
        if (sub == 0) {
            const float l = live ? a.lse[z * a.at.z + h * a.at.h + t * a.at.t] : -INFINITY;
            float* s = a.stats + tile * kStatTile + r;
            if (kF16) s[kStatDot] = x;
            s[kStatLse] = l == -INFINITY ? -INFINITY : -l * kLog2e + (kF16 ? (float)kPUp : 0.f);
            s[kStatDelta] = kF16 ? 0.f : x;
        }
    }
    if constexpr (kF16) {
        float v2 = 0.f;
        const int z = rep / a.Hkv, hk = rep % a.Hkv, head = imin(a.sinks, a.zlo);
        for (int64_t j = (int64_t)part * 32 + (threadIdx.x >> 3); j < (int64_t)head + a.Sk - a.zlo; j += (int64_t)a.parts * 32) {
            const int64_t t = j < head ? j : j - head + a.zlo;
            const T* v = static_cast<const T*>(a.V.ptr) + z * a.V.s[0] + hk * a.V.s[1] + t * a.V.s[2];
            float y = 0.f;
            for (int c = sub * N; c < a.D; c += 8 * N) {
                float u[N];
                Vec16<T>::load(v + c, u);
#pragma unroll
                for (int k = 0; k < N; ++k) y = fmaf(u[k], u[k], y);
            }
#pragma unroll
            for (int k = 4; k; k >>= 1) y += __shfl_xor_sync(group, y, k);
            if (y < INFINITY) v2 = fmaxf(v2, y);
        }
        __shared__ float most[2][8];
        o2 = block_most(o2, most[0]);
        v2 = block_most(v2, most[1]);
        if (threadIdx.x == 0) a.range[blockIdx.x] = RangePart{o2, v2};
    }
}

// What the fp16 gradient scales dS by: a warp per (batch entry, KV head).
__global__ void __launch_bounds__(256) factor_kernel(const RangePart* range, int parts, DsFactor* factor, int rep) {
    const int lane = threadIdx.x & 31, r = blockIdx.x * 8 + (threadIdx.x >> 5);
    cudaGridDependencySynchronize();
    if (r >= rep) return;
    float o2 = 0.f, v2 = 0.f;
    for (int i = lane; i < parts; i += 32) {
        const RangePart x = range[(int64_t)r * parts + i];
        o2 = fmaxf(o2, x.dO2), v2 = fmaxf(v2, x.V2);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) {
        o2 = fmaxf(o2, __shfl_xor_sync(0xffffffffu, o2, k));
        v2 = fmaxf(v2, __shfl_xor_sync(0xffffffffu, v2, k));
    }
    const float most = 2.0f * sqrtf(o2) * sqrtf(v2);  // of |dP - delta|
    // most < 2^(e + 1): times 2^(14 - e) below 2^15
    const int e = most > 0.f ? ilogbf(most) : 14;
    if (lane == 0) factor[r] = DsFactor{scalbnf(1.0f, 14 - kPUp - e), scalbnf(1.0f, e - 14)};
}

// K and V rows of new tokens to their pages' slots: token t of sequence s goes
// to position kv_len[s] - (new tokens of s) + its index.  A warp per token, 16
// bytes per lane and copy.  Moves each byte once in and once out; the rows are
// on their way into registers while the warp finds the sequence (by a 32-way
// search of q_start), its length and its page, three dependent reads.
struct AppendArgs {
    View Kn, Vn, Kc, Vc;
    Prob p;
    int row16;  // 16-byte pieces per head row
};

constexpr int kAhead = 4;  // pieces of K and of V that a lane holds

__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendArgs a) {
    cudaGridDependencySynchronize();
    const Prob& p = a.p;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int s = threadIdx.x; s < p.nseg; s += blockDim.x)
            if (p.bad_seg(p.q_start[s], p.q_start[s + 1], p.kv_len[s])) set_status(p.status, BSP_ERR_DEVICE_CHECK);
    const int n = p.Hkv * a.row16, stride = gridDim.y * 32;  // gridDim.y blocks share a token's row
    for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < p.T; t += (int64_t)gridDim.x * 8) {
        uint4 k[kAhead], v[kAhead];
        auto fetch = [&](int first) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = first + j * stride, h = i / a.row16, c = i - h * a.row16;
                if (i < n) {
                    k[j] = static_cast<const uint4*>(a.Kn.ptr)[h * a.Kn.s[1] + t * a.Kn.s[2] + c];
                    v[j] = static_cast<const uint4*>(a.Vn.ptr)[h * a.Vn.s[1] + t * a.Vn.s[2] + c];
                }
            }
        };
        const int i0 = blockIdx.y * 32 + lane;
        fetch(i0);
        // last s in [0, nseg) with q_start[s] <= t: each round asks 32 places
        int lo = 0, hi = p.nseg;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int s = lo + lane * step;
            const bool le = s < hi && p.q_start[s] <= t;
            const unsigned m = __ballot_sync(0xffffffffu, le);
            if (m == 0) break;  // t lies before the first sequence
            const int last = 31 - __clz(m);
            const int nlo = lo + last * step;
            hi = imin(hi, nlo + step);
            lo = nlo;
        }
        const int q0 = p.q_start[lo], q1 = p.q_start[lo + 1], kv = p.kv_len[lo];
        if (p.bad_seg(q0, q1, kv) || t < q0 || t >= q1) continue;
        const int pos = kv - q1 + (int)t;
        if (pos < 0) continue;
        const int pg = p.table[(int64_t)lo * p.max_pages + (pos >> p.page_shift)];
        if ((unsigned)pg >= (unsigned)p.n_pages) {
            if (lane == 0) set_status(p.status, BSP_ERR_DEVICE_CHECK);
            continue;
        }
        const int slot = pos & ((1 << p.page_shift) - 1);
        uint4* kd = static_cast<uint4*>(a.Kc.ptr) + pg * a.Kc.s[0] + slot * a.Kc.s[2];
        uint4* vd = static_cast<uint4*>(a.Vc.ptr) + pg * a.Vc.s[0] + slot * a.Vc.s[2];
        for (int first = i0; first < n; first += kAhead * stride) {
            if (first != i0) fetch(first);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = first + j * stride, h = i / a.row16, c = i - h * a.row16;
                if (i < n) {
                    kd[h * a.Kc.s[1] + c] = k[j];
                    vd[h * a.Vc.s[1] + c] = v[j];
                }
            }
        }
    }
}

__global__ void take_status_kernel(int* status) { status[1] = atomicExch(status, 0); }

// zeros rows of row16 16-byte pieces of a strided tensor (strides in pieces)
__global__ void __launch_bounds__(256) zero_kernel(const View v, int64_t pieces, int64_t n1, int64_t n2, int row16) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
        const int64_t c = i % row16, r = i / row16, k = r % n2, jk = r / n2, j = jk % n1, z = jk / n1;
        static_cast<uint4*>(v.ptr)[z * v.s[0] + j * v.s[1] + k * v.s[2] + c] = make_uint4(0u, 0u, 0u, 0u);
    }
}

template <typename T>
int join_t(const JoinArgs& a, int n_cta, bool is_dq, cudaStream_t s) {
    return launch_behind(is_dq ? join_kernel<T, true> : join_kernel<T, false>, dim3(n_cta, kJoinParts), kJoinT, 0, s, a);
}

template <typename T>
int delta_t(const Call& c) {
    const int64_t rows = (int64_t)c.Z * c.p.Hq * c.p.Sq;
    const int64_t blocks = (rows + 31) / 32, most = (int64_t)sm_count() * 16;
    delta_kernel<T><<<(int)(blocks < most ? blocks : most), 256, 0, c.stream>>>(
        c.O, c.dO, c.stats, RowStrides{c.lz, c.lh, c.lt}, rows, c.p.Hq, c.p.Sq, c.D);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

template <typename T>
int tile_stats_t(const Call& c) {
    constexpr bool kF16 = std::is_same<T, __half>::value;
    const Prob& p = c.p;
    const int tq = kStatRows / p.G, ntiles = (p.Sq + tq - 1) / tq;
    const int64_t per = (int64_t)ntiles * kStatRows, most = (int64_t)sm_count() * 16;
    const int64_t rows = kF16 ? per : per * p.rep;  // of a part's share
    int64_t parts = (rows + 31) / 32;
    if (kF16) {
        parts = p.Sk / 32 > parts ? p.Sk / 32 : parts;  // V may have many more rows than Q
        parts = parts < range_parts(p.rep) ? parts : range_parts(p.rep);
    } else {
        parts = parts < most ? parts : most;
    }
    const StatsArgs a{c.O, c.dO, c.V, c.lse, RowStrides{c.lz, c.lh, c.lt}, c.stats, c.range, (int)parts, rows, ntiles,
                      p.G, tq, p.Hkv, p.Sq, c.D, p.Sk, window_low(p.Sk - p.Sq, p.window), p.sinks};
    const int64_t grid = kF16 ? parts * p.rep : parts;
    int rc = launch_behind(tile_stats_kernel<T>, dim3((uint32_t)grid), 256, 0, c.stream, a);
    if (kF16 && !rc)
        rc = launch_behind(factor_kernel, dim3((p.rep + 7) / 8), 256, 0, c.stream, (const RangePart*)c.range, (int)parts,
                           c.factor, p.rep);
    return rc;
}

View in_16(const View& v, int elt) {
    View r = v;
    for (int64_t& s : r.s) s = s * elt / 16;
    return r;
}

}  // namespace

#define BSP_WIN_TYPES(call_f32, call_bf16, call_f16) \
    switch (c.dtype) {                               \
        case BSP_F32: return call_f32;               \
        case BSP_BF16: return call_bf16;             \
        case BSP_F16: return call_f16;               \
        default: return BSP_ERR_INVALID_ARG;         \
    }

int launch_join(const Call& c, int rows, int n_cta, bool is_dq) {
    JoinArgs a{c.cuts, c.slots, c.p, is_dq ? c.dQ : c.O, View{}, c.lse, c.lz, c.lh, c.lt, c.D, rows, c.scale};
    BSP_WIN_TYPES(join_t<float>(a, n_cta, is_dq, c.stream), join_t<__nv_bfloat16>(a, n_cta, is_dq, c.stream),
                  join_t<__half>(a, n_cta, is_dq, c.stream))
}

int launch_join_kv(const Call& c, const KProb& kp, int rows, int n_cta) {
    JoinArgs a{c.cuts, c.slots, c.p, c.dK, c.dV, nullptr, 0, 0, 0, c.D, rows, c.scale};
    BSP_WIN_TYPES(launch_behind(join_kv_kernel<float>, dim3(n_cta, 2 * kJoinParts), kJoinT, 0, c.stream, a, kp),
                  launch_behind(join_kv_kernel<__nv_bfloat16>, dim3(n_cta, 2 * kJoinParts), kJoinT, 0, c.stream, a, kp),
                  launch_behind(join_kv_kernel<__half>, dim3(n_cta, 2 * kJoinParts), kJoinT, 0, c.stream, a, kp))
}

int launch_delta(const Call& c) { BSP_WIN_TYPES(delta_t<float>(c), delta_t<__nv_bfloat16>(c), delta_t<__half>(c)) }

int launch_tile_stats(const Call& c) {
    BSP_WIN_TYPES(BSP_ERR_UNSUPPORTED, tile_stats_t<__nv_bfloat16>(c), tile_stats_t<__half>(c))
}

int launch_take_status(const bsp_window_s* w, cudaStream_t s) {
    take_status_kernel<<<1, 1, 0, s>>>(w->status);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

int launch_zero(const View& v, int elt, int64_t n0, int64_t n1, int64_t n2, int row16, cudaStream_t s) {
    const int64_t pieces = n0 * n1 * n2 * row16, blocks = (pieces + 255) / 256, most = (int64_t)sm_count() * 8;
    if (pieces == 0) return BSP_OK;
    zero_kernel<<<(int)(blocks < most ? blocks : most), 256, 0, s>>>(in_16(v, elt), pieces, n1, n2, row16);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

int launch_append(const bsp_window_s* w, int dtype, const View& Kn, const View& Vn, const View& Kc, const View& Vc,
                  const Prob& p, int D, cudaStream_t s) {
    const int elt = dtype == BSP_F32 ? 4 : 2;
    AppendArgs a{in_16(Kn, elt), in_16(Vn, elt), in_16(Kc, elt), in_16(Vc, elt), p, D * elt / 16};
    // few tokens: several blocks copy one token's heads, so that a batch of
    // single tokens still spreads over the SMs (64 tokens: 3.3 us, 3.7 without)
    const int64_t blocks = ((int64_t)p.T + 7) / 8, most = (int64_t)sm_count() * 8;
    const int pieces = (p.Hkv * a.row16 + 31) / 32;
    const int share = imax(1, imin(pieces, (int)(sm_count() / blocks)));
    return launch_behind(append_kernel, dim3((int)(blocks < most ? blocks : most), share), 256, 0, s, a);
}

}  // namespace win
}  // namespace bsp
