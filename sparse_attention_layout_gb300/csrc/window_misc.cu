// Small kernels around the windowed attention: joining the pieces of cut
// tiles, the rows' dO . O, and the append of new tokens' keys and values to
// the pages.
#include "common.cuh"
#include "window.h"

namespace bsp {
namespace win {
namespace {

constexpr int kJoinParts = 8;  // blocks per cut tile, each an eighth of its rows
constexpr int kJoinT = 128;    // a warp per row, four columns per lane

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

// Rows of cut query tiles.  Forward: the pieces' outputs are relative to each
// piece's own maximum m_i (in log2 units): with m = max m_i,
// o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.  dQ: their sum, scaled.
// The order of the sums is fixed, whoever wrote the pieces first.
//
// A tile of many rows has few pieces: a warp per row.  A tile of many pieces
// (a long history under a small batch) has few rows: the block's warps share a
// row, each every fourth piece, and add up in shared memory (16000 keys, one
// token, 38 pieces: a warp alone spent 12 us of the call's 30 on its reads).
template <typename T, bool DQ>
__global__ void __launch_bounds__(kJoinT) join_kernel(const JoinArgs a) {
    cudaGridDependencySynchronize();
    constexpr int NW = kJoinT / 32;
    const Cut cut = a.cuts[blockIdx.x];
    if (cut.pieces == 0) return;
    const Prob& p = a.p;
    const Seg g = p.seg(cut.seg);
    const QTile q = p.qtile(g, cut.tile);
    const int z = p.paged ? 0 : cut.rep / p.Hkv, hk = p.paged ? cut.rep : cut.rep % p.Hkv;
    const int rows = q.nt * p.G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool shared_row = cut.pieces > 4;
    const int first = shared_row ? 0 : warp, per = shared_row ? 1 : NW;  // rows of a block at a time
    __shared__ float part_m[NW], part_l[NW];
    __shared__ float4 part_o[NW][32];
    for (int r = blockIdx.y * per + first; r < rows; r += kJoinParts * per) {
        const size_t row = (size_t)r * kSlotD + 4 * lane, ms = (size_t)a.R * kSlotD + r;
        const int i0 = shared_row ? warp : 0, step = shared_row ? NW : 1;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float m = -INFINITY, l = 0.f;
        if (!DQ) {
            // maxima of this warp's pieces, a lane each
            for (int i = i0 + lane * step; i < cut.pieces; i += 32 * step)
                m = fmaxf(m, a.slots[piece_slot(i) * slot_floats(a.R) + ms]);
#pragma unroll
            for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        }
#pragma unroll 4
        for (int i = i0; i < cut.pieces; i += step) {
            const float* sl = a.slots + piece_slot(i) * slot_floats(a.R);
            float w = 1.f;
            if (!DQ) {
                const float mi = sl[ms];
                w = mi == -INFINITY ? 0.f : exp2f(mi - m);
                l += w * sl[ms + a.R];
            }
            if (4 * lane < a.D && w != 0.f) {  // a piece that saw nothing may hold anything
                const float4 v = *reinterpret_cast<const float4*>(sl + row);
                o.x += w * v.x, o.y += w * v.y, o.z += w * v.z, o.w += w * v.w;
            }
        }
        if (shared_row) {
            __syncthreads();  // the last row's parts have been read
            part_o[warp][lane] = o;
            if (lane == 0) part_m[warp] = m, part_l[warp] = l;
            __syncthreads();
            if (warp) continue;
            o = make_float4(0.f, 0.f, 0.f, 0.f);
            l = 0.f;
            m = -INFINITY;
            if (!DQ)
                for (int k = 0; k < NW; ++k) m = fmaxf(m, part_m[k]);
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const float w = DQ ? 1.f : (part_m[k] == -INFINITY ? 0.f : exp2f(part_m[k] - m));
                const float4 v = part_o[k][lane];
                l += w * part_l[k];
                o.x += w * v.x, o.y += w * v.y, o.z += w * v.z, o.w += w * v.w;
            }
        }
        const float f = DQ ? a.scale : (l != 0.f ? 1.0f / l : 0.f);  // l may be no number
        const int64_t h = (int64_t)hk * p.G + r % p.G, t = (int64_t)g.t0 + q.tok0 + r / p.G;
        if (4 * lane < a.D) {
            T* dst = static_cast<T*>(a.out.ptr) + z * a.out.s[0] + h * a.out.s[1] + t * a.out.s[2] + 4 * lane;
            dst[0] = from_f32<T>(o.x * f), dst[1] = from_f32<T>(o.y * f);
            dst[2] = from_f32<T>(o.z * f), dst[3] = from_f32<T>(o.w * f);
        }
        if (!DQ && a.lse && lane == 0)
            a.lse[z * a.lz + h * a.lh + t * a.lt] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
}

// Keys of cut key tiles: dK (scaled) and dV as the sums of their pieces.
template <typename T>
__global__ void __launch_bounds__(kJoinT) join_kv_kernel(const JoinArgs a, const KProb kp) {
    cudaGridDependencySynchronize();
    const Cut cut = a.cuts[blockIdx.x];
    if (cut.pieces == 0) return;
    const int z = cut.rep / kp.Hkv, hk = cut.rep % kp.Hkv, lane = threadIdx.x & 31;
    const int kb = cut.tile << kp.kshift, rows = imin(a.R, kp.Sk - kb);
    if (4 * lane >= a.D) return;
    for (int r = blockIdx.y * (kJoinT / 32) + (threadIdx.x >> 5); r < rows; r += kJoinParts * (kJoinT / 32)) {
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
#pragma unroll 4
        for (int i = 0; i < cut.pieces; ++i) {
            const float* sl = a.slots + piece_slot(i) * kv_slot_floats(a.R) + 4 * lane;
            const float4 x = *reinterpret_cast<const float4*>(sl + (size_t)r * kSlotD);
            const float4 y = *reinterpret_cast<const float4*>(sl + (size_t)(a.R + r) * kSlotD);
            k.x += x.x, k.y += x.y, k.z += x.z, k.w += x.w;
            v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
        }
        const int64_t j = kb + r;
        T* dk = static_cast<T*>(a.out.ptr) + z * a.out.s[0] + hk * a.out.s[1] + j * a.out.s[2] + 4 * lane;
        T* dv = static_cast<T*>(a.out2.ptr) + z * a.out2.s[0] + hk * a.out2.s[1] + j * a.out2.s[2] + 4 * lane;
        dk[0] = from_f32<T>(k.x * a.scale), dk[1] = from_f32<T>(k.y * a.scale);
        dk[2] = from_f32<T>(k.z * a.scale), dk[3] = from_f32<T>(k.w * a.scale);
        dv[0] = from_f32<T>(v.x), dv[1] = from_f32<T>(v.y), dv[2] = from_f32<T>(v.z), dv[3] = from_f32<T>(v.w);
    }
}

// delta[z][h][t] = dO . O of the row, fp32: a group of 8 lanes per row, 16
// bytes per lane and step.  Reads both tensors once: HBM-bound.
template <typename T>
__global__ void __launch_bounds__(256) delta_kernel(const View O, const View dO, float* delta, int64_t rows, int Hq, int S,
                                                    int D) {
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
        if (sub == 0) delta[r] = x;
    }
}

// The same per tile of kStatRows rows (row r: token r / G, head r % G, as the
// tensor-core kernels lay them out): tile i's values of -lse log2(e), then of
// dO . O, so that one bulk copy brings a tile's statistics.  Rows beyond the
// sequence and rows that see nothing get -inf: their P is then 0.
template <typename T>
__global__ void __launch_bounds__(256) tile_stats_kernel(const View O, const View dO, const float* lse, float* stats,
                                                         int64_t rows, int ntiles, int G, int TQ, int Hkv, int S, int D) {
    constexpr int N = Vec16<T>::N;
    const int sub = threadIdx.x & 7;
    cudaGridDependencySynchronize();
    for (int64_t i = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3); i < rows; i += (int64_t)gridDim.x * 32) {
        const int r = (int)(i % kStatRows);
        const int64_t tile = i / kStatRows, zh = tile / ntiles;
        const int z = (int)(zh / Hkv), t = (int)(tile % ntiles) * TQ + r / G;
        const int64_t h = zh % Hkv * G + r % G;
        const bool live = r < TQ * G && t < S;
        float x = 0.f;
        if (live) {
            const T* o = static_cast<const T*>(O.ptr) + z * O.s[0] + h * O.s[1] + t * O.s[2];
            const T* g = static_cast<const T*>(dO.ptr) + z * dO.s[0] + h * dO.s[1] + t * dO.s[2];
            for (int c = sub * N; c < D; c += 8 * N) {
                float a[N], b[N];
                Vec16<T>::load(o + c, a);
                Vec16<T>::load(g + c, b);
#pragma unroll
                for (int k = 0; k < N; ++k) x = fmaf(a[k], b[k], x);
            }
        }
        const unsigned group = 0xffu << (threadIdx.x & 24);  // the row's 8 lanes
#pragma unroll
        for (int k = 4; k; k >>= 1) x += __shfl_xor_sync(group, x, k);
        if (sub == 0) {
            const float l = live ? lse[(z * (int64_t)Hkv * G + h) * S + t] : -INFINITY;
            stats[tile * 2 * kStatRows + r] = l == -INFINITY ? -INFINITY : -l * kLog2e;
            stats[tile * 2 * kStatRows + kStatRows + r] = x;
        }
    }
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

template <typename T>
int join_t(const JoinArgs& a, int n_cta, bool is_dq, cudaStream_t s) {
    return launch_behind(is_dq ? join_kernel<T, true> : join_kernel<T, false>, dim3(n_cta, kJoinParts), kJoinT, 0, s, a);
}

template <typename T>
int delta_t(const Call& c) {
    const int64_t rows = (int64_t)c.Z * c.p.Hq * c.p.Sq;
    const int64_t blocks = (rows + 31) / 32, most = (int64_t)sm_count() * 16;
    delta_kernel<T><<<(int)(blocks < most ? blocks : most), 256, 0, c.stream>>>(c.O, c.dO, c.stats, rows, c.p.Hq, c.p.Sq,
                                                                                 c.D);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

template <typename T>
int tile_stats_t(const Call& c) {
    const int tq = kStatRows / c.p.G, ntiles = (c.p.Sq + tq - 1) / tq;
    const int64_t rows = (int64_t)c.Z * c.p.Hkv * ntiles * kStatRows;
    const int64_t blocks = (rows + 31) / 32, most = (int64_t)sm_count() * 16;
    return launch_behind(tile_stats_kernel<T>, dim3((int)(blocks < most ? blocks : most)), 256, 0, c.stream, c.O, c.dO,
                         (const float*)c.lse, c.stats, rows, ntiles, c.p.G, tq, c.p.Hkv, c.p.Sq, c.D);
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
    BSP_WIN_TYPES(launch_behind(join_kv_kernel<float>, dim3(n_cta, kJoinParts), kJoinT, 0, c.stream, a, kp),
                  launch_behind(join_kv_kernel<__nv_bfloat16>, dim3(n_cta, kJoinParts), kJoinT, 0, c.stream, a, kp),
                  launch_behind(join_kv_kernel<__half>, dim3(n_cta, kJoinParts), kJoinT, 0, c.stream, a, kp))
}

int launch_delta(const Call& c) { BSP_WIN_TYPES(delta_t<float>(c), delta_t<__nv_bfloat16>(c), delta_t<__half>(c)) }

int launch_tile_stats(const Call& c) {
    BSP_WIN_TYPES(BSP_ERR_UNSUPPORTED, tile_stats_t<__nv_bfloat16>(c), tile_stats_t<__half>(c))
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
