// Windowed attention on the CUDA cores (fp32 products and sums): forward over
// dense tensors or pages, and the gradient.  It serves fp32, whose accuracy
// 16-bit tensor-core operands would lose, and every type when
// BSP_FORCE_SIMT=1.
//
// Tiles of 64 query rows x 64 keys, 256 threads; a thread holds a 4 x 4 patch
// of scores (rows ty + 16 u, keys tx + 16 v) and 4 rows x D / 16 columns of the
// output.  Shared-memory rows are padded by 4 floats, so the float4 reads of 16
// neighbouring rows meet no bank twice.  fp32 tiles are copied asynchronously,
// each as soon as the product that read its place is done, so that one product
// or the softmax covers every copy (24 heads of 4096 tokens, D 64, window 512:
// forward 494 -> 437 us, gradient 1585 -> 1425; pages of 32 sequences of 2000
// keys, D 128: 443 -> 268).
//
// Bound by shared memory: per four steps of the contraction a thread reads 8
// float4 for 64 multiply-adds, three wavefronts a read: the pipe is 73..78 %
// busy, that of the multiply-adds 54 %.  4 x 8 patches read less (0.19 float4 a
// pair of multiply-adds, not 0.25) but leave 8 warps an SM, and take as long
// (435 and 1510 us; D 128: 997 and 3740 for 914 and 3039); 8 x 8 spill.
#include <type_traits>

#include "common.cuh"
#include "window.h"

namespace bsp {
namespace win {
namespace {

__device__ float4 kNothing[1];  // where copies of no row point

constexpr int kT = 256;
constexpr int R = kSimtRows;      // query rows, and keys, per tile
constexpr int kShift = 6;
constexpr int PP = R + 4;         // pitch of P

struct Args {
    Prob p;
    View Q, K, V, O, dO, dQ, dK, dV;
    float* lse;
    int64_t lz, lh, lt;
    const float* delta;
    int D;
    float scale, c2;  // c2 = scale * log2(e)
    Cut* cuts;
    float* slots;
};

struct Where {  // a segment repetition's batch entry and KV head
    int z, hk;
};
__device__ __forceinline__ Where where(const Prob& p, int rep) {
    if (p.paged) return Where{0, rep};
    return Where{rep / p.Hkv, rep % p.Hkv};
}

template <typename T>
__device__ __forceinline__ T* at(const View& v, int64_t i, int64_t j, int64_t k) {
    return static_cast<T*>(v.ptr) + i * v.s[0] + j * v.s[1] + k * v.s[2];
}

// 64 rows of `DP` columns into shared memory (pitch DP + 4); row r from
// rowptr(r), or zeros where that is null.  fp32 rows are copied behind the
// thread's back: landed() and a barrier make them visible.
template <typename T, int DP, typename F>
__device__ __forceinline__ void load_tile(float* dst, int D, F rowptr) {
    constexpr int N = Vec16<T>::N, C = DP / N;
#pragma unroll 4
    for (int i = threadIdx.x; i < R * C; i += kT) {
        const int r = i / C, c = (i % C) * N;
        const T* src = rowptr(r);
        const bool live = src && c < D;
        float* to = dst + r * (DP + 4) + c;
        if constexpr (std::is_same<T, float>::value) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
                         "l"(live ? src + c : reinterpret_cast<const T*>(kNothing)), "r"(live ? 16 : 0)
                         : "memory");
        } else {
            float v[N];
            if (live) {
                Vec16<T>::load(src + c, v);
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < N; k += 4)
                *reinterpret_cast<float4*>(to + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        }
    }
}
// ends a group of copies; waits until all but the last n groups have landed
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void landed() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// s[u][v] = sum_d A[ty + 16 u][d] B[tx + 16 v][d]
template <int DP>
__device__ __forceinline__ void dots(const float* A, const float* B, int ty, int tx, float (&s)[4][4]) {
    float2 acc[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) a[u] = *reinterpret_cast<const float4*>(A + (ty + 16 * u) * (DP + 4) + d);
#pragma unroll
        for (int v = 0; v < 4; ++v) b[v] = *reinterpret_cast<const float4*>(B + (tx + 16 * v) * (DP + 4) + d);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                acc[u][v] = __ffma2_rn(make_float2(a[u].x, a[u].y), make_float2(b[v].x, b[v].y), acc[u][v]);
                acc[u][v] = __ffma2_rn(make_float2(a[u].z, a[u].w), make_float2(b[v].z, b[v].w), acc[u][v]);
            }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) s[u][v] = acc[u][v].x + acc[u][v].y;
}

// acc[u][g] (columns 64 g + 4 tx ..) += sum_k P[ty + 16 u][k] B[k][..]
template <int DP>
__device__ __forceinline__ void accumulate(const float* P, const float* B, int ty, int tx,
                                           float2 (&acc)[4][DP / 64][2]) {
    constexpr int NG = DP / 64;
#pragma unroll 2
    for (int k4 = 0; k4 < R; k4 += 4) {
        float4 pa[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) pa[u] = *reinterpret_cast<const float4*>(P + (ty + 16 * u) * PP + k4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float4 b[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g)
                b[g] = *reinterpret_cast<const float4*>(B + (k4 + k) * (DP + 4) + 64 * g + 4 * tx);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float w = k == 0 ? pa[u].x : k == 1 ? pa[u].y : k == 2 ? pa[u].z : pa[u].w;
                const float2 ww = make_float2(w, w);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    acc[u][g][0] = __ffma2_rn(ww, make_float2(b[g].x, b[g].y), acc[u][g][0]);
                    acc[u][g][1] = __ffma2_rn(ww, make_float2(b[g].z, b[g].w), acc[u][g][1]);
                }
            }
        }
    }
}

// sums over the 16 threads (tx) of a row
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
    for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ bool visible(int p, int j, const Prob& P) {
    return j <= p && (p - j < P.window || j < P.sinks);
}

template <typename T>
__device__ __forceinline__ void store4(T* dst, float a, float b, float c, float d) {
    dst[0] = from_f32<T>(a);
    dst[1] = from_f32<T>(b);
    dst[2] = from_f32<T>(c);
    dst[3] = from_f32<T>(d);
}

// Sequences with impossible lengths count as empty; one CTA reports them.
__device__ __forceinline__ void report_bad_segs(const Prob& p) {
    if (!p.paged || blockIdx.x) return;
    for (int s = threadIdx.x; s < p.nseg; s += blockDim.x)
        if (p.bad_seg(p.q_start[s], p.q_start[s + 1], p.kv_len[s])) set_status(p.status, BSP_ERR_DEVICE_CHECK);
}

template <typename T, int DP, bool PAGED>
__global__ void __launch_bounds__(kT, DP == 64 ? 2 : 1) forward_kernel(const __grid_constant__ Args A,
                                                     const __grid_constant__ SimtPlan plan) {
    constexpr int NG = DP / 64, PITCH = DP + 4;
    extern __shared__ float sm[];
    float *Qs = sm, *Ks = Qs + R * PITCH, *Vs = Ks + R * PITCH, *Ps = Vs + R * PITCH;
    __shared__ Start start;
    __shared__ uint32_t red[32];
    __shared__ int pages[2][R];  // page of each key's slot, of this step and the next
    const Prob& p = A.p;
    report_bad_segs(p);
    if constexpr (PAGED) locate<kT>(p, 1, reinterpret_cast<int*>(sm), red, &start);
    if (threadIdx.x == 0) A.cuts[blockIdx.x].pieces = 0;
    __syncthreads();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    Walk<Prob, PAGED ? kRagged : kDense> walk(p, PAGED ? start.tab : plan.tab, PAGED ? start.cta : plan.s[blockIdx.x]);
    Item it;
    while (walk.next(it)) {
        const Where w = where(p, it.rep);
        const QTile q = p.qtile(it.g, it.tile);
        const Span sp = p.span(q);
        const int lo = window_low(q.a, p.window);
        const int rows = q.nt * p.G;
        __syncthreads();
        load_tile<T, DP>(Qs, A.D, [&](int r) -> const T* {
            if (r >= rows) return nullptr;
            return at<const T>(A.Q, w.z, (int64_t)w.hk * p.G + r % p.G, (int64_t)it.g.t0 + q.tok0 + r / p.G);
        });
        float m[4], l[4];
        int pos[4];
        float2 acc[4][NG][2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = ty + 16 * u;
            pos[u] = r < rows ? q.a + r / p.G : -1;  // dead rows see nothing
            m[u] = -INFINITY;
            l[u] = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) acc[u][g][0] = acc[u][g][1] = make_float2(0.f, 0.f);
        }
        // keys that some row of the tile sees; the others (behind the sequence,
        // before every row's window) are not read at all
        auto wanted = [&](int j) { return j <= q.b && (j >= lo || j < p.sinks); };
        auto first_key = [&](int n) { return sp.tile(it.s0 + n) << kShift; };
        auto find_pages = [&](int n) {  // by the barrier before the step's copies
            if (!PAGED || threadIdx.x >= R || n >= it.ns) return;
            const int j = first_key(n) + threadIdx.x;
            int pg = -1;
            if (wanted(j)) {
                pg = p.table[(int64_t)it.seg * p.max_pages + (j >> p.page_shift)];
                if ((unsigned)pg >= (unsigned)p.n_pages) {
                    set_status(p.status, BSP_ERR_DEVICE_CHECK);
                    pg = -1;
                }
            }
            pages[n & 1][threadIdx.x] = pg;
        };
        auto copy = [&](float* dst, const View& v, int n) {
            const int kb = first_key(n);
            if (n < it.ns)
                load_tile<T, DP>(dst, A.D, [&](int r) -> const T* {
                    const int j = kb + r;
                    if (PAGED) {
                        const int pg = pages[n & 1][r];
                        return pg < 0 ? nullptr : at<const T>(v, pg, w.hk, j & ((1 << p.page_shift) - 1));
                    }
                    return wanted(j) ? at<const T>(v, w.z, w.hk, j) : nullptr;
                });
            copies_end();
        };
        find_pages(0);
        if (PAGED) __syncthreads();
        copy(Ks, A.K, 0);
        copy(Vs, A.V, 0);
        // K's next tile is on its way from the scores on, V's from the product on
        for (int n = 0; n < it.ns; ++n) {
            const int kb = first_key(n);
            find_pages(n + 1);
            landed<1>();
            __syncthreads();
            float s[4][4];
            dots<DP>(Qs, Ks, ty, tx, s);
            __syncthreads();
            copy(Ks, A.K, n + 1);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float cm = -INFINITY;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    s[u][v] = visible(pos[u], kb + tx + 16 * v, p) ? s[u][v] * A.c2 : -INFINITY;
                    cm = fmaxf(cm, s[u][v]);
                }
                cm = row_max(cm);
                const float mn = fmaxf(m[u], cm);
                const float ms = mn == -INFINITY ? 0.f : mn;
                const float alpha = m[u] == -INFINITY ? 0.f : exp2f(m[u] - ms);
                float rs = 0.f;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    s[u][v] = exp2f(s[u][v] - ms);
                    rs += s[u][v];
                    Ps[(ty + 16 * u) * PP + tx + 16 * v] = s[u][v];
                }
                l[u] = l[u] * alpha + row_sum(rs);
                m[u] = mn;
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int c = 0; c < 2; ++c) acc[u][g][c] = __fmul2_rn(acc[u][g][c], make_float2(alpha, alpha));
            }
            landed<1>();
            __syncthreads();
            accumulate<DP>(Ps, Vs, ty, tx, acc);
            __syncthreads();
            copy(Vs, A.V, n + 1);
        }
        float* slot = A.slots + (size_t)it.slot() * slot_floats(R);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = ty + 16 * u;
            if (r >= rows) continue;
            if (!it.whole()) {
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    *reinterpret_cast<float4*>(slot + SlotRows(rows).at(r, 64 * g + 4 * tx)) =
                        make_float4(acc[u][g][0].x, acc[u][g][0].y, acc[u][g][1].x, acc[u][g][1].y);
                if (tx == 0) {
                    slot[R * kSlotD + r] = m[u];
                    slot[R * kSlotD + R + r] = l[u];
                }
                continue;
            }
            const int h = w.hk * p.G + r % p.G, t = it.g.t0 + q.tok0 + r / p.G;
            const float inv = l[u] != 0.f ? 1.0f / l[u] : 0.f;  // l may be no number
            T* dst = at<T>(A.O, w.z, h, t);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int c = 64 * g + 4 * tx;
                if (c < A.D)
                    store4(dst + c, acc[u][g][0].x * inv, acc[u][g][0].y * inv, acc[u][g][1].x * inv, acc[u][g][1].y * inv);
            }
            if (A.lse && tx == 0)
                A.lse[w.z * A.lz + h * A.lh + t * A.lt] = l[u] != 0.f ? (m[u] + log2f(l[u])) * kLn2 : -INFINITY;
        }
        if (threadIdx.x == 0 && it.s0 == 0 && !it.whole())
            write_cut(A.cuts, it.seg, it.rep, it.tile, it.n - it.ns,
                      [&](int c) { return PAGED ? start.shares.of(c) : plan.s[c].count; });
    }
}

// dQ = scale dS K with dS = P (dO V^T - delta), P = exp(scale Q K^T - lse)
template <typename T, int DP>
__global__ void __launch_bounds__(kT, DP == 64 ? 2 : 1) dq_kernel(const __grid_constant__ Args A, const __grid_constant__ SimtPlan plan) {
    constexpr int NG = DP / 64, PITCH = DP + 4;
    extern __shared__ float sm[];
    float *Qs = sm, *Gs = Qs + R * PITCH, *Ks = Gs + R * PITCH, *Vs = Ks + R * PITCH, *Ps = Vs + R * PITCH;
    const Prob& p = A.p;
    if (threadIdx.x == 0) A.cuts[blockIdx.x].pieces = 0;
    __syncthreads();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    Walk<Prob, kDense> walk(p, plan.tab, plan.s[blockIdx.x]);
    Item it;
    while (walk.next(it)) {
        const Where w = where(p, it.rep);
        const QTile q = p.qtile(it.g, it.tile);
        const Span sp = p.span(q);
        const int lo = window_low(q.a, p.window);
        const int rows = q.nt * p.G;
        __syncthreads();
        auto qrow = [&](const View& v, int r) -> const T* {
            return r < rows ? at<const T>(v, w.z, (int64_t)w.hk * p.G + r % p.G, q.tok0 + r / p.G) : nullptr;
        };
        load_tile<T, DP>(Qs, A.D, [&](int r) { return qrow(A.Q, r); });
        load_tile<T, DP>(Gs, A.D, [&](int r) { return qrow(A.dO, r); });
        float lse2[4], dl[4];
        int pos[4];
        float2 acc[4][NG][2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = ty + 16 * u;
            pos[u] = -1;
            lse2[u] = INFINITY;  // P = 0
            dl[u] = 0.f;
            if (r < rows) {
                const int64_t o = w.z * A.lz + (w.hk * p.G + r % p.G) * A.lh + (q.tok0 + r / p.G) * A.lt;
                pos[u] = q.a + r / p.G;
                const float x = A.lse[o];
                lse2[u] = x == -INFINITY ? INFINITY : x * kLog2e;
                dl[u] = A.delta[o];
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) acc[u][g][0] = acc[u][g][1] = make_float2(0.f, 0.f);
        }
        auto first_key = [&](int n) { return sp.tile(it.s0 + n) << kShift; };
        auto copy = [&](float* dst, const View& v, int n) {
            const int kb = first_key(n);
            if (n < it.ns)
                load_tile<T, DP>(dst, A.D, [&](int r) -> const T* {
                    const int j = kb + r;
                    return j <= q.b && (j >= lo || j < p.sinks) ? at<const T>(v, w.z, w.hk, j) : nullptr;
                });
            copies_end();
        };
        copy(Vs, A.V, 0);
        copy(Ks, A.K, 0);
        // V's next tile is on its way from dP on, K's from the product on
        for (int n = 0; n < it.ns; ++n) {
            const int kb = first_key(n);
            float s[4][4], d[4][4];
            landed<1>();
            __syncthreads();
            dots<DP>(Gs, Vs, ty, tx, d);
            landed<0>();
            __syncthreads();
            copy(Vs, A.V, n + 1);
            dots<DP>(Qs, Ks, ty, tx, s);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const bool vis = visible(pos[u], kb + tx + 16 * v, p);
                    const float e = exp2f(s[u][v] * A.c2 - lse2[u]);
                    Ps[(ty + 16 * u) * PP + tx + 16 * v] = vis ? e * (d[u][v] - dl[u]) : 0.f;
                }
            __syncwarp();  // a warp's rows of dS are its own
            accumulate<DP>(Ps, Ks, ty, tx, acc);
            __syncthreads();
            copy(Ks, A.K, n + 1);
        }
        float* slot = A.slots + (size_t)it.slot() * slot_floats(R);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = ty + 16 * u;
            if (r >= rows) continue;
            T* dst = at<T>(A.dQ, w.z, (int64_t)w.hk * p.G + r % p.G, q.tok0 + r / p.G);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int c = 64 * g + 4 * tx;
                const float2 a = acc[u][g][0], b = acc[u][g][1];
                if (!it.whole())
                    *reinterpret_cast<float4*>(slot + SlotRows(rows).at(r, c)) = make_float4(a.x, a.y, b.x, b.y);
                else if (c < A.D)
                    store4(dst + c, a.x * A.scale, a.y * A.scale, b.x * A.scale, b.y * A.scale);
            }
        }
        if (threadIdx.x == 0 && it.s0 == 0 && !it.whole())
            write_cut(A.cuts, it.seg, it.rep, it.tile, it.n - it.ns, [&](int c) { return plan.s[c].count; });
    }
}

// dV = P^T dO, dK = scale dS^T Q per key tile, over the query tiles that see
// it and the heads that share it
template <typename T, int DP>
__global__ void __launch_bounds__(kT, DP == 64 ? 2 : 1) dkv_kernel(const __grid_constant__ Args A, const __grid_constant__ KProb kp,
                                                 const __grid_constant__ SimtPlan plan) {
    constexpr int NG = DP / 64, PITCH = DP + 4;
    extern __shared__ float sm[];
    float *Qs = sm, *Gs = Qs + R * PITCH, *Ks = Gs + R * PITCH, *Vs = Ks + R * PITCH;
    float *Ps = Vs + R * PITCH, *Ds = Ps + R * PP;  // P and dS, [key][row]
    __shared__ float lse_s[R], del_s[R];
    const Prob& p = A.p;
    if (threadIdx.x == 0) A.cuts[blockIdx.x].pieces = 0;
    __syncthreads();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    Walk<KProb, kDense> walk(kp, plan.tab, plan.s[blockIdx.x]);
    Item it;
    while (walk.next(it)) {
        const Where w = where(p, it.rep);
        const int kb = it.tile << kShift;
        int first, nq;
        kp.qrange(it.tile, &first, &nq);
        __syncthreads();
        auto keyrow = [&](const View& v, int r) -> const T* {
            return kb + r < p.Sk ? at<const T>(v, w.z, w.hk, kb + r) : nullptr;
        };
        load_tile<T, DP>(Ks, A.D, [&](int r) { return keyrow(A.K, r); });
        load_tile<T, DP>(Vs, A.D, [&](int r) { return keyrow(A.V, r); });
        float2 ak[4][NG][2], av[4][NG][2];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int g = 0; g < NG; ++g)
                ak[u][g][0] = ak[u][g][1] = av[u][g][0] = av[u][g][1] = make_float2(0.f, 0.f);
        auto qtile = [&](int n) { return p.qtile(Seg{0, p.Sq, p.Sk, 0}, first + it.s0 + n); };
        auto copy = [&](float* dst, const View& v, int n) {
            const QTile q = qtile(n);
            const int rows = q.nt * p.G;
            if (n < it.ns)
                load_tile<T, DP>(dst, A.D, [&](int r) -> const T* {
                    return r < rows ? at<const T>(v, w.z, (int64_t)w.hk * p.G + r % p.G, q.tok0 + r / p.G) : nullptr;
                });
            copies_end();
        };
        copy(Gs, A.dO, 0);
        copy(Qs, A.Q, 0);
        // dO's next tile is on its way from dV's product on, Q's from dK's on
        for (int n = 0; n < it.ns; ++n) {
            const QTile q = qtile(n);
            const int rows = q.nt * p.G;
            if (threadIdx.x < R) {
                const int r = threadIdx.x;
                float x = INFINITY, dl = 0.f;
                if (r < rows) {
                    const int64_t o = w.z * A.lz + (w.hk * p.G + r % p.G) * A.lh + (q.tok0 + r / p.G) * A.lt;
                    x = A.lse[o];
                    x = x == -INFINITY ? INFINITY : x * kLog2e;
                    dl = A.delta[o];
                }
                lse_s[r] = x;
                del_s[r] = dl;
            }
            float s[4][4], d[4][4];
            landed<1>();
            __syncthreads();
            dots<DP>(Vs, Gs, ty, tx, d);
            landed<0>();
            __syncthreads();
            dots<DP>(Ks, Qs, ty, tx, s);  // keys ty + 16 u, rows tx + 16 v
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int r = tx + 16 * v;
                const int pos = r < rows ? q.a + r / p.G : -1;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float e = visible(pos, kb + ty + 16 * u, p) ? exp2f(s[u][v] * A.c2 - lse_s[r]) : 0.f;
                    Ps[(ty + 16 * u) * PP + r] = e;
                    Ds[(ty + 16 * u) * PP + r] = e == 0.f ? 0.f : e * (d[u][v] - del_s[r]);
                }
            }
            __syncwarp();
            accumulate<DP>(Ps, Gs, ty, tx, av);
            __syncthreads();
            copy(Gs, A.dO, n + 1);
            accumulate<DP>(Ds, Qs, ty, tx, ak);
            __syncthreads();
            copy(Qs, A.Q, n + 1);
        }
        float* slot = A.slots + (size_t)it.slot() * kv_slot_floats(R);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = ty + 16 * u;
            if (kb + r >= p.Sk) continue;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int c = 64 * g + 4 * tx;
                const float2 a = ak[u][g][0], b = ak[u][g][1], e = av[u][g][0], f = av[u][g][1];
                if (!it.whole()) {
                    *reinterpret_cast<float4*>(slot + SlotRows(R).at(r, c)) = make_float4(a.x, a.y, b.x, b.y);
                    *reinterpret_cast<float4*>(slot + R * kSlotD + SlotRows(R).at(r, c)) = make_float4(e.x, e.y, f.x, f.y);
                } else if (c < A.D) {
                    store4(at<T>(A.dK, w.z, w.hk, kb + r) + c, a.x * A.scale, a.y * A.scale, b.x * A.scale, b.y * A.scale);
                    store4(at<T>(A.dV, w.z, w.hk, kb + r) + c, e.x, e.y, f.x, f.y);
                }
            }
        }
        if (threadIdx.x == 0 && it.s0 == 0 && !it.whole())
            write_cut(A.cuts, it.seg, it.rep, it.tile, it.n - it.ns, [&](int c) { return plan.s[c].count; });
    }
}

Args make_args(const Call& c) {
    Args a{};
    a.p = c.p;
    a.p.kshift = kShift;
    a.p.TQ = imin(R / c.p.G, imax(1, c.p.paged && c.p.T <= c.p.nseg ? 1 : R));
    a.Q = c.Q, a.K = c.K, a.V = c.V, a.O = c.O, a.dO = c.dO, a.dQ = c.dQ, a.dK = c.dK, a.dV = c.dV;
    a.lse = c.lse, a.lz = c.lz, a.lh = c.lh, a.lt = c.lt, a.delta = c.stats;
    a.D = c.D;
    a.scale = c.scale;
    a.c2 = c.scale * kLog2e;
    a.cuts = c.cuts;
    a.slots = c.slots;
    return a;
}

template <typename K, typename... A>
int launch(K kern, int grid, size_t smem, cudaStream_t s, const A&... args) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return BSP_ERR_CUDA;
    kern<<<grid, kT, smem, s>>>(args...);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

template <int DP>
constexpr size_t tiles_bytes(int tiles, int patches) {
    return sizeof(float) * ((size_t)tiles * R * (DP + 4) + (size_t)patches * R * PP);
}

template <typename T, int DP>
int forward_t(Call& c, const Args& a, int grid) {
    c.p.TQ = a.p.TQ, c.p.kshift = a.p.kshift;
    size_t smem = tiles_bytes<DP>(3, 1);
    if (smem < (size_t)c.p.nseg * sizeof(int)) smem = (size_t)c.p.nseg * sizeof(int);
    SimtPlan plan{};
    bool cut = true;
    int rc = c.p.paged ? BSP_OK : query_plan(c, grid, &plan.tab, plan.s, &cut);
    if (rc) return rc;
    rc = c.p.paged ? launch(forward_kernel<T, DP, true>, grid, smem, c.stream, a, plan)
                   : launch(forward_kernel<T, DP, false>, grid, smem, c.stream, a, plan);
    return rc || !cut ? rc : launch_join(c, R, grid, false);
}

template <typename T, int DP>
int backward_t(Call& c, const Args& a, int grid) {
    c.p.TQ = a.p.TQ, c.p.kshift = a.p.kshift;
    const KProb kp{1, c.p.rep, c.p.G, a.p.TQ, kShift, c.p.Hq, c.p.Hkv, c.p.Sq, c.p.Sk, c.p.window, c.p.sinks};
    SimtPlan plan, kplan;
    bool cut = false, kcut = false;
    int rc = query_plan(c, grid, &plan.tab, plan.s, &cut);
    if (!rc) rc = key_plan(c, kp, grid, &kplan.tab, kplan.s, &kcut);
    if (!rc) rc = launch_delta(c);
    if (!rc) rc = launch(dq_kernel<T, DP>, grid, tiles_bytes<DP>(4, 1), c.stream, a, plan);
    if (!rc && cut) rc = launch_join(c, R, grid, true);
    if (!rc) rc = launch(dkv_kernel<T, DP>, grid, tiles_bytes<DP>(4, 2), c.stream, a, kp, kplan);
    return rc || !kcut ? rc : launch_join_kv(c, kp, R, grid);
}

}  // namespace

#define BSP_WIN_DISPATCH(fn)                                                                    \
    const Args a = make_args(c);                                                                \
    const int grid = imin(kSimtPerSm * sm_count(), SimtPlan::kCtas);                                                   \
    switch (c.dtype) {                                                                          \
        case BSP_F32: return c.D <= 64 ? fn<float, 64>(c, a, grid) : fn<float, 128>(c, a, grid); \
        case BSP_BF16: return c.D <= 64 ? fn<__nv_bfloat16, 64>(c, a, grid) : fn<__nv_bfloat16, 128>(c, a, grid); \
        case BSP_F16: return c.D <= 64 ? fn<__half, 64>(c, a, grid) : fn<__half, 128>(c, a, grid); \
        default: return BSP_ERR_INVALID_ARG;                                                    \
    }

int launch_forward_simt(Call& c) { BSP_WIN_DISPATCH(forward_t) }
int launch_backward_simt(Call& c) { BSP_WIN_DISPATCH(backward_t) }

}  // namespace win
}  // namespace bsp
