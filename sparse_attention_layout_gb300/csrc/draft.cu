// Drafted tokens: the shape of their trees (bsp_draft_tree) and their
// verification against the target's probabilities (bsp_draft_verify).
//
// A tree's node 0 is the sequence's last known token; parents come before their
// children.
#include <cooperative_groups.h>

#include <type_traits>

#include "common.cuh"
#include "window_args.h"

namespace cg = cooperative_groups;

namespace bsp {
namespace win {
namespace {

// ------------------------------------------------------------------ tree --

struct TreeArgs {
    const int* q_start;
    const int* kv_len;
    const int* parent;
    int* pos;
    uint32_t* bits;
    int T, words, window, sinks;
    int* status;
};

// A node's ancestors by walking up: a thread per node, the parents in shared
// memory.  Node a at depth e is seen by node i below it at depth d when
// d - e < window or the position of a is one of the sinks.  Bound by latency
// (three dependent reads and the walk).
__global__ void __launch_bounds__(256) draft_tree_kernel(const __grid_constant__ TreeArgs a) {
    __shared__ int up[kMaxNodes];
    cudaGridDependencySynchronize();
    const int s = blockIdx.x, q0 = a.q_start[s], q1 = a.q_start[s + 1], kv = a.kv_len[s], n = q1 - q0;
    if (q0 < 0 || q1 < q0 || q1 > a.T || n > 32 * a.words || kv < n || kv > kMaxLen) {
        if (threadIdx.x == 0) set_status(a.status, BSP_ERR_DEVICE_CHECK);
        return;
    }
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        int p = a.parent[q0 + i];
        if (p < -1 || p >= i) {
            set_status(a.status, BSP_ERR_DEVICE_CHECK);
            p = -1;
        }
        up[i] = p;
    }
    __syncthreads();
    const int ctx = kv - n;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        int depth = 0;
#pragma unroll 1
        for (int x = up[i]; x >= 0; x = up[x]) ++depth;
        a.pos[q0 + i] = ctx + depth;
        // words from the last down: ancestors come in falling order
        uint32_t* row = a.bits + (int64_t)(q0 + i) * a.words;
        int x = i, back = 0;
#pragma unroll 1
        for (int w = a.words - 1; w >= 0; --w) {
            uint32_t v = 0;
#pragma unroll 1
            for (; x >= 32 * w; x = up[x], ++back)  // (-1 ends it: w >= 0)
                if (back < a.window || ctx + depth - back < a.sinks) v |= 1u << (x & 31);
            row[w] = v;
        }
    }
}

// ---------------------------------------------------------- verification --

struct VerifyArgs {
    const void* target;
    const void* draft;
    int64_t target_row, draft_row;  // elements from a row to the next
    const int* tokens;
    const int* q_start;
    const int* parent;
    const float* accept;
    const float* sample;
    int* path;
    int* count;
    int* token;
    int T, V;
    int* status;
};

constexpr int kVerifyT = 512, kVerifyWarps = kVerifyT / 32;
constexpr int kMaxCluster = 8;

// What the walk needs of a tree.  One CTA of the cluster reads it and hands it to
// all, so that their walks, and with them their barriers, cannot part.
struct Tree {
    int n, q0;
    int up[kMaxNodes], tok[kMaxNodes];
    float px[kMaxNodes], qx[kMaxNodes], u[kMaxNodes];
};

// A sum in two fp32 parts: the rounding error of every addition goes to the
// second, so a sum of some thousand terms is off by 2^-46 of itself.
struct Sum2 {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x, float e) {
        const float t = hi + x, b = t - hi;
        lo += ((hi - (t - b)) + (x - b)) + e;
        hi = t;
    }
    __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

// The rows at the node where the walk stands.
template <typename T, bool DRAWN>
struct Rows {
    static constexpr int N = 16 / sizeof(T);
    const T *p, *q;  // q: null while nothing was rejected
    float ch, cl;    // what of q is taken away, in two parts
    const int* out;  // tokens taken out of p, n_out of them
    int n_out;
    int V, off;      // a 16-byte piece k holds entries k N - off ..

    // The piece's probabilities that are left, in two parts; entries of nothing
    // (outside the row, not positive, no number) are 0.
    __device__ __forceinline__ void load(int k, float (&a)[N], float (&b)[N]) const {
        const int i0 = k * N - off;
        if (i0 >= 0 && i0 + N <= V) {
            Vec16<T>::load(p + i0, a);
            if (DRAWN && q) {
                if (((uintptr_t)(q + i0) & 15) == 0) {
                    Vec16<T>::load(q + i0, b);
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) b[j] = to_f32(q[i0 + j]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const bool in = i0 + j >= 0 && i0 + j < V;
                a[j] = in ? to_f32(p[i0 + j]) : 0.f;
                if (DRAWN && q) b[j] = in ? to_f32(q[i0 + j]) : 0.f;
            }
        }
    }
    __device__ __forceinline__ void left(int k, float (&a)[N], float (&b)[N]) const {
        if (DRAWN && q) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                // p - c q, every rounding error kept
                const float m = ch * b[j], e = fmaf(cl, b[j], fmaf(ch, b[j], -m));
                const float d = a[j] - m, t = d - a[j];
                const float r = ((a[j] - (d - t)) - (m + t)) - e;
                const bool on = d + r > 0.f;
                a[j] = on ? d : 0.f;
                b[j] = on ? r : 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                a[j] = a[j] > 0.f ? a[j] : 0.f;
                b[j] = 0.f;
            }
            if (!DRAWN) {
                const int i0 = k * N - off;
#pragma unroll 1
                for (int x = 0; x < n_out; ++x) {
                    const unsigned at = (unsigned)(out[x] - i0);
                    if (at < (unsigned)N) {
#pragma unroll
                        for (int j = 0; j < N; ++j) a[j] = at == (unsigned)j ? 0.f : a[j];
                    }
                }
            }
        }
    }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The walk from node 0 down, by every warp of a sequence's cluster alike.  At a
// node with the target's row p and the draft's row q, before its k-th child,
//     r_0 = p, s_0 = 1;  r_(k+1) = max(r_k - s_k q, 0), s_(k+1) = sum r_(k+1)
// and the child x is taken when u q(x) s_k < r_k(x).  Since r_k is where it is
// not zero p - (s_0 + .. + s_(k-1)) q, one number c_k = s_0 + .. + s_(k-1) stands
// for all rejections so far: r_k = max(p - c_k q, 0), and a rejection costs one
// pass over the two rows for s_(k+1).  Drafts that were chosen, not drawn, have
// no row: u s_k < r_k(x), and r_(k+1) is r_k without x.  Where no child is taken,
// the next token is the first one up to which r_k adds up to more than u sum r_k.
//
// Each warp of the cluster holds a run of the vocabulary; their sums, in fp64,
// go to every CTA through the cluster's shared memory, and the warp that the
// number falls to looks for the token in its run.
template <typename T, bool DRAWN>
__global__ void __launch_bounds__(kVerifyT) draft_verify_kernel(const __grid_constant__ VerifyArgs a) {
    using R = Rows<T, DRAWN>;
    constexpr int N = R::N;
    __shared__ Tree tree;
    __shared__ double sums[2][kMaxCluster * kVerifyWarps];
    __shared__ int out[kMaxNodes];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), C = (int)cluster.num_blocks();
    const int s = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int W = C * kVerifyWarps, me = rank * kVerifyWarps + warp;
    const T* target = static_cast<const T*>(a.target);
    const T* draft = static_cast<const T*>(a.draft);
    cudaGridDependencySynchronize();
    if (rank == 0) {
        int q0 = 0, n = 0;
        if (warp == 0) {
            q0 = a.q_start[s];
            n = a.q_start[s + 1] - q0;
            if (q0 < 0 || n < 0 || n > kMaxNodes || q0 > a.T - n) {
                if (lane == 0) set_status(a.status, BSP_ERR_DEVICE_CHECK);
                n = 0;
            }
            if (lane < C) {
                Tree* to = lane == 0 ? &tree : cluster.map_shared_rank(&tree, lane);
                to->n = n;
                to->q0 = q0;
            }
        }
        __syncthreads();
        n = tree.n, q0 = tree.q0;
        for (int i = tid; i < n; i += kVerifyT) {
            int up = a.parent[q0 + i], tok = a.tokens[q0 + i];
            // (-1 past node 0: a place without a token)
            if (up < -1 || up >= i || (up >= 0 && (unsigned)tok >= (unsigned)a.V)) {
                set_status(a.status, BSP_ERR_DEVICE_CHECK);
                up = -1;
            }
            float p = 0.f, q = 0.f;
            if (up >= 0) {
                p = to_f32(target[(q0 + up) * a.target_row + tok]);
                if (DRAWN) q = to_f32(draft[(q0 + up) * a.draft_row + tok]);
            }
            const float u = a.accept[q0 + i];
            for (int r = 0; r < C; ++r) {
                Tree* to = cluster.map_shared_rank(&tree, r);
                to->up[i] = up;
                to->tok[i] = tok;
                to->px[i] = p;
                to->qx[i] = q;
                to->u[i] = u;
            }
        }
    }
    cluster.sync();
    const int n = tree.n, q0 = tree.q0;
    const bool writer = rank == 0 && tid == 0;
    if (n == 0) {
        if (writer) {
            a.count[s] = 0;
            a.token[s] = -1;
        }
        return;
    }
    int passes = 0;
    R rows;
    rows.V = a.V;
    rows.out = out;
    rows.n_out = 0;
    // pieces of the row, 32 a step, and this warp's run of steps
    int first = 0, last = 0;
    auto at_node = [&](int node) {
        rows.p = target + (q0 + node) * a.target_row;
        rows.q = nullptr;
        rows.n_out = 0;
        rows.off = (int)(((uintptr_t)rows.p & 15) / sizeof(T));
        const int steps = (int)(((int64_t)a.V + rows.off + 32 * N - 1) / (32 * N));
        first = (int)((int64_t)steps * me / W);
        last = (int)((int64_t)steps * (me + 1) / W);
    };
    // sum of what is left of the row, the same in every thread of the cluster
    auto pass = [&]() -> double {
        Sum2 sum;
        int k = first;
#pragma unroll 1
        for (; k + 4 <= last; k += 4) {
            float x[4][N], y[4][N];
#pragma unroll
            for (int j = 0; j < 4; ++j) rows.load((k + j) * 32 + lane, x[j], y[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                rows.left((k + j) * 32 + lane, x[j], y[j]);
#pragma unroll
                for (int i = 0; i < N; ++i) sum.add(x[j][i], y[j][i]);
            }
        }
#pragma unroll 1
        for (; k < last; ++k) {
            float x[N], y[N];
            rows.load(k * 32 + lane, x, y);
            rows.left(k * 32 + lane, x, y);
#pragma unroll
            for (int i = 0; i < N; ++i) sum.add(x[i], y[i]);
        }
        const double mine = warp_sum(sum.value());
        double* buf = sums[passes++ & 1];
        if (lane < C) cluster.map_shared_rank(buf, lane)[me] = mine;
        cluster.sync();
        double all = 0.0;
#pragma unroll 1
        for (int i = lane; i < W; i += 32) all += buf[i];
        return warp_sum(all);
    };
    auto next_child = [&](int node, int after) {
#pragma unroll 1
        for (int i0 = after + 1; i0 < n; i0 += 32) {
            const unsigned m = __ballot_sync(0xffffffffu, i0 + lane < n && tree.up[i0 + lane] == node);
            if (m) return i0 + __ffs(m) - 1;
        }
        return -1;
    };
    int node = 0, depth = 0;
    double c, mass;
    bool fresh;  // the cluster's sums are of what is left now
    while (true) {
        if (writer) a.path[q0 + depth] = node;
        at_node(node);
        c = 0.0, mass = 1.0, fresh = false;
        int child = next_child(node, node);
#pragma unroll 1
        for (; child >= 0; child = next_child(node, child)) {
            const double u = tree.u[child], px = tree.px[child];
            if (DRAWN) {
                const double qx = tree.qx[child];
                if (u * qx * mass < px - c * qx) break;
                c += mass;
                rows.q = draft + (q0 + node) * a.draft_row;
                rows.ch = (float)c;
                rows.cl = (float)(c - (double)rows.ch);
                mass = pass();
                fresh = true;
            } else {
                const int x = tree.tok[child];
                double have = px;
                for (int i = 0; i < rows.n_out; ++i)
                    if (out[i] == x) have = 0.0;
                if (u * mass < have) break;
                __syncthreads();  // out[]'s readers of the last rejection are done
                if (tid == 0) out[rows.n_out] = x;
                ++rows.n_out;
                __syncthreads();
                // later ones only take their own share away
                fresh = rows.n_out == 1;
                mass = fresh ? pass() : fmax(mass - have, 0.0);
            }
        }
        if (child < 0) break;
        node = child;
        ++depth;
    }
    if (!fresh) mass = pass();
    if (!(mass > 0.0) && (rows.q || rows.n_out)) {
        // rounding left nothing: the target's own row
        rows.q = nullptr;
        rows.n_out = 0;
        mass = pass();
    }
    if (rank == 0)
        for (int i = depth + 1 + tid; i < n; i += kVerifyT) a.path[q0 + i] = -1;
    if (writer) {
        a.count[s] = depth + 1;
        if (!(mass > 0.0)) a.token[s] = -1;
    }
    if (!(mass > 0.0)) return;
    // the warp whose run the number falls to: the first up to which the sums are
    // above it (none, for a number of 1 or more: the last with anything)
    const double* buf = sums[(passes - 1) & 1];
    const double want = (double)a.sample[s] * mass;
    double before = 0.0;
    int mine = -1;
    double mine_before = 0.0;
#pragma unroll 1
    for (int i = 0; i < W; ++i) {
        if (buf[i] > 0.0) mine = i, mine_before = before;
        before += buf[i];
        if (before > want) break;
    }
    if (mine != me) return;
    int found = -1, some = -1;  // the token; the last with anything
    double run = mine_before;
#pragma unroll 1
    for (int k = first; k < last && found < 0; ++k) {
        const int piece = k * 32 + lane;
        float x[N], y[N];
        rows.load(piece, x, y);
        rows.left(piece, x, y);
        Sum2 sum;
        int any = -1;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            sum.add(x[i], y[i]);
            if (x[i] + y[i] > 0.f) any = piece * N - rows.off + i;
        }
        const double v = sum.value();
        double incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double z = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += z;
        }
        const unsigned have = __ballot_sync(0xffffffffu, any >= 0);
        if (have) some = __shfl_sync(0xffffffffu, any, 31 - __clz(have));
        const unsigned over = __ballot_sync(0xffffffffu, any >= 0 && run + incl > want);
        if (over) {
            double at = run + (incl - v);
            int i_at = any;
#pragma unroll
            for (int i = N - 1; i >= 0; --i) {
                // the entry's own end: the sum up to it, from the front
                double end = at;
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (j <= i) end += (double)x[j] + (double)y[j];
                if (end > want && x[i] + y[i] > 0.f) i_at = piece * N - rows.off + i;
            }
            found = __shfl_sync(0xffffffffu, i_at, __ffs(over) - 1);
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) a.token[s] = found >= 0 ? found : some;
}

template <typename T>
int verify_t(const VerifyArgs& a, int n_seq, int cluster, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(n_seq * cluster);
    cfg.blockDim = dim3(kVerifyT);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, a.draft ? draft_verify_kernel<T, true> : draft_verify_kernel<T, false>, a) == cudaSuccess
               ? BSP_OK : BSP_ERR_CUDA;
}

}  // namespace
}  // namespace win
}  // namespace bsp

using namespace bsp::win;

extern "C" int bsp_draft_tree(bsp_window_t w, const int32_t* q_start, const int32_t* kv_len, const int32_t* parent,
                              int32_t* positions, uint32_t* bits, int T, int n_seq, int words, void* stream) {
    int rc = check_handle(w, BSP_F32);
    if (rc) return rc;
    if (T < 0 || n_seq < 0 || words < 1) return BSP_ERR_INVALID_ARG;
    if (T > kMaxLen || n_seq > kMaxSeqs || words > kMaxNodes / 32) return BSP_ERR_UNSUPPORTED;
    if (T == 0 || n_seq == 0) return BSP_OK;
    if (!q_start || !kv_len || !parent || !positions || !bits) return BSP_ERR_INVALID_ARG;
    if (((uintptr_t)q_start | (uintptr_t)kv_len | (uintptr_t)parent | (uintptr_t)positions | (uintptr_t)bits) & 3u)
        return BSP_ERR_ALIGNMENT;
    TreeArgs a{q_start, kv_len, parent, positions, bits, T, words, 0, 0, w->status};
    set_rule(w, &a.window, &a.sinks);
    return launch_behind(draft_tree_kernel, dim3(n_seq), 256, 0, (cudaStream_t)stream, a);
}

extern "C" int bsp_draft_verify(bsp_window_t w, int dtype, const void* target, int64_t target_stride, const void* draft,
                                int64_t draft_stride, const int32_t* tokens, const int32_t* q_start,
                                const int32_t* parent, const float* accept, const float* sample, int32_t* path,
                                int32_t* count, int32_t* token, int T, int n_seq, int V, void* stream) {
    int rc = check_handle(w, dtype);
    if (rc) return rc;
    if (T < 0 || n_seq < 0 || V < 1) return BSP_ERR_INVALID_ARG;
    if (T > kMaxLen || n_seq > kMaxSeqs || V > kMaxLen) return BSP_ERR_UNSUPPORTED;
    if (n_seq == 0) return BSP_OK;
    if (!q_start || !sample || !count || !token) return BSP_ERR_INVALID_ARG;
    if (T > 0) {
        if (!target || !tokens || !parent || !accept || !path) return BSP_ERR_INVALID_ARG;
        if (T > 1 && (target_stride < V || (draft && draft_stride < V))) return BSP_ERR_INVALID_ARG;
        if (T > 1 && (target_stride > (int64_t)1 << 38 || (draft && draft_stride > (int64_t)1 << 38)))
            return BSP_ERR_UNSUPPORTED;
    }
    if (((uintptr_t)target | (uintptr_t)draft) & (uintptr_t)(elt_bytes(dtype) - 1)) return BSP_ERR_ALIGNMENT;
    if (((uintptr_t)tokens | (uintptr_t)q_start | (uintptr_t)parent | (uintptr_t)accept | (uintptr_t)sample |
         (uintptr_t)path | (uintptr_t)count | (uintptr_t)token) & 3u)
        return BSP_ERR_ALIGNMENT;
    const VerifyArgs a{target, draft, target_stride, draft_stride, tokens, q_start, parent, accept, sample,
                       path, count, token, T, V, w->status};
    // few sequences: eight SMs share each one's vocabulary
    const int cluster = n_seq <= 4 * bsp::sm_count() ? 8 : n_seq <= 16 * bsp::sm_count() ? 2 : 1;
    cudaStream_t s = (cudaStream_t)stream;
    switch (dtype) {
        case BSP_F32: return verify_t<float>(a, n_seq, cluster, s);
        case BSP_BF16: return verify_t<__nv_bfloat16>(a, n_seq, cluster, s);
        default: return verify_t<__half>(a, n_seq, cluster, s);
    }
}
