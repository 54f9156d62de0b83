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

// Threads of a CTA, four CTAs an SM: while one waits for the reads that its walk or its
// search asks for, others pass over their rows (64 sequences of 128000 entries 19.3
// us, 200 53.8, 2000 of 4000 33; with 512 threads, two CTAs an SM, 20.1, 61.3 and 59; with
// 128 23.0, 57.6 and 24).
constexpr int kVerifyT = 256;
constexpr int kMaxCluster = 8;

// What the walk needs of a tree.  One CTA of the cluster reads it and hands it to
// all, so that their walks, and with them their barriers, cannot part.
struct Tree {
    int n, q0;
    int up[kMaxNodes], tok[kMaxNodes];
    float px[kMaxNodes], qx[kMaxNodes], u[kMaxNodes];
};

// A number in two fp32 parts, the second the rounding error of the first, and a
// sum whose additions' errors all go to its second part (the error of a sum as Knuth
// finds it, that of a product by a fused multiply-add).  The second part rounds too,
// the more the longer it is: of the m terms since the parts were last made whole, the
// j-th adds an error of at most (2 j + 3) 2^-48 of the sum.  Made whole after every 8 or
// 16, n terms are off by less than n 2^-43 of it; never (as first built), 65536 equal
// ones were by 2^-22.  (GB300 has two fp64 lanes an SM, and an fp64
// operation takes over 100 cycles: with them for the walk and the sums of the
// warps, 64 sequences of 128000 entries took 27 us, not 23.5, and with every warp
// adding up all sums 230.)
struct Two {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ Two() {}
    __device__ __forceinline__ Two(float h) : hi(h) {}
    __device__ __forceinline__ Two(float h, float l) : hi(h), lo(l) {}
    __device__ __forceinline__ void add(float x, float e) {
        const float t = hi + x, b = t - hi;
        lo += ((hi - (t - b)) + (x - b)) + e;
        hi = t;
    }
    __device__ __forceinline__ Two whole() const {  // parts that do not overlap
        const float h = hi + lo;
        return Two(h, lo - (h - hi));
    }
    __device__ __forceinline__ bool above(Two x) const { return (hi - x.hi) + (lo - x.lo) > 0.f; }
};
__device__ __forceinline__ Two operator+(Two a, Two b) {
    a.add(b.hi, b.lo);
    return a.whole();
}
__device__ __forceinline__ Two operator-(Two a, Two b) { return a + Two(-b.hi, -b.lo); }
__device__ __forceinline__ Two operator*(Two a, Two b) {
    const float h = __fmul_rn(a.hi, b.hi);  // (not to be joined with an addition)
    return Two(h, fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, fmaf(a.hi, b.hi, -h)))).whole();
}
__device__ __forceinline__ Two from_lane(Two x, int lane) {
    return Two(__shfl_sync(0xffffffffu, x.hi, lane), __shfl_sync(0xffffffffu, x.lo, lane));
}
// the sum over a warp, in lane 0 (other lanes' may be rounded otherwise)
__device__ __forceinline__ Two over_warp(Two x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x.add(__shfl_down_sync(0xffffffffu, x.hi, o), __shfl_down_sync(0xffffffffu, x.lo, o));
    return x.whole();
}
// inclusive prefix over the lanes of a warp
__device__ __forceinline__ Two warp_scan(Two x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two z(__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o));
        if (lane >= o) x = z + x;
    }
    return x;
}

// What an entry of a row counts as: one that is negative or no number, 0.
__device__ __forceinline__ float weight(float x) { return fmaxf(x, 0.f); }

// What is left of a row of the target: p - c q where that is positive, or p
// without some tokens.
template <typename T, bool DRAWN>
struct Rows {
    static constexpr int N = 16 / sizeof(T);
    const T *p, *q;  // q: null while nothing was rejected
    Two c;
    const int* out;  // tokens taken out of p, n_out of them
    int n_out;
    int V, off;      // a 16-byte piece k holds entries k N - off ..

    __device__ __forceinline__ uint4 piece(const T* row, int i0) const {
        if (i0 >= 0 && i0 + N <= V && ((uintptr_t)(row + i0) & 15) == 0) return *reinterpret_cast<const uint4*>(row + i0);
        return edge(row, i0, V);
    }
    static __device__ __noinline__ uint4 edge(const T* row, int i0, int V) {
        uint32_t w[4] = {};
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (i0 + j >= 0 && i0 + j < V) {
                if constexpr (sizeof(T) == 4)
                    w[j] = __float_as_uint(row[i0 + j]);
                else
                    w[j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[i0 + j] << (j & 1) * 16;
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void load(int k, uint4& a, uint4& b) const {
        a = piece(p, k * N - off);
        if (DRAWN && q) b = piece(q, k * N - off);
    }
    // the piece's entries in two parts; entries of nothing (outside the row, not
    // positive, no number) are 0
    __device__ __forceinline__ void left(int k, const uint4& a, const uint4& b, float (&x)[N], float (&y)[N]) const {
        const T *pe = reinterpret_cast<const T*>(&a), *qe = reinterpret_cast<const T*>(&b);
        if (DRAWN && q) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                // p - c q, every rounding error kept
                const float u = to_f32(pe[j]), v = weight(to_f32(qe[j]));
                const float m = __fmul_rn(c.hi, v), e = fmaf(c.lo, v, fmaf(c.hi, v, -m));
                const float d = u - m, t = d - u;
                const float r = ((u - (d - t)) - (m + t)) - e;
                const bool on = d + r > 0.f;
                x[j] = on ? d : 0.f;
                y[j] = on ? r : 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                x[j] = weight(to_f32(pe[j]));
                y[j] = 0.f;
            }
            if (!DRAWN) {
                const int i0 = k * N - off;
#pragma unroll 1
                for (int o = 0; o < n_out; ++o) {
                    const unsigned at = (unsigned)(out[o] - i0);
                    if (at < (unsigned)N) {
#pragma unroll
                        for (int j = 0; j < N; ++j) x[j] = at == (unsigned)j ? 0.f : x[j];
                    }
                }
            }
        }
    }
};

__device__ __forceinline__ void block_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kVerifyT) : "memory"); }

// The walk from node 0 down, by the first warp of each CTA of a sequence's cluster
// alike.  At a node with the target's row p and the draft's row q, before its k-th
// child,
//     r_0 = p, s_0 = 1;  r_(k+1) = max(r_k - s_k q, 0), s_(k+1) = sum r_(k+1)
// and the child x is taken when u q(x) s_k < r_k(x).  Since r_k is where it is
// not zero p - (s_0 + .. + s_(k-1)) q, one number c_k = s_0 + .. + s_(k-1) stands
// for all rejections so far: r_k = max(p - c_k q, 0), and a rejection costs one
// pass over the two rows for s_(k+1).  Drafts that were chosen, not drawn, have
// no row: u s_k < r_k(x), and r_(k+1) is r_k without x.  Where no child is taken,
// the next token is the first one up to which r_k adds up to more than u sum r_k.
//
// Each warp of the cluster holds a run of the vocabulary.  The sums of the runs go
// to every CTA through the cluster's shared memory; the CTA that the number falls
// to looks for the token in that run, a step of 32 pieces to a warp.
//
// Bound by the chain of what follows one another, most of all the reads: offsets,
// parents and tokens, their probabilities (2.5 us), the pass (64 sequences of
// 128000 fp32 entries: 65 MB of two rows each, 9.2 us with what L2 holds of them, for
// 9.6 from memory at a copy's rate), the sums (1.7) and the search (2.1); with the
// launch 19.6 us, and 7 for one sequence of 32000.  The walk's code stands once, and so does the pass': the first
// instructions come from memory too, and with a copy of the pass wherever one is
// asked for, one sequence took 18 us under the profiler, not 9.5.
template <typename T, bool DRAWN>
__global__ void __launch_bounds__(kVerifyT, 1024 / kVerifyT) draft_verify_kernel(const __grid_constant__ VerifyArgs a) {
    using R = Rows<T, DRAWN>;
    constexpr int N = R::N, NW = kVerifyT / 32;
    __shared__ Tree tree;
    __shared__ float2 sums[2][kMaxCluster * NW];  // Two's of the cluster's warps, of this pass and the last
    __shared__ int out[kMaxNodes];
    __shared__ struct {
        int node, n_out, walking, winner;
        float2 c;
        float2 before, want;  // the sum in front of the winner's run, and what is looked for
    } now;
    __shared__ float2 step_sum[NW];
    auto two = [](float2 x) { return Two(x.x, x.y); };
    auto pair = [](Two x) { return make_float2(x.hi, x.lo); };
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), C = (int)cluster.num_blocks();
    const int s = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int W = C * NW;
    const T* target = static_cast<const T*>(a.target);
    const T* draft = static_cast<const T*>(a.draft);
    cluster.sync();  // all of them have begun: their shared memory may be written
    cudaGridDependencySynchronize();
    const float number = a.sample[s];
    if (rank == 0) {
        if (warp == 0) {
            const int q0 = a.q_start[s];
            int n = a.q_start[s + 1] - q0;
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
        const int n = tree.n, q0 = tree.q0;
        for (int i = tid; i < n; i += kVerifyT) {
            int up = a.parent[q0 + i], tok = a.tokens[q0 + i];
            // (-1 past node 0: a place without a token)
            if (up < -1 || up >= i || (up >= 0 && (unsigned)tok >= (unsigned)a.V)) {
                set_status(a.status, BSP_ERR_DEVICE_CHECK);
                up = -1;
            }
            float p = 0.f, q = 0.f;
            if (up >= 0) {
                p = weight(to_f32(target[(q0 + up) * a.target_row + tok]));
                if (DRAWN) q = weight(to_f32(draft[(q0 + up) * a.draft_row + tok]));
            }
            const float u = a.accept[q0 + i];
            for (int r = 0; r < C; ++r) {
                Tree* to = r == 0 ? &tree : cluster.map_shared_rank(&tree, r);
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
    if (n == 0) {
        if (rank == 0 && tid == 0) {
            a.count[s] = 0;
            a.token[s] = -1;
        }
        return;
    }
    // the rows that `now` tells of, and a warp's run of steps of 32 pieces
    auto rows_now = [&]() {
        R r;
        r.V = a.V;
        r.p = target + (q0 + now.node) * a.target_row;
        r.c = two(now.c);
        r.q = DRAWN && now.c.x > 0.f ? draft + (q0 + now.node) * a.draft_row : nullptr;
        r.out = out, r.n_out = now.n_out;
        r.off = (int)(((uintptr_t)r.p & 15) / sizeof(T));
        return r;
    };
    auto steps_of = [&](const R& r) { return ((uint32_t)a.V + r.off + 32 * N - 1) / (32 * N); };  // at most 2^23
    auto run_of = [&](const R& r, int w, int* first, int* last) {
        const uint32_t steps = steps_of(r);
        *first = (int)(steps * w / W);
        *last = (int)(steps * (w + 1) / W);
    };
    // one pass over what is left: every warp's sum to every CTA
    int parity = 1;
    auto pass = [&]() {
        const R rows = rows_now();
        const int me = rank * NW + warp;
        int k, last;
        run_of(rows, me, &k, &last);
        Two sum;
        constexpr int kAhead = 2;
#pragma unroll 1
        for (; k < last; k += kAhead) {
            uint4 x[kAhead], y[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (k + j < last) rows.load((k + j) * 32 + lane, x[j], y[j]);
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (k + j < last) {
                    float u[N], v[N];
                    rows.left((k + j) * 32 + lane, x[j], y[j], u, v);
#pragma unroll
                    for (int i = 0; i < N; ++i) sum.add(u[i], v[i]);
                }
            sum = sum.whole();  // (1 % of the pass; a third part for the second's errors 8 %)
        }
        parity ^= 1;
        const float2 mine = pair(from_lane(over_warp(sum), 0));  // the same bits for every CTA
        if (lane < C) cluster.map_shared_rank(&sums[parity][0], lane)[me] = mine;
        cluster.sync();
    };
    Two c, mass(1.f);
    int n_out = 0;
    // the sums in front of the lane's runs, and each of theirs
    constexpr int kRuns = kMaxCluster * NW / 32;
    static_assert(kRuns * 32 == kMaxCluster * NW, "a lane holds a whole number of runs");
    Two front, run[kRuns];
    auto add_up = [&]() {
        Two mine;
#pragma unroll
        for (int j = 0; j < kRuns; ++j) {
            const int i = lane * kRuns + j;
            run[j] = i < W ? two(sums[parity][i]) : Two();
            mine = mine + run[j];
        }
        const Two incl = warp_scan(mine, lane);
        front = incl - mine;
        mass = from_lane(incl, 31);
    };
    auto next_child = [&](int node, int after) {
#pragma unroll 1
        for (int i0 = after + 1; i0 < n; i0 += 32) {
            const unsigned m = __ballot_sync(0xffffffffu, i0 + lane < n && tree.up[i0 + lane] == node);
            if (m) return i0 + __ffs(m) - 1;
        }
        return -1;
    };
    int node = 0, depth = 0, child = 0;
    bool fresh = false;   // the cluster's sums are of what is left now
    bool later = false;   // shares were taken away behind the sums' pass
    bool summed = false;  // nothing is taken any more, the sums are on their way
    if (rank == 0 && lane == 0) a.path[q0] = 0;
    // one turn for each pass that the walk asks for
#pragma unroll 1
    while (true) {
        if (warp == 0) {
            bool ask = false;
#pragma unroll 1
            while (!summed && !ask) {
                child = next_child(node, child);
                if (child < 0) {
                    summed = true;
                    ask = !fresh;
                    break;
                }
                const Two u(tree.u[child]), px(tree.px[child]);
                bool take;
                Two have = px;
                if (DRAWN) {
                    const Two qx(tree.qx[child]);
                    take = (px - c * qx).above(u * qx * mass);
                } else {
                    const int x = tree.tok[child];
#pragma unroll 1
                    for (int i = 0; i < n_out; ++i)
                        if (out[i] == x) have = Two();
                    take = have.above(u * mass);
                }
                if (take) {
                    node = child;
                    ++depth;
                    c = Two(), mass = Two(1.f), n_out = 0, fresh = later = false;
                    if (rank == 0 && lane == 0) a.path[q0 + depth] = node;
                } else if (DRAWN) {
                    c = c + mass;
                    ask = fresh = true;
                } else {
                    // the first one's pass sums up what is left; later ones take their
                    // own share away, from the sum of the run that holds them too
                    const int x = tree.tok[child];
                    __syncwarp();
                    if (lane == 0) {
                        out[n_out] = x;
                        if (n_out) {
                            const R r = rows_now();
                            const uint32_t step = (uint32_t)(x + r.off) / (32 * N);
                            float2& sum = sums[parity][((step + 1) * W - 1) / steps_of(r)];
                            sum = have.above(two(sum)) ? make_float2(0.f, 0.f) : pair(two(sum) - have);
                        }
                    }
                    __syncwarp();
                    ask = fresh = true;
                    if (n_out++ > 0) {
                        ask = false;
                        mass = have.above(mass) ? Two() : mass - have;
                        later = true;
                    }
                }
            }
            bool done = false;
            if (!ask) {
                if (!DRAWN && later) add_up();
                later = false;
                done = mass.hi > 0.f || !(c.hi > 0.f || n_out);
                // rounding left nothing: the target's own row
                if (!done) c = Two(), n_out = 0;
            }
            if (lane == 0) {
                now.node = node, now.n_out = n_out, now.walking = !done;
                now.c = pair(c);
            }
            if (done) {
                if (rank == 0) {
                    if (lane == 0) {
                        a.count[s] = depth + 1;
                        if (!(mass.hi > 0.f)) a.token[s] = -1;
                    }
                    for (int i = depth + 1 + lane; i < n; i += 32) a.path[q0 + i] = -1;
                }
                // the run that the number falls to: the first up to which the sums are above
                // it (none, for a number of 1 or more: the last with anything)
                const Two want = Two(number) * mass;
                int over = -1, some = -1;
                Two over_front, some_front, at = front;
#pragma unroll
                for (int j = 0; j < kRuns; ++j) {
                    if (run[j].hi > 0.f) {
                        some = lane * kRuns + j, some_front = at;
                        at = at + run[j];
                        if (over < 0 && at.above(want)) over = some, over_front = some_front;
                    }
                }
                const unsigned any_over = __ballot_sync(0xffffffffu, over >= 0), any = __ballot_sync(0xffffffffu, some >= 0);
                const int src = any_over ? __ffs(any_over) - 1 : any ? 31 - __clz(any) : 0;
                const int winner = __shfl_sync(0xffffffffu, any_over ? over : some, src);
                const Two before = from_lane(any_over ? over_front : some_front, src);
                if (lane == 0) {
                    now.winner = mass.hi > 0.f ? winner : -1;
                    now.before = pair(before), now.want = pair(want);
                }
            }
            __syncwarp();
        }
        block_barrier();
        if (!now.walking) break;
        pass();
        if (warp == 0) add_up();
    }
    if (now.winner < 0 || now.winner / NW != rank) return;
    // from the winner's run on, NW steps at a time, each by a warp; its token stands
    // behind the run only where rounding says so (a run whose tokens were all taken
    // away may keep a sum above 0)
    const R rows = rows_now();
    int first, last;
    run_of(rows, now.winner, &first, &last);
    last = (int)steps_of(rows);
    const Two want = two(now.want);
    Two reached = two(now.before);
    int some = -1;  // the last entry with anything, of this thread
#pragma unroll 1
    for (int k0 = first; k0 < last; k0 += NW) {
        const int piece = (k0 + warp) * 32 + lane;
        float x[N], y[N];
        Two sum;
        if (k0 + warp < last) {
            uint4 p, q;
            rows.load(piece, p, q);
            rows.left(piece, p, q, x, y);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                sum.add(x[i], y[i]);
                if (x[i] + y[i] > 0.f) some = piece * N - rows.off + i;
            }
        }
        sum = sum.whole();
        const Two all = over_warp(sum);
        if (lane == 0) step_sum[warp] = pair(all);
        __syncthreads();
        // the first step up to which the sums are above the number
        const Two mine = lane < NW ? two(step_sum[lane]) : Two(), upto = reached + warp_scan(mine, lane);
        const unsigned hits = __ballot_sync(0xffffffffu, mine.hi > 0.f && upto.above(want));
        if (hits) {
            const int hit = __ffs(hits) - 1;
            if (hit != warp) return;
            Two at = from_lane(upto - mine, hit) + (warp_scan(sum, lane) - sum);
            int found = -1;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                at.add(x[i], y[i]);
                if (found < 0 && at.above(want) && x[i] + y[i] > 0.f) found = piece * N - rows.off + i;
            }
            // (rounding may put the border behind the step's last entry: that one then)
            const unsigned m = __ballot_sync(0xffffffffu, found >= 0), have = __ballot_sync(0xffffffffu, sum.hi > 0.f);
            const int tok = m ? __shfl_sync(0xffffffffu, found, __ffs(m) - 1) : __shfl_sync(0xffffffffu, some, 31 - __clz(have));
            if (lane == 0) a.token[s] = tok;
            return;
        }
        reached = from_lane(upto, 31);
        __syncthreads();
    }
    // rounding, or a number of 1 or more: the last entry with anything
    int* last_of = reinterpret_cast<int*>(step_sum);
    auto over_block = [&]() {
        some = __reduce_max_sync(0xffffffffu, some);
        if (lane == 0) last_of[warp] = some;
        __syncthreads();
        for (int i = 0; i < NW; ++i) some = imax(some, last_of[i]);
        __syncthreads();
    };
    over_block();
    if (some < 0) {  // in front of the run, then
#pragma unroll 1
        for (int k = warp; k < first; k += NW) {
            const int piece = k * 32 + lane;
            uint4 p, q;
            float x[N], y[N];
            rows.load(piece, p, q);
            rows.left(piece, p, q, x, y);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (x[i] + y[i] > 0.f) some = piece * N - rows.off + i;
        }
        over_block();
    }
    if (tid == 0) a.token[s] = some;
}

template <typename T>
int verify_t(const VerifyArgs& a, int n_seq, cudaStream_t s) {
    // As many CTAs to a sequence as run at once, while each warp of theirs has a step
    // of its own: 1, 2, 4, 8 CTAs for one sequence of 128000 entries 55, 30, 17, 11 us, for
    // 200 of them 86, 53, 53, 51, for 2000 of 4000 32, 48, 83, 155.
    const int at_once = 1024 / kVerifyT * sm_count(), per_step = kVerifyT * 16 / (int)sizeof(T);
    int cluster = 1;
    while (cluster < kMaxCluster && 2 * cluster * n_seq <= at_once && cluster * per_step < a.V) cluster *= 2;
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
    cudaStream_t s = (cudaStream_t)stream;
    switch (dtype) {
        case BSP_F32: return verify_t<float>(a, n_seq, s);
        case BSP_BF16: return verify_t<__nv_bfloat16>(a, n_seq, s);
        default: return verify_t<__half>(a, n_seq, s);
    }
}
