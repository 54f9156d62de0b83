// Windowed attention forward on tcgen05 tensor cores (bf16 / fp16 in, fp32
// accumulate), over dense tensors or a paged cache: one pass over the visible
// key tiles with a running maximum and sum per row.
//
// A tile is 128 rows -- consecutive tokens of one sequence times the query
// heads that share a KV head -- against steps of 128 keys.  Persistent CTAs,
// one per SM, each take an equal run of the launch's steps (window.cuh), so
// that ragged batches, long histories and few rows load the SMs evenly; a
// tile cut between CTAs leaves its raw output, maxima and sums for the join.
//
// Roles (512 threads):
//   warps 0, 3  TMA producers of Q and K, and of V.  Dense: one copy per 64
//               columns; pages: one per page and 64 columns, each by its own
//               lane, the page numbers read a step ahead.  Only pages with a
//               key that a row of the tile sees are touched.
//   warp 1      one thread issues S[g % 3] = Q K^T (M = N = 128, K = D)
//   warp 2      one thread issues O += P V, P from TMEM, in pieces of 16 keys:
//               those no row of the tile sees are left out
//   warps 4..7  epilogue: O / l of a finished tile to memory while the next
//               tile's softmax runs
//   warps 8..15 softmax: thread = row, each warpgroup one half of its 128 keys;
//               half-row maxima are swapped through shared memory
// TMEM columns: S buffers at 0, 128, 256, each step's P over its own scores;
// O at 384.
//
// P is rounded to the call's type, which the product takes; its sum l is of the
// unrounded values, in fp32, as O is.  Against an fp64 softmax O is off by 2.0 to
// 2.4e-3 (bf16) and 2.7 to 2.9e-4 (fp16), 1.6e-3 and 2.0e-4 of it its own
// rounding.
//
// V rows that no query of the sequence sees but that share a piece of 16 keys
// with visible ones (the tail of the last page, keys before every window) are
// zeroed in shared memory before the product, since 0 * NaN is NaN.
#include "tc_window.cuh"

namespace bsp {
namespace win {
namespace {

// O is rescaled only when a row's maximum grew by more than 2^8 (log2 units);
// P stays below 2^8 then, and O / l is exact either way.
constexpr float kRescaleThreshold = 8.0f;
// Ragged batches: steps below which a CTA is not worth starting for a part of a
// tile (one token over 1000 / 4000 keys: 12.9 / 22 us with 1, 13.1 / 17 with 2,
// 15.4 / 17 with 4).
constexpr int kMinShare = 2;

// A dense launch's split comes with it; a ragged one's is found in the kernel.
struct None {};
template <int MODE>
using Split = std::conditional_t<MODE == kDense, TcPlan, None>;
template <bool TREE>
using Problem = std::conditional_t<TREE, TreeProb, Prob>;

template <int DP>
struct Smem {
    static constexpr int KP = DP / 64;
    static constexpr int kTile = 128 * DP * 2;
    static constexpr int QST = 2;
    static constexpr int KVST = DP == 128 ? 2 : 3;  // at most 3: a stage is freed by a ring of 3 barriers
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + QST * kTile;
    static constexpr int kV = kK + KVST * kTile;
    static constexpr int kEpi = kV + KVST * kTile;  // one 32 x 64 panel per epilogue warp
    static constexpr int kBytes = kEpi + 4 * 4096;
    static constexpr int kAlloc = kBytes + 1024;
};

template <typename P>
struct Args {
    P p;
    View O;
    float* lse;
    int64_t lz, lh, lt;
    int D;
    float c2;  // scale * log2(e)
    Cut* cuts;
    float* slots;
};

// TREE: the tokens are nodes of trees (a ragged batch), each with a position and
// bits of its own; keys before a tree's first slot follow the rule at the node's
// position, the others the node's bits.  Only the tiles that hold a tree's slots,
// the last of each sequence, are looked at bit by bit.
template <typename T, int DP, int MODE, bool TREE>
__global__ void __launch_bounds__(kThreads, 1)
window_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Args<Problem<TREE>> args,
                 const __grid_constant__ Split<MODE> plan) {
    using SM = Smem<DP>;
    constexpr bool PAGED = MODE != kDense;
    constexpr int KP = SM::KP, QST = SM::QST, NST = SM::KVST;
    constexpr uint32_t kTileBytes = SM::kTile;
    constexpr uint32_t kIdescQK = idesc_f16(128, 128, std::is_same<T, __nv_bfloat16>::value, 0, 0);
    constexpr uint32_t kIdescPV = idesc_f16(128, DP, std::is_same<T, __nv_bfloat16>::value, 0, 1);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    // K and V of step g sit in stage g % NST; S buffer g % 3 has s_full (Q K^T
    // done, which also frees the step's K stage), p_full (P written) and
    // pv_done (P V done, which frees the buffer and the V stage).
    __shared__ uint64_t q_full[QST], q_empty[QST], k_full[NST], v_full[NST], v_land;
    __shared__ uint64_t s_full[3], p_full[3], pv_done[3];
    __shared__ uint64_t o_full, o_empty, l_full[2], l_empty[2];
    __shared__ float lsum[2][2][128], lref[2][2][128];
    __shared__ float xm[2][2][128];
    __shared__ uint64_t x_full[2][4];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ uint32_t issued[5];  // K steps, Q tiles, V steps, Q K^T steps, P V steps: drained after an abort
    __shared__ Start start;
    __shared__ uint32_t red[32];
    __shared__ Ring ring;
    __shared__ Work cut;  // the tile that begins here and is cut at the end of the share

    using P = Problem<TREE>;
    const P& p = args.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Stop ab{&abort_flag};

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < 5; ++i) issued[i] = 0;
        for (int i = 0; i < QST; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < NST; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&v_full[i], 1);
        }
        mbar_init(&v_land, 1);
        for (int i = 0; i < 3; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&pv_done[i], 1);
            mbar_init(&p_full[i], 8);
        }
        mbar_init(&o_full, 1);
        mbar_init(&o_empty, 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&l_full[i], 8);
            mbar_init(&l_empty[i], 4);
            for (int q = 0; q < 4; ++q) mbar_init(&x_full[i][q], 2);
        }
        ring.init();
        fence_barrier_init();
        cut.ns = 0;
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    cudaGridDependencySynchronize();
    if (PAGED && blockIdx.x == 0)
        for (int s = threadIdx.x; s < p.nseg; s += kThreads)
            if (p.bad_seg(p.q_start[s], p.q_start[s + 1], p.kv_len[s])) set_status(p.status, BSP_ERR_DEVICE_CHECK);
    tc_fence_before();
    if constexpr (MODE == kPlain) locate_plain<kThreads>(p, kMinShare, red, &start);
    if constexpr (MODE == kRagged) {
        locate<kThreads>(p, kMinShare, reinterpret_cast<int*>(smem), red, &start);
        fence_proxy_async_smem();  // locate's scratch is where the copies land next
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tS = tmem_base;
    const uint32_t tO = tmem_base + 384;

    if (warp < 4) {
    regs_dec<kRegsCtl>();
    if (warp == 0 || warp == 3) {
        // ----------------------------------------------- TMA producers ----
        // warp 0 walks the share and hands the tiles out
        const bool is_v = warp == 3;
        const CUtensorMap* tm = is_v ? &tmV : &tmK;
        if (lane == 0) {
            if (!is_v) tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(tm);
        }
        uint32_t i = 0, g = 0, tiles = 0, lands = 0;  // Q tiles, steps, tiles handed out, scrubbed tiles
        const uint32_t q_bytes = (uint32_t)(p.TQ * p.G) * 128 * KP;
        const int pages = PAGED ? 128 >> p.page_shift : 1;  // copies per 64 columns
        const int my_page = lane % pages, my_panel = lane / pages;
        const uint32_t page_bytes = PAGED ? 128u << p.page_shift : 128u * 128u;
        auto begin = [&] {
            if constexpr (PAGED) return Walk<P, MODE>(p, start);
            else return Walk<P, MODE>(p, plan.tab, plan.s[blockIdx.x]);
        };
        Walk<P, MODE> walk = begin();
        Work w;
        // one step is loaded while the next one's place, and its page number,
        // are on their way
        struct Step {
            int kb, pg, hk, z, row0, zlo, zhi;
            Keys keys;
            bool first;  // of its tile
        } cur, nxt;
        bool have = false;
        int n = 0;
        w.ns = 0;
#pragma unroll 1
        while (true) {
            bool more = true;
            if (n >= w.ns) {
                if (is_v) {
                    more = ring.take(tiles, w, lane == 0, true, ab);
                } else {
                    Item it;
                    w.ns = 0;
                    if (walk.next(it)) w = make_work(p, it);
                    more = ring.put(tiles, w, lane, ab) && w.ns > 0;
                }
                ++tiles;
                n = 0;
            }
            if (more) {
                nxt.kb = w.key_tile(n) << 7;
                nxt.hk = w.hk, nxt.z = w.z, nxt.row0 = w.row0, nxt.zlo = w.zlo, nxt.zhi = w.zhi;
                nxt.keys = tile_keys(p, w);
                nxt.first = n == 0;
                if (PAGED) {  // -1: hidden (not copied), -2: a bad page
                    const int a = nxt.kb + (my_page << p.page_shift);
                    nxt.pg = -1;
                    if (nxt.keys.any(a, a + (1 << p.page_shift) - 1)) {
                        nxt.pg = p.table[(int64_t)w.seg * p.max_pages + (a >> p.page_shift)];
                        if ((unsigned)nxt.pg >= (unsigned)p.n_pages) nxt.pg = -2;
                    }
                }
            }
            if (have) {
                if (!is_v && cur.first) {
                    const uint32_t qs = i % QST;
                    bool ok = wait(&q_empty[qs], ((i / QST) & 1) ^ 1, ab);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&q_full[qs], q_bytes);
#pragma unroll 1
                        for (int c = 0; c < KP; ++c)
                            tma_load_4d(smem_u32(smem + SM::kQ + qs * kTileBytes + c * 16384), &tmQ, c * 64, cur.hk * p.G,
                                        cur.row0, cur.z, &q_full[qs]);
                    }
                    ++i;
                }
                if (PAGED && __any_sync(0xffffffffu, cur.pg == -2)) {
                    if (lane == 0) ab.fail(BSP_ERR_DEVICE_CHECK);
                    break;
                }
                const bool want = PAGED ? cur.pg >= 0 && my_panel < KP : lane < KP;
                const uint32_t st = g % NST;
                if (g >= NST) {
                    const uint32_t gp = g - NST;
                    uint64_t* freed = is_v ? &pv_done[gp % 3] : &s_full[gp % 3];
                    bool ok = wait(freed, (gp / 3) & 1, ab);
                    if (!__all_sync(0xffffffffu, ok)) break;
                }
                const uint32_t bytes = PAGED ? page_bytes * __popc(__ballot_sync(0xffffffffu, want)) : kTileBytes;
                uint64_t* full = is_v ? &v_full[st] : &k_full[st];
                // rows of this V tile that no query of the sequence sees
                const bool scrub = is_v && bytes > 0 &&
                                   ((cur.kb + 127 > cur.zhi && PAGED) || (cur.kb < cur.zlo && !(cur.kb + 127 < p.sinks)));
                uint64_t* bar = scrub ? &v_land : full;
                if (lane == 0) {
                    if (bytes) mbar_arrive_expect_tx(bar, bytes);
                    else mbar_arrive(bar);
                }
                __syncwarp();
                const uint32_t base = smem_u32(smem + (is_v ? SM::kV : SM::kK) + st * kTileBytes);
                if (want) {
                    if (PAGED)
                        tma_load_4d(base + my_panel * 16384 + my_page * page_bytes, tm, my_panel * 64, 0, cur.hk, cur.pg, bar);
                    else
                        tma_load_4d(base + lane * 16384, tm, lane * 64, cur.kb, cur.hk, cur.z, bar);
                }
                if (scrub) {
                    bool ok = wait(&v_land, lands & 1, ab);
                    if (!__all_sync(0xffffffffu, ok)) {
                        if (lane == 0) drain_wait(&v_land, lands & 1);
                        break;
                    }
                    ++lands;
#pragma unroll 1
                    for (int r = lane; r < 128; r += 32) {
                        const int j = cur.kb + r, j16 = cur.kb + (r & ~15);
                        const bool used = j <= cur.zhi && (j >= cur.zlo || j < p.sinks);
                        if (!used && cur.keys.any(j16, j16 + 15))
#pragma unroll 1
                            for (int k = 0; k < KP * 8; ++k)
                                *reinterpret_cast<uint4*>(smem + SM::kV + st * kTileBytes + (k >> 3) * 16384 + r * 128 +
                                                          (k & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full);
                }
                ++g;
            }
            if (!more) break;
            cur = nxt;
            have = true;
            ++n;
        }
        if (lane == 0) {
            if (is_v) {
                issued[2] = g;
            } else {
                issued[0] = g;
                issued[1] = i;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------- Q K^T issuer (one thread) ----
        if (lane == 0) {
            const uint64_t dq = smem_desc(smem_u32(smem + SM::kQ), 16, 1024, kSw128);
            const uint64_t dk = smem_desc(smem_u32(smem + SM::kK), 16, 1024, kSw128);
            uint32_t i = 0, g = 0;
            Work w;
            for (; ring.take(i, w, true, false, ab); ++i) {
                const uint32_t qs = i % QST;
                const int ns = w.ns;
                if (!wait(&q_full[qs], (i / QST) & 1, ab)) goto qk_done;
#pragma unroll 1
                for (int n = 0; n < ns; ++n, ++g) {
                    const uint32_t st = g % NST, sb = g % 3;
                    if (g >= 3 && !wait(&pv_done[sb], ((g - 3) / 3) & 1, ab)) goto qk_done;
                    if (!wait(&k_full[st], (g / NST) & 1, ab)) goto qk_done;
                    tc_fence_after();
                    const uint64_t aq = dq + ((qs * kTileBytes) >> 4), bk = dk + ((st * kTileBytes) >> 4);
#pragma unroll 1
                    for (uint32_t c = 0; c < KP; ++c)
#pragma unroll
                        for (uint32_t ks = 0; ks < 4; ++ks) {
                            const uint32_t off = (c * 16384 + ks * 32) >> 4;
                            mma_f16(tS + sb * 128, aq + off, bk + off, kIdescQK, ks > 0 ? 1u : c);
                        }
                    mma_commit(&s_full[sb]);
                    if (n == ns - 1) mma_commit(&q_empty[qs]);
                }
            }
        qk_done:
            issued[3] = g;
        }
    } else if (warp == 2) {
        // --------------------------------------------- P V issuer (one thread) ----
        if (lane == 0) {
            const uint64_t dv = smem_desc(smem_u32(smem + SM::kV), 128 * 128, 1024, kSw128);
            uint32_t g = 0, tc = 0;
            Work w;
            while (ring.take(tc, w, true, false, ab)) {
                const Keys keys = tile_keys(p, w);
                if (tc > 0 && !wait(&o_empty, (tc - 1) & 1, ab)) goto pv_done_label;
                uint32_t acc = 0;
#pragma unroll 1
                for (int n = 0; n < w.ns; ++n, ++g) {
                    const uint32_t st = g % NST, sb = g % 3;
                    const int kb = w.key_tile(n) << 7;
                    const uint64_t bv = dv + ((st * kTileBytes) >> 4);
                    uint32_t pieces = keys.pieces(kb);
                    if (!wait(&v_full[st], (g / NST) & 1, ab)) goto pv_done_label;
                    if (!wait(&p_full[sb], (g / 3) & 1, ab)) goto pv_done_label;
                    tc_fence_after();
#pragma unroll 1
                    for (uint32_t h = 0; h < 2; ++h, pieces >>= 4)
#pragma unroll
                        for (uint32_t ks = 0; ks < 4; ++ks)
                            if ((pieces >> ks) & 1) {
                                mma_f16_tmem_a(tO, tS + sb * 128 + h * 64 + ks * 8,
                                               bv + (((h * 4 + ks) * 2048) >> 4), kIdescPV, acc);
                                acc = 1;
                            }
                    mma_commit(&pv_done[sb]);
                }
                mma_commit(&o_full);
                ++tc;
            }
        pv_done_label:
            issued[4] = g;
        }
    }
    } else if (warp < 8) {
        // ---------------------------------------------------- epilogue ----
        const int quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        uint8_t* stage = smem + SM::kEpi + quad * 4096;
        const uint32_t inv_g = 65536u / p.G + 1;  // r / G = r * inv_g >> 16 for r < 128
        uint32_t tc = 0;
        Work w;
        while (ring.take(tc, w, lane == 0, true, ab)) {
            const int rows = w.nt * p.G, hk = w.hk, z = w.z, t0 = w.row0;
            const uint32_t lb = tc & 1;
            bool ok = wait(&l_full[lb], (tc >> 1) & 1, ab, p.attempts);
            if (!__all_sync(0xffffffffu, ok)) break;
            const float m0 = lref[lb][0][row], m1 = lref[lb][1][row];
            const float l0 = lsum[lb][0][row], l1 = lsum[lb][1][row];
            __syncwarp();
            if (lane == 0) mbar_arrive(&l_empty[lb]);
            const float mf = fmaxf(m0, m1);
            const float lt = mf == -INFINITY ? l0 + l1 : l0 * ex2_approx(m0 - mf) + l1 * ex2_approx(m1 - mf);
            const bool seen = lt != 0.f;  // also where a score was no number: the row is none then
            const float inv = seen ? 1.0f / lt : 0.f;
            ok = wait(&o_full, tc & 1, ab);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            ++tc;
            if (quad * 32 >= rows) {  // no live row in this quadrant
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_empty);
                continue;
            }
            if (!w.whole()) {
                // a piece: raw O (relative to mf), mf and the sum, for the join
                float* slot = args.slots + (size_t)w.slot() * slot_floats(kTcRows);
                // (unrolled by 1 or 4, the whole kernel was 1..4 % slower, cut tiles or not)
                const SlotRows sr(rows);
                float* at = slot + sr.at(row, 0);
#pragma unroll 2
                for (int c = 0; c < DP / 32; ++c) {
                    uint32_t r[32];
                    tmem_ld32_sync(tO + lane_base + c * 32, r);
                    if (row < rows) {
#pragma unroll
                        for (int k = 0; k < 8; ++k, at += sr.step)
                            *reinterpret_cast<uint4*>(at) = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_empty);
                if (row < rows) {
                    slot[kTcRows * kSlotD + row] = mf;
                    slot[kTcRows * kSlotD + kTcRows + row] = lt;
                }
                if (threadIdx.x == 128 && w.s0 == 0) cut = w;
                continue;
            }
            if (args.lse && row < rows) {
                const int t = (row * inv_g) >> 16, h = row - t * p.G;
                args.lse[z * args.lz + (hk * p.G + h) * args.lh + (t0 + t) * args.lt] =
                    seen ? (mf + log2f(lt)) * kLn2 : -INFINITY;
            }
            // O is read out of TMEM, scaled and packed before anything is stored, and
            // the accumulator handed to the next tile (after the first panel's
            // stores instead, its first product waited 5400 cycles)
            uint32_t pk[KP][32];
#pragma unroll
            for (int c = 0; c < KP; ++c) read_panel<T>(tO + lane_base + c * 64, inv, pk[c]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty);
            // a row that saw nothing: 0, whatever its accumulator holds
            T* out = static_cast<T*>(args.O.ptr) + z * args.O.s[0] + hk * p.G * args.O.s[1] + t0 * args.O.s[2];
            store_panels<T, KP>(stage, pk, seen ? ~0u : 0u, lane, args.D, [&](int i) -> T* {
                const int r = quad * 32 + i, t = (r * inv_g) >> 16, h = r - t * p.G;
                return r < rows ? out + h * args.O.s[1] + t * args.O.s[2] : nullptr;
            });
        }
    } else {
        regs_inc<kRegsSoftmax>();
        // ---------------------------------------------------- softmax ----
        const int wg = (warp - 8) >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t inv_g = 65536u / p.G + 1;
        uint32_t g = 0, tc = 0, xg = 0;  // xg: half-row exchanges so far
        while (true) {
            int ns, s0, n_s, lo_tile, rows, pos;
            int ctx = 0, end = 0, node = 0;  // TREE: its first slot, the last one's successor, the row's token
            Seen seen;
            {
                Work w;
                if (!ring.take(tc, w, lane == 0, true, ab)) break;
                ns = w.ns, s0 = w.s0, n_s = w.n_s, lo_tile = w.lo;
                rows = w.nt * p.G;
                // rows past the tile's last see what its last row sees; they are not stored
                pos = w.a + (int)((imin(row, rows - 1) * inv_g) >> 16);
                if constexpr (TREE) {
                    ctx = w.a, end = w.zhi + 1;
                    node = w.row0 + pos - w.a;
                    pos = tree_position(p, node, ctx);
                    seen.first = __reduce_min_sync(0xffffffffu, pos);
                    seen.last = __reduce_max_sync(0xffffffffu, pos);
                } else {
                    seen.first = w.a + (int)((imin(quad * 32, rows - 1) * inv_g) >> 16);
                    seen.last = w.a + (int)((imin(quad * 32 + 31, rows - 1) * inv_g) >> 16);
                }
            }
            const bool idle = quad * 32 >= rows;  // no live row in this warp's lanes
            const int low = pos - p.window + 1;
            float l = 0.f, m = -INFINITY;
#pragma unroll 1
            for (int n = 0; n < ns; ++n, ++g) {
                const uint32_t sb = g % 3;
                const int kt = s0 + n < n_s ? s0 + n : lo_tile + (s0 + n - n_s);
                const int kb = (kt << 7) + wg * 64;  // first key of this half
                bool full = seen.all(p, kb), skip = seen.none(p, kb);
                unsigned long long vis = 0;
                if constexpr (TREE) {
                    if (kb + 64 > ctx) {  // slots of the tree's nodes among these
                        full = false;
                        skip = kb >= end;
                        if (!skip && !idle)
                            vis = (row_keys(ctx - 1, low, p.sinks, kb) |
                                   bits_at(p.bits + (int64_t)node * p.words, p.words, kb - ctx)) & below(imin(end - kb, 64));
                    } else if (!full) {
                        vis = row_keys(pos, low, p.sinks, kb);
                    }
                }
                bool ok = wait(&s_full[sb], (g / 3) & 1, ab);
                if (!__all_sync(0xffffffffu, ok)) goto softmax_done;
                if (idle) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[sb]);
                    continue;
                }
                tc_fence_after();
                const uint32_t srow = tS + sb * 128 + wg * 64 + lane_base;
                const uint32_t xb = xg & 1, xph = (xg >> 1) & 1;
                ++xg;
                float x[64];
                float mx = -INFINITY;
                if (!skip) {
                    tmem_ld64_sync(srow, srow + 32, *reinterpret_cast<uint32_t(*)[64]>(x));
                    if (!full) hide(x, TREE ? vis : row_keys(pos, low, p.sinks, kb));
                    float m8[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) m8[k] = fmax3(x[k], x[k + 8], x[k + 16]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) m8[k] = fmax3(m8[k], x[k + 24], x[k + 32]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) m8[k] = fmax3(fmaxf(m8[k], x[k + 40]), x[k + 48], x[k + 56]);
                    mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                }
                xm[xb][wg][row] = mx;
                __syncwarp();
                if (lane == 0) mbar_arrive(&x_full[xb][quad]);
                ok = wait(&x_full[xb][quad], xph, ab);
                if (!__all_sync(0xffffffffu, ok)) goto softmax_done;
                const float mrow = fmaxf(mx, xm[xb][wg ^ 1][row]);
                const float m_new = fmaxf(m, mrow * args.c2);
                const bool need = m_new > m + kRescaleThreshold;  // also true for the first finite max
                const float mnext = need ? m_new : m;
                const float msub = (mnext == -INFINITY) ? 0.f : mnext;
                uint32_t pk[32];
                float rs = 0.f;
                if (!skip) {
                    const float2 c2v = make_float2(args.c2, args.c2), nm = make_float2(-msub, -msub);
                    float2 rs4[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) rs4[k] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float2 y = __ffma2_rn(make_float2(x[2 * k], x[2 * k + 1]), c2v, nm);
                        const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                        rs4[k & 3] = __fadd2_rn(rs4[k & 3], e);
                        pk[k] = Pack2<T>::pack(e.x, e.y);
                    }
                    const float2 r2 = __fadd2_rn(__fadd2_rn(rs4[0], rs4[1]), __fadd2_rn(rs4[2], rs4[3]));
                    rs = r2.x + r2.y;
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) pk[k] = 0u;
                }
                tmem_st32_sync(srow, pk);
                // rows that saw nothing yet have O = 0, which no factor changes
                const bool grew = need && m != -INFINITY;
                if (__any_sync(0xffffffffu, grew)) {
                    ok = wait(&pv_done[(g - 1) % 3], ((g - 1) / 3) & 1, ab);
                    if (!__all_sync(0xffffffffu, ok)) goto softmax_done;
                    tc_fence_after();
                    const float alpha = grew ? ex2_approx(m - mnext) : 1.f;
#pragma unroll 1
                    for (int cc = 0; cc < DP / 64; ++cc) {
                        uint32_t r[32];
                        const uint32_t ta = tO + lane_base + wg * (DP / 2) + cc * 32;
                        tmem_ld32_sync(ta, r);
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const float2 v = __fmul2_rn(make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])),
                                                        make_float2(alpha, alpha));
                            r[k] = __float_as_uint(v.x);
                            r[k + 1] = __float_as_uint(v.y);
                        }
                        tmem_st32_sync(ta, r);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[sb]);
                l = l * ex2_approx(m - msub) + rs;
                m = mnext;
            }
            {
                const uint32_t lb = tc & 1;
                if (tc >= 2) {
                    bool ok = wait(&l_empty[lb], ((tc - 2) >> 1) & 1, ab);
                    if (!__all_sync(0xffffffffu, ok)) goto softmax_done;
                }
                lsum[lb][wg][row] = l;
                lref[lb][wg][row] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(&l_full[lb]);
                ++tc;
            }
        }
    softmax_done:;
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        if (abort_flag) set_status(p.status, abort_flag);
        args.cuts[blockIdx.x].pieces = 0;
        if (cut.ns)
            write_cut(args.cuts, cut.seg, cut.rep, cut.tile, cut.n - cut.ns, [&](int c) {
                if constexpr (PAGED) return start.shares.of(c);
                else return plan.s[c].count;
            });
    }
    if (abort_flag) {
        // the copies and products issued before the stop land before the CTA
        // lets go of its shared memory and TMEM
        if (threadIdx.x == 0) {
            drain_ring(k_full, NST, issued[0]);
            drain_ring(q_full, QST, issued[1]);
            drain_ring(v_full, NST, issued[2]);
            if (issued[3]) drain_wait(&s_full[(issued[3] - 1) % 3], ((issued[3] - 1) / 3) & 1);
            if (issued[4]) drain_wait(&pv_done[(issued[4] - 1) % 3], ((issued[4] - 1) / 3) & 1);
            drain_end();
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

template <typename T, int DP, int MODE, bool TREE>
int launch(Call& c) {
    constexpr bool PAGED = MODE != kDense;
    const int is_bf16 = std::is_same<T, __nv_bfloat16>::value;
    const Prob& p = c.p;
    CUtensorMap mq, mk, mv;
    const int rows = PAGED ? 1 << p.page_shift : 128;
    int rc = query_map(&mq, c.Q, c, is_bf16, PAGED ? p.T : p.Sq, p.TQ);
    if (!rc) rc = key_map(&mk, c.K, c, is_bf16, rows);
    if (!rc) rc = key_map(&mv, c.V, c, is_bf16, rows);
    if (rc) return rc;
    auto kern = window_tc_kernel<T, DP, MODE, TREE>;
    constexpr int smem = Smem<DP>::kAlloc;
    static std::atomic<uint64_t> prepared{0};
    if ((rc = prepare_kernel(kern, smem, prepared))) return rc;
    const int grid = imin(sm_count(), TcPlan::kCtas);
    const Args<Problem<TREE>> a{Problem<TREE>{p}, c.O, c.lse, c.lz, c.lh, c.lt, c.D, c.scale * kLog2e, c.cuts, c.slots};
    Split<MODE> plan;
    bool cut = true;
    if constexpr (!PAGED)
        if ((rc = query_plan(c, grid, &plan.tab, plan.s, &cut))) return rc;
    if ((rc = launch_behind(kern, dim3(grid), kThreads, smem, c.stream, mq, mk, mv, a, plan))) return rc;
    return cut ? launch_join(c, kTcRows, grid, false) : BSP_OK;
}

template <typename T, int MODE, bool TREE = false>
int by_width(Call& c) {
    return c.D <= 64 ? launch<T, 64, MODE, TREE>(c) : launch<T, 128, MODE, TREE>(c);
}

template <typename T>
int by_mode(Call& c) {
    if (!c.p.paged) return by_width<T, kDense>(c);
    if (c.p.words) return by_width<T, kRagged, true>(c);
    return c.p.TQ == 1 && c.p.nseg <= kThreads ? by_width<T, kPlain>(c) : by_width<T, kRagged>(c);
}

}  // namespace

int launch_forward_tc(Call& c) {
    // one new token per sequence (as far as the host can know): a tile is one
    // token's heads, and its copies are no wider (64 such tokens 180 us, with
    // 128-row tiles 185; one over 1000 keys 13.1 and 16.2); else as many tokens
    // as fill 128 rows
    c.p.kshift = 7;
    c.p.TQ = c.p.paged && c.p.T <= c.p.nseg ? 1 : kTcRows / c.p.G;
    if (c.p.words) c.p.TQ = imin(c.p.TQ, 32 * c.p.words);  // no sequence has more
    const int64_t keys = c.p.paged ? (int64_t)c.p.max_pages << c.p.page_shift : c.p.Sk;
    c.p.attempts = wait_attempts(c, (keys >> 7) + 2);
    return c.dtype == BSP_BF16 ? by_mode<__nv_bfloat16>(c) : by_mode<__half>(c);
}

}  // namespace win
}  // namespace bsp
