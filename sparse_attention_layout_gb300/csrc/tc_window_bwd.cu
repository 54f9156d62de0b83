// Gradient of the windowed attention on tcgen05 tensor cores (bf16 / fp16 in,
// fp32 accumulate).  With P = exp(scale Q K^T - lse) on the visible pairs and
// dS = P (dO V^T - dO . O):
//     dq kernel   per query tile, over the key tiles it sees:   dQ = scale dS K
//     dkv kernel  per key tile, over the query tiles that see it (all heads of
//                 the group in a tile's rows): dV = P^T dO, dK = scale dS^T Q
// S and dP are computed in both, seven products where five would do with dQ
// added up in memory: no atomics, so the same inputs give the same bits, and no
// fp32 dQ in memory.  The dkv kernel forms the transposes S^T = K Q^T and
// dP^T = V dO^T (thread = key), so that P^T and dS^T are tensor-memory operands
// of the two products that contract over the rows, and nothing but the 16-bit
// tiles passes through shared memory.  Persistent CTAs take equal runs of
// steps, as in the forward; the tile with the sinks, which every query sees, is
// cut among many.
//
// P and dS are rounded to the call's type on their way to the products that
// contract over them, which take no fp32 operands; all sums stay in fp32.  fp16
// holds both times powers of two (window.h, DsFactor).
//
// K and V rows that no query sees but that share a tile with visible ones are
// zeroed in shared memory where a product sums over them or their dP enters a
// product, since 0 * NaN is NaN.
#include "tc_window.cuh"

namespace bsp {
namespace win {
namespace {

struct Args {
    Prob p;
    View dQ, dK, dV;
    float* stats;        // kStatTile floats per tile of kStatRows rows
    const DsFactor* factor;  // fp16: per (batch entry, KV head)
    int D, ntiles;       // such tiles per (batch entry, KV head)
    float scale, c2;     // c2 = scale * log2(e)
    Cut* cuts;
    float* slots;
};

template <int DP>
struct Smem {
    static constexpr int KP = DP / 64;
    static constexpr int kTile = 128 * DP * 2;
    // dq: Q, dO one stage, K, V two; dkv: K, V one stage, Q, dO (64 rows) four
    static constexpr int kA = 0, kB = kTile;            // the tile's own operands
    static constexpr int kX = 2 * kTile, kY = 4 * kTile;  // the steps' operands, two (four) stages each
    static constexpr int kEpi = 6 * kTile;              // one 32 x 64 panel per epilogue warp
    static constexpr int kStats = kEpi + 4 * 4096;      // dkv: four stages of 2 * kStatRows floats
    static constexpr int kBytes = kStats + 4 * 2 * kStatRows * 4;
    static constexpr int kAlloc = kBytes + 1024;
};

// 128 x DP accumulator columns of a warp's 32 rows to the partial-result slot
// (raw fp32) or, scaled and rounded, to memory; arrives on `empty` as soon as
// the columns are in registers.  down: what takes fp16's factors out.
template <typename T, int DP, typename F>
__device__ __forceinline__ void drain(uint32_t tacc, uint64_t* empty, int lane, int row, int rows, float* slot,
                                      float scale, float down, int D, uint8_t* stage, F dst) {
    constexpr bool kF16 = std::is_same<T, __half>::value;
    if (slot) {
        const SlotRows sr(rows);
        float* at = slot + sr.at(row, 0);
#pragma unroll 1
        for (int c = 0; c < DP / 32; ++c) {
            uint32_t r[32];
            tmem_ld32_sync(tacc + c * 32, r);
            if (kF16) {
#pragma unroll
                for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * down);
            }
            if (row < rows) {
#pragma unroll
                for (int k = 0; k < 8; ++k, at += sr.step)
                    *reinterpret_cast<uint4*>(at) = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(empty);
        return;
    }
    uint32_t pk[DP / 64][32];
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) read_panel<T>(tacc + c * 64, kF16 ? scale * down : scale, pk[c]);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(empty);
    store_panels<T, DP / 64>(stage, pk, ~0u, lane, D, dst);
}

// ------------------------------------------------------------------- dQ ----
// Roles: warp 0 copies; warp 1 issues S = Q K^T into buffer g % 2, warp 3
// dP = dO V^T, warp 2 dQ += dS K (dS from TMEM over its own scores, K as it
// lies); warps 4..7 write dQ; warps 8..15 form dS, thread = row, each warpgroup
// half of the step's keys.  Three issuing threads, because each spends more
// time on its barriers (200 cycles for one that has long completed, while the
// other warps load the shared-memory pipe) than on its products.
// TMEM columns: S 0 and 128, dP 256, dQ 384.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
dq_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
             const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
             const __grid_constant__ Args args, const __grid_constant__ TcPlan plan) {
    using SM = Smem<DP>;
    constexpr int KP = SM::KP;
    constexpr uint32_t kTile = SM::kTile;
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t kIdescS = idesc_f16(128, 128, kBf, 0, 0), kIdescD = idesc_f16(128, DP, kBf, 0, 1);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t a_full, a_free, k_full[2], v_full[2], s_full[2], dp_full, dp_free, ds_full[2], dq_done[2];
    __shared__ uint64_t land;  // K and V of a step with rows to be zeroed
    __shared__ uint64_t acc_full, acc_empty;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ uint32_t issued[5];  // K steps, V steps, S steps, dQ steps, dP steps
    __shared__ uint32_t issued_a;
    __shared__ Ring ring;
    __shared__ Work cut;  // the tile that begins here and is cut at the end of the share

    const Prob& p = args.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Stop ab{&abort_flag};
    if (threadIdx.x == 0) {
        abort_flag = 0;
        issued_a = 0;
        for (int i = 0; i < 5; ++i) issued[i] = 0;
        mbar_init(&a_full, 1);
        mbar_init(&a_free, 2);  // S has read Q, dP has read dO
        mbar_init(&dp_full, 1);
        mbar_init(&dp_free, 8);
        mbar_init(&land, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&ds_full[i], 8);
            mbar_init(&dq_done[i], 1);
        }
        mbar_init(&acc_full, 1);
        mbar_init(&acc_empty, 4);
        ring.init();
        fence_barrier_init();
        cut.ns = 0;
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    cudaGridDependencySynchronize();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tS = tmem_base, tP = tmem_base + 256, tA = tmem_base + 384;

    if (warp < 4) {
        regs_dec<kRegsCtl>();
        if (warp == 0) {
            // ------------------------------------------------- producer ----
            // walks the share and hands the tiles out
            if (lane == 0) {
                tma_prefetch_desc(&tmQ);
                tma_prefetch_desc(&tmG);
                tma_prefetch_desc(&tmK);
                tma_prefetch_desc(&tmV);
            }
            const uint32_t a_bytes = (uint32_t)(p.TQ * p.G) * 128 * KP;
            const int zlo = window_low(p.Sk - p.Sq, p.window);
            uint32_t g = 0, tiles = 0, lands = 0;
            Walk<Prob, kDense> walk(p, plan.tab, plan.s[blockIdx.x]);
            Item it;
            Work w;
            while (true) {
                w.ns = 0;
                if (walk.next(it)) w = make_work(p, it);
                if (!ring.put(tiles, w, lane, ab) || w.ns == 0) break;
                // the previous tile's S and dP products have read Q and dO
                if (tiles > 0) {
                    const bool ok = wait(&a_free, (tiles - 1) & 1, ab);
                    if (!__all_sync(0xffffffffu, ok)) goto load_done;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&a_full, 2 * a_bytes);
                    for (int c = 0; c < KP; ++c) {
                        tma_load_4d(smem_u32(smem + SM::kA + c * 16384), &tmQ, c * 64, w.hk * p.G, w.row0, w.z, &a_full);
                        tma_load_4d(smem_u32(smem + SM::kB + c * 16384), &tmG, c * 64, w.hk * p.G, w.row0, w.z, &a_full);
                    }
                }
                ++tiles;
#pragma unroll 1
                for (int n = 0; n < w.ns; ++n, ++g) {
                    const uint32_t st = g & 1;
                    // K of step g - 2 is free after its dQ product, V after its dP product,
                    // which the same step's dS follows
                    if (g >= 2) {
                        const bool ok = wait(&dq_done[st], ((g - 2) >> 1) & 1, ab);
                        if (!__all_sync(0xffffffffu, ok)) goto load_done;
                    }
                    const int kb = w.key_tile(n) << 7;
                    const Unseen un(kb, p.sinks, zlo);
                    uint64_t* const kbar = un.any() ? &land : &k_full[st];
                    uint64_t* const vbar = un.any() ? &land : &v_full[st];
                    if (lane == 0) {
                        if (un.any()) mbar_expect_tx(&land, kTile);
                        else mbar_arrive_expect_tx(kbar, kTile);
                        for (int c = 0; c < KP; ++c)
                            tma_load_4d(smem_u32(smem + SM::kX + st * kTile + c * 16384), &tmK, c * 64, kb, w.hk, w.z, kbar);
                        mbar_arrive_expect_tx(vbar, kTile);
                        for (int c = 0; c < KP; ++c)
                            tma_load_4d(smem_u32(smem + SM::kY + st * kTile + c * 16384), &tmV, c * 64, kb, w.hk, w.z, vbar);
                    }
                    if (un.any()) {
                        __syncwarp();
                        const bool ok = wait(&land, lands & 1, ab);
                        if (!__all_sync(0xffffffffu, ok)) {
                            if (lane == 0) drain_wait(&land, lands & 1);
                            goto load_done;
                        }
                        ++lands;
                        zero_rows<KP>(smem + SM::kX + st * kTile, un.r0, un.r1, lane);
                        zero_rows<KP>(smem + SM::kY + st * kTile, un.r0, un.r1, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&k_full[st]);
                            mbar_arrive(&v_full[st]);
                        }
                    }
                }
            }
        load_done:
            if (lane == 0) {
                issued[0] = issued[1] = g;
                issued_a = tiles;
            }
        } else if ((warp == 1 || warp == 3) && lane == 0) {
            // ---------------------------------- S (warp 1), dP (warp 3) ----
            const bool is_s = warp == 1;
            const uint64_t da = smem_desc(smem_u32(smem + (is_s ? SM::kA : SM::kB)), 16, 1024, kSw128);
            const uint64_t dx = smem_desc(smem_u32(smem + (is_s ? SM::kX : SM::kY)), 16, 1024, kSw128);
            uint32_t g = 0, tiles = 0;
            Work w;
            while (ring.take(tiles, w, true, false, ab)) {
                const int ns = w.ns;
                if (!wait(&a_full, tiles & 1, ab)) goto score_done;
#pragma unroll 1
                for (int n = 0; n < ns; ++n, ++g) {
                    const uint32_t st = g & 1;
                    // S buffer free: dQ of step g - 2; dP's: step g - 1 has been read
                    if (is_s ? g >= 2 : g >= 1)
                        if (!wait(is_s ? &dq_done[st] : &dp_free, (is_s ? (g - 2) >> 1 : g - 1) & 1, ab)) goto score_done;
                    if (!wait(is_s ? &k_full[st] : &v_full[st], (g >> 1) & 1, ab)) goto score_done;
                    tc_fence_after();
                    const uint32_t d = is_s ? tS + st * 128 : tP;
#pragma unroll
                    for (uint32_t c = 0; c < KP; ++c)
#pragma unroll
                        for (uint32_t ks = 0; ks < 4; ++ks) {
                            const uint32_t off = (c * 16384 + ks * 32) >> 4;
                            mma_f16(d, da + off, dx + ((st * kTile) >> 4) + off, kIdescS, c + ks > 0 ? 1u : 0u);
                        }
                    mma_commit(is_s ? &s_full[st] : &dp_full);
                    if (n == ns - 1) mma_commit(&a_free);
                }
                ++tiles;
            }
        score_done:
            issued[is_s ? 2 : 4] = g;
        } else if (warp == 2 && lane == 0) {
            // ------------------------------------------- dQ product ----
            const uint64_t dx = smem_desc(smem_u32(smem + SM::kX), 128 * 128, 1024, kSw128);
            uint32_t g = 0, tiles = 0;
            Work w;
            while (ring.take(tiles, w, true, false, ab)) {
                const int ns = w.ns;
                if (tiles > 0 && !wait(&acc_empty, (tiles - 1) & 1, ab)) goto dq_end;
#pragma unroll 1
                for (int n = 0; n < ns; ++n, ++g) {
                    const uint32_t st = g & 1;
                    if (!wait(&ds_full[st], (g >> 1) & 1, ab)) goto dq_end;
                    tc_fence_after();
#pragma unroll 1
                    for (uint32_t h = 0; h < 2; ++h)
#pragma unroll
                        for (uint32_t ks = 0; ks < 4; ++ks)
                            mma_f16_tmem_a(tA, tS + st * 128 + h * 64 + ks * 8, dx + ((st * kTile + (h * 4 + ks) * 2048) >> 4),
                                           kIdescD, ks > 0 ? 1u : h + n);
                    mma_commit(&dq_done[st]);
                }
                mma_commit(&acc_full);
                ++tiles;
            }
        dq_end:
            issued[3] = g;
        }
    } else if (warp < 8) {
        // ---------------------------------------------------- epilogue ----
        const int quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t inv_g = 65536u / p.G + 1;  // r / G = r * inv_g >> 16 for r < 128
        uint32_t tiles = 0;
        Work w;
        while (ring.take(tiles, w, lane == 0, true, ab)) {
            const int rows = w.nt * p.G, hk = w.hk, z = w.z;
            const bool ok = wait(&acc_full, tiles & 1, ab, p.attempts);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            ++tiles;
            float* slot = w.whole() ? nullptr : args.slots + (size_t)w.slot() * slot_floats(kTcRows);
            T* out = static_cast<T*>(args.dQ.ptr) + z * args.dQ.s[0] + hk * p.G * args.dQ.s[1] + w.row0 * args.dQ.s[2];
            const float down = kBf ? 1.0f : args.factor[w.rep].down;
            drain<T, DP>(tA + lane_base, &acc_empty, lane, row, rows, slot, args.scale, down, args.D,
                         smem + SM::kEpi + quad * 4096, [&](int i) -> T* {
                             const int r = quad * 32 + i, t = (r * inv_g) >> 16, h = r - t * p.G;
                             return r < rows ? out + h * args.dQ.s[1] + t * args.dQ.s[2] : nullptr;
                         });
            if (threadIdx.x == 128 && w.s0 == 0 && !w.whole()) cut = w;
        }
    } else {
        regs_inc<kRegsSoftmax>();
        // -------------------------------------------------------- dS ----
        const int wg = (warp - 8) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t inv_g = 65536u / p.G + 1;
        uint32_t g = 0;
        for (uint32_t i = 0;; ++i) {
            int ns, s0, n_s, lo_tile, pos;
            float nlse, delta, up = 1.f;
            Seen seen;
            {
                Work w;
                if (!ring.take(i, w, lane == 0, true, ab)) break;
                ns = w.ns, s0 = w.s0, n_s = w.n_s, lo_tile = w.lo;
                const int end = w.nt * p.G - 1;
                const int t = (imin(row, end) * inv_g) >> 16, h = row - t * p.G;
                const int tq = kStatRows / p.G, tok = w.row0 + t;
                float* s = args.stats + ((int64_t)w.rep * args.ntiles + tok / tq) * kStatTile + tok % tq * p.G + h;
                nlse = row <= end ? s[kStatLse] : -INFINITY;  // rows past the tile's last: P = 0
                delta = row <= end ? s[kBf ? kStatDelta : kStatDot] : 0.f;
                if (!kBf) {
                    up = args.factor[w.rep].up;
                    delta *= up;
                    if (wg == 0 && row <= end) s[kStatDelta] = delta;  // for the dkv kernel
                }
                pos = w.a + t;
                seen.first = w.a + (int)((imin(quad * 32, end) * inv_g) >> 16);
                seen.last = w.a + (int)((imin(quad * 32 + 31, end) * inv_g) >> 16);
            }
            const int low = pos - p.window + 1;
#pragma unroll 1
            for (int n = 0; n < ns; ++n, ++g) {
                const uint32_t st = g & 1;
                const int kt = s0 + n < n_s ? s0 + n : lo_tile + (s0 + n - n_s);
                const int kb = (kt << 7) + wg * 64;
                const bool full = seen.all(p, kb);
                bool ok = wait(&s_full[st], (g >> 1) & 1, ab);
                if (!__all_sync(0xffffffffu, ok)) goto ds_done;
                tc_fence_after();
                const uint32_t ts = tS + st * 128 + lane_base + wg * 64;
                float x[64];
                tmem_ld64_sync(ts, ts + 32, *reinterpret_cast<uint32_t(*)[64]>(x));
                if (!full) hide(x, row_keys(pos, low, p.sinks, kb));
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    const float2 y = __ffma2_rn(make_float2(x[j], x[j + 1]), make_float2(args.c2, args.c2),
                                                make_float2(nlse, nlse));
                    x[j] = ex2_approx(y.x);
                    x[j + 1] = ex2_approx(y.y);
                }
                ok = wait(&dp_full, g & 1, ab);
                if (!__all_sync(0xffffffffu, ok)) goto ds_done;
                tc_fence_after();
                uint32_t pk[32];
                const float2 nd = make_float2(-delta, -delta);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t r[32];
                    tmem_ld32_sync(tP + lane_base + wg * 64 + c * 32, r);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 dp = make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1]));
                        const float2 d = kBf ? __fadd2_rn(dp, nd) : __ffma2_rn(dp, make_float2(up, up), nd);
                        const float2 e = __fmul2_rn(d, make_float2(x[c * 32 + j], x[c * 32 + j + 1]));
                        pk[c * 16 + j / 2] = Pack2<T>::pack(e.x, e.y);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&dp_free);
                tmem_st32_sync(ts, pk);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ds_full[st]);
            }
        }
    ds_done:;
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        if (abort_flag) set_status(p.status, abort_flag);
        args.cuts[blockIdx.x].pieces = 0;
        if (cut.ns)
            write_cut(args.cuts, cut.seg, cut.rep, cut.tile, cut.n - cut.ns, [&](int c) { return plan.s[c].count; });
    }
    if (abort_flag) {
        if (threadIdx.x == 0) {
            drain_ring(k_full, 2, issued[0]);
            drain_ring(v_full, 2, issued[1]);
            if (issued_a) drain_wait(&a_full, (issued_a - 1) & 1);
            if (issued[2]) drain_wait(&s_full[(issued[2] - 1) & 1], ((issued[2] - 1) >> 1) & 1);
            if (issued[4]) drain_wait(&dp_full, (issued[4] - 1) & 1);
            if (issued[3]) drain_wait(&dq_done[(issued[3] - 1) & 1], ((issued[3] - 1) >> 1) & 1);
            drain_end();
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// --------------------------------------------------------------- dK, dV ----
// Roles: warp 0 copies; warp 1 issues S^T = K Q^T, warp 3 dP^T = V dO^T, warp 2
// dV += P^T dO and dK += dS^T Q; warps 4..7 write dV and dK; warps 8..15 form P^T and dS^T,
// thread = key, the warpgroups taking turns at the steps.
// A step is 64 query rows: P^T lies over S^T and dS^T over dP^T, so a product of
// the next scores has to wait for the products that read them, and with both
// accumulators of D = 128 tensor memory has room for two steps of 64 rows but
// only one of 128 (measured with those: 4150 cycles per 128 rows, the tensor
// core idle half of the time).
// TMEM columns: S^T 0 and 64, dP^T 128 and 192, dV 256, dK 384.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
dkv_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
              const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
              const __grid_constant__ Args args, const __grid_constant__ KProb kp,
              const __grid_constant__ TcPlan plan) {
    using SM = Smem<DP>;
    constexpr int KP = SM::KP;
    constexpr uint32_t kTile = SM::kTile, kStep = kTile / 2, kPanel = kStatRows * 128;
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t kIdescS = idesc_f16(128, kStatRows, kBf, 0, 0), kIdescD = idesc_f16(128, DP, kBf, 0, 1);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    // stages of Q, dO and the rows' statistics: step % 4; scores: step % 2
    __shared__ uint64_t a_full, a_free, x_full[4], dk_done[4];
    __shared__ uint64_t land;  // V of a tile with rows to be zeroed
    __shared__ uint64_t s_full[2], p_full[2], dv_done[2], dp_full[2], ds_full[2];
    __shared__ uint64_t dv_full, dv_empty, dk_full, dk_empty;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ uint32_t issued[5];  // steps: copied, -, S^T, dP^T, dV
    __shared__ uint32_t issued_a, issued_k;
    __shared__ Ring ring;
    __shared__ Work cut;  // the tile that begins here and is cut at the end of the share

    const Prob& p = args.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Stop ab{&abort_flag};
    if (threadIdx.x == 0) {
        abort_flag = 0;
        issued_a = issued_k = 0;
        for (int i = 0; i < 5; ++i) issued[i] = 0;
        mbar_init(&a_full, 1);
        mbar_init(&a_free, 2);  // S^T has read K, dP^T has read V
        mbar_init(&land, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&x_full[i], 1);
            mbar_init(&dk_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&dv_done[i], 1);
            mbar_init(&dp_full[i], 1);
            mbar_init(&ds_full[i], 4);
        }
        mbar_init(&dv_full, 1);
        mbar_init(&dk_full, 1);
        mbar_init(&dv_empty, 4);
        mbar_init(&dk_empty, 4);
        ring.init();
        fence_barrier_init();
        cut.ns = 0;
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    cudaGridDependencySynchronize();
    tc_fence_before();
    // rows past TQ * G, which no copy writes, enter the products over the rows
    // with P = 0: they must not hold NaN
    if (kp.TQ * p.G < kStatRows)
        for (int i = threadIdx.x; i < 4 * (int)kTile / 16; i += kThreads)
            *reinterpret_cast<uint4*>(smem + SM::kX + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    __syncthreads();
    tc_fence_after();
    const uint32_t tS = tmem_base, tP = tmem_base + 128, tV = tmem_base + 256, tK = tmem_base + 384;

    if (warp < 4) {
        regs_dec<kRegsCtl>();
        if (warp == 0) {
            // ------------------------------------------------- producer ----
            if (lane == 0) {
                tma_prefetch_desc(&tmQ);
                tma_prefetch_desc(&tmG);
                tma_prefetch_desc(&tmK);
                tma_prefetch_desc(&tmV);
            }
            const uint32_t bytes = (uint32_t)(kp.TQ * p.G) * 128 * KP;
            const int zlo = window_low(p.Sk - p.Sq, p.window);
            uint32_t g = 0, tiles = 0, lands = 0;
            Walk<KProb, kDense> walk(kp, plan.tab, plan.s[blockIdx.x]);
            Item it;
            Work w;
            while (true) {
                w = Work{};
                if (walk.next(it)) {
                    w.ns = it.ns, w.s0 = it.s0, w.n = it.n, w.tile = it.tile;
                    w.lo = it.sp.lo + it.s0;
                    w.z = it.rep / p.Hkv, w.hk = it.rep % p.Hkv, w.rep = it.rep;
                }
                if (!ring.put(tiles, w, lane, ab) || w.ns == 0) break;
                // the previous tile's score products have read K and V
                if (tiles > 0) {
                    const bool ok = wait(&a_free, (tiles - 1) & 1, ab);
                    if (!__all_sync(0xffffffffu, ok)) goto load_done;
                }
                const Unseen un(w.tile << 7, p.sinks, zlo);
                uint64_t* const vbar = un.any() ? &land : &a_full;
                if (lane == 0) {
                    if (un.any()) mbar_arrive_expect_tx(&land, kTile);
                    else mbar_expect_tx(&a_full, kTile);
                    for (int c = 0; c < KP; ++c)
                        tma_load_4d(smem_u32(smem + SM::kB + c * 16384), &tmV, c * 64, w.tile << 7, w.hk, w.z, vbar);
                }
                if (un.any()) {
                    __syncwarp();
                    const bool ok = wait(&land, lands & 1, ab);
                    if (!__all_sync(0xffffffffu, ok)) {
                        if (lane == 0) drain_wait(&land, lands & 1);
                        goto load_done;
                    }
                    ++lands;
                    zero_rows<KP>(smem + SM::kB, un.r0, un.r1, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&a_full, kTile);
                    for (int c = 0; c < KP; ++c)
                        tma_load_4d(smem_u32(smem + SM::kA + c * 16384), &tmK, c * 64, w.tile << 7, w.hk, w.z, &a_full);
                }
                ++tiles;
#pragma unroll 1
                for (int n = 0; n < w.ns; ++n, ++g) {
                    const uint32_t st = g & 3;
                    if (g >= 4) {
                        const bool ok = wait(&dk_done[st], ((g - 4) >> 2) & 1, ab);
                        if (!__all_sync(0xffffffffu, ok)) goto load_done;
                    }
                    if (lane == 0) {
                        const int tok = (w.lo + n) * kp.TQ;
                        mbar_arrive_expect_tx(&x_full[st], 2 * bytes + 8u * kStatRows);
                        for (int c = 0; c < KP; ++c)
                            tma_load_4d(smem_u32(smem + SM::kX + st * kStep + c * kPanel), &tmQ, c * 64, w.hk * p.G, tok,
                                        w.z, &x_full[st]);
                        bulk_load(smem_u32(smem + SM::kStats + st * 8 * kStatRows),
                                  args.stats + ((int64_t)w.rep * args.ntiles + w.lo + n) * kStatTile + kStatLse, 8 * kStatRows,
                                  &x_full[st]);
                        for (int c = 0; c < KP; ++c)
                            tma_load_4d(smem_u32(smem + SM::kY + st * kStep + c * kPanel), &tmG, c * 64, w.hk * p.G, tok,
                                        w.z, &x_full[st]);
                    }
                }
            }
        load_done:
            if (lane == 0) {
                issued[0] = g;
                issued_a = tiles;
            }
        } else if ((warp == 1 || warp == 3) && lane == 0) {
            // ------------------------------ S^T (warp 1), dP^T (warp 3) ----
            const bool is_s = warp == 1;
            const uint64_t da = smem_desc(smem_u32(smem + (is_s ? SM::kA : SM::kB)), 16, 1024, kSw128);
            const uint64_t dx = smem_desc(smem_u32(smem + (is_s ? SM::kX : SM::kY)), 16, 1024, kSw128);
            uint64_t* const out = is_s ? s_full : dp_full;
            const uint32_t d = is_s ? tS : tP;
            uint32_t g = 0, tiles = 0;
            Work w;
            while (ring.take(tiles, w, true, false, ab)) {
                const int ns = w.ns;
                if (!wait(&a_full, tiles & 1, ab)) goto score_done;
#pragma unroll 1
                for (int n = 0; n < ns; ++n, ++g) {
                    const uint32_t st = g & 3, sb = g & 1;
                    if (!wait(&x_full[st], (g >> 2) & 1, ab)) goto score_done;
                    // the buffer's previous step has been read: P^T by dV, dS^T by dK
                    if (g >= 2) {
                        uint64_t* used = is_s ? &dv_done[sb] : &dk_done[(g - 2) & 3];
                        if (!wait(used, (is_s ? (g - 2) >> 1 : (g - 2) >> 2) & 1, ab)) goto score_done;
                    }
                    tc_fence_after();
#pragma unroll
                    for (uint32_t c = 0; c < KP; ++c)
#pragma unroll
                        for (uint32_t ks = 0; ks < 4; ++ks)
                            mma_f16(d + sb * 64, da + ((c * 16384 + ks * 32) >> 4),
                                    dx + ((st * kStep + c * kPanel + ks * 32) >> 4), kIdescS, c + ks > 0 ? 1u : 0u);
                    mma_commit(&out[sb]);
                    if (n == ns - 1) mma_commit(&a_free);
                }
                ++tiles;
            }
        score_done:
            issued[is_s ? 2 : 3] = g;
        } else if (warp == 2 && lane == 0) {
            // ----------------------------------- dV and dK products ----
            const uint64_t dx = smem_desc(smem_u32(smem + SM::kX), kPanel, 1024, kSw128);
            const uint64_t dy = smem_desc(smem_u32(smem + SM::kY), kPanel, 1024, kSw128);
            uint32_t g = 0, gk = 0, tiles = 0;
            Work w;
            while (ring.take(tiles, w, true, false, ab)) {
                const int ns = w.ns;
#pragma unroll 1
                for (int n = 0; n < ns; ++n) {
                    const uint32_t st = g & 3, sb = g & 1;
                    if (n == 0 && tiles > 0 && !wait(&dv_empty, (tiles - 1) & 1, ab)) goto grad_done;
                    // (the softmax has seen the step's copies land before it wrote P^T)
                    if (!wait(&p_full[sb], (g >> 1) & 1, ab)) goto grad_done;
                    tc_fence_after();
#pragma unroll
                    for (uint32_t ks = 0; ks < kStatRows / 16; ++ks)
                        mma_f16_tmem_a(tV, tS + sb * 64 + ks * 8, dy + ((st * kStep + ks * 2048) >> 4), kIdescD,
                                       ks > 0 ? 1u : n);
                    mma_commit(&dv_done[sb]);
                    if (n == ns - 1) mma_commit(&dv_full);
                    ++g;
                    if (n == 0 && tiles > 0 && !wait(&dk_empty, (tiles - 1) & 1, ab)) goto grad_done;
                    if (!wait(&ds_full[sb], (gk >> 1) & 1, ab)) goto grad_done;
                    tc_fence_after();
#pragma unroll
                    for (uint32_t ks = 0; ks < kStatRows / 16; ++ks)
                        mma_f16_tmem_a(tK, tP + sb * 64 + ks * 8, dx + ((st * kStep + ks * 2048) >> 4), kIdescD,
                                       ks > 0 ? 1u : n);
                    mma_commit(&dk_done[st]);
                    if (n == ns - 1) mma_commit(&dk_full);
                    ++gk;
                }
                ++tiles;
            }
        grad_done:
            issued[4] = g;
            issued_k = gk;
        }
    } else if (warp < 8) {
        // ---------------------------------------------------- epilogue ----
        const int quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        uint8_t* stage = smem + SM::kEpi + quad * 4096;
        uint32_t tiles = 0;
        Work w;
        while (ring.take(tiles, w, lane == 0, true, ab)) {
            const int hk = w.hk, z = w.z, kb = w.tile << 7;
            float* slot = w.whole() ? nullptr : args.slots + (size_t)w.slot() * kv_slot_floats(kTcRows);
            auto rows_of = [&](const View& v) {
                T* out = static_cast<T*>(v.ptr) + z * v.s[0] + hk * v.s[1] + (kb + quad * 32) * v.s[2];
                const int64_t row_stride = v.s[2];
                const int end = p.Sk - kb - quad * 32;
                return [=](int i) -> T* { return i < end ? out + i * row_stride : nullptr; };
            };
            bool ok = wait(&dv_full, tiles & 1, ab, p.attempts);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            drain<T, DP>(tV + lane_base, &dv_empty, lane, row, kTcRows, slot ? slot + (size_t)kTcRows * kSlotD : nullptr,
                         1.0f, 1.0f / (1 << kPUp), args.D, stage, rows_of(args.dV));
            ok = wait(&dk_full, tiles & 1, ab, p.attempts);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const float down = kBf ? 1.0f : args.factor[w.rep].down;
            drain<T, DP>(tK + lane_base, &dk_empty, lane, row, kTcRows, slot, args.scale, down, args.D, stage,
                         rows_of(args.dK));
            ++tiles;
            if (threadIdx.x == 128 && w.s0 == 0 && !w.whole()) cut = w;
        }
    } else {
        regs_inc<kRegsSoftmax>();
        // ------------------------------------------------ P^T and dS^T ----
        const int wg = (warp - 8) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        uint32_t g = 0;
        for (uint32_t i = 0;; ++i) {
            int ns, first, j;
            float up = 1.f;
            {
                Work w;
                if (!ring.take(i, w, lane == 0, true, ab)) break;
                ns = w.ns, first = w.lo;
                j = (w.tile << 7) + row;  // this thread's key
                if (!kBf) up = args.factor[w.rep].up;
            }
            const int j_first = j - lane, j_last = j_first + 31;
#pragma unroll 1
            for (int n = 0; n < ns; ++n, ++g) {
                if ((g & 1) != (uint32_t)wg) continue;
                const uint32_t st = g & 3, ph = (g >> 1) & 1;
                // rows that see the key: tokens from the key's own to window - 1
                // later ones (a sink: all later ones), G rows each
                const int tok = p.Sk - p.Sq + (first + n) * kp.TQ;  // position of row 0
                // the warp's keys against the first and last row
                const bool full =
                    (tok >= j_last) & ((tok + kp.TQ - 1 - j_first < p.window) | (j_last < p.sinks));
                const float* stats = reinterpret_cast<const float*>(smem + SM::kStats + st * 8 * kStatRows);
                bool ok = wait(&x_full[st], (g >> 2) & 1, ab);
                ok = ok && wait(&s_full[wg], ph, ab);
                if (!__all_sync(0xffffffffu, ok)) goto ds_done;
                tc_fence_after();
                float x[64];
                tmem_ld64_sync(tS + lane_base + wg * 64, tS + lane_base + wg * 64 + 32,
                               *reinterpret_cast<uint32_t(*)[64]>(x));
                if (!full) {
                    const int c0 = imin(imin(imax(j - tok, 0), 64) * p.G, 64);
                    const int c1 = j < p.sinks ? 64 : imin(imin(imax(j - tok + p.window, 0), 64) * p.G, 64);
                    hide(x, below(c1) & ~below(c0));
                }
                {
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 64; i += 4) {
                        const float4 nl = *reinterpret_cast<const float4*>(stats + i);
                        const float2 c2v = make_float2(args.c2, args.c2);
                        const float2 y0 = __ffma2_rn(make_float2(x[i], x[i + 1]), c2v, make_float2(nl.x, nl.y));
                        const float2 y1 = __ffma2_rn(make_float2(x[i + 2], x[i + 3]), c2v, make_float2(nl.z, nl.w));
                        x[i] = ex2_approx(y0.x);
                        x[i + 1] = ex2_approx(y0.y);
                        x[i + 2] = ex2_approx(y1.x);
                        x[i + 3] = ex2_approx(y1.y);
                        pk[i / 2] = Pack2<T>::pack(x[i], x[i + 1]);
                        pk[i / 2 + 1] = Pack2<T>::pack(x[i + 2], x[i + 3]);
                    }
                    tmem_st32_sync(tS + lane_base + wg * 64, pk);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[wg]);
                ok = wait(&dp_full[wg], ph, ab);
                if (!__all_sync(0xffffffffu, ok)) goto ds_done;
                tc_fence_after();
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t r[32];
                    tmem_ld32_sync(tP + lane_base + wg * 64 + c * 32, r);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 dl = *reinterpret_cast<const float4*>(stats + kStatRows + c * 32 + i);
                        const float2 dp0 = make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                        const float2 dp1 = make_float2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
                        const float2 n0 = make_float2(-dl.x, -dl.y), n1 = make_float2(-dl.z, -dl.w);
                        const float2 d0 = kBf ? __fadd2_rn(dp0, n0) : __ffma2_rn(dp0, make_float2(up, up), n0);
                        const float2 d1 = kBf ? __fadd2_rn(dp1, n1) : __ffma2_rn(dp1, make_float2(up, up), n1);
                        const float2 e0 = __fmul2_rn(d0, make_float2(x[c * 32 + i], x[c * 32 + i + 1]));
                        const float2 e1 = __fmul2_rn(d1, make_float2(x[c * 32 + i + 2], x[c * 32 + i + 3]));
                        pk[c * 16 + i / 2] = Pack2<T>::pack(e0.x, e0.y);
                        pk[c * 16 + i / 2 + 1] = Pack2<T>::pack(e1.x, e1.y);
                    }
                }
                tmem_st32_sync(tP + lane_base + wg * 64, pk);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ds_full[wg]);
            }
        }
    ds_done:;
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        if (abort_flag) set_status(p.status, abort_flag);
        args.cuts[blockIdx.x].pieces = 0;
        if (cut.ns)
            write_cut(args.cuts, cut.seg, cut.rep, cut.tile, cut.n - cut.ns, [&](int c) { return plan.s[c].count; });
    }
    if (abort_flag) {
        if (threadIdx.x == 0) {
            drain_ring(x_full, 4, issued[0]);
            if (issued_a) drain_wait(&a_full, (issued_a - 1) & 1);
            drain_ring(s_full, 2, issued[2]);
            drain_ring(dp_full, 2, issued[3]);
            drain_ring(dv_done, 2, issued[4]);
            drain_ring(dk_done, 4, issued_k);
            drain_end();
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

template <typename T, int DP>
int launch(Call& c) {
    const int is_bf16 = std::is_same<T, __nv_bfloat16>::value;
    const Prob& p = c.p;
    CUtensorMap mq, mk, mv, mg, mq2, mg2;
    const int tq2 = kStatRows / p.G;
    int rc = query_map(&mq, c.Q, c, is_bf16, p.Sq, p.TQ);
    if (!rc) rc = query_map(&mg, c.dO, c, is_bf16, p.Sq, p.TQ);
    if (!rc) rc = query_map(&mq2, c.Q, c, is_bf16, p.Sq, tq2);
    if (!rc) rc = query_map(&mg2, c.dO, c, is_bf16, p.Sq, tq2);
    if (!rc) rc = key_map(&mk, c.K, c, is_bf16, 128);
    if (!rc) rc = key_map(&mv, c.V, c, is_bf16, 128);
    if (rc) return rc;
    constexpr int smem = Smem<DP>::kAlloc;
    static std::atomic<uint64_t> prepared[2];
    if ((rc = prepare_kernel(dq_tc_kernel<T, DP>, smem, prepared[0]))) return rc;
    if ((rc = prepare_kernel(dkv_tc_kernel<T, DP>, smem, prepared[1]))) return rc;
    const int grid = imin(sm_count(), TcPlan::kCtas);
    Args a{p, c.dQ, c.dK, c.dV, c.stats, c.factor, c.D, (p.Sq + tq2 - 1) / tq2, c.scale, c.scale * kLog2e, c.cuts, c.slots};
    const KProb kp{1, p.rep, p.G, tq2, p.kshift, p.Hq, p.Hkv, p.Sq, p.Sk, p.window, p.sinks};
    TcPlan plan, kplan;
    bool cut, kcut;
    if ((rc = query_plan(c, grid, &plan.tab, plan.s, &cut))) return rc;
    if ((rc = key_plan(c, kp, grid, &kplan.tab, kplan.s, &kcut))) return rc;
    if ((rc = launch_tile_stats(c))) return rc;
    if ((rc = launch_behind(dq_tc_kernel<T, DP>, dim3(grid), kThreads, smem, c.stream, mq, mk, mv, mg, a, plan)))
        return rc;
    if (cut && (rc = launch_join(c, kTcRows, grid, true))) return rc;
    if ((rc = launch_behind(dkv_tc_kernel<T, DP>, dim3(grid), kThreads, smem, c.stream, mq2, mk, mv, mg2, a, kp, kplan)))
        return rc;
    return kcut ? launch_join_kv(c, kp, kTcRows, grid) : BSP_OK;
}

}  // namespace

int launch_backward_tc(Call& c) {
    c.p.kshift = 7;
    c.p.TQ = kTcRows / c.p.G;
    // a tile's steps: key tiles, or half tiles of query rows
    const int64_t keys = c.p.Sk >> 7, rows = c.p.Sq / (kStatRows / c.p.G);
    c.p.attempts = wait_attempts(c, (keys > rows ? keys : rows) + 2);
    if (c.dtype == BSP_BF16) return c.D <= 64 ? launch<__nv_bfloat16, 64>(c) : launch<__nv_bfloat16, 128>(c);
    return c.D <= 64 ? launch<__half, 64>(c) : launch<__half, 128>(c);
}

}  // namespace win
}  // namespace bsp
