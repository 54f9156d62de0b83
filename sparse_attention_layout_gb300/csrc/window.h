// Host-side declarations of the windowed attention operators.
#pragma once

#include <atomic>
#include <mutex>

#include "bsp_internal.h"
#include "window.cuh"

namespace bsp {
namespace win {
// Splits of dense launches, by their sizes (window_plan.cpp); the oldest give
// way.
struct Plans;
}  // namespace win
}  // namespace bsp

struct bsp_window_s {
    int window = 0, sinks = 0;  // as given (window 0: no limit)
    int device = -1;
    int* status = nullptr;      // device status word, and where it is read from
    std::mutex reading;
    bsp::win::Plans* plans = nullptr;
    std::atomic<int> attempts{0};  // of the wait for a tile, 0: as many as the call's sizes ask for
    std::atomic<int> family{0};  // kernels of the last call: 1 tensor cores, 2 CUDA cores
};

namespace bsp {
namespace win {

// A launch that may be set up while the kernel before it in the stream still
// runs; the kernel waits for that one's end (cudaGridDependencySynchronize)
// before it touches memory, so the order of a stream holds and only the
// launch's own latency is hidden.
template <typename... P, typename... A>
int launch_behind(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

// The tensor cores take P and dS in the call's type.  fp16 ends at 65504 and
// 2^-24 (its last full-precision value is 2^-14), and dS = P (dP - delta) leaves
// it on either side: over 16384 keys P is 2^-14, and dO may be 1e-4 or 1e4.  So
// the fp16 gradient holds P times 2^15, which its last position 1 allows, and dS
// times a power of two, one per (batch entry, KV head) since dK sums over the
// rows: |dP - delta| <= 2 |dO| |V| over the longest rows of dO and V, which
// leaves the largest dS below 2^15.  Both factors are taken out of the fp32 sums
// at the end, and are exact.  (Relative error of dQ over 6000 keys, dO of 1, 1e-2,
// 1e-3: 3.0e-4, 2.1e-4 of it the result's own rounding; unscaled 3.0e-4, 9.3e-4,
// 9.1e-3.  Cost: a pass over V and one small launch, 4 us of 41 for 1037 rows of
// 12 heads, 8 of 475 for 8192 rows of 32.)
constexpr int kPUp = 15;
struct DsFactor {
    float up;    // of dP - delta, which P times 2^kPUp then multiplies
    float down;  // 1 / (up 2^kPUp)
};
// Blocks that look for the longest rows of one of `rep` (batch entry, KV head)
// pairs: together enough to fill the GPU.
constexpr int kRangeParts = 512;
inline int range_parts(int64_t rep) {
    const int64_t fill = (16 * (int64_t)sm_count() + rep - 1) / rep;
    return fill < kRangeParts ? (int)fill : kRangeParts;
}
struct RangePart {
    float dO2, V2;  // largest sum of squares of a row
};

// One call's tensors and sizes, checked.
struct Call {
    const bsp_window_s* w;
    int dtype, D;
    float scale;
    View Q, K, V, O, dO, dQ, dK, dV;
    float* lse;
    int64_t lz, lh, lt;  // strides of lse (batch entry, head, row)
    // backward: rows' dO . O, with the strides of lse (CUDA cores), or kStatTile
    // floats per tile of kStatRows rows (tensor cores)
    float* stats;
    // fp16 gradient on the tensor cores: of each (batch entry, KV head) up to
    // range_parts() partial results, and the factors
    RangePart* range;
    DsFactor* factor;
    Prob p;              // TQ and kshift set by the launcher
    int Z;
    // workspace: partial results of cut tiles
    Cut* cuts;
    float* slots;
    cudaStream_t stream;
};

// Floats of one partial-result slot: the rows' raw output, running maxima and
// sums (forward), or raw dQ; the keys' raw dK and dV (backward).
constexpr int kSlotD = 128;
constexpr size_t slot_floats(int rows) { return (size_t)rows * (kSlotD + 2); }
constexpr size_t kv_slot_floats(int rows) { return (size_t)rows * kSlotD * 2; }
// Place in a slot of column col (a multiple of 4) of one of the tile's `rows`
// rows.  Many rows: four columns of all rows, then the next four, so that a warp
// whose threads are rows writes and reads 512 contiguous bytes (row after row,
// 16 bytes of 32 rows at a time: the gradient of 1037 tokens of 12 heads took 60
// us, not 37).  Few rows (a new token's heads): row after row (31 such tokens'
// join 5.1 us; by columns 7.1).
constexpr int kManyRows = 32;
struct SlotRows {
    int row, step;  // floats from a row to the next, from four columns to the next
    BSP_HD explicit SlotRows(int rows) : row(rows >= kManyRows ? 4 : kSlotD), step(rows >= kManyRows ? 4 * rows : 4) {}
    BSP_HD int at(int r, int col) const { return r * row + (col >> 2) * step; }
};
// CTAs per SM of the CUDA-core kernels (64-row tiles) and the tensor-core ones
// (128-row tiles); both need the same workspace
constexpr int kSimtPerSm = 2, kSimtRows = 64, kTcRows = 128;
static_assert(kSimtPerSm * kSimtRows <= kTcRows, "the workspace holds two slots of kTcRows rows per SM");
// query rows of a step of the tensor-core dK / dV kernel
constexpr int kStatRows = 64;
// such a step's statistics: fp16's dO . O, -lse log2(e), and dO . O as the dK /
// dV kernel takes it (fp16: with the factor of dS, which the dQ kernel puts in)
constexpr int kStatDot = 0, kStatLse = kStatRows, kStatDelta = 2 * kStatRows, kStatTile = 3 * kStatRows;

int launch_forward_simt(Call& c);
int launch_backward_simt(Call& c);
inline int wait_attempts(const Call& c, int64_t steps) {
    const int n = c.w->attempts.load();
    return n ? n : wait_attempts(steps);
}
int launch_forward_tc(Call& c);  // 16-bit types
int launch_backward_tc(Call& c);
int launch_append(const bsp_window_s* w, int dtype, const View& Kn, const View& Vn, const View& Kc, const View& Vc,
                  const Prob& p, int D, cudaStream_t s);
// the status word to its neighbour, and 0 in its place
int launch_take_status(const bsp_window_s* w, cudaStream_t s);
// zeros n0 x n1 x n2 rows of row16 16-byte pieces (elt: bytes of an element of v)
int launch_zero(const View& v, int elt, int64_t n0, int64_t n1, int64_t n2, int row16, cudaStream_t s);
// The split of a dense launch's query tiles (p) or key tiles (k) over `ctas`
// CTAs; *cut: some tile is shared between CTAs, so that a join has to follow.
// BSP_ERR_UNSUPPORTED: more steps than 31 bits count; BSP_ERR_OOM: the host has no
// memory for it.
Plans* plans_create();
void plans_destroy(Plans* p);
int query_plan(const Call& c, int ctas, Table* tab, CtaStart* starts, bool* cut);
int key_plan(const Call& c, const KProb& k, int ctas, Table* tab, CtaStart* starts, bool* cut);

// stats = rowsum(dO .* O) per row; the same and the rows' -lse log2(e), per
// tile, and fp16's factors
int launch_delta(const Call& c);
int launch_tile_stats(const Call& c);
// joins the pieces of cut tiles: forward / dQ (rows of query tiles) and dK, dV
int launch_join(const Call& c, int rows, int n_cta, bool is_dq);
int launch_join_kv(const Call& c, const KProb& kp, int rows, int n_cta);

}  // namespace win
}  // namespace bsp
