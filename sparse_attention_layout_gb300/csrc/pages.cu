// Pages of a cache: which sequences hold which (fork, reserve, free, compact), and
// the moves of their contents (copy, keep).
//
// refs[x] is the number of table entries that hold page x, 0 for a free one; a
// table entry below 0 holds none.  The bookkeeping is on whole numbers, and pages
// are given out lowest first, so that results do not depend on timing.  It is
// small work bound by latency: a turn's tables are some thousand entries.
#include <cooperative_groups.h>

#include "common.cuh"
#include "window_args.h"

namespace cg = cooperative_groups;

namespace bsp {
namespace win {
namespace {

// ------------------------------------------------------------- bookkeeping --

struct Book {
    int* refs;
    int* table;
    int* kv_len;
    int n_seq, max_pages, n_pages, page_shift;
    int* status;

    __device__ __forceinline__ bool bad_len(int n) const { return n < 0 || n > (max_pages << page_shift); }
    __device__ __forceinline__ int held(int n) const { return (n + (1 << page_shift) - 1) >> page_shift; }
    // an entry's page, or -1
    __device__ __forceinline__ int page_of(int e) const {
        if (e < 0) return -1;
        if (e >= n_pages) {
            set_status(status, BSP_ERR_DEVICE_CHECK);
            return -1;
        }
        return e;
    }
};

constexpr int kT = 256;

// An entry per thread.
__global__ void __launch_bounds__(kT) free_kernel(const __grid_constant__ Book b) {
    cudaGridDependencySynchronize();
    const int n = b.n_seq * b.max_pages;
    for (int i = blockIdx.x * kT + threadIdx.x; i < n; i += gridDim.x * kT) {
        const int s = i / b.max_pages, j = i - s * b.max_pages, len = b.kv_len[s];
        if (b.bad_len(len)) {
            if (j == 0) set_status(b.status, BSP_ERR_DEVICE_CHECK);
            continue;
        }
        if (j < b.held(len)) continue;
        const int e = b.table[i];
        if (e < 0) continue;
        const int x = b.page_of(e);
        if (x >= 0) atomicSub(&b.refs[x], 1);
        b.table[i] = -1;
    }
}

// The tables and lengths as they were, for forks that read rows that others
// write.  (Both steps in one block over shared memory: 4.5 us for 96 tables of 48
// entries; this 3.1, and 2.5 for 8 of 40, where that took 1.9.)
__global__ void __launch_bounds__(kT) snapshot_kernel(const __grid_constant__ Book b, int* table, int* kv_len) {
    cudaGridDependencySynchronize();
    const int n = b.n_seq * b.max_pages;
    for (int i = blockIdx.x * kT + threadIdx.x; i < n; i += gridDim.x * kT) {
        table[i] = b.table[i];
        if (i < b.n_seq) kv_len[i] = b.kv_len[i];
    }
}

// Entry i of the table becomes its parent's entry.
__device__ __forceinline__ void fork_entry(const Book& b, int i, const int* parent, const int* table, const int* kv_len) {
    const int s = i / b.max_pages, j = i - s * b.max_pages, p = parent[s];
    if (p == s) return;
    const int len = p >= 0 && p < b.n_seq ? kv_len[p] : 0;
    if (p < -1 || p >= b.n_seq || b.bad_len(len)) {
        if (j == 0) set_status(b.status, BSP_ERR_DEVICE_CHECK);
        return;
    }
    const int old = b.page_of(table[i]);
    const int now = j < b.held(len) ? b.page_of(table[p * b.max_pages + j]) : -1;
    if (old >= 0) atomicSub(&b.refs[old], 1);
    if (now >= 0) atomicAdd(&b.refs[now], 1);
    b.table[i] = now;
    if (j == 0) b.kv_len[s] = len;
}

__global__ void __launch_bounds__(kT) fork_kernel(const __grid_constant__ Book b, const int* parent, const int* table,
                                                  const int* kv_len) {
    cudaGridDependencySynchronize();
    const int n = b.n_seq * b.max_pages;
    for (int i = blockIdx.x * kT + threadIdx.x; i < n; i += gridDim.x * kT) fork_entry(b, i, parent, table, kv_len);
}

// The threads of one block, or of a cluster of blocks, that work through a book
// together, phase after phase.
constexpr int kBig = 1024;
constexpr int kSteps = 4;  // pages of a thread and scan
constexpr int kTeam = 8;   // blocks of a cluster
struct Team {
    cg::cluster_group cluster;
    int rank, blocks;
    int parity = 0;
    uint32_t* red;          // 32 words of the block's shared memory
    int (*totals)[kTeam];   // of this scan and the last
    __device__ __forceinline__ Team(uint32_t* scratch, int (*both)[kTeam])
        : cluster(cg::this_cluster()), rank((int)cluster.block_rank()), blocks((int)cluster.num_blocks()), red(scratch),
          totals(both) {
        if (blocks > 1) cluster.sync();  // all of them have begun: their shared memory may be written
    }
    __device__ __forceinline__ int size() const { return blocks * kBig; }
    __device__ __forceinline__ int thread() const { return rank * kBig + threadIdx.x; }
    __device__ __forceinline__ void sync() {
        if (blocks == 1) __syncthreads();
        else cluster.sync();
    }
    // exclusive prefix over the block's threads; *total: the block's sum
    __device__ __forceinline__ int block_prefix(int v, int* total) {
        uint32_t all;
        const int x = (int)block_scan<kBig>((uint32_t)v, red, &all);
        *total = (int)all;
        return x;
    }
    // The same over the whole team.  Every block gets the same totals, so that loops
    // bounded by them, and with them the barriers, are the same in all.
    __device__ __forceinline__ int prefix(int v, int* total) {
        int x = block_prefix(v, total);
        if (blocks == 1) return x;
        int* mine = totals[parity];
        parity ^= 1;
        if (threadIdx.x < blocks) cluster.map_shared_rank(mine, threadIdx.x)[rank] = *total;
        cluster.sync();
        *total = 0;
        for (int r = 0; r < blocks; ++r) {
            if (r < rank) x += mine[r];
            *total += mine[r];
        }
        return x;
    }
    __device__ __forceinline__ int count(bool v) {
        if (blocks == 1) return __syncthreads_count(v);
        int total;
        prefix(v, &total);
        return total;
    }
};

struct ReserveArgs {
    Book b;
    const int* lengths;
    int *src, *dst;
    int *users, *first, *list;  // of each page
};

// Pages for the positions kv_len .. lengths - 1 of each sequence.  An item is a
// table entry that such a position falls into; items stand in the order of
// (sequence, entry).  An item without a page, or whose page others hold too, gets
// the next free page; of the items that share a page that nobody else holds, the
// first keeps it.  Its phases need each other's results, so a team works through
// them: one block for a turn's some hundred items, bound by the latency of a read or
// an atomic in each (200 sequences of 2 items among 5000 pages: 5.4 us).
__global__ void __launch_bounds__(kBig) reserve_kernel(const __grid_constant__ ReserveArgs a) {
    extern __shared__ int ends[];  // items up to each sequence's end
    __shared__ uint32_t red[32];
    __shared__ int totals[2][kTeam], items_of_first;
    const Book& b = a.b;
    Team team(red, totals);
    const int tid = team.thread();
    cudaGridDependencySynchronize();
    int head[kSteps];  // the first pages' holders, on their way early
#pragma unroll
    for (int k = 0; k < kSteps; ++k) head[k] = kSteps * tid + k < b.n_pages ? b.refs[kSteps * tid + k] : 1;
    // (by every block for itself)
    int items = 0;
    for (int s0 = 0; s0 < b.n_seq; s0 += kBig) {
        const int s = s0 + threadIdx.x;
        int n = 0;
        if (s < b.n_seq) {
            const int len = b.kv_len[s], want = a.lengths[s];
            if (b.bad_len(len) || b.bad_len(want)) set_status(b.status, BSP_ERR_DEVICE_CHECK);
            else if (want > len) n = b.held(want) - (len >> b.page_shift);
            if (team.rank == 0) a.src[s] = a.dst[s] = -1;
        }
        int total;
        const int at = team.block_prefix(n, &total);
        if (s < b.n_seq) ends[s] = items + at + n;
        items += total;
    }
    if (team.blocks > 1) {
        // the first block's number for all: their barriers must not part
        if (team.rank == 0 && threadIdx.x < team.blocks) *team.cluster.map_shared_rank(&items_of_first, threadIdx.x) = items;
        team.sync();
        items = items_of_first;
    } else {
        __syncthreads();
    }
    if (items == 0) return;
    // item i: its sequence, place in the row, what the entry holds, and the length
    struct Item {
        int s, j, e, len;
    };
    auto look_up = [&](int i) {
        int lo = 0, hi = b.n_seq - 1;
#pragma unroll 1
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (ends[mid] > i) hi = mid;
            else lo = mid + 1;
        }
        Item it;
        it.s = lo, it.len = b.kv_len[lo];
        it.j = imin((it.len >> b.page_shift) + i - (lo ? ends[lo - 1] : 0), b.max_pages - 1);
        it.e = b.table[lo * b.max_pages + it.j];
        return it;
    };
    // (each thread keeps its first one: looked up again in every phase, and with the
    // first pages' holders read where they are needed, a turn of 96 beams took 17.2 us,
    // not 14.6)
    const Item mine = tid < items ? look_up(tid) : Item{};
    auto item = [&](int i) { return i == tid ? mine : look_up(i); };
    bool shared = false;
    for (int i = tid; i < items; i += team.size()) {
        const int x = b.page_of(item(i).e);
        if (x < 0) continue;
        a.users[x] = 0;
        a.first[x] = INT32_MAX;
        shared |= b.refs[x] > 1;
    }
    shared = team.count(shared) > 0;
    if (shared) {
        for (int i = tid; i < items; i += team.size()) {
            const int x = b.page_of(item(i).e);
            if (x < 0) continue;
            atomicAdd(&a.users[x], 1);
            atomicMin(&a.first[x], i);
        }
        team.sync();
        // the first item of each page says what becomes of it: 0, it keeps the
        // page; 1, all of them leave it to others
        for (int i = tid; i < items; i += team.size()) {
            const int x = b.page_of(item(i).e);
            if (x < 0 || a.first[x] != i) continue;
            const int holders = b.refs[x], here = a.users[x];
            const bool leave = holders > here;
            if (holders > 1) b.refs[x] = leave ? holders - here : 1;
            a.users[x] = leave && holders > 1;
        }
        team.sync();
    }
    auto needs = [&](int i, int e) {
        if (e >= b.n_pages) return false;  // reported; left as it is
        return e < 0 || (shared && (a.users[e] != 0 || a.first[e] != i));
    };
    int need = 0;
    for (int i0 = 0; i0 < items; i0 += team.size()) {
        const int i = i0 + tid;
        need += team.count(i < items && needs(i, item(i).e));
    }
    // free pages, as many as there are needs (a page that is left is never free)
    int have = 0;
    for (int x0 = 0; x0 < b.n_pages && have < need; x0 += kSteps * team.size()) {
        const int x = x0 + kSteps * tid;
        bool is[kSteps];
        int n = 0;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            is[k] = x + k < b.n_pages && (x0 == 0 ? head[k] : b.refs[x + k]) <= 0;
            n += is[k];
        }
        int total;
        int at = have + team.prefix(n, &total);
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
            if (is[k]) a.list[at++] = x + k;
        have += total;
    }
    team.sync();
    int given = 0;
    for (int i0 = 0; i0 < items; i0 += team.size()) {
        const int i = i0 + tid;
        const Item it = i < items ? item(i) : Item{};
        const bool on = i < items && needs(i, it.e);
        int total;
        const int at = given + team.prefix(on, &total);
        given += total;
        if (!on) continue;
        if (at >= have) {
            // none left: a shared page stays shared
            if (it.e >= 0) atomicAdd(&b.refs[it.e], 1);
            set_status(b.status, BSP_ERR_OOM);
            continue;
        }
        const int x = a.list[at];
        b.table[it.s * b.max_pages + it.j] = x;
        b.refs[x] = 1;
        if (it.e >= 0 && it.j == it.len >> b.page_shift && (it.len & ((1 << b.page_shift) - 1))) {
            a.src[it.s] = it.e;
            a.dst[it.s] = x;
        }
    }
}

struct CompactArgs {
    Book b;  // refs and table as they are
    int *refs_out, *table_out;
    int *src, *dst;
    int *map, *live;  // of each page; one number
};

// Where the pages go: the k-th page in use behind the first n_live to the k-th
// free one among them.
__global__ void __launch_bounds__(kBig) compact_kernel(const __grid_constant__ CompactArgs a) {
    __shared__ uint32_t red[32];
    __shared__ int totals[2][kTeam];
    const Book& b = a.b;
    Team team(red, totals);
    const int tid = team.thread(), size = team.size(), half = b.n_pages / 2;
    cudaGridDependencySynchronize();
    int n = 0, live;
    for (int x = tid; x < b.n_pages; x += size) n += b.refs[x] > 0;
    team.prefix(n, &live);
    int moved = 0, holes = 0;
    for (int x0 = 0; x0 < b.n_pages; x0 += kSteps * size) {
        const int x = x0 + kSteps * tid;
        bool high[kSteps], low[kSteps];
        int mine = 0;  // (a chunk's two counts, 32768 at the most, in one scan)
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const bool in = x + k < b.n_pages, used = in && b.refs[x + k] > 0;
            high[k] = used && x + k >= live;
            low[k] = x + k < live && !used;
            mine += (int)high[k] | (int)low[k] << 16;
            if (in && x + k >= live) a.map[x + k] = x + k;
        }
        int total;
        const int before = team.prefix(mine, &total);
        int m = moved + (before & 0xffff), h = holes + (int)((uint32_t)before >> 16);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            if (high[k] && m < half) a.src[m++] = x + k;
            if (low[k] && h < half) a.dst[h++] = x + k;
        }
        moved += total & 0xffff;
        holes += (int)((uint32_t)total >> 16);
    }
    moved = imin(imin(moved, holes), half);  // equal, and no more, unless refs change under the call
    if (tid == 0) *a.live = live;
    for (int k = moved + tid; k < half; k += size) a.src[k] = a.dst[k] = -1;
    if (a.refs_out != b.refs)
        for (int x = tid; x < b.n_pages; x += size) a.refs_out[x] = b.refs[x];
    team.sync();
    for (int k = tid; k < moved; k += size) {
        const int x = a.src[k], y = a.dst[k];
        a.map[x] = y;
        a.refs_out[y] = b.refs[x];
        a.refs_out[x] = 0;
    }
}

__global__ void __launch_bounds__(kT) renumber_kernel(const __grid_constant__ CompactArgs a) {
    cudaGridDependencySynchronize();
    const Book& b = a.b;
    const int n = b.n_seq * b.max_pages, live = *a.live;
    for (int i = blockIdx.x * kT + threadIdx.x; i < n; i += gridDim.x * kT) {
        const int e = b.table[i], x = b.page_of(e);
        a.table_out[i] = x >= live ? a.map[x] : e;
    }
}

// ---------------------------------------------------------------- contents --

struct CopyArgs {
    View K, V;  // strides in 16-byte pieces
    const int *src, *dst;
    int n, n_pages, page, Hkv, row16;
    int* status;
};

constexpr int kAhead = 4;
constexpr int kCopyT = 128;

// blockIdx.x: a pair of pages; blockIdx.y: a share of the pieces of K's page, or
// (odd) of V's.  HBM-bound: 1122 pages of 32 slots of 8 heads of 128 columns, bf16,
// 294 MB: 48 us (6.2 TB/s); pages of 128 slots 6.6 TB/s.  (256 threads a block 51 us,
// 512 58; twice the pieces of a thread on their way 50, half as many 49; both
// caches by one thread 57.)
__global__ void __launch_bounds__(kCopyT) copy_kernel(const __grid_constant__ CopyArgs a) {
    cudaGridDependencySynchronize();
    const int pieces = a.Hkv * a.page * a.row16, step = (gridDim.y >> 1) * kCopyT;
    const View& v = blockIdx.y & 1 ? a.V : a.K;
    for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
        const int x = a.src[i], y = a.dst[i];
        if (x < 0 || y < 0) continue;
        if (x >= a.n_pages || y >= a.n_pages) {
            if (threadIdx.x == 0) set_status(a.status, BSP_ERR_DEVICE_CHECK);
            continue;
        }
        if (x == y) continue;
        const uint4* from = static_cast<const uint4*>(v.ptr) + x * v.s[0];
        uint4* to = static_cast<uint4*>(v.ptr) + y * v.s[0];
#pragma unroll 1
        for (int k0 = (blockIdx.y >> 1) * kCopyT + threadIdx.x; k0 < pieces; k0 += kAhead * step) {
            uint4 row[kAhead];
            int64_t at[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int k = k0 + j * step;
                if (k >= pieces) break;
                const int r = (uint32_t)k / (uint32_t)a.row16, c = k - r * a.row16;
                const int h = (uint32_t)r / (uint32_t)a.page, slot = r - h * a.page;
                at[j] = h * v.s[1] + slot * v.s[2] + c;
                row[j] = from[at[j]];
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (k0 + j * step < pieces) to[at[j]] = row[j];
        }
    }
}

struct KeepArgs {
    View K, V;  // strides in 16-byte pieces
    Prob p;
    const int *path, *count;
    int row16;
};

// The accepted nodes' rows to the positions behind the context: a thread moves
// one 16-byte column of all of them, in their order, so no row is overwritten
// before it was read (node d of the path has at least d nodes before it).
__global__ void __launch_bounds__(kT) keep_kernel(const __grid_constant__ KeepArgs a) {
    __shared__ int64_t from[kMaxNodes];  // a node; then its page and slot, or -1
    __shared__ int64_t to[kMaxNodes];
    const Prob& p = a.p;
    cudaGridDependencySynchronize();
    const int s = blockIdx.x, q0 = p.q_start[s], q1 = p.q_start[s + 1], kv = p.kv_len[s], n = q1 - q0, m = a.count[s];
    if (p.bad_seg(q0, q1, kv) || n > kMaxNodes || kv < n || m < 0 || m > n) {
        if (threadIdx.x == 0) set_status(p.status, BSP_ERR_DEVICE_CHECK);
        return;
    }
    const int ctx = kv - n, mask = (1 << p.page_shift) - 1;
    for (int d = threadIdx.x; d < m; d += kT) from[d] = a.path[q0 + d];
    __syncthreads();
    bool bad = false;
    for (int d = threadIdx.x; d < m; d += kT) bad |= from[d] < d || from[d] >= n || (d > 0 && from[d - 1] >= from[d]);
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) set_status(p.status, BSP_ERR_DEVICE_CHECK);
        return;
    }
    for (int d = threadIdx.x; d < m; d += kT) {
        const int x = (int)from[d];
        int64_t f = -1, t = -1;
        if (x != d) {
            const int pf = p.table[(int64_t)s * p.max_pages + ((ctx + x) >> p.page_shift)];
            const int pt = p.table[(int64_t)s * p.max_pages + ((ctx + d) >> p.page_shift)];
            if ((unsigned)pf >= (unsigned)p.n_pages || (unsigned)pt >= (unsigned)p.n_pages) {
                set_status(p.status, BSP_ERR_DEVICE_CHECK);
            } else {
                f = (int64_t)pf << 32 | ((ctx + x) & mask);
                t = (int64_t)pt << 32 | ((ctx + d) & mask);
            }
        }
        from[d] = f;
        to[d] = t;
    }
    __syncthreads();
    const int columns = 2 * p.Hkv * a.row16;
    for (int k = blockIdx.y * kT + threadIdx.x; k < columns; k += gridDim.y * kT) {
        const bool is_v = k >= p.Hkv * a.row16;
        const int r = is_v ? k - p.Hkv * a.row16 : k, h = r / a.row16, c = r - h * a.row16;
        const View& v = is_v ? a.V : a.K;
        uint4* base = static_cast<uint4*>(v.ptr) + h * v.s[1] + c;
        constexpr int kB = 8;
#pragma unroll 1
        for (int d0 = 0; d0 < m; d0 += kB) {
            uint4 x[kB];
#pragma unroll
            for (int i = 0; i < kB; ++i)
                if (d0 + i < m && from[d0 + i] >= 0)
                    x[i] = base[(from[d0 + i] >> 32) * v.s[0] + (int)from[d0 + i] * v.s[2]];
#pragma unroll
            for (int i = 0; i < kB; ++i)
                if (d0 + i < m && from[d0 + i] >= 0) base[(to[d0 + i] >> 32) * v.s[0] + (int)to[d0 + i] * v.s[2]] = x[i];
        }
    }
}

int blocks_for(int64_t n) {
    const int64_t b = (n + kT - 1) / kT, most = (int64_t)sm_count() * 8;
    return (int)(b < most ? b : most);
}

View in_16(const View& v, int elt) {
    View r = v;
    for (int64_t& s : r.s) s = s * elt / 16;
    return r;
}

int page_shift(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1; }

int check_sizes(int n_seq, int max_pages, int n_pages, int page) {
    if (n_seq < 0 || max_pages < 1 || n_pages < 1 || page_shift(page) < 0) return BSP_ERR_INVALID_ARG;
    if (n_seq > kMaxSeqs || (int64_t)max_pages * page > kMaxLen || (int64_t)n_seq * max_pages > kMaxLen ||
        n_pages > kMaxLen)
        return BSP_ERR_UNSUPPORTED;
    return BSP_OK;
}

template <typename... P>
int check_ints(P... ptr) {
    for (const void* p : {static_cast<const void*>(ptr)...}) {
        if (!p) return BSP_ERR_INVALID_ARG;
        if ((uintptr_t)p & 3u) return BSP_ERR_ALIGNMENT;
    }
    return BSP_OK;
}

// A book's team: one block, or a cluster where its pages are many scans of one.
// Compaction of 5000 pages 7.7 us with one block, 9.0 with eight; of 65536 48 and 14; of
// a million 700 and 124.  Reserving two pages for each of 200 sequences 5 and 10 us
// whatever the pages, until only the last ones are free (65536: 18 and 11, a million:
// 245 and 65); 128 pages for each of 256 prompts 103 and 26.  (The rule asks for the
// pages alone, since how many items there are is known on the device only: many
// prompts among few pages stay on one block.)
int team_of(int n_pages, int scans) { return n_pages > scans * kSteps * kBig ? kTeam : 1; }

template <typename A>
int launch_team(void (*kern)(const A), int blocks, size_t smem, cudaStream_t s, const A& a) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kBig);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = blocks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

size_t page_ints(int n_pages) { return round_up((size_t)n_pages * sizeof(int)); }

}  // namespace
}  // namespace win
}  // namespace bsp

using namespace bsp::win;

extern "C" size_t bsp_pages_workspace(int n_seq, int max_pages, int n_pages) {
    if (check_sizes(n_seq, max_pages, n_pages, 16)) return 0;
    const size_t fork = round_up((size_t)n_seq * max_pages * sizeof(int)) + round_up((size_t)n_seq * sizeof(int));
    const size_t reserve = 3 * page_ints(n_pages), compact = page_ints(n_pages) + 256;
    size_t n = fork > reserve ? fork : reserve;
    return n > compact ? n : compact;
}

extern "C" int bsp_pages_free(bsp_window_t w, int32_t* refs, int32_t* table, const int32_t* kv_len, int n_seq,
                              int max_pages, int n_pages, int page, void* stream) {
    int rc = check_handle(w, BSP_F32);
    if (!rc) rc = check_sizes(n_seq, max_pages, n_pages, page);
    if (rc || n_seq == 0) return rc;
    if ((rc = check_ints(refs, table, kv_len))) return rc;
    const Book b{refs, table, const_cast<int*>(kv_len), n_seq, max_pages, n_pages, page_shift(page), w->status};
    return launch_behind(free_kernel, dim3(blocks_for((int64_t)n_seq * max_pages)), kT, 0, (cudaStream_t)stream, b);
}

extern "C" int bsp_pages_fork(bsp_window_t w, int32_t* refs, int32_t* table, int32_t* kv_len, const int32_t* parent,
                              int n_seq, int max_pages, int n_pages, int page, void* workspace, size_t workspace_bytes,
                              void* stream) {
    int rc = check_handle(w, BSP_F32);
    if (!rc) rc = check_sizes(n_seq, max_pages, n_pages, page);
    if (rc || n_seq == 0) return rc;
    if ((rc = check_ints(refs, table, kv_len, parent))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, bsp_pages_workspace(n_seq, max_pages, n_pages)))) return rc;
    const Book b{refs, table, kv_len, n_seq, max_pages, n_pages, page_shift(page), w->status};
    int* was = static_cast<int*>(workspace);
    int* len = reinterpret_cast<int*>(static_cast<char*>(workspace) + round_up((size_t)n_seq * max_pages * sizeof(int)));
    const dim3 grid(blocks_for((int64_t)n_seq * max_pages));
    cudaStream_t s = (cudaStream_t)stream;
    if ((rc = launch_behind(snapshot_kernel, grid, kT, 0, s, b, was, len))) return rc;
    return launch_behind(fork_kernel, grid, kT, 0, s, b, parent, (const int*)was, (const int*)len);
}

extern "C" int bsp_pages_reserve(bsp_window_t w, int32_t* refs, int32_t* table, const int32_t* kv_len,
                                 const int32_t* lengths, int32_t* src, int32_t* dst, int n_seq, int max_pages,
                                 int n_pages, int page, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_handle(w, BSP_F32);
    if (!rc) rc = check_sizes(n_seq, max_pages, n_pages, page);
    if (rc || n_seq == 0) return rc;
    if ((rc = check_ints(refs, table, kv_len, lengths, src, dst))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, bsp_pages_workspace(n_seq, max_pages, n_pages)))) return rc;
    char* ws = static_cast<char*>(workspace);
    ReserveArgs a{};
    a.b = Book{refs, table, const_cast<int*>(kv_len), n_seq, max_pages, n_pages, page_shift(page), w->status};
    a.lengths = lengths;
    a.src = src, a.dst = dst;
    a.users = reinterpret_cast<int*>(ws);
    a.first = reinterpret_cast<int*>(ws + page_ints(n_pages));
    a.list = reinterpret_cast<int*>(ws + 2 * page_ints(n_pages));
    const int smem = n_seq * (int)sizeof(int);
    if (smem > 40 * 1024 && cudaFuncSetAttribute(reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kMaxSeqs * (int)sizeof(int)) != cudaSuccess)
        return BSP_ERR_CUDA;
    return launch_team(reserve_kernel, team_of(n_pages, 16), smem, (cudaStream_t)stream, a);
}

extern "C" int bsp_pages_compact(bsp_window_t w, const int32_t* refs, const int32_t* table, int32_t* refs_out,
                                 int32_t* table_out, int32_t* src, int32_t* dst, int n_seq, int max_pages, int n_pages,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_handle(w, BSP_F32);
    if (!rc) rc = check_sizes(n_seq, max_pages, n_pages, 16);
    if (rc) return rc;
    if ((rc = check_ints(refs, refs_out))) return rc;
    if (n_pages > 1 && (rc = check_ints(src, dst))) return rc;
    if (n_seq > 0 && (rc = check_ints(table, table_out))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, bsp_pages_workspace(n_seq, max_pages, n_pages)))) return rc;
    char* ws = static_cast<char*>(workspace);
    CompactArgs a{};
    a.b = Book{const_cast<int*>(refs), const_cast<int*>(table), nullptr, n_seq, max_pages, n_pages, 4, w->status};
    a.refs_out = refs_out, a.table_out = table_out;
    a.src = src, a.dst = dst;
    a.map = reinterpret_cast<int*>(ws);
    a.live = reinterpret_cast<int*>(ws + page_ints(n_pages));
    cudaStream_t s = (cudaStream_t)stream;
    if ((rc = launch_team(compact_kernel, team_of(n_pages, 4), 0, s, a)) || n_seq == 0) return rc;
    return launch_behind(renumber_kernel, dim3(blocks_for((int64_t)n_seq * max_pages)), kT, 0, s, a);
}

extern "C" int bsp_paged_copy(bsp_window_t w, int dtype, const bsp_tensor_t* K_cache, const bsp_tensor_t* V_cache,
                              const int32_t* src, const int32_t* dst, int n, int n_pages, int page, int Hkv, int D,
                              void* stream) {
    int rc = check_handle(w, dtype);
    if (rc) return rc;
    if (n < 0 || n_pages < 1 || Hkv < 1 || page_shift(page) < 0 || !valid_d(D)) return BSP_ERR_INVALID_ARG;
    if (n > kMaxLen || n_pages > kMaxLen || (int64_t)Hkv * page * D * 4 > kMaxLen) return BSP_ERR_UNSUPPORTED;
    const int elt = elt_bytes(dtype);
    View k, v;
    if ((rc = make_view(K_cache, n_pages, Hkv, page, D, elt, true, &k))) return rc;
    if ((rc = make_view(V_cache, n_pages, Hkv, page, D, elt, true, &v))) return rc;
    if (K_cache->ptr == V_cache->ptr) return BSP_ERR_INVALID_ARG;
    if (n == 0) return BSP_OK;
    if ((rc = check_ints(src, dst))) return rc;
    const CopyArgs a{in_16(k, elt), in_16(v, elt), src, dst, n, n_pages, page, Hkv, D * elt / 16, w->status};
    const int pieces = Hkv * page * a.row16, parts = 2 * imax(1, imin(pieces / (kCopyT * kAhead), 32));
    const int most = 16 * bsp::sm_count();
    return launch_behind(copy_kernel, dim3(imin(n, most), parts), kCopyT, 0, (cudaStream_t)stream, a);
}

extern "C" int bsp_paged_keep(bsp_window_t w, int dtype, const bsp_tensor_t* K_cache, const bsp_tensor_t* V_cache,
                              const int32_t* q_start, const int32_t* kv_len, const int32_t* table, const int32_t* path,
                              const int32_t* count, int T, int n_seq, int max_pages, int n_pages, int page, int Hkv,
                              int D, void* stream) {
    int rc = check_handle(w, dtype);
    if (rc) return rc;
    if (T < 0 || n_seq < 0 || max_pages < 1 || n_pages < 1 || Hkv < 1 || page_shift(page) < 0 || !valid_d(D))
        return BSP_ERR_INVALID_ARG;
    if (T > kMaxLen || n_seq > kMaxSeqs || (int64_t)max_pages * page > kMaxLen || (int64_t)Hkv * D > kMaxLen / 8)
        return BSP_ERR_UNSUPPORTED;
    const int elt = elt_bytes(dtype);
    KeepArgs a{};
    if ((rc = make_view(K_cache, n_pages, Hkv, page, D, elt, true, &a.K))) return rc;
    if ((rc = make_view(V_cache, n_pages, Hkv, page, D, elt, true, &a.V))) return rc;
    if (K_cache->ptr == V_cache->ptr) return BSP_ERR_INVALID_ARG;
    if (T == 0 || n_seq == 0) return BSP_OK;
    if ((rc = check_ints(q_start, kv_len, table, path, count))) return rc;
    a.K = in_16(a.K, elt), a.V = in_16(a.V, elt);
    a.p.T = T, a.p.nseg = n_seq, a.p.Hkv = Hkv;
    a.p.max_pages = max_pages, a.p.n_pages = n_pages, a.p.page_shift = page_shift(page);
    a.p.q_start = q_start, a.p.kv_len = kv_len, a.p.table = table, a.p.status = w->status;
    a.path = path, a.count = count;
    a.row16 = D * elt / 16;
    const int parts = imax(1, imin((2 * Hkv * a.row16 + kT - 1) / kT, 1024));
    return launch_behind(keep_kernel, dim3(n_seq, parts), kT, 0, (cudaStream_t)stream, a);
}
