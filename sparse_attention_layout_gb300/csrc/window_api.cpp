// C ABI entry points of the windowed attention operators: the handle, argument
// checks, workspace layout and dispatch between the tensor-core and CUDA-core
// kernels.
#include <cstdint>
#include <cstdlib>
#include <new>

#include "window_args.h"

namespace {

using bsp::win::Call;
using bsp::win::check_handle;
using bsp::win::check_workspace;
using bsp::win::clash;
using bsp::win::kMaxGroup;
using bsp::win::kMaxLen;
using bsp::win::kMaxSeqs;
using bsp::win::make_view;
using bsp::win::Prob;
using bsp::win::round_up;
using bsp::win::valid_d;
using bsp::win::valid_dtype;
using bsp::win::View;

bool valid_scale(float s) { return s > 0.f && s <= 3.0e38f; }
bool force_simt() {
    const char* e = std::getenv("BSP_FORCE_SIMT");
    return e && e[0] == '1';
}

// The type alone decides the kernels: whatever keeps the tensor-core ones from
// running is an error, not a reason to take 15 to 37 times as long.
bool on_tensor_cores(bsp_window_t w, int dtype) {
    const bool tc = dtype != BSP_F32 && !force_simt();
    w->family = tc ? 1 : 2;
    return tc;
}

// Workspace: one record per CTA, two partial-result slots per CTA, and for the
// backward the query rows' statistics, in tiles, and what fp16 scales dS by.
size_t cuts_bytes() { return round_up(sizeof(bsp::win::Cut) * bsp::win::kSimtPerSm * bsp::sm_count()); }
size_t slots_bytes(bool backward) {
    const size_t rows = bsp::win::kTcRows;
    const size_t f = backward ? bsp::win::kv_slot_floats(rows) : bsp::win::slot_floats(rows);
    return round_up(f * sizeof(float) * 2 * bsp::sm_count());
}

size_t range_bytes(int Z, int Hkv) {
    const int64_t rep = (int64_t)Z * Hkv;
    return rep == 0 ? 0 : round_up((size_t)rep * bsp::win::range_parts(rep) * sizeof(bsp::win::RangePart));
}
size_t factor_bytes(int Z, int Hkv) { return round_up((size_t)Z * Hkv * sizeof(bsp::win::DsFactor)); }
// of each tile's rows (more than the one float per row that the CUDA-core kernels
// keep)
size_t stats_bytes(int Z, int Hq, int Hkv, int Sq) {
    const size_t rows = bsp::win::kStatRows, tq = rows / (Hq / Hkv);
    return round_up((size_t)Z * Hkv * ((Sq + tq - 1) / tq) * bsp::win::kStatTile * sizeof(float));
}

void set_rule(const bsp_window_s* w, Prob* p) {
    bsp::win::set_rule(w, &p->window, &p->sinks);
    p->status = w->status;
}

int check_dense(int Z, int Hq, int Hkv, int Sq, int Sk, int D, float scale) {
    if (Z < 0 || Hq < 1 || Hkv < 1 || Sq < 0 || Sk < 0 || !valid_d(D) || !valid_scale(scale)) return BSP_ERR_INVALID_ARG;
    if (Hq % Hkv) return BSP_ERR_INVALID_ARG;
    // (the split refuses what has more steps than 32 bits count)
    if (Hq / Hkv > kMaxGroup || Sq > kMaxLen || Sk > kMaxLen || (int64_t)Z * Hkv > kMaxLen) return BSP_ERR_UNSUPPORTED;
    return BSP_OK;
}

void dense_prob(const bsp_window_s* w, int Z, int Hq, int Hkv, int Sq, int Sk, Prob* p) {
    set_rule(w, p);
    p->paged = 0;
    p->nseg = 1;
    p->rep = Z * Hkv;
    p->G = Hq / Hkv;
    p->Hq = Hq, p->Hkv = Hkv, p->Sq = Sq, p->Sk = Sk;
}

}  // namespace

extern "C" int bsp_window_create(int window, int sinks, void* stream, bsp_window_t* out) {
    if (!out || window < 0 || sinks < 0) return BSP_ERR_INVALID_ARG;
    *out = nullptr;
    bsp_window_s* w = new (std::nothrow) bsp_window_s;
    if (!w) return BSP_ERR_OOM;
    w->window = window;
    w->sinks = sinks;
    if (!(w->plans = bsp::win::plans_create())) {
        delete w;
        return BSP_ERR_OOM;
    }
    int rc = BSP_OK;
    if (cudaGetDevice(&w->device) != cudaSuccess) {
        rc = BSP_ERR_CUDA;
    } else if (cudaMalloc(&w->status, 2 * sizeof(int)) != cudaSuccess) {
        (void)cudaGetLastError();
        rc = BSP_ERR_OOM;
    } else if (cudaMemsetAsync(w->status, 0, 2 * sizeof(int), (cudaStream_t)stream) != cudaSuccess) {
        cudaFree(w->status);
        rc = BSP_ERR_CUDA;
    }
    if (rc) {
        bsp::win::plans_destroy(w->plans);
        delete w;
        return rc;
    }
    *out = w;
    return BSP_OK;
}

extern "C" int bsp_window_destroy(bsp_window_t w) {
    if (!w) return BSP_OK;
    cudaFree(w->status);  // waits for the device's work
    bsp::win::plans_destroy(w->plans);
    delete w;
    return BSP_OK;
}

extern "C" int bsp_window_info(bsp_window_t w, int* window, int* sinks) {
    if (!w) return BSP_ERR_INVALID_ARG;
    if (window) *window = w->window;
    if (sinks) *sinks = w->sinks;
    return BSP_OK;
}

extern "C" int bsp_window_status(bsp_window_t w, void* stream) {
    int rc = check_handle(w, BSP_F32);
    if (rc) return rc;
    // read and cleared in one step on the stream: what a call on another stream
    // reports meanwhile stays for the next reader
    std::lock_guard<std::mutex> lock(w->reading);
    cudaStream_t s = (cudaStream_t)stream;
    int word = 0;
    if ((rc = bsp::win::launch_take_status(w, s))) return rc;
    if (cudaMemcpyAsync(&word, w->status + 1, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return BSP_ERR_CUDA;
    return cudaStreamSynchronize(s) == cudaSuccess ? word : BSP_ERR_CUDA;
}

extern "C" size_t bsp_window_attention_workspace(int Z, int Hq, int Hkv, int Sq, int backward) {
    if (Z < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq / Hkv > kMaxGroup || Sq < 0) return 0;
    size_t n = cuts_bytes() + slots_bytes(backward != 0);
    if (backward) n += range_bytes(Z, Hkv) + factor_bytes(Z, Hkv) + stats_bytes(Z, Hq, Hkv, Sq);
    return n;
}

extern "C" size_t bsp_paged_attention_workspace(void) { return cuts_bytes() + slots_bytes(false); }

extern "C" int bsp_window_attention(bsp_window_t w, int dtype, const bsp_tensor_t* Q, const bsp_tensor_t* K,
                                    const bsp_tensor_t* V, const bsp_tensor_t* O, float* lse, int Z, int Hq, int Hkv,
                                    int Sq, int Sk, int D, float scale, void* workspace, size_t workspace_bytes,
                                    void* stream) {
    int rc = check_handle(w, dtype);
    if (!rc) rc = check_dense(Z, Hq, Hkv, Sq, Sk, D, scale);
    if (rc) return rc;
    if (Z == 0 || Sq == 0) return BSP_OK;
    Call c{};
    const int elt = dtype == BSP_F32 ? 4 : 2;
    if ((rc = make_view(Q, Z, Hq, Sq, D, elt, false, &c.Q))) return rc;
    if (Sk > 0) {
        if ((rc = make_view(K, Z, Hkv, Sk, D, elt, false, &c.K))) return rc;
        if ((rc = make_view(V, Z, Hkv, Sk, D, elt, false, &c.V))) return rc;
    }
    if ((rc = make_view(O, Z, Hq, Sq, D, elt, true, &c.O))) return rc;
    if (Sk > 0 ? clash({O}, {Q, K, V}) : clash({O}, {Q})) return BSP_ERR_INVALID_ARG;
    if ((uintptr_t)lse & 15u) return BSP_ERR_ALIGNMENT;
    if ((rc = check_workspace(workspace, workspace_bytes, bsp_window_attention_workspace(Z, Hq, Hkv, Sq, 0)))) return rc;
    if (Sk == 0) c.K = c.V = c.Q;  // no key at all: zeros and -inf, by the kernels' hidden step over Q's own first rows
    c.w = w, c.dtype = dtype, c.D = D, c.scale = scale, c.Z = Z;
    c.lse = lse;
    c.lz = (int64_t)Hq * Sq, c.lh = Sq, c.lt = 1;
    dense_prob(w, Z, Hq, Hkv, Sq, Sk, &c.p);
    c.cuts = static_cast<bsp::win::Cut*>(workspace);
    c.slots = reinterpret_cast<float*>(static_cast<char*>(workspace) + cuts_bytes());
    c.stream = (cudaStream_t)stream;
    return on_tensor_cores(w, dtype) ? bsp::win::launch_forward_tc(c) : bsp::win::launch_forward_simt(c);
}

extern "C" int bsp_window_attention_backward(bsp_window_t w, int dtype, const bsp_tensor_t* Q, const bsp_tensor_t* K,
                                             const bsp_tensor_t* V, const bsp_tensor_t* O, const bsp_tensor_t* dO,
                                             const float* lse, const bsp_tensor_t* dQ, const bsp_tensor_t* dK,
                                             const bsp_tensor_t* dV, int Z, int Hq, int Hkv, int Sq, int Sk, int D,
                                             float scale, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_handle(w, dtype);
    if (!rc) rc = check_dense(Z, Hq, Hkv, Sq, Sk, D, scale);
    if (rc) return rc;
    if (Z == 0) return BSP_OK;
    Call c{};
    const int elt = dtype == BSP_F32 ? 4 : 2;
    cudaStream_t s = (cudaStream_t)stream;
    if (Sk > 0) {
        if ((rc = make_view(K, Z, Hkv, Sk, D, elt, false, &c.K))) return rc;
        if ((rc = make_view(V, Z, Hkv, Sk, D, elt, false, &c.V))) return rc;
        if ((rc = make_view(dK, Z, Hkv, Sk, D, elt, true, &c.dK))) return rc;
        if ((rc = make_view(dV, Z, Hkv, Sk, D, elt, true, &c.dV))) return rc;
    }
    if (Sq > 0) {
        if ((rc = make_view(Q, Z, Hq, Sq, D, elt, false, &c.Q))) return rc;
        if ((rc = make_view(O, Z, Hq, Sq, D, elt, false, &c.O))) return rc;
        if ((rc = make_view(dO, Z, Hq, Sq, D, elt, false, &c.dO))) return rc;
        if ((rc = make_view(dQ, Z, Hq, Sq, D, elt, true, &c.dQ))) return rc;
        if (!lse) return BSP_ERR_INVALID_ARG;
        if ((uintptr_t)lse & 15u) return BSP_ERR_ALIGNMENT;
    }
    if (Sq == 0 && Sk == 0) return BSP_OK;
    if (Sq == 0   ? clash({dK, dV}, {K, V})
        : Sk == 0 ? clash({dQ}, {Q, O, dO})
                  : clash({dQ, dK, dV}, {Q, K, V, O, dO}))
        return BSP_ERR_INVALID_ARG;
    // no pair at all: every gradient is 0
    const int row16 = D * elt / 16;
    if (Sq == 0) {
        rc = bsp::win::launch_zero(c.dK, elt, Z, Hkv, Sk, row16, s);
        return rc ? rc : bsp::win::launch_zero(c.dV, elt, Z, Hkv, Sk, row16, s);
    }
    if (Sk == 0) return bsp::win::launch_zero(c.dQ, elt, Z, Hq, Sq, row16, s);
    if ((rc = check_workspace(workspace, workspace_bytes, bsp_window_attention_workspace(Z, Hq, Hkv, Sq, 1)))) return rc;
    c.w = w, c.dtype = dtype, c.D = D, c.scale = scale, c.Z = Z;
    c.lse = const_cast<float*>(lse);
    c.lz = (int64_t)Hq * Sq, c.lh = Sq, c.lt = 1;
    const View all = c.dQ;
    const int none = Sq > Sk ? Sq - Sk : 0;
    if (none > 0) {
        // the first queries stand before position 0: their dQ is 0, and the
        // kernels never meet their rows, which may hold anything
        for (View* v : {&c.Q, &c.O, &c.dO, &c.dQ}) v->ptr = static_cast<char*>(v->ptr) + v->s[2] * none * elt;
        c.lse += none;
        Sq = Sk;
    }
    dense_prob(w, Z, Hq, Hkv, Sq, Sk, &c.p);
    char* ws = static_cast<char*>(workspace);
    c.cuts = reinterpret_cast<bsp::win::Cut*>(ws);
    c.slots = reinterpret_cast<float*>(ws + cuts_bytes());
    ws += cuts_bytes() + slots_bytes(true);
    c.range = reinterpret_cast<bsp::win::RangePart*>(ws);
    c.factor = reinterpret_cast<bsp::win::DsFactor*>(ws + range_bytes(Z, Hkv));
    c.stats = reinterpret_cast<float*>(ws + range_bytes(Z, Hkv) + factor_bytes(Z, Hkv));
    c.stream = s;
    rc = on_tensor_cores(w, dtype) ? bsp::win::launch_backward_tc(c) : bsp::win::launch_backward_simt(c);
    return rc || none == 0 ? rc : bsp::win::launch_zero(all, elt, Z, Hq, none, row16, s);
}

namespace {
// `nodes`: the most a tree may have, 0 for plain new tokens.
int paged_prob(bsp_window_t w, const int32_t* q_start, const int32_t* kv_len, const int32_t* table, int T, int n_seq,
               int max_pages, int n_pages, int page, int Hq, int Hkv, int D, int nodes, Prob* p) {
    if (T < 0 || n_seq < 0 || max_pages < 1 || n_pages < 1 || Hq < 1 || Hkv < 1 || !valid_d(D)) return BSP_ERR_INVALID_ARG;
    if (page != 16 && page != 32 && page != 64 && page != 128) return BSP_ERR_INVALID_ARG;
    if (Hq % Hkv) return BSP_ERR_INVALID_ARG;
    if (Hq / Hkv > kMaxGroup || T > kMaxLen || n_seq > kMaxSeqs || (int64_t)max_pages * page > kMaxLen)
        return BSP_ERR_UNSUPPORTED;
    set_rule(w, p);
    // tiles and steps are counted in 32 bits; a tile holds 64 rows and a step 64
    // keys at the least, but a sequence's last tile may hold one row, and a tile's
    // steps go over the tables' keys or, if they are fewer, its sinks and windows
    const int64_t tq = 64 / (Hq / Hkv), qt = T <= n_seq ? T : (T + tq - 1) / tq + n_seq;
    const int64_t all = ((int64_t)max_pages * page + 63) / 64 + 1;
    const int64_t span = nodes > tq ? nodes : tq;  // of the rows' own slots
    const int64_t near = ((int64_t)p->sinks + 63) / 64 + ((int64_t)p->window + span + 63) / 64 + 1;
    const int64_t kt = near < all ? near : all;
    if (qt > 0 && (kt > (1ll << 31) / qt || Hkv > (1ll << 31) / (qt * kt) - 1)) return BSP_ERR_UNSUPPORTED;
    if (T == 0 || n_seq == 0) return BSP_OK;
    if (!q_start || !kv_len || !table) return BSP_ERR_INVALID_ARG;
    if (((uintptr_t)q_start | (uintptr_t)kv_len | (uintptr_t)table) & 3u) return BSP_ERR_ALIGNMENT;
    p->paged = 1;
    p->nseg = n_seq;
    p->rep = Hkv;
    p->G = Hq / Hkv;
    p->Hq = Hq, p->Hkv = Hkv;
    p->T = T, p->max_pages = max_pages, p->n_pages = n_pages;
    p->page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    p->q_start = q_start, p->kv_len = kv_len, p->table = table;
    return BSP_OK;
}
}  // namespace

extern "C" int bsp_paged_append(bsp_window_t w, int dtype, const bsp_tensor_t* K, const bsp_tensor_t* V,
                                const bsp_tensor_t* K_cache, const bsp_tensor_t* V_cache, const int32_t* q_start,
                                const int32_t* kv_len, const int32_t* table, int T, int n_seq, int max_pages,
                                int n_pages, int page, int Hkv, int D, void* stream) {
    int rc = check_handle(w, dtype);
    Prob p{};
    if (!rc) rc = paged_prob(w, q_start, kv_len, table, T, n_seq, max_pages, n_pages, page, Hkv, Hkv, D, 0, &p);
    if (rc || T == 0 || n_seq == 0) return rc;
    const int elt = dtype == BSP_F32 ? 4 : 2;
    View kn, vn, kc, vc;
    // new rows [T][Hkv][D]: token, head
    if ((rc = make_view(K, 1, Hkv, T, D, elt, false, &kn))) return rc;
    if ((rc = make_view(V, 1, Hkv, T, D, elt, false, &vn))) return rc;
    if ((rc = make_view(K_cache, n_pages, Hkv, page, D, elt, true, &kc))) return rc;
    if ((rc = make_view(V_cache, n_pages, Hkv, page, D, elt, true, &vc))) return rc;
    if (clash({K_cache, V_cache}, {K, V})) return BSP_ERR_INVALID_ARG;
    return bsp::win::launch_append(w, dtype, kn, vn, kc, vc, p, D, (cudaStream_t)stream);
}

namespace {
// Attention over pages: of plain new tokens, or (words > 0) of trees.
int paged_attention(bsp_window_t w, int dtype, const bsp_tensor_t* Q, const bsp_tensor_t* K_cache,
                    const bsp_tensor_t* V_cache, const bsp_tensor_t* O, float* lse, const int32_t* q_start,
                    const int32_t* kv_len, const int32_t* table, const int32_t* pos, const uint32_t* bits, int words, int T,
                    int n_seq, int max_pages, int n_pages, int page, int Hq, int Hkv, int D, float scale, void* workspace,
                    size_t workspace_bytes, void* stream) {
    int rc = check_handle(w, dtype);
    Call c{};
    if (!rc) rc = paged_prob(w, q_start, kv_len, table, T, n_seq, max_pages, n_pages, page, Hq, Hkv, D, 32 * words, &c.p);
    if (rc) return rc;
    if (!valid_scale(scale)) return BSP_ERR_INVALID_ARG;
    if (T == 0 || n_seq == 0) return BSP_OK;
    if (words) {
        if (!pos || !bits) return BSP_ERR_INVALID_ARG;
        if (((uintptr_t)pos | (uintptr_t)bits) & 3u) return BSP_ERR_ALIGNMENT;
        c.p.pos = pos, c.p.bits = bits, c.p.words = words;
    }
    const int elt = dtype == BSP_F32 ? 4 : 2;
    if ((rc = make_view(Q, 1, Hq, T, D, elt, false, &c.Q))) return rc;
    if ((rc = make_view(K_cache, n_pages, Hkv, page, D, elt, false, &c.K))) return rc;
    if ((rc = make_view(V_cache, n_pages, Hkv, page, D, elt, false, &c.V))) return rc;
    if ((rc = make_view(O, 1, Hq, T, D, elt, true, &c.O))) return rc;
    if (clash({O}, {Q, K_cache, V_cache})) return BSP_ERR_INVALID_ARG;
    if ((uintptr_t)lse & 15u) return BSP_ERR_ALIGNMENT;
    if ((rc = check_workspace(workspace, workspace_bytes, bsp_paged_attention_workspace()))) return rc;
    c.w = w, c.dtype = dtype, c.D = D, c.scale = scale, c.Z = 1;
    c.lse = lse;
    c.lz = 0, c.lh = 1, c.lt = Hq;
    c.cuts = static_cast<bsp::win::Cut*>(workspace);
    c.slots = reinterpret_cast<float*>(static_cast<char*>(workspace) + cuts_bytes());
    c.stream = (cudaStream_t)stream;
    return on_tensor_cores(w, dtype) ? bsp::win::launch_forward_tc(c) : bsp::win::launch_forward_simt(c);
}
}  // namespace

extern "C" int bsp_paged_attention(bsp_window_t w, int dtype, const bsp_tensor_t* Q, const bsp_tensor_t* K_cache,
                                   const bsp_tensor_t* V_cache, const bsp_tensor_t* O, float* lse,
                                   const int32_t* q_start, const int32_t* kv_len, const int32_t* table, int T,
                                   int n_seq, int max_pages, int n_pages, int page, int Hq, int Hkv, int D, float scale,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    return paged_attention(w, dtype, Q, K_cache, V_cache, O, lse, q_start, kv_len, table, nullptr, nullptr, 0, T, n_seq,
                           max_pages, n_pages, page, Hq, Hkv, D, scale, workspace, workspace_bytes, stream);
}

extern "C" int bsp_paged_tree_attention(bsp_window_t w, int dtype, const bsp_tensor_t* Q, const bsp_tensor_t* K_cache,
                                        const bsp_tensor_t* V_cache, const bsp_tensor_t* O, float* lse,
                                        const int32_t* q_start, const int32_t* kv_len, const int32_t* table,
                                        const int32_t* positions, const uint32_t* bits, int T, int n_seq, int max_pages,
                                        int n_pages, int page, int Hq, int Hkv, int D, int words, float scale,
                                        void* workspace, size_t workspace_bytes, void* stream) {
    if (words < 1) return BSP_ERR_INVALID_ARG;
    if (words > bsp::win::kMaxNodes / 32) return BSP_ERR_UNSUPPORTED;
    return paged_attention(w, dtype, Q, K_cache, V_cache, O, lse, q_start, kv_len, table, positions, bits, words, T, n_seq,
                           max_pages, n_pages, page, Hq, Hkv, D, scale, workspace, workspace_bytes, stream);
}

extern "C" int bsp_diag_window_wait_limit(bsp_window_t w, int attempts) {
    if (!w || attempts < 0) return BSP_ERR_INVALID_ARG;
    w->attempts = attempts;
    return BSP_OK;
}

extern "C" int bsp_diag_window_attempts(int64_t steps) { return steps < 0 ? 0 : bsp::win::wait_attempts(steps); }

extern "C" int bsp_diag_window_family(bsp_window_t w) { return w ? w->family.load() : BSP_ERR_INVALID_ARG; }

extern "C" int bsp_diag_window_tiles(int window, int sinks, int a, int b, int shift, int* n, int* tiles, int cap) {
    if (window < 0 || sinks < 0 || b < a || b - a >= 128 || shift < 4 || shift > 7 || !n || cap < 0 || (cap && !tiles))
        return BSP_ERR_INVALID_ARG;
    if (a < -kMaxLen || b > kMaxLen) return BSP_ERR_UNSUPPORTED;
    bsp_window_s w;
    w.window = window, w.sinks = sinks;
    Prob p{};
    set_rule(&w, &p);
    const bsp::win::Span s = bsp::win::span_of(a, b, p.window, p.sinks, shift);
    *n = s.n;
    for (int i = 0; i < s.n && i < cap; ++i) tiles[i] = s.tile(i);
    return BSP_OK;
}

extern "C" int bsp_diag_window_queries(int window, int sinks, int Sq, int Sk, int tokens, int shift, int t, int* first,
                                       int* n) {
    if (window < 0 || sinks < 0 || Sq < 1 || Sk < 1 || tokens < 1 || tokens > 128 || shift < 4 || shift > 7 || t < 0 ||
        !first || !n)
        return BSP_ERR_INVALID_ARG;
    if (Sq > kMaxLen || Sk > kMaxLen) return BSP_ERR_UNSUPPORTED;
    if (((int64_t)t << shift) >= Sk) return BSP_ERR_INVALID_ARG;
    bsp_window_s w;
    w.window = window, w.sinks = sinks;
    Prob p{};
    set_rule(&w, &p);
    const bsp::win::KProb k{1, 1, 1, tokens, shift, 1, 1, Sq, Sk, p.window, p.sinks};
    k.qrange(t, first, n);
    return BSP_OK;
}
