// Argument checks that the C entry points of the windowed attention, the paged
// cache and the operators beside them share.
#pragma once

#include <cstdint>
#include <initializer_list>

#include "window.h"

namespace bsp {
namespace win {

inline bool valid_dtype(int d) { return d == BSP_F32 || d == BSP_BF16 || d == BSP_F16; }
inline bool valid_d(int D) { return D >= 16 && D <= 128 && D % 16 == 0; }
inline int elt_bytes(int dtype) { return dtype == BSP_F32 ? 4 : 2; }
inline size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

inline int check_handle(bsp_window_t w, int dtype) {
    if (!w || !valid_dtype(dtype)) return BSP_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return BSP_ERR_CUDA;
    return dev == w->device ? BSP_OK : BSP_ERR_INVALID_ARG;
}

// A tensor of extents n0, n1, n2 and D contiguous elements: pointer and the
// strides that are used must be multiples of 16 bytes, strides positive (a
// stride whose extent is 1 is never used).  Outputs must not overlap
// themselves: taken from the smallest, each stride covers what lies below it.
inline int make_view(const bsp_tensor_t* t, int64_t n0, int64_t n1, int64_t n2, int D, int elt, bool out, View* v) {
    if (!t || !t->ptr) return BSP_ERR_INVALID_ARG;
    if ((uintptr_t)t->ptr & 15u) return BSP_ERR_ALIGNMENT;
    const int64_t n[3] = {n0, n1, n2};
    v->ptr = t->ptr;
    for (int i = 0; i < 3; ++i) {
        int64_t s = t->stride[i];
        if (n[i] <= 1) {
            s = D;  // any legal value: the index is always 0
        } else {
            if (s <= 0 || s > (int64_t)1 << 38) return BSP_ERR_INVALID_ARG;
            if (s * elt % 16) return BSP_ERR_ALIGNMENT;
        }
        v->s[i] = s;
    }
    if (out) {
        int64_t below = D;  // elements from the first to the last of the dimensions so far, plus one
        bool used[3] = {false, false, false};
        for (int k = 0; k < 3; ++k) {
            int at = -1;
            for (int i = 0; i < 3; ++i)
                if (!used[i] && n[i] > 1 && (at < 0 || v->s[i] < v->s[at])) at = i;
            if (at < 0) break;
            used[at] = true;
            if (v->s[at] < below) return BSP_ERR_INVALID_ARG;
            below += v->s[at] * (n[at] - 1);
        }
    }
    return BSP_OK;
}

// An output in an input's place (or another output's) would be overwritten
// while other blocks still read it.
inline bool clash(std::initializer_list<const bsp_tensor_t*> out, std::initializer_list<const bsp_tensor_t*> in) {
    for (auto o = out.begin(); o != out.end(); ++o) {
        if (!(*o)->ptr) continue;
        for (const bsp_tensor_t* i : in)
            if (i->ptr == (*o)->ptr) return true;
        for (auto q = out.begin(); q != o; ++q)
            if ((*q)->ptr == (*o)->ptr) return true;
    }
    return false;
}

// window and sinks as the kernels take them
inline void set_rule(const bsp_window_s* w, int* window, int* sinks) {
    *window = w->window == 0 || w->window > kMaxLen ? kMaxLen : w->window;
    *sinks = w->sinks > kMaxLen ? kMaxLen : w->sinks;
}

inline int check_workspace(const void* ws, size_t have, size_t need) {
    if (!ws) return BSP_ERR_INVALID_ARG;
    if ((uintptr_t)ws & 255u) return BSP_ERR_ALIGNMENT;
    return have < need ? BSP_ERR_INVALID_ARG : BSP_OK;
}

}  // namespace win
}  // namespace bsp
