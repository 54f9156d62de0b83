// Rotary positions of Q and K: pair i of a head (x_a, x_b) at position p turns by
// the angle p * f_i,
//     y_a = A (x_a cos - x_b sin),   y_b = A (x_b cos + x_a sin),
// pairs (i, i + R / 2) or (2 i, 2 i + 1) of the head's first R columns; the
// others are copied.  The gradient is the transposed map: the same with the
// angle's sign changed.
//
// Angles: f_i / 2 pi is held as a 64-bit fraction of a turn, so that p times it,
// modulo 2^64, is the exact fraction of a turn at any position (in fp32 the angle
// of position 10^6 is off by 0.03).  The nearest quarter turn comes off as the
// top two bits, what is left, at most an eighth of a turn either way, is exact to
// 2^-24 of itself in fp32.
#include <cmath>
#include <cstring>
#include <new>
#include <type_traits>

#include "common.cuh"
#include "window_args.h"

struct bsp_rotary_s {
    int device = -1;
    int pairs = 0;
    int interleaved = 0;
    double amplitude = 1.0;
    uint64_t turns[64] = {};  // fraction of a turn per position, in units of 2^-64
};

namespace bsp {
namespace win {
namespace {

constexpr int kMaxPairs = 64;
constexpr int kThreads = 256;
constexpr int kHeads = 16;  // of a thread, at most: what its sines serve (8: 113 us, 40: 105, with fewer blocks)

struct Args {
    uint64_t turns[kMaxPairs];
    View Q, K, Qo, Ko;
    const int* pos;
    int64_t pz;       // from one batch entry's positions to the next's
    float amplitude, sign;
    int Hq, H;        // query heads, and all
    int S;
    uint32_t tokens;  // Z * S
    int R, D;
    int units, turned;  // vectors of a head a thread group takes, those of them that turn
    int heads;          // per thread
};

// N elements as one access
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
    T x[N];
};

// cos and sin of 2 pi turn / 2^32
__device__ __forceinline__ float2 unit_at(uint32_t turn) {
    const uint32_t q = (turn + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(turn - (q << 30)) * 0x1p-31f;  // half turns, |x| <= 1/4
    float s, c;
    sincospif(x, &s, &c);
    const float a = q & 1 ? s : c, b = q & 1 ? c : s;
    return make_float2((q + 1) & 2 ? -a : a, q & 2 ? -b : b);
}

// How a thread's pairs lie: kPairs, within its vector; kHalves, over two vectors R / 2
// columns apart; kSwap, the same, but the thread has one of the two and the
// other comes from a thread of its warp.
enum Kind { kPairs, kHalves, kSwap };

// A thread owns one vector of VE columns (kHalves: the two vectors of VE pairs) of
// one token in some heads, so its sines serve all of those.
//
// HBM-bound: each element is read and written once.  32768 tokens of 40 heads of 128
// columns, bf16, 671 MB: 105 us (6.4 TB/s, 94 % of a copy's rate) with halves, 107
// with pairs.  Halves as two vectors a thread (kHalves: 128 bytes of a row per
// access, not 256) took 127; rows of a few heads per block, or one access of a
// thread on its way at a time, 130 to 150.
template <typename T, int VE, Kind KIND>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Args a) {
    constexpr int NP = KIND == kPairs ? VE / 2 : VE;  // pairs of a thread
    // heads on their way at once (kPairs in 16 bits: 107 us with 2, 110 with 4; kSwap
    // 110 and 105; kHalves 127 and 157, by its registers)
    constexpr int kAhead = KIND == kHalves || (KIND == kPairs && sizeof(T) == 2) ? 2 : 4;
    __shared__ uint64_t turns[kMaxPairs];
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    for (int i = tid; i < a.R / 2; i += blockDim.x * blockDim.y) turns[i] = a.turns[i];
    __syncthreads();
    cudaGridDependencySynchronize();
    // (threads without a token go along with the last one's, for the warp's sake)
    const uint32_t token = blockIdx.x * blockDim.y + threadIdx.y, t = min(token, a.tokens - 1);
    const bool live = token < a.tokens;
    if (KIND != kSwap && !live) return;
    const uint32_t z = t / (uint32_t)a.S, s = t - z * (uint32_t)a.S;
    const int u = threadIdx.x;
    const bool turned = u < a.turned;
    const int half = a.turned / 2;  // kSwap: vectors of one half of the pairs
    float cs[NP], sn[NP];
    if (turned) {
        const int64_t p = a.pos ? a.pos[z * a.pz + s] : (int64_t)s;
        const int first = (KIND == kSwap && u >= half ? u - half : u) * NP;
        const float sign = KIND == kSwap && u < half ? -a.sign : a.sign;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const uint64_t f = (uint64_t)p * turns[first + k];
            const float2 e = unit_at((uint32_t)(f >> 32));
            cs[k] = e.x * a.amplitude;
            sn[k] = e.y * a.amplitude * sign;
        }
    }
    using P = Pack<T, VE>;
    // columns of the thread's first vector; kHalves: the other is R / 2 further
    const int c0 = !turned ? a.R + (u - a.turned) * VE : u * VE;
    const int h0 = blockIdx.y * a.heads, h1 = min(h0 + a.heads, a.H);
    // heads h .. e - 1 of one tensor, kAhead of them on their way at once (a tensor
    // may be turned in its own place, so the compiler keeps loads behind stores)
    auto heads = [&](const View& in, const View& out, int h, int e) {
        const T* x = static_cast<const T*>(in.ptr) + z * in.s[0] + h * in.s[1] + s * in.s[2] + c0;
        T* y = static_cast<T*>(out.ptr) + z * out.s[0] + h * out.s[1] + s * out.s[2] + c0;
#pragma unroll 1
        for (; h < e; h += kAhead, x += kAhead * in.s[1], y += kAhead * out.s[1]) {
            P v[kAhead], w[KIND == kHalves ? kAhead : 1];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (h + j < e) {
                    v[j] = *reinterpret_cast<const P*>(x + j * in.s[1]);
                    if constexpr (KIND == kHalves)
                        if (turned) w[j] = *reinterpret_cast<const P*>(x + j * in.s[1] + a.R / 2);
                }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (h + j < e) {
                    P& f = v[j];
                    if constexpr (KIND == kSwap) {
                        constexpr int NW = sizeof(P) / 4;
                        P g;
                        uint32_t fw[NW], gw[NW];
                        memcpy(fw, &f, sizeof(P));
#pragma unroll
                        for (int k = 0; k < NW; ++k) gw[k] = __shfl_xor_sync(0xffffffffu, fw[k], half);
                        memcpy(&g, gw, sizeof(P));
                        if (turned)
#pragma unroll
                            for (int k = 0; k < NP; ++k)
                                f.x[k] = from_f32<T>(fmaf(to_f32(f.x[k]), cs[k], to_f32(g.x[k]) * sn[k]));
                    } else if (turned) {
                        if constexpr (KIND == kPairs) {
#pragma unroll
                            for (int k = 0; k < NP; ++k) {
                                const float xa = to_f32(f.x[2 * k]), xb = to_f32(f.x[2 * k + 1]);
                                f.x[2 * k] = from_f32<T>(fmaf(xa, cs[k], -(xb * sn[k])));
                                f.x[2 * k + 1] = from_f32<T>(fmaf(xb, cs[k], xa * sn[k]));
                            }
                        } else {
                            P& g = w[j];
#pragma unroll
                            for (int k = 0; k < NP; ++k) {
                                const float xa = to_f32(f.x[k]), xb = to_f32(g.x[k]);
                                f.x[k] = from_f32<T>(fmaf(xa, cs[k], -(xb * sn[k])));
                                g.x[k] = from_f32<T>(fmaf(xb, cs[k], xa * sn[k]));
                            }
                            *reinterpret_cast<P*>(y + j * out.s[1] + a.R / 2) = g;
                        }
                    }
                    if (KIND != kSwap || live) *reinterpret_cast<P*>(y + j * out.s[1]) = f;
                }
        }
    };
    if (h0 < a.Hq) heads(a.Q, a.Qo, h0, min(h1, a.Hq));
    if (h1 > a.Hq) heads(a.K, a.Ko, max(h0 - a.Hq, 0), h1 - a.Hq);
}

template <typename T, int VE>
int launch(Args a, bool pairs, bool rest, cudaStream_t s) {
    // kSwap where a token's vectors fill a power of two of a warp's lanes, so that the
    // other half is an exclusive or away
    const int vectors = a.R / VE, others = rest ? (a.D - a.R) / VE : 0;
    const bool swap = VE * sizeof(T) >= 4 && !pairs && (vectors & (vectors - 1)) == 0 && others % vectors == 0 &&
                      32 % (vectors + others) == 0;
    a.turned = pairs || swap ? vectors : vectors / 2;
    a.units = a.turned + others;
    const int rows = kThreads / a.units;
    const uint32_t blocks = (a.tokens + rows - 1) / rows;
    // few tokens: their heads go to several blocks, as many as fill the GPU
    const int64_t fill = 4 * (int64_t)sm_count();
    const int groups = (int)(blocks >= fill ? 1 : (fill + blocks - 1) / blocks);
    a.heads = imin(kHeads, imax(1, (a.H + groups - 1) / groups));
    const dim3 grid(blocks, (a.H + a.heads - 1) / a.heads);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(a.units, rows);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    void (*kern)(const Args) = rotary_kernel<T, VE, kHalves>;
    if constexpr (VE > 1)
        if (pairs) kern = rotary_kernel<T, VE, kPairs>;
    if constexpr (VE * sizeof(T) >= 4)
        if (swap) kern = rotary_kernel<T, VE, kSwap>;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

// The widest vector that the rotated columns divide into.
template <typename T>
int by_vector(const Args& a, bool pairs, bool rest, cudaStream_t s) {
    const int n = pairs ? a.R : a.R / 2;
    if constexpr (sizeof(T) == 2)
        if (n % 8 == 0) return launch<T, 8>(a, pairs, rest, s);
    if (n % 4 == 0) return launch<T, 4>(a, pairs, rest, s);
    if (n % 2 == 0) return launch<T, 2>(a, pairs, rest, s);
    return launch<T, 1>(a, false, rest, s);  // (pairs are always two columns)
}

bool same_view(const View& a, const View& b) {
    return a.ptr == b.ptr && a.s[0] == b.s[0] && a.s[1] == b.s[1] && a.s[2] == b.s[2];
}

}  // namespace
}  // namespace win
}  // namespace bsp

using namespace bsp::win;

extern "C" int bsp_rotary_create(const double* frequencies, int n_pairs, double amplitude, int interleaved,
                                 bsp_rotary_t* out) {
    if (!out) return BSP_ERR_INVALID_ARG;
    *out = nullptr;
    if (!frequencies || n_pairs < 1 || !std::isfinite((float)amplitude) || (interleaved != 0 && interleaved != 1))
        return BSP_ERR_INVALID_ARG;
    if (n_pairs > kMaxPairs) return BSP_ERR_UNSUPPORTED;
    for (int i = 0; i < n_pairs; ++i)
        if (!std::isfinite(frequencies[i])) return BSP_ERR_INVALID_ARG;
    bsp_rotary_s* r = new (std::nothrow) bsp_rotary_s;
    if (!r) return BSP_ERR_OOM;
    if (cudaGetDevice(&r->device) != cudaSuccess) {
        delete r;
        return BSP_ERR_CUDA;
    }
    r->pairs = n_pairs;
    r->interleaved = interleaved;
    r->amplitude = amplitude;
    constexpr long double kTurn = 6.283185307179586476925286766559005768L;
    for (int i = 0; i < n_pairs; ++i) {
        const long double x = (long double)frequencies[i] / kTurn;
        const long double f = (x - floorl(x)) * 18446744073709551616.0L;  // 2^64; may round up to it
        r->turns[i] = f >= 18446744073709551616.0L ? 0 : (uint64_t)f;
    }
    *out = r;
    return BSP_OK;
}

extern "C" int bsp_rotary_destroy(bsp_rotary_t r) {
    delete r;
    return BSP_OK;
}

extern "C" int bsp_rotary(bsp_rotary_t r, int dtype, const bsp_tensor_t* Q, const bsp_tensor_t* Q_out,
                          const bsp_tensor_t* K, const bsp_tensor_t* K_out, const int32_t* positions,
                          int64_t position_stride, int inverse, int Z, int Hq, int Hkv, int S, int D, void* stream) {
    if (!r || !valid_dtype(dtype) || (inverse != 0 && inverse != 1)) return BSP_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return BSP_ERR_CUDA;
    if (dev != r->device) return BSP_ERR_INVALID_ARG;
    if (Z < 0 || Hq < 1 || Hkv < 0 || S < 0 || !valid_d(D) || 2 * r->pairs > D) return BSP_ERR_INVALID_ARG;
    if (S > kMaxLen || (int64_t)Z * S > kMaxLen || (int64_t)Hq + Hkv > 65535) return BSP_ERR_UNSUPPORTED;
    if (Z == 0 || S == 0) return BSP_OK;
    if ((uintptr_t)positions & 3u) return BSP_ERR_ALIGNMENT;
    if (positions && Z > 1 && position_stride < 0) return BSP_ERR_INVALID_ARG;
    Args a{};
    const int elt = elt_bytes(dtype);
    int rc = make_view(Q, Z, Hq, S, D, elt, false, &a.Q);
    if (!rc) rc = make_view(Q_out, Z, Hq, S, D, elt, true, &a.Qo);
    if (!rc && Hkv) rc = make_view(K, Z, Hkv, S, D, elt, false, &a.K);
    if (!rc && Hkv) rc = make_view(K_out, Z, Hkv, S, D, elt, true, &a.Ko);
    if (rc) return rc;
    // in its own place a tensor may turn; over another one, or itself in another
    // order, not
    const bool q_in = same_view(a.Q, a.Qo), k_in = Hkv && same_view(a.K, a.Ko);
    if (a.Q.ptr == a.Qo.ptr && !q_in) return BSP_ERR_INVALID_ARG;
    if (Hkv && ((a.K.ptr == a.Ko.ptr && !k_in) || a.Qo.ptr == a.Ko.ptr || a.Qo.ptr == a.K.ptr || a.Ko.ptr == a.Q.ptr))
        return BSP_ERR_INVALID_ARG;
    for (int i = 0; i < r->pairs; ++i) a.turns[i] = r->turns[i];
    a.pos = positions;
    a.pz = Z > 1 ? position_stride : 0;
    a.amplitude = (float)r->amplitude;
    a.sign = inverse ? -1.f : 1.f;
    a.Hq = Hq, a.H = Hq + Hkv;
    a.S = S, a.tokens = (uint32_t)Z * (uint32_t)S;
    a.R = 2 * r->pairs, a.D = D;
    const bool pairs = r->interleaved != 0, rest = a.R < D && !(q_in && (k_in || !Hkv));
    cudaStream_t s = (cudaStream_t)stream;
    switch (dtype) {
        case BSP_F32: return by_vector<float>(a, pairs, rest, s);
        case BSP_BF16: return by_vector<__nv_bfloat16>(a, pairs, rest, s);
        default: return by_vector<__half>(a, pairs, rest, s);
    }
}
