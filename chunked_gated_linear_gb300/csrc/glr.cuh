// glr.cuh -- gated linear recurrence h_t = a_t h_{t-1} + m(a_t) u_t: what its kernels share.
#pragma once

#include "dla.cuh"

namespace gcl {
namespace glr {

using dla::Rows;

constexpr int kSave = 64;          // tokens between the states of h_save

struct Kind {                      // which a, m and u
    const float *rate;
    int32_t decay, mix;
};

// A lane's consecutive channels of a row: four bytes, so that a warp takes 128.
template <typename T>
struct Lane {
    static constexpr int V = 4 / sizeof(T);
    static constexpr int CB = 32 * V;                  // channels of a warp
    static __device__ __forceinline__ void get(uint32_t w, float *v) {
        if constexpr (V == 1) {
            v[0] = __uint_as_float(w);
        } else {
            const T *h = reinterpret_cast<const T *>(&w);
            v[0] = (float)h[0];
            v[1] = (float)h[1];
        }
    }
    static __device__ __forceinline__ uint32_t put(const float *v) {
        if constexpr (V == 1) {
            return __float_as_uint(v[0]);
        } else {
            uint32_t w;
            T *h = reinterpret_cast<T *>(&w);
            h[0] = (T)v[0];
            h[1] = (T)v[1];
            return w;
        }
    }
};

// exp, 1 / x and the square root: the accurate ones for fp32 rows; for 16-bit rows, whose own rounding is 2^13 ulp, the
// special-function unit's, off by a few ulp.  (Flushing subnormals: without it each takes three instructions more, 40 of
// the forward's 108 a value.)
template <typename T>
__device__ __forceinline__ float fexp(float x) {
    if (sizeof(T) == 4) return expf(x);
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}
template <typename T>
__device__ __forceinline__ float frcp(float x) {
    if (sizeof(T) == 4) return 1.f / x;
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <typename T>
__device__ __forceinline__ float root(float x) {
    x = fmaxf(x, 0.f);
    if (sizeof(T) == 4) return sqrtf(x);
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// sigmoid(x) and sigmoid(-x), neither by a difference.
template <typename T>
__device__ __forceinline__ void sigmoids(float x, float &s, float &c) {
    const float e = fexp<T>(-fabsf(x)), hi = frcp<T>(1.f + e), lo = e * hi;
    s = x >= 0.f ? hi : lo;
    c = x >= 0.f ? lo : hi;
}

// sigmoid(x) alone.  (exp(-x) = infinity gives 0.)
template <typename T>
__device__ __forceinline__ float sigmoid(float x) { return frcp<T>(1.f + fexp<T>(-x)); }

// a = exp(l) and q = 1 - a.  Near l = 0 the difference loses q's digits and the fast exp's error, some units of
// 2^-24 with one sign, would add up over all the tokens that a close to 1 remembers: for 0 <= y = -l < 0.7 q is
// y P(y), P the polynomial of degree 5 that meets (1 - exp(-y)) / y at the Chebyshev points of [0, 0.7] (off by 1.2e-8 of
// its value), and a = 1 - q, rounded once.
template <typename T>
__device__ __forceinline__ void exps(float l, float &a, float &q) {
    a = fexp<T>(l);
    if (sizeof(T) == 4) {
        q = -expm1f(l);
        return;
    }
    const float y = -l;
    float s = fmaf(y, -1.0332434e-3f, 8.0679525e-3f);
    s = fmaf(y, s, -4.1572765e-2f);
    s = fmaf(y, s, 1.6665146e-1f);
    s = fmaf(y, s, -4.9999911e-1f);
    s = fmaf(y, s, 1.f);
    const bool near = __float_as_uint(y) < __float_as_uint(0.7f);          // (y < 0 and NaN have larger bits)
    q = near ? y * s : 1.f - a;
    a = near ? 1.f - q : a;
}

// a and q = 1 - a of N values of r (N / V tokens of the lane's V channels); the kind is the same for the grid.
template <typename T, int N>
__device__ __forceinline__ void decays(const Kind &k, const float *rate, const float *r, float *a, float *q) {
    constexpr int V = Lane<T>::V;
    if (k.decay == GCL_DECAY_SIGMOID) {
#pragma unroll
        for (int e = 0; e < N; ++e) sigmoids<T>(r[e], a[e], q[e]);
    } else if (k.decay == GCL_DECAY_POWER) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            exps<T>(-rate[e % V] * sigmoid<T>(r[e]), a[e], q[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            exps<T>(r[e], a[e], q[e]);
        }
    }
}

// m(a) in place of q = 1 - a.
template <typename T, int N>
__device__ __forceinline__ void mixes(const Kind &k, const float *a, float *q) {
    if (k.mix == GCL_MIX_ONE) {
#pragma unroll
        for (int e = 0; e < N; ++e) q[e] = 1.f;
    } else if (k.mix == GCL_MIX_ROOT) {                // 1 - a^2 = (1 - a) (1 + a)
#pragma unroll
        for (int e = 0; e < N; ++e) q[e] = root<T>(q[e] * (1.f + a[e]));
    }
}

// What the launches of a call leave each other at the front of the workspace.
struct Header {
    int32_t blocked;               // the call does nothing (status word set, or cu_seqlens invalid)
    int32_t live;                  // cu_seqlens[n_max]
    uint32_t ticket;               // tiles taken
    int32_t pad;
};

// The states between tiles, by tile in the order of the recurrence and block of channels.
struct Chain {
    int32_t *flag;                 // [n_cb, tiles]: 0, kOwn (a and own are there), kDone (out is there)
    float *a, *own;                // [tiles, D]: product of the tile's decays, its state from zero
    float *out;                    // [tiles, D]: the state that leaves the tile
};
constexpr int32_t kOwn = 1, kDone = 2;

struct Params {
    Rows x, r, i, o, d_o, dx, dr, di;
    Kind kind;
    const float *h0, *dht;
    float *ht, *dh0, *h_save, *drate;
    const int32_t *cu;
    int32_t *status;
    Header *head;
    int32_t *first;                // [tiles]: the first sequence that starts at or behind the tile's first token
    Chain chain;
    float *drate_part;             // [tiles, D]
    int64_t t_max, tiles;
    int32_t n_max, D, n_cb;        // n_cb: blocks of channels
};

}  // namespace glr
}  // namespace gcl
