// glr.cuh -- gated linear recurrence h_t = a_t h_{t-1} + m(a_t) u_t: what its kernels share.
#pragma once

#include <type_traits>

#include "dla.cuh"

namespace gcl {
namespace glr {

using dla::Rows;

constexpr int kSave = 64;          // tokens between the states of h_save

struct Kind {                      // which a, m and u
    const float *rate;
    int32_t decay, mix;
};

// exp and 1 / x: the accurate ones for fp32 rows; for 16-bit rows, whose own rounding is 2^13 ulp, the
// special-function unit's, off by a few ulp.  (Flushing subnormals: without it each takes three instructions more.)
template <typename T>
__device__ __forceinline__ float fexp2(float x) {          // 2^x; fp32 rows: e^x
    if (sizeof(T) == 4) return expf(x);
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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
__device__ __forceinline__ float froot(float x) {
    if (sizeof(T) == 4) return sqrtf(x);
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The smaller of x and a bound, NaN where x is (fminf would answer with the bound: a gate that is not a number would count as closed).
__device__ __forceinline__ float at_most(float x, float bound) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(bound));
    return y;
}

// A lane's channels of a row, four bytes: two values of 16 bits, held as a pair whose arithmetic is one instruction,
// or one of fp32.  A warp takes 128 bytes of the row.
template <typename T>
struct Lane {
    static constexpr int V = 2;
    static constexpr int CB = 64;                          // channels of a warp
    using P = float2;
    static __device__ __forceinline__ P get(uint32_t w) {
        const T *h = reinterpret_cast<const T *>(&w);
        return make_float2((float)h[0], (float)h[1]);
    }
    static __device__ __forceinline__ uint32_t put(P x) {
        uint32_t w;
        T *h = reinterpret_cast<T *>(&w);
        h[0] = (T)x.x;
        h[1] = (T)x.y;
        return w;
    }
    static __device__ __forceinline__ P all(float x) { return make_float2(x, x); }
    static __device__ __forceinline__ P load(const float *p) {
        return *reinterpret_cast<const float2 *>(p);
    }
    static __device__ __forceinline__ void store(float *p, P x) { *reinterpret_cast<float2 *>(p) = x; }
    static __device__ __forceinline__ P mul(P a, P b) { return __fmul2_rn(a, b); }
    static __device__ __forceinline__ P add(P a, P b) { return __fadd2_rn(a, b); }
    static __device__ __forceinline__ P fma(P a, P b, P c) { return __ffma2_rn(a, b, c); }
    template <typename F>
    static __device__ __forceinline__ P map(P x, F f) {
        return make_float2(f(x.x), f(x.y));
    }
    template <typename F>
    static __device__ __forceinline__ P map(P x, P y, F f) {
        return make_float2(f(x.x, y.x), f(x.y, y.y));
    }
    template <typename F>
    static __device__ __forceinline__ P map(P x, P y, P z, F f) {
        return make_float2(f(x.x, y.x, z.x), f(x.y, y.y, z.y));
    }
    template <typename F>
    static __device__ __forceinline__ bool every(P x, F f) {
        return f(x.x) && f(x.y);
    }
};
template <>
struct Lane<float> {
    static constexpr int V = 1;
    static constexpr int CB = 32;
    using P = float;
    static __device__ __forceinline__ P get(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t put(P x) { return __float_as_uint(x); }
    static __device__ __forceinline__ P all(float x) { return x; }
    static __device__ __forceinline__ P load(const float *p) { return *p; }
    static __device__ __forceinline__ void store(float *p, P x) { *p = x; }
    static __device__ __forceinline__ P mul(P a, P b) { return a * b; }
    static __device__ __forceinline__ P add(P a, P b) { return a + b; }
    static __device__ __forceinline__ P fma(P a, P b, P c) { return fmaf(a, b, c); }
    template <typename F>
    static __device__ __forceinline__ P map(P x, F f) { return f(x); }
    template <typename F>
    static __device__ __forceinline__ P map(P x, P y, F f) { return f(x, y); }
    template <typename F>
    static __device__ __forceinline__ P map(P x, P y, P z, F f) { return f(x, y, z); }
    template <typename F>
    static __device__ __forceinline__ bool every(P x, F f) { return f(x); }
};

// e^x of each value.
template <typename T>
__device__ __forceinline__ typename Lane<T>::P exps(typename Lane<T>::P x) {
    if (sizeof(T) == 2) x = Lane<T>::mul(x, Lane<T>::all(1.4426950408889634f));
    return Lane<T>::map(x, [](float v) { return fexp2<T>(v); });
}
// sigmoid(x) and sigmoid(-x) = exp(-x) sigmoid(x), neither by a difference.
template <typename T>
__device__ __forceinline__ void sigmoids(typename Lane<T>::P x, typename Lane<T>::P &s, typename Lane<T>::P &c) {
    using L = Lane<T>;
    typename L::P e;
    if (sizeof(T) == 2) e = L::map(L::mul(x, L::all(-1.4426950408889634f)), [](float v) { return fexp2<T>(at_most(v, 126.f)); });
    else e = L::map(x, [](float v) { return fexp2<T>(at_most(-v, 87.f)); });
    s = L::map(L::add(e, L::all(1.f)), [](float v) { return frcp<T>(v); });
    c = L::mul(e, s);
}
// The same of x and z.  16-bit rows: by one reciprocal, that of (1 + exp(-x)) (1 + exp(-z)), since a reciprocal takes the
// special-function unit as long as two exponentials.  Below 2^-63 (x < -43.6) they stay at 2^-63, so that the product is finite.  A NaN
// of either makes all four NaN; with APART one of z leaves x's alone.
template <typename T, bool APART = false>
__device__ __forceinline__ void sigmoids(typename Lane<T>::P x, typename Lane<T>::P z, typename Lane<T>::P &sx, typename Lane<T>::P &cx,
                                         typename Lane<T>::P &sz, typename Lane<T>::P &cz) {
    using L = Lane<T>;
    if (sizeof(T) == 4) {
        sigmoids<T>(x, sx, cx);
        sigmoids<T>(z, sz, cz);
        return;
    }
    auto ex = [](typename L::P v) { return L::map(L::mul(v, L::all(-1.4426950408889634f)), [](float u) { return fexp2<T>(at_most(u, 63.f)); }); };
    const typename L::P e = ex(x), f = ex(z), a = L::add(e, L::all(1.f));
    const typename L::P b = L::add(APART ? L::map(f, [](float u) { return fminf(u, 0x1p63f); }) : f, L::all(1.f));
    const typename L::P r = L::map(L::mul(a, b), [](float u) { return frcp<T>(u); });
    sx = L::mul(b, r);
    sz = L::mul(APART ? L::fma(f, L::all(0.f), a) : a, r);
    cx = L::mul(e, sx);
    cz = L::mul(f, sz);
}

// q = 1 - exp(-y) for 0 <= y <= kNear: y P(y), P the polynomial of degree 6 that meets (1 - exp(-y)) / y at the Chebyshev points
// of [0, 0.9] (off by 5e-9 of its value).  N values at a time: a pair of constants then serves N instructions.  Rates of a warp's channels that
// are all in that range leave the exponential out (65,536 tokens of 2,048 channels 247 us, with rates of 0.01 to 8 in every warp 264; backward
// of 32,768 277 and 286).
constexpr float kNear = 0.9f;
template <typename T, int N>
__device__ __forceinline__ void one_minus_exp(const typename Lane<T>::P *y, typename Lane<T>::P *q) {
    using L = Lane<T>;
    constexpr float C[7] = {1.3465580e-4f, -1.3153803e-3f, 8.2897432e-3f, -4.1653194e-2f, 1.6666466e-1f, -4.9999988e-1f, 1.f};
#pragma unroll
    for (int e = 0; e < N; ++e) q[e] = L::fma(y[e], L::all(C[0]), L::all(C[1]));
#pragma unroll
    for (int c = 2; c < 7; ++c)
#pragma unroll
        for (int e = 0; e < N; ++e) q[e] = L::fma(y[e], q[e], L::all(C[c]));
#pragma unroll
    for (int e = 0; e < N; ++e) q[e] = L::mul(y[e], q[e]);
}

// a = exp(-y) and q = 1 - a of the N values y in q.  16-bit rows: the difference loses q's digits near y = 0, and the fast exp's
// error, some units of 2^-24 with one sign, would add up over all the tokens that a close to 1 remembers: there a = 1 - q from the
// polynomial, rounded once.  NEAR: all y lie in [0, kNear].
template <typename T, bool NEAR, int N>
__device__ __forceinline__ void decay_of(typename Lane<T>::P *a, typename Lane<T>::P *q) {
    using L = Lane<T>;
    using P = typename L::P;
    if (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            a[e] = L::map(q[e], [](float v) { return expf(-v); });
            q[e] = L::map(q[e], [](float v) { return -expm1f(-v); });
        }
        return;
    }
    P p[N];
    one_minus_exp<T, N>(q, p);
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (NEAR) {
            q[e] = p[e];
            a[e] = L::fma(p[e], L::all(-1.f), L::all(1.f));
        } else {
            const P y = q[e], far = L::map(L::mul(y, L::all(-1.4426950408889634f)), [](float v) { return fexp2<T>(v); });
            auto pick = [](float v, float n, float f) {    // (y < 0 and NaN have larger bits)
                return __float_as_uint(v) <= __float_as_uint(kNear) ? n : f;
            };
            q[e] = L::map(y, p[e], L::fma(far, L::all(-1.f), L::all(1.f)), pick);
            a[e] = L::map(y, L::fma(p[e], L::all(-1.f), L::all(1.f)), far, pick);
        }
    }
}

// The gates of N tokens: a, m(a) and the input gate's sigmoid from r and g (g is not read without gate: GATE false, sg = 1).
// rate: of the lane's channels; near: all the warp's rates lie in [0, kNear].  APART: a and m do not take a NaN from g (forwards the
// state is NaN by either; the gradient that a token passes on does not depend on g).
template <typename T, int DECAY, int MIX, bool GATE, int N, bool APART = false>
__device__ __forceinline__ void gates(typename Lane<T>::P rate, bool near, const typename Lane<T>::P *r, const typename Lane<T>::P *g,
                                      typename Lane<T>::P *a, typename Lane<T>::P *m, typename Lane<T>::P *sg) {
    using L = Lane<T>;
    using P = typename L::P;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        P s = L::all(0.f), c = L::all(0.f), cg;
        if (DECAY == GCL_DECAY_LOG) {
            if (GATE) sigmoids<T>(g[e], sg[e], cg);
            m[e] = L::mul(r[e], L::all(-1.f));
        } else {
            if (GATE) sigmoids<T, APART>(r[e], g[e], s, c, sg[e], cg);
            else sigmoids<T>(r[e], s, c);
            // a >= 1/2 from c: one rounding, where s carries those of its sum, its reciprocal and their product (r of 6 to 10: 3e-8
            // instead of up to 1.6e-7, which 1 / (1 - a) tokens add up)
            a[e] = s;
            if (DECAY == GCL_DECAY_SIGMOID)
                a[e] = L::map(c, s, L::fma(c, L::all(-1.f), L::all(1.f)), [](float u, float v, float w) { return u <= 0.5f ? w : v; });
            m[e] = DECAY == GCL_DECAY_SIGMOID ? c : L::mul(rate, s);
        }
        if (!GATE) sg[e] = L::all(1.f);
    }
    if (DECAY != GCL_DECAY_SIGMOID) {                      // from y = -log a in m
        if (DECAY == GCL_DECAY_POWER && sizeof(T) == 2 && near) decay_of<T, true, N>(a, m);
        else decay_of<T, false, N>(a, m);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (MIX == GCL_MIX_ONE) m[e] = L::all(1.f);
        if (MIX == GCL_MIX_ROOT) {                         // 1 - a^2 = (1 - a) (1 + a); a > 1 counts as 1
            if (DECAY == GCL_DECAY_LOG) m[e] = L::map(m[e], [](float v) { return fmaxf(v, 0.f); });
            m[e] = L::map(L::fma(m[e], a[e], m[e]), [](float v) { return froot<T>(v); });
        }
    }
}

// Calls f(integral_constant decay, integral_constant mix, integral_constant gate) for the kind.
template <typename F>
inline auto for_kind(int decay, int mix, bool gate, F f) {
    auto with_mix = [&](auto d) {
        auto with_gate = [&](auto m) { return gate ? f(d, m, std::true_type()) : f(d, m, std::false_type()); };
        if (mix == GCL_MIX_ONE) return with_gate(std::integral_constant<int, GCL_MIX_ONE>());
        if (mix == GCL_MIX_COMPLEMENT) return with_gate(std::integral_constant<int, GCL_MIX_COMPLEMENT>());
        return with_gate(std::integral_constant<int, GCL_MIX_ROOT>());
    };
    if (decay == GCL_DECAY_LOG) return with_mix(std::integral_constant<int, GCL_DECAY_LOG>());
    if (decay == GCL_DECAY_SIGMOID) return with_mix(std::integral_constant<int, GCL_DECAY_SIGMOID>());
    return with_mix(std::integral_constant<int, GCL_DECAY_POWER>());
}

// What the launches of a call leave each other at the front of the workspace.
struct Header {
    int32_t blocked;               // the call does nothing (status word set, or cu_seqlens invalid)
    int32_t live;                  // cu_seqlens[n_max]
    uint32_t ticket;               // spans taken
    int32_t pad;
};

// What spans of tiles leave each other, a packet a channel of 16 bytes that is written and read as one: the product of the span's decays
// and its state from zero (tag kOwn), and the state that leaves it (tag kDone).
struct __align__(16) Packet {
    float a, own, out;
    uint32_t tag;
};
constexpr uint32_t kOwn = 1, kDone = 2;

struct Params {
    Rows x, r, i, o, d_o, dx, dr, di;
    Kind kind;
    const float *h0, *dht;
    float *ht, *dh0, *h_save, *drate;
    const int32_t *cu;
    int32_t *status;
    Header *head;
    int32_t *first;                // [tiles]: the first sequence that starts at or behind the tile's first token; NULL: solo, a call of one
                                   // span, whose launch does the set-up's work itself
    Packet *chain;                 // [spans, D], in the order of the recurrence
    float *drate_part;             // [tiles, D]
    int64_t t_max, tiles;
    int32_t n_max, D, n_cb, tile;  // n_cb: blocks of channels; tokens of a tile
};

// Launchers, one pair for each type of the rows.
template <typename T>
cudaError_t launch_fwd(const Params &p, cudaStream_t s);
template <typename T>
cudaError_t launch_bwd(const Params &p, cudaStream_t s);

constexpr int kTileF = 128, kTileB = 64;               // tokens of a tile, forward and backward
constexpr int kRanks = 2;                              // tiles of a span (65,536 tokens of 2,048 channels: 246 us; four 251, eight 297;
                                                       // of 1,024 channels, twice the tokens, 282 and 268)

}  // namespace glr
}  // namespace gcl
