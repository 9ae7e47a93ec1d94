// block_norm.cuh -- the norms after and before a block with its gate, dropout, residual scale and sum.
//
//   v = scale drop(act(gate) n w_post), n = y r_y;   xo = x + v;   z = xo r w_pre
// Backward, with u = dz w_pre and the row's sums S = sum(xo^2) and M = sum(u xo):
//   d = dxo + r (u - xo r^2 M / D),   dy = r_y (d v / n - n P / D),   P = sum(d v)
// P is linear in d, so its three parts sum(dxo v), sum(u v), sum(xo v) cross the row's threads together with S and M: a row
// has two reductions (y's own length first, on which xo depends).
// Rows are read and written once.  A row is held by TPR threads, VPT vectors of eight values each; a block's next row comes into shared
// memory by asynchronous copies while one is worked on (each thread its own vectors, so that no barrier belongs to it).  Bound by HBM and
// issue together forwards (46 instructions a value, 62% of slots; a third are conversions, Philox and the sums), so
// arithmetic goes by fp32 pairs, choices are made for a vector and not for a value, and weights stay in shared memory over a
// block's rows.  Backwards by latency: 86 instructions a value take 55% of the slots and rows 42% of HBM's peak, with 12 warps an SM and two
// reductions a row one after the other.  bf16, both norms, gate and dropout: 32,768 tokens of 2,048 129 us, 77% of copy bandwidth;
// backward 262 us, 60%; gated norms of heads (no x, no z) 72 us, 83%.  On the way: rows loaded when needed 190 and 440; copied a row ahead, pairs, sums
// side by side 136 and 279.  Not kept: one vector a thread (195, backward 279 to 304); more blocks of fewer registers (spills, 291 to 399).
#pragma once

#include <atomic>

#include "dla.cuh"
#include "dla_simt.cuh"

namespace gcl {
namespace blk {

// A gcl_rows, and how far (in bytes) a thread moves from one of its rows to the next: by d, and by w more where the head index
// wraps.  (Here, not in registers: two for each of eight arrays.)
struct Rows : dla::Rows {
    int64_t d, w;
    Rows() = default;
    Rows(const gcl_rows &r) : dla::Rows(dla::rows(r)), d(0), w(0) {}
    void step(int64_t rows, int H, int esize) {
        d = (rows / H * st + rows % H * sh) * esize;
        w = (st - H * sh) * esize;
    }
};

struct Params {
    Rows y, gate, x, xo, z, dxo, dz, dy, dgate, dx;
    const void *w_post, *w_pre;
    float *part_post, *part_pre;   // [blocks, D] sums of the weights' gradients, or NULL
    float *dw_post, *dw_pre;
    const int64_t *rng;
    const int32_t *cu;
    int32_t *status;
    int64_t t_max;
    int32_t n_max, H, D;
    float scale, eps;
    int32_t cut;                   // dropout: half-words below are dropped (0: none)
    int32_t post, pre, act;
    int32_t dh;                    // heads from a thread's row to its next, modulo H
};

// Philox4x32-10 of a 64-bit counter half, offset and key.
__device__ __forceinline__ uint4 philox(uint64_t at, uint64_t offset, uint64_t seed) {
    uint32_t c0 = (uint32_t)at, c1 = (uint32_t)(at >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = (uint64_t)0xD2511F53u * c0, q = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)q;
        c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

using P = float2;                  // two fp32 values
constexpr int kPairs = 4;          // of a vector

__device__ __forceinline__ P mul2(P a, P b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ P add2(P a, P b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ P fma2(P a, P b, P c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ P both(float x) { return make_float2(x, x); }
template <typename F>
__device__ __forceinline__ P map(P x, F f) { return make_float2(f(x.x), f(x.y)); }

// Zeros in place of a vector's dropped values: value e is kept where half-word e of its block is at least `cut`.
// (cut16: cut in the upper half; an upper half-word is compared with the lower one still below it.)
__device__ __forceinline__ void drop(const uint4 &w, uint32_t cut16, P *x) {
    const uint32_t word[kPairs] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        if (word[k] << 16 < cut16) x[k].x = 0.f;
        if (word[k] < cut16) x[k].y = 0.f;
    }
}

// exp(-x) and 1 / x: the accurate ones for fp32 rows, the special-function unit's (subnormals flushed) for 16-bit rows.
template <typename T>
__device__ __forceinline__ float exp_minus(float x) {
    if (sizeof(T) == 4) return expf(-x);
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * -1.4426950408889634f));
    return y;
}
template <typename T>
__device__ __forceinline__ float reciprocal(float x) {
    if (sizeof(T) == 4) return 1.f / x;
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// act(g) of a vector, and with SLOPE its derivative.
template <typename T, bool SLOPE>
__device__ __forceinline__ void activation(int act, const P *g, P *a, P *da) {
    if (act == GCL_ACT_NONE) {
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            a[k] = g[k];
            if (SLOPE) da[k] = both(1.f);
        }
        return;
    }
    P s[kPairs], c[kPairs];                                // sigmoid(g) and sigmoid(-g) = exp(-g) sigmoid(g), neither by a difference
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        // (exp(-g) may be infinite: then s = 0, and c is 1 from where it rounds to that; a NaN passes)
        const P e = map(g[k], [](float v) { return exp_minus<T>(v); });
        s[k] = map(add2(e, both(1.f)), [](float v) { return reciprocal<T>(v); });
        if (SLOPE) {
            c[k] = mul2(e, s[k]);
            if (e.x > 0x1p26f) c[k].x = 1.f;
            if (e.y > 0x1p26f) c[k].y = 1.f;
        }
    }
    if (act == GCL_ACT_SILU) {
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            a[k] = mul2(g[k], s[k]);
            if (SLOPE) da[k] = mul2(s[k], fma2(g[k], c[k], both(1.f)));
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            a[k] = s[k];
            if (SLOPE) da[k] = mul2(s[k], c[k]);
        }
    }
}

// Eight consecutive values of a row as loaded.
template <typename T>
struct Vec {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p, bool on) {
#pragma unroll
        for (int e = 0; e < (int)sizeof(T) / 2; ++e) v[e] = on ? reinterpret_cast<const uint4 *>(p)[e] : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(P *f) const {
        float x[8];
        dla::load8f(reinterpret_cast<const T *>(v), x);
#pragma unroll
        for (int k = 0; k < kPairs; ++k) f[k] = make_float2(x[2 * k], x[2 * k + 1]);
    }
    static __device__ __forceinline__ void store(T *p, const P *f) {
        float x[8];
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            x[2 * k] = f[k].x;
            x[2 * k + 1] = f[k].y;
        }
        Vec o;
        dla::store4f(reinterpret_cast<T *>(o.v), x);
        dla::store4f(reinterpret_cast<T *>(o.v) + 4, x + 4);
#pragma unroll
        for (int e = 0; e < (int)sizeof(T) / 2; ++e) reinterpret_cast<uint4 *>(p)[e] = o.v[e];
    }
};

constexpr int threads_of(int tpr) { return tpr > 128 ? tpr : 128; }

// Sums over a row's threads.  Rows of several warps pass through shared memory; `turn` alternates two buffers, so that
// one barrier a reduction is enough.  Of five sums four cross a warp together: lanes first part the sums among them (6 shuffles
// instead of 20), and the warps' sums are added by lanes side by side.
template <int TPR, int NS>
struct RowSum {
    static constexpr int W = TPR / 32 > 0 ? TPR / 32 : 1;          // warps of a row
    static constexpr int R = threads_of(TPR) / TPR;                // rows of a block
    float (*buf)[R][NS][W];
    int turn;
    static __device__ __forceinline__ float across(float x, int most) {
#pragma unroll
        for (int d = most / 2; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        return x;
    }
    template <int N>
    __device__ __forceinline__ void operator()(float *s) {
        if (TPR <= 32) {
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = across(s[i], TPR);
            return;
        }
        const int row = threadIdx.x / TPR, warp = threadIdx.x % TPR / 32, lane = threadIdx.x & 31;
        float (*b)[W] = buf[turn][row];
        if (N == 5) {
            const bool hi = lane & 16, mid = lane & 8;
            float u = hi ? s[2] : s[0], v = hi ? s[3] : s[1];
            u += __shfl_xor_sync(0xffffffffu, hi ? s[0] : s[2], 16);
            v += __shfl_xor_sync(0xffffffffu, hi ? s[1] : s[3], 16);
            float c = mid ? v : u;
            c += __shfl_xor_sync(0xffffffffu, mid ? u : v, 8);
            c = across(c, 8);
            const float last = across(s[4], 32);
            if (lane % 8 == 0) b[lane / 8][warp] = c;      // (8 hi + mid: the sum's number)
            if (lane == 0) b[4][warp] = last;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float c = across(s[i], 32);
                if (lane == 0) b[i][warp] = c;
            }
        }
        __syncthreads();
        constexpr int G = 32 / W;                          // sums that a warp adds up side by side
        if (N == 1) {
            s[0] = across(b[0][lane % W], W);
        } else {
#pragma unroll
            for (int i0 = 0; i0 < N; i0 += G) {
                const int i = i0 + lane / W;
                const float c = across(i < N ? b[i][lane % W] : 0.f, W);
#pragma unroll
                for (int j = i0; j < N && j < i0 + G; ++j) s[j] = __shfl_sync(0xffffffffu, c, (j - i0) * W);
            }
        }
        turn ^= 1;
    }
};
__device__ __forceinline__ float sum_of(P x) {
    return x.x + x.y;
}

__device__ __forceinline__ float inverse_length(int norm, float ss, float inv_d, float eps) {
    return norm == GCL_NORM_NONE ? 1.f : rsqrtf((norm == GCL_NORM_RMS ? ss * inv_d : ss) + eps);
}

// The live rows; false: the call does nothing.  Every thread of the block calls it.
__device__ __forceinline__ bool live_rows(const Params &p, int64_t &rows) {
    if (status_blocks_cta(p.status)) return false;
    int64_t t = p.t_max;
    if (p.cu) {
        t = p.cu[p.n_max];
        if (t < 0 || t > p.t_max) {
            if (threadIdx.x == 0) status_set(p.status, GCL_DEV_BAD_RANGE);
            return false;
        }
    }
    rows = t * p.H;
    return true;
}

// A thread's place in an array: its first vector of row t, h.
template <typename T>
__device__ __forceinline__ char *place(const Rows &r, int64_t t, int h, int l) {
    return static_cast<char *>(r.p) + (t * r.st + h * r.sh + l * 8) * (int)sizeof(T);
}
__device__ __forceinline__ void advance(char *&at, const Rows &r, bool wrap) {
    at += r.d;
    if (wrap) at += r.w;
}
// (debug build) Whether the row of a thread's cursor lies in its array.
template <typename T>
__device__ __forceinline__ bool row_in(const Params &p, const Rows &r, const char *at, int l) {
    return !r.p || GCL_RANGE_IN_BOUNDS(at - static_cast<const char *>(r.p) - l * 8 * (int)sizeof(T),
                                       at - static_cast<const char *>(r.p) + (p.D - l * 8) * (int)sizeof(T) - 1,
                                       ((p.t_max - 1) * r.st + (p.H - 1) * r.sh + p.D) * (int)sizeof(T), p.status);
}
template <typename T>
__device__ __forceinline__ T *vec_at(char *at, int v, int tpr) { return reinterpret_cast<T *>(at) + v * tpr * 8; }

// Vectors of eight values in shared memory, each thread's own: copied there a row ahead (asynchronously), read when needed.
// Rows too wide for that (STAGED false) are read from memory each time.
template <typename T, bool STAGED, int THREADS>
__device__ __forceinline__ void stage_copy(uint4 *at, int chunk, const T *src, bool on) {
    if constexpr (STAGED) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             static_cast<uint32_t>(__cvta_generic_to_shared(at + (chunk + i) * THREADS))),
                         "l"(reinterpret_cast<const uint4 *>(src) + i), "r"(on ? 16 : 0)
                         : "memory");
    }
}
template <typename T, bool STAGED, int THREADS>
__device__ __forceinline__ void stage_get(const uint4 *at, int chunk, const T *src, bool on, P *f) {
    Vec<T> r;
    if (STAGED) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = at[(chunk + i) * THREADS];
    } else {
        r.load(src, on);
    }
    r.get(f);
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void stage_wait_prev() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// 16-byte chunks of a thread's row: y, the gate, x; backwards dxo and dz too.
template <typename T, typename S, int VPT, bool BWD>
struct Chunks {
    static constexpr int t = sizeof(T) / 2, s = sizeof(S) / 2;
    static constexpr int y = 0, g = VPT * t, x = 2 * VPT * t, dxo = x + VPT * s, dz = dxo + VPT * s;
    static constexpr int all = BWD ? dz + VPT * t : dxo;
    static constexpr int weights = 2 * VPT * t;
    static constexpr bool staged(int threads) { return (weights + 2 * all) * threads * 16 <= 224 * 1024; }
};

// A thread's vectors of the weights, in slots of its own (registers would be 16 to 32 a thread).
template <typename T, int TPR, int VPT, int THREADS>
__device__ __forceinline__ void keep_weights(const Params &p, int l, uint4 *at) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const T *w = static_cast<const T *>(i ? p.w_pre : p.w_post);
            Vec<T> r;
            r.load(w + (l + v * TPR) * 8, w && l + v * TPR < p.D / 8);
#pragma unroll
            for (int k = 0; k < (int)sizeof(T) / 2; ++k) at[((i * VPT + v) * (int)sizeof(T) / 2 + k) * THREADS] = r.v[k];
        }
}
template <typename T, int TPR, bool STAGED, int THREADS>
__device__ __forceinline__ void weight(const uint4 *at, int v, const void *w, int vec, int nv, P *f) {
    Vec<T> r;
    if (STAGED) {
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) r.v[k] = at[(v * (int)sizeof(T) / 2 + k) * THREADS];
    } else {
        r.load(static_cast<const T *>(w) + vec * 8, vec < nv);
    }
    r.get(f);
}

namespace {                        // (of each library its own: the caches of launch_kernel too)

constexpr int fwd_blocks(int tpr, int vpt) { return vpt > 2 ? 1 : 640 / threads_of(tpr); }
constexpr int bwd_blocks(int tpr, int vpt) { return vpt > 2 ? 1 : tpr > 256 ? 1 : tpr > 128 ? 2 : 3; }

template <typename T, typename S, int TPR, int VPT>
__global__ void __launch_bounds__(threads_of(TPR), fwd_blocks(TPR, VPT)) block_fwd_kernel(const Params p) {
    constexpr int R = threads_of(TPR) / TPR;
    __shared__ float s_sum[2][R][1][TPR / 32 > 0 ? TPR / 32 : 1];
    int64_t rows;
    if (!live_rows(p, rows)) return;
    RowSum<TPR, 1> sum{s_sum, 0};
    const int l = threadIdx.x % TPR, nv = p.D / 8;
    const float inv_d = 1.f / p.D;
    uint64_t seed = 0, offset = 0;
    if (p.cut) { seed = (uint64_t)p.rng[0]; offset = (uint64_t)p.rng[1]; }
    const float keep = p.cut ? p.scale * (65536.f / (65536 - p.cut)) : p.scale;
    using C = Chunks<T, S, VPT, false>;
    constexpr int TH = threads_of(TPR);
    constexpr bool ST = C::staged(TH);
    extern __shared__ __align__(16) uint4 s_rows[];        // weights [2 VPT t][TH], rows [2][chunks][TH]
    uint4 *weights = s_rows + threadIdx.x, *staged = weights + C::weights * TH;
    if (ST) keep_weights<T, TPR, VPT, TH>(p, l, weights);
    const int64_t step = (int64_t)gridDim.x * R;
    int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / TPR;
    int64_t t = p.H == 1 ? row : row / p.H;
    int h = p.H == 1 ? 0 : (int)(row - t * p.H);
    char *cy = place<T>(p.y, t, h, l), *cg = place<T>(p.gate, t, h, l), *cx = place<S>(p.x, t, h, l);
    char *co = place<S>(p.xo, t, h, l), *cz = place<T>(p.z, t, h, l);
    auto stage = [&](int64_t r, int buf) {                 // row r, at the cursors; moves them on
        uint4 *to = staged + buf * C::all * TH;
        if (r - threadIdx.x / TPR < rows) {                // (the same for the block)
            const bool live = r < rows && row_in<T>(p, p.y, cy, l) && row_in<T>(p, p.gate, cg, l) && row_in<S>(p, p.x, cx, l);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const bool on = live && l + v * TPR < nv;
                const T *none = static_cast<const T *>(p.y.p);
                stage_copy<T, ST, TH>(to, C::y + v * C::t, on ? vec_at<const T>(cy, v, TPR) : none, on);
                if (p.gate.p) stage_copy<T, ST, TH>(to, C::g + v * C::t, on ? vec_at<const T>(cg, v, TPR) : none, on);
                if (p.x.p) stage_copy<S, ST, TH>(to, C::x + v * C::s, on ? vec_at<const S>(cx, v, TPR) : reinterpret_cast<const S *>(none), on);
            }
        }
        stage_commit();
    };
    stage(row, 0);
    int buf = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * R; row0 < rows; row0 += step, buf ^= 1) {
        const bool live = row < rows && row_in<T>(p, p.y, cy, l) && row_in<T>(p, p.gate, cg, l) && row_in<S>(p, p.x, cx, l) &&
                          row_in<S>(p, p.xo, co, l) && row_in<T>(p, p.z, cz, l);
        const bool wrap = (h += p.dh) >= p.H;
        if (wrap) h -= p.H;
        char *here_cy = cy, *here_cg = cg, *here_cx = cx;  // (of this row, where it is read from memory)
        advance(cy, p.y, wrap);
        advance(cg, p.gate, wrap);
        advance(cx, p.x, wrap);
        stage(row + step, buf ^ 1);
        stage_wait_prev();
        const uint4 *in = staged + buf * C::all * TH;
        float scale = keep;
        if (p.post != GCL_NORM_NONE) {
            P q = both(0.f);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                P f[kPairs];
                stage_get<T, ST, TH>(in, C::y + v * C::t, vec_at<const T>(here_cy, v, TPR), live && l + v * TPR < nv, f);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) q = fma2(f[k], f[k], q);
            }
            float ss = sum_of(q);
            sum.template operator()<1>(&ss);
            scale *= inverse_length(p.post, ss, inv_d, p.eps);
        }
        P xo[VPT][kPairs], q = both(0.f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const bool on = live && l + v * TPR < nv;
            P w[kPairs];
            stage_get<T, ST, TH>(in, C::y + v * C::t, vec_at<const T>(here_cy, v, TPR), live && l + v * TPR < nv, xo[v]);
            if (p.w_post) {
                weight<T, TPR, ST, TH>(weights, v, p.w_post, l + v * TPR, nv, w);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) xo[v][k] = mul2(xo[v][k], w[k]);
            }
            if (p.gate.p) {
                P a[kPairs];
                stage_get<T, ST, TH>(in, C::g + v * C::t, vec_at<const T>(here_cg, v, TPR), live && l + v * TPR < nv, w);
                activation<T, false>(p.act, w, a, nullptr);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) xo[v][k] = mul2(xo[v][k], a[k]);
            }
            if (p.cut) drop(philox((uint64_t)(row * nv + l + v * TPR), offset, seed), (uint32_t)p.cut << 16, xo[v]);
            if (p.x.p) {
                stage_get<S, ST, TH>(in, C::x + v * C::s, vec_at<const S>(here_cx, v, TPR), live && l + v * TPR < nv && p.x.p, w);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) xo[v][k] = fma2(xo[v][k], both(scale), w[k]);
            } else {
#pragma unroll
                for (int k = 0; k < kPairs; ++k) xo[v][k] = mul2(xo[v][k], both(scale));
            }
            if (on && p.xo.p) Vec<S>::store(vec_at<S>(co, v, TPR), xo[v]);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) q = fma2(xo[v][k], xo[v][k], q);
        }
        float r = 1.f;
        if (p.z.p && p.pre != GCL_NORM_NONE) {
            float ss = sum_of(q);
            sum.template operator()<1>(&ss);
            r = inverse_length(p.pre, ss, inv_d, p.eps);
        }
        if (p.z.p)
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
#pragma unroll
            for (int k = 0; k < kPairs; ++k) xo[v][k] = mul2(xo[v][k], both(r));
            if (p.w_pre) {
                P w[kPairs];
                weight<T, TPR, ST, TH>(weights, VPT + v, p.w_pre, l + v * TPR, nv, w);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) xo[v][k] = mul2(xo[v][k], w[k]);
            }
            if (live && l + v * TPR < nv) Vec<T>::store(vec_at<T>(cz, v, TPR), xo[v]);
        }
        advance(co, p.xo, wrap);
        advance(cz, p.z, wrap);
        row += step;
    }
}

// The widest rows keep the sums of the weights' gradients in shared memory (each thread its own values), others in registers.
constexpr bool sums_in_smem(int vpt) { return vpt > 2; }

template <typename T, typename S, int TPR, int VPT>
__global__ void __launch_bounds__(threads_of(TPR), bwd_blocks(TPR, VPT)) block_bwd_kernel(const Params p) {
    constexpr int R = threads_of(TPR) / TPR;
    constexpr bool SM = sums_in_smem(VPT);
    __shared__ float s_sum[2][R][5][TPR / 32 > 0 ? TPR / 32 : 1];
    __shared__ P s_dw[R > 1 ? R : 1][R > 1 ? TPR * VPT * kPairs : 1];
    using C = Chunks<T, S, VPT, true>;
    constexpr int TH = threads_of(TPR);
    constexpr bool ST = C::staged(TH);
    extern __shared__ __align__(16) uint4 s_rows[];        // weights [2 VPT t][TH], rows [2][chunks][TH]
    uint4 *weights = s_rows + threadIdx.x, *staged = weights + C::weights * TH;
    P *s_wide = reinterpret_cast<P *>(s_rows + (ST ? C::weights + 2 * C::all : 0) * TH);           // [2][VPT][kPairs][TPR]
    launch_dependents();                                   // (the weights' sums wait for this grid's end)
    int64_t rows;
    if (!live_rows(p, rows)) return;
    RowSum<TPR, 5> sum{s_sum, 0};
    const int l = threadIdx.x % TPR, nv = p.D / 8;
    const float inv_d = 1.f / p.D;
    uint64_t seed = 0, offset = 0;
    if (p.cut) { seed = (uint64_t)p.rng[0]; offset = (uint64_t)p.rng[1]; }
    const float keep = p.cut ? p.scale * (65536.f / (65536 - p.cut)) : p.scale;
    if (ST) keep_weights<T, TPR, VPT, TH>(p, l, weights);
    P dw[2][SM ? 1 : VPT][kPairs];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                if (SM) s_wide[((i * VPT + v) * kPairs + k) * TPR + l] = both(0.f);
                else dw[i][SM ? 0 : v][k] = both(0.f);
            }
    }
    auto add = [&](int i, int v, int k, P a, P b) {        // += a b
        if (SM) {
            P &d = s_wide[((i * VPT + v) * kPairs + k) * TPR + l];
            d = fma2(a, b, d);
        } else {
            dw[i][SM ? 0 : v][k] = fma2(a, b, dw[i][SM ? 0 : v][k]);
        }
    };
    const int64_t step = (int64_t)gridDim.x * R;
    int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / TPR;
    int64_t t = p.H == 1 ? row : row / p.H;
    int h = p.H == 1 ? 0 : (int)(row - t * p.H);
    char *cy = place<T>(p.y, t, h, l), *cg = place<T>(p.gate, t, h, l), *cx = place<S>(p.x, t, h, l);
    char *cdo = place<S>(p.dxo, t, h, l), *cdz = place<T>(p.dz, t, h, l);
    char *cdy = place<T>(p.dy, t, h, l), *cdg = place<T>(p.dgate, t, h, l), *cdx = place<S>(p.dx, t, h, l);
    auto stage = [&](int64_t r, int buf) {                 // row r, at the cursors
        uint4 *to = staged + buf * C::all * TH;
        if (r - threadIdx.x / TPR < rows) {                // (the same for the block)
            const bool live = r < rows && row_in<T>(p, p.y, cy, l) && row_in<T>(p, p.gate, cg, l) && row_in<S>(p, p.x, cx, l) &&
                              row_in<S>(p, p.dxo, cdo, l) && row_in<T>(p, p.dz, cdz, l);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const bool on = live && l + v * TPR < nv;
                const T *none = static_cast<const T *>(p.y.p);
                const S *none_s = reinterpret_cast<const S *>(none);
                stage_copy<T, ST, TH>(to, C::y + v * C::t, on ? vec_at<const T>(cy, v, TPR) : none, on);
                if (p.gate.p) stage_copy<T, ST, TH>(to, C::g + v * C::t, on ? vec_at<const T>(cg, v, TPR) : none, on);
                stage_copy<S, ST, TH>(to, C::dxo + v * C::s, on && p.dxo.p ? vec_at<const S>(cdo, v, TPR) : none_s, on && p.dxo.p);
                if (p.dz.p) {
                    stage_copy<T, ST, TH>(to, C::dz + v * C::t, on ? vec_at<const T>(cdz, v, TPR) : none, on);
                    stage_copy<S, ST, TH>(to, C::x + v * C::s, on && p.x.p ? vec_at<const S>(cx, v, TPR) : none_s, on && p.x.p);
                }
            }
        }
        stage_commit();
    };
    stage(row, 0);
    int buf = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * R; row0 < rows; row0 += step, buf ^= 1) {
        const bool live = row < rows && row_in<T>(p, p.y, cy, l) && row_in<T>(p, p.gate, cg, l) && row_in<S>(p, p.x, cx, l) &&
                          row_in<S>(p, p.dxo, cdo, l) && row_in<T>(p, p.dz, cdz, l) && row_in<T>(p, p.dy, cdy, l) &&
                          row_in<T>(p, p.dgate, cdg, l) && row_in<S>(p, p.dx, cdx, l);
        const bool wrap = (h += p.dh) >= p.H;
        if (wrap) h -= p.H;
        char *here_cy = cy, *here_cg = cg, *here_cx = cx, *here_cdo = cdo, *here_cdz = cdz;        // (of this row, where it is read from memory)
        advance(cy, p.y, wrap);
        advance(cg, p.gate, wrap);
        advance(cx, p.x, wrap);
        advance(cdo, p.dxo, wrap);
        advance(cdz, p.dz, wrap);
        stage(row + step, buf ^ 1);
        stage_wait_prev();
        const uint4 *in = staged + buf * C::all * TH;
        float ry = 1.f;
        if (p.post != GCL_NORM_NONE) {
            P q = both(0.f);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                P f[kPairs];
                stage_get<T, ST, TH>(in, C::y + v * C::t, vec_at<const T>(here_cy, v, TPR), live && l + v * TPR < nv, f);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) q = fma2(f[k], f[k], q);
            }
            float ss = sum_of(q);
            sum.template operator()<1>(&ss);
            ry = live ? inverse_length(p.post, ss, inv_d, p.eps) : 0.f;       // (a row past the last adds 0 to the weights' sums)
        }
        // per vector: act and its slope, times scale and dropout's factor; then xo (v without dz), which the outputs use again
        P a[VPT][kPairs], da[VPT][kPairs], xo[VPT][kPairs];
        P s0 = both(0.f), s1 = s0, s2 = s0, s3 = s0, s4 = s0;          // sums of dxo v, xo^2, u xo, u v, xo v
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            P f[kPairs], w[kPairs];
            stage_get<T, ST, TH>(in, C::y + v * C::t, vec_at<const T>(here_cy, v, TPR), live && l + v * TPR < nv, f);
            if (p.w_post) {
                weight<T, TPR, ST, TH>(weights, v, p.w_post, l + v * TPR, nv, w);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) f[k] = mul2(f[k], w[k]);
            }
            if (p.gate.p) {
                stage_get<T, ST, TH>(in, C::g + v * C::t, vec_at<const T>(here_cg, v, TPR), live && l + v * TPR < nv, w);
                activation<T, true>(p.act, w, a[v], da[v]);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    a[v][k] = mul2(a[v][k], both(keep));
                    da[v][k] = mul2(da[v][k], both(keep));
                }
            } else {
#pragma unroll
                for (int k = 0; k < kPairs; ++k) a[v][k] = both(keep);
            }
            if (p.cut) {
                const uint4 words = philox((uint64_t)(row * nv + l + v * TPR), offset, seed);
                drop(words, (uint32_t)p.cut << 16, a[v]);
                if (p.gate.p) drop(words, (uint32_t)p.cut << 16, da[v]);
            }
            stage_get<S, ST, TH>(in, C::dxo + v * C::s, vec_at<const S>(here_cdo, v, TPR), live && l + v * TPR < nv && p.dxo.p, w);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                f[k] = mul2(mul2(f[k], both(ry)), a[v][k]);                    // v
                s0 = fma2(w[k], f[k], s0);
            }
            if (p.dz.p) {
                P u[kPairs];
                stage_get<T, ST, TH>(in, C::dz + v * C::t, vec_at<const T>(here_cdz, v, TPR), live && l + v * TPR < nv, u);
                if (p.w_pre) {
                    weight<T, TPR, ST, TH>(weights, VPT + v, p.w_pre, l + v * TPR, nv, w);
#pragma unroll
                    for (int k = 0; k < kPairs; ++k) u[k] = mul2(u[k], w[k]);
                }
                stage_get<S, ST, TH>(in, C::x + v * C::s, vec_at<const S>(here_cx, v, TPR), live && l + v * TPR < nv && p.x.p, w);     // (zeros without x)
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    const P o = add2(w[k], f[k]);
                    xo[v][k] = o;
                    s1 = fma2(o, o, s1);
                    s2 = fma2(u[k], o, s2);
                    s3 = fma2(u[k], f[k], s3);
                    s4 = fma2(o, f[k], s4);
                }
            }
        }
        float s5[5] = {sum_of(s0), sum_of(s1), sum_of(s2), sum_of(s3), sum_of(s4)};
        float r = 1.f, m = 0.f, mean = 0.f;                // r, r^3 M / D, P / D
        if (p.dz.p) {
            sum.template operator()<5>(s5);
            if (p.pre != GCL_NORM_NONE) {
                r = live ? inverse_length(p.pre, s5[1], inv_d, p.eps) : 0.f;
                m = r * (r * (r * s5[2])) * (p.pre == GCL_NORM_RMS ? inv_d : 1.f);      // (r^3 alone leaves fp32's range)
            }
            mean = s5[0] + r * s5[3] - m * s5[4];
        } else if (p.post != GCL_NORM_NONE) {
            sum.template operator()<1>(s5);
            mean = s5[0];
        }
        mean = p.post == GCL_NORM_NONE ? 0.f : p.post == GCL_NORM_RMS ? mean * inv_d : mean;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const bool on = live && l + v * TPR < nv;
            P d[kPairs], w[kPairs], q[kPairs], n[kPairs];
            stage_get<S, ST, TH>(in, C::dxo + v * C::s, vec_at<const S>(here_cdo, v, TPR), live && l + v * TPR < nv && p.dxo.p, d);
            if (p.dz.p) {
                stage_get<T, ST, TH>(in, C::dz + v * C::t, vec_at<const T>(here_cdz, v, TPR), live && l + v * TPR < nv, q);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    q[k] = mul2(q[k], both(r));
                    add(1, v, k, q[k], xo[v][k]);
                    d[k] = fma2(xo[v][k], both(-m), d[k]);
                }
                if (p.w_pre) {
                    weight<T, TPR, ST, TH>(weights, VPT + v, p.w_pre, l + v * TPR, nv, w);
#pragma unroll
                    for (int k = 0; k < kPairs; ++k) q[k] = mul2(q[k], w[k]);
                }
#pragma unroll
                for (int k = 0; k < kPairs; ++k) d[k] = add2(d[k], q[k]);
            }
            if (on && p.dx.p) Vec<S>::store(vec_at<S>(cdx, v, TPR), d);
            stage_get<T, ST, TH>(in, C::y + v * C::t, vec_at<const T>(here_cy, v, TPR), live && l + v * TPR < nv, n);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) n[k] = mul2(n[k], both(ry));
            if (p.gate.p) {
#pragma unroll
                for (int k = 0; k < kPairs; ++k) q[k] = mul2(mul2(d[k], da[v][k]), n[k]);
                if (p.w_post) {
                    weight<T, TPR, ST, TH>(weights, v, p.w_post, l + v * TPR, nv, w);
#pragma unroll
                    for (int k = 0; k < kPairs; ++k) q[k] = mul2(q[k], w[k]);
                }
                if (on) Vec<T>::store(vec_at<T>(cdg, v, TPR), q);
            }
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                d[k] = mul2(d[k], a[v][k]);
                add(0, v, k, d[k], n[k]);
            }
            if (p.w_post) {
                weight<T, TPR, ST, TH>(weights, v, p.w_post, l + v * TPR, nv, w);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) d[k] = mul2(d[k], w[k]);
            }
#pragma unroll
            for (int k = 0; k < kPairs; ++k) q[k] = mul2(fma2(n[k], both(-mean), d[k]), both(ry));
            if (on) Vec<T>::store(vec_at<T>(cdy, v, TPR), q);
        }
        advance(cdy, p.dy, wrap);
        advance(cdg, p.dgate, wrap);
        advance(cdx, p.dx, wrap);
        row += step;
    }
    // the block's sums of the weights' gradients, its rows side by side first
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float *part = i ? p.part_pre : p.part_post;
        if (!part) continue;
        part += (int64_t)blockIdx.x * p.D;
        if (R > 1) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int k = 0; k < kPairs; ++k) s_dw[R > 1 ? threadIdx.x / TPR : 0][R > 1 ? (l + v * TPR) * kPairs + k : 0] = dw[i][SM ? 0 : v][k];
            __syncthreads();
            for (int c = threadIdx.x; c < p.D / 2; c += threads_of(TPR)) {
                P s = both(0.f);
                for (int j = 0; j < R; ++j) s = add2(s, s_dw[j][R > 1 ? c : 0]);
                reinterpret_cast<P *>(part)[c] = s;
            }
        } else {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
                if (l + v * TPR < nv)
#pragma unroll
                    for (int k = 0; k < kPairs; ++k)
                        reinterpret_cast<P *>(part)[(l + v * TPR) * kPairs + k] =
                            SM ? s_wide[((i * VPT + v) * kPairs + k) * TPR + l] : dw[i][SM ? 0 : v][k];
        }
    }
}

constexpr int kFwdBlocks = 8, kBwdBlocks = 3;          // blocks an SM at most (the backward's leave sums in the workspace)

// Resident blocks on the current device (each then walks rows); 0: an error.  Looked up once a kernel and device, in `cache`.
template <typename K>
inline int resident(K kernel, int threads, size_t smem, int most, std::atomic<int> *cache) {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if ((n = cache[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess)
        return 0;
    n = (n < most ? n : most) * num_sms();
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <typename T, typename S, int TPR, int VPT, bool BWD>
cudaError_t launch_kernel(Params p, int *blocks, cudaStream_t s) {
    constexpr int R = threads_of(TPR) / TPR;
    using C = Chunks<T, S, VPT, BWD>;
    const size_t smem = sizeof(uint4) * (C::staged(threads_of(TPR)) ? C::weights + 2 * C::all : 0) * threads_of(TPR) +
                        (BWD && sums_in_smem(VPT) ? sizeof(P) * 2 * VPT * kPairs * TPR : 0);
    static std::atomic<int> cache[64];                     // zero-initialised (static storage)
    auto launch = [&](auto kernel) {
        const int most = resident(kernel, threads_of(TPR), smem, BWD ? kBwdBlocks : kFwdBlocks, cache);
        if (most < 1) return cudaErrorInvalidConfiguration;
        const int64_t need = (p.t_max * p.H + R - 1) / R;
        *blocks = (int)(need < most ? need : most);
        const int64_t step = (int64_t)*blocks * R;
        for (Rows *r : {&p.y, &p.gate, &p.z, &p.dz, &p.dy, &p.dgate}) r->step(step, p.H, sizeof(T));
        for (Rows *r : {&p.x, &p.xo, &p.dxo, &p.dx}) r->step(step, p.H, sizeof(S));
        p.dh = (int32_t)(step % p.H);
        kernel<<<*blocks, threads_of(TPR), smem, s>>>(p);
        return cudaGetLastError();
    };
    if constexpr (BWD) return launch(block_bwd_kernel<T, S, TPR, VPT>);
    else return launch(block_fwd_kernel<T, S, TPR, VPT>);
}

// Threads of a row by its width: two vectors a thread (fp32 rows one, which takes the same registers), more where 512
// threads do not hold the row so.
template <typename T, typename S, bool BWD>
cudaError_t launch_ts(const Params &p, int *blocks, cudaStream_t s) {
    constexpr int V = sizeof(T) == 4 ? 1 : 2;
    if (p.D <= 32 * V) return launch_kernel<T, S, 4, V, BWD>(p, blocks, s);
    if (p.D <= 64 * V) return launch_kernel<T, S, 8, V, BWD>(p, blocks, s);
    if (p.D <= 128 * V) return launch_kernel<T, S, 16, V, BWD>(p, blocks, s);
    if (p.D <= 256 * V) return launch_kernel<T, S, 32, V, BWD>(p, blocks, s);
    if (p.D <= 512 * V) return launch_kernel<T, S, 64, V, BWD>(p, blocks, s);
    if (p.D <= 1024 * V) return launch_kernel<T, S, 128, V, BWD>(p, blocks, s);
    if (p.D <= 2048 * V) return launch_kernel<T, S, 256, V, BWD>(p, blocks, s);
    if (p.D <= 4096 * V) return launch_kernel<T, S, 512, V, BWD>(p, blocks, s);
    if (V == 1 && p.D <= 8192) return launch_kernel<T, S, 512, 2, BWD>(p, blocks, s);
    return launch_kernel<T, S, 512, 4, BWD>(p, blocks, s);
}

}  // namespace

// One pair of these for each type of the rows and of the stream (block_norm_*.cu); *blocks: the backward's blocks.
template <typename T, typename S>
cudaError_t launch_fwd(const Params &p, cudaStream_t s);
template <typename T, typename S>
cudaError_t launch_bwd(const Params &p, int *blocks, cudaStream_t s);

#define GCL_BLOCK_NORM(T, S)                                                         \
    template <>                                                                      \
    cudaError_t launch_fwd<T, S>(const Params &p, cudaStream_t s) {                  \
        int blocks;                                                                  \
        return launch_ts<T, S, false>(p, &blocks, s);                                \
    }                                                                                \
    template <>                                                                      \
    cudaError_t launch_bwd<T, S>(const Params &p, int *blocks, cudaStream_t s) {     \
        return launch_ts<T, S, true>(p, blocks, s);                                  \
    }

}  // namespace blk
}  // namespace gcl
