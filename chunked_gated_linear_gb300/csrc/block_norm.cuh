// block_norm.cuh -- the norms after and before a block with its gate, dropout, residual scale and sum.
//
//   v = scale drop(act(gate) n w_post), n = y r_y;   xo = x + v;   z = xo r w_pre
// Backward, with u = dz w_pre and the row's sums S = sum(xo^2) and M = sum(u xo):
//   d = dxo + r (u - xo r^2 M / D),   dy = r_y (d v / n - n P / D),   P = sum(d v)
// P is linear in d, so its three parts sum(dxo v), sum(u v), sum(xo v) cross the row's threads together with S and M: a row
// has two reductions (y's own length first, on which xo depends).
// HBM-bound: rows are read and written once.  A row is held by TPR threads, VPT vectors of eight values each, as loaded.
#pragma once

#include "dla.cuh"
#include "dla_simt.cuh"

namespace gcl {
namespace blk {

using dla::Rows;
using dla::row_ptr;

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

// The mask of a vector's eight values, bit e set where value e is kept.
__device__ __forceinline__ uint32_t kept(int32_t cut, int64_t vec, uint64_t seed, uint64_t offset) {
    if (!cut) return 0xFFu;
    const uint4 w = philox((uint64_t)vec, offset, seed);
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t half = e & 1 ? word[e / 2] >> 16 : word[e / 2] & 0xFFFFu;
        m |= (half >= (uint32_t)cut ? 1u : 0u) << e;
    }
    return m;
}

// act(g) and its derivative.
template <typename T>
__device__ __forceinline__ void activation(int act, float g, float &a, float &da) {
    if (act == GCL_ACT_NONE) {
        a = g;
        da = 1.f;
        return;
    }
    // sigmoid(g) and sigmoid(-g), neither by a difference
    const float e = sizeof(T) == 4 ? expf(-fabsf(g)) : __expf(-fabsf(g));
    const float hi = sizeof(T) == 4 ? 1.f / (1.f + e) : __fdividef(1.f, 1.f + e), lo = e * hi;
    const float s = g >= 0.f ? hi : lo, c = g >= 0.f ? lo : hi;
    a = act == GCL_ACT_SILU ? g * s : s;
    da = act == GCL_ACT_SILU ? s * fmaf(g, c, 1.f) : s * c;
}

// Eight consecutive values of a row as loaded.
template <typename T>
struct Vec {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p, bool on) {
#pragma unroll
        for (int e = 0; e < (int)sizeof(T) / 2; ++e) v[e] = on ? reinterpret_cast<const uint4 *>(p)[e] : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float *f) const { dla::load8f(reinterpret_cast<const T *>(v), f); }
    static __device__ __forceinline__ void store(T *p, const float *f) {
        Vec o;
        dla::store4f(reinterpret_cast<T *>(o.v), f);
        dla::store4f(reinterpret_cast<T *>(o.v) + 4, f + 4);
#pragma unroll
        for (int e = 0; e < (int)sizeof(T) / 2; ++e) reinterpret_cast<uint4 *>(p)[e] = o.v[e];
    }
};

constexpr int threads_of(int tpr) { return tpr > 256 ? tpr : 256; }

// Sums over a row's threads.  Rows of several warps pass through shared memory; `turn` alternates two buffers, so that
// one barrier a reduction is enough.
template <int TPR, int NS>
struct RowSum {
    static constexpr int W = TPR / 32 > 0 ? TPR / 32 : 1;          // warps of a row
    static constexpr int R = threads_of(TPR) / TPR;                // rows of a block
    float (*buf)[R][W][NS];
    int turn;
    template <int N>
    __device__ __forceinline__ void operator()(float *s) {
#pragma unroll
        for (int d = (TPR < 32 ? TPR : 32) / 2; d; d >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
        if (TPR <= 32) return;
        const int row = threadIdx.x / TPR, warp = threadIdx.x % TPR / 32;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) buf[turn][row][warp][i] = s[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            s[i] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) s[i] += buf[turn][row][w][i];
        }
        turn ^= 1;
    }
};

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

// A vector of a weight as floats; ones without weight.
template <typename T>
__device__ __forceinline__ void weight(const void *w, int at, bool on, float *f) {
    if (w) {
        Vec<T> r;
        r.load(static_cast<const T *>(w) + at * 8, on);
        r.get(f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 1.f;
    }
}

template <typename T, typename S, int TPR, int VPT>
__global__ void __launch_bounds__(threads_of(TPR)) block_fwd_kernel(const Params p) {
    constexpr int R = threads_of(TPR) / TPR;
    __shared__ float s_sum[2][R][TPR / 32 > 0 ? TPR / 32 : 1][1];
    int64_t rows;
    if (!live_rows(p, rows)) return;
    RowSum<TPR, 1> sum{s_sum, 0};
    const int l = threadIdx.x % TPR, nv = p.D / 8;
    const float inv_d = 1.f / p.D;
    uint64_t seed = 0, offset = 0;
    if (p.cut) { seed = (uint64_t)p.rng[0]; offset = (uint64_t)p.rng[1]; }
    const float keep = p.cut ? p.scale * (65536.f / (65536 - p.cut)) : p.scale;
    for (int64_t row0 = (int64_t)blockIdx.x * R; row0 < rows; row0 += (int64_t)gridDim.x * R) {
        const int64_t row = row0 + threadIdx.x / TPR, t = p.H == 1 ? row : row / p.H;
        const int h = p.H == 1 ? 0 : (int)(row - t * p.H);
        const bool live = row < rows;
        Vec<T> y[VPT], g[VPT];
        Vec<S> x[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int at = l + v * TPR;
            const bool on = live && at < nv && GCL_IN_BOUNDS(t, p.t_max, p.status);
            y[v].load(row_ptr<const T>(p.y, t, h) + at * 8, on);
            if (p.gate.p) g[v].load(row_ptr<const T>(p.gate, t, h) + at * 8, on);
            if (p.x.p) x[v].load(row_ptr<const S>(p.x, t, h) + at * 8, on);
        }
        float ry = 1.f;
        if (p.post != GCL_NORM_NONE) {
            float ss = 0.f;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                float f[8];
                y[v].get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
            }
            sum.template operator()<1>(&ss);
            ry = inverse_length(p.post, ss, inv_d, p.eps);
        }
        float xo[VPT][8], ss = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int at = l + v * TPR;
            const bool on = live && at < nv;
            float w[8];
            y[v].get(xo[v]);
            const uint32_t mask = kept(p.cut, row * nv + at, seed, offset);
            weight<T>(p.w_post, at, on, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) xo[v][e] *= ry * (mask >> e & 1 ? keep : 0.f) * w[e];
            if (p.gate.p) {
                g[v].get(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float a, da;
                    activation<T>(p.act, w[e], a, da);
                    xo[v][e] *= a;
                }
            }
            if (p.x.p) {
                x[v].get(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) xo[v][e] += w[e];
            }
            if (on && p.xo.p) Vec<S>::store(row_ptr<S>(p.xo, t, h) + at * 8, xo[v]);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(xo[v][e], xo[v][e], ss);
        }
        if (!p.z.p) continue;
        float r = 1.f;
        if (p.pre != GCL_NORM_NONE) {
            sum.template operator()<1>(&ss);
            r = inverse_length(p.pre, ss, inv_d, p.eps);
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int at = l + v * TPR;
            const bool on = live && at < nv;
            float w[8];
            weight<T>(p.w_pre, at, on, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) xo[v][e] *= r * w[e];
            if (on) Vec<T>::store(row_ptr<T>(p.z, t, h) + at * 8, xo[v]);
        }
    }
}

// Wide rows keep the sums of the weights' gradients in shared memory (each thread its own values), others in registers.
constexpr bool sums_in_smem(int vpt) { return vpt > 1; }

template <typename T, typename S, int TPR, int VPT>
__global__ void __launch_bounds__(threads_of(TPR)) block_bwd_kernel(const Params p) {
    constexpr int R = threads_of(TPR) / TPR;
    constexpr bool SM = sums_in_smem(VPT);
    __shared__ float s_sum[2][R][TPR / 32 > 0 ? TPR / 32 : 1][5];
    __shared__ float s_dw[R > 1 ? R : 1][R > 1 ? TPR * 8 : 1];
    extern __shared__ __align__(16) float s_wide[];        // [2][VPT][8][TPR]
    launch_dependents();                                   // (the weights' sums wait for this grid's end)
    int64_t rows;
    if (!live_rows(p, rows)) return;
    RowSum<TPR, 5> sum{s_sum, 0};
    const int l = threadIdx.x % TPR, nv = p.D / 8;
    const float inv_d = 1.f / p.D;
    const float post_d = p.post == GCL_NORM_RMS ? inv_d : 1.f, pre_d = p.pre == GCL_NORM_RMS ? inv_d : 1.f;
    uint64_t seed = 0, offset = 0;
    if (p.cut) { seed = (uint64_t)p.rng[0]; offset = (uint64_t)p.rng[1]; }
    const float keep = p.cut ? p.scale * (65536.f / (65536 - p.cut)) : p.scale;
    float dw[2][SM ? 1 : VPT][8];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (SM) s_wide[((k * VPT + v) * 8 + e) * TPR + l] = 0.f;
                else dw[k][SM ? 0 : v][e] = 0.f;
            }
    auto add = [&](int k, int v, int e, float a) {
        if (SM) s_wide[((k * VPT + v) * 8 + e) * TPR + l] += a;
        else dw[k][SM ? 0 : v][e] += a;
    };
    for (int64_t row0 = (int64_t)blockIdx.x * R; row0 < rows; row0 += (int64_t)gridDim.x * R) {
        const int64_t row = row0 + threadIdx.x / TPR, t = p.H == 1 ? row : row / p.H;
        const int h = p.H == 1 ? 0 : (int)(row - t * p.H);
        const bool live = row < rows;
        Vec<T> y[VPT], g[VPT], dz[VPT];
        Vec<S> x[VPT], dxo[VPT];
        uint32_t mask[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int at = l + v * TPR;
            const bool on = live && at < nv && GCL_IN_BOUNDS(t, p.t_max, p.status);
            y[v].load(row_ptr<const T>(p.y, t, h) + at * 8, on);
            if (p.gate.p) g[v].load(row_ptr<const T>(p.gate, t, h) + at * 8, on);
            dxo[v].load(row_ptr<const S>(p.dxo, t, h) + at * 8, on && p.dxo.p);
            if (p.dz.p) {
                dz[v].load(row_ptr<const T>(p.dz, t, h) + at * 8, on);
                x[v].load(row_ptr<const S>(p.x, t, h) + at * 8, on && p.x.p);
            }
        }
        float ry = 1.f;
        if (p.post != GCL_NORM_NONE) {
            float ss = 0.f;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                float f[8];
                y[v].get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
            }
            sum.template operator()<1>(&ss);
            ry = inverse_length(p.post, ss, inv_d, p.eps);
        }
        // n = y ry, w_post, act and its slope of a vector (formed again for the outputs: registers)
        auto branch = [&](int v, float *n, float *w, float *a, float *da) {
            const int at = l + v * TPR;
            y[v].get(n);
#pragma unroll
            for (int e = 0; e < 8; ++e) { n[e] *= ry; a[e] = 1.f; da[e] = 0.f; }
            weight<T>(p.w_post, at, live && at < nv, w);
            if (p.gate.p) {
                float q[8];
                g[v].get(q);
#pragma unroll
                for (int e = 0; e < 8; ++e) activation<T>(p.act, q[e], a[e], da[e]);
            }
        };
        float s5[5] = {0.f, 0.f, 0.f, 0.f, 0.f};           // sums of dxo v, xo^2, u xo, u v, xo v
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float n[8], w[8], a[8], da[8], q[8], u[8];
            mask[v] = kept(p.cut, row * nv + l + v * TPR, seed, offset);
            branch(v, n, w, a, da);
            dxo[v].get(q);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                n[e] *= w[e] * (mask[v] >> e & 1 ? keep : 0.f) * a[e];          // v
                s5[0] = fmaf(q[e], n[e], s5[0]);
            }
            if (p.dz.p) {
                dz[v].get(u);
                weight<T>(p.w_pre, l + v * TPR, live && l + v * TPR < nv, w);
                if (p.x.p) x[v].get(q);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xo = p.x.p ? q[e] + n[e] : n[e];
                    u[e] *= w[e];
                    s5[1] = fmaf(xo, xo, s5[1]);
                    s5[2] = fmaf(u[e], xo, s5[2]);
                    s5[3] = fmaf(u[e], n[e], s5[3]);
                    s5[4] = fmaf(xo, n[e], s5[4]);
                }
            }
        }
        float r = 1.f, m = 0.f, P = 0.f;                   // r, r^3 M / D, P / D
        if (p.dz.p) {
            sum.template operator()<5>(s5);
            if (p.pre != GCL_NORM_NONE) {
                r = inverse_length(p.pre, s5[1], inv_d, p.eps);
                m = r * r * r * s5[2] * pre_d;
            }
            P = s5[0] + r * s5[3] - m * s5[4];
        } else if (p.post != GCL_NORM_NONE) {
            sum.template operator()<1>(s5);
            P = s5[0];
        }
        P = p.post != GCL_NORM_NONE ? P * post_d : 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int at = l + v * TPR;
            const bool on = live && at < nv;
            float n[8], w[8], a[8], da[8], d[8], q[8];
            branch(v, n, w, a, da);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = mask[v] >> e & 1 ? keep : 0.f;
                a[e] *= f;
                da[e] *= f;
            }
            dxo[v].get(d);
            if (p.dz.p) {
                float u[8], w2[8];
                if (p.x.p) x[v].get(q);
                dz[v].get(u);
                weight<T>(p.w_pre, at, on, w2);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xo = fmaf(n[e] * w[e], a[e], p.x.p ? q[e] : 0.f);
                    add(1, v, e, u[e] * xo * r);
                    d[e] += u[e] * w2[e] * r - xo * m;
                }
            }
            if (on && p.dx.p) Vec<S>::store(row_ptr<S>(p.dx, t, h) + at * 8, d);
            if (p.gate.p) {
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = d[e] * n[e] * w[e] * da[e];
                if (on) Vec<T>::store(row_ptr<T>(p.dgate, t, h) + at * 8, q);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dn = d[e] * a[e];
                add(0, v, e, dn * n[e]);
                q[e] = ry * (dn * w[e] - n[e] * P);
            }
            if (on) Vec<T>::store(row_ptr<T>(p.dy, t, h) + at * 8, q);
        }
    }
    // the block's sums of the weights' gradients, its rows side by side first
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float *part = k ? p.part_pre : p.part_post;
        if (!part) continue;
        if (R > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) s_dw[R > 1 ? threadIdx.x / TPR : 0][R > 1 ? l * 8 + e : 0] = dw[k][0][e];
            __syncthreads();
            for (int c = threadIdx.x; c < p.D; c += threads_of(TPR)) {
                float s = 0.f;
                for (int i = 0; i < R; ++i) s += s_dw[i][R > 1 ? c : 0];
                part[(int64_t)blockIdx.x * p.D + c] = s;
            }
        } else {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
                if (l + v * TPR < nv)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        part[(int64_t)blockIdx.x * p.D + (l + v * TPR) * 8 + e] =
                            SM ? s_wide[((k * VPT + v) * 8 + e) * TPR + l] : dw[k][SM ? 0 : v][e];
        }
    }
}

constexpr int kMaxBlocks = 8;      // resident blocks an SM at most (256 threads of the SM's 2,048)

// Resident blocks on the current device (each then walks rows); 0: an error.
template <typename K>
inline int resident(K kernel, int threads, size_t smem) {
    int n = 0;
    if (smem > 48 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess) return 0;
    return (n < kMaxBlocks ? n : kMaxBlocks) * num_sms();
}

template <typename T, typename S, int TPR, int VPT, bool BWD>
cudaError_t launch_kernel(const Params &p, int *blocks, cudaStream_t s) {
    constexpr int R = threads_of(TPR) / TPR;
    const auto kernel = BWD ? block_bwd_kernel<T, S, TPR, VPT> : block_fwd_kernel<T, S, TPR, VPT>;
    const size_t smem = BWD && sums_in_smem(VPT) ? sizeof(float) * 2 * VPT * 8 * TPR : 0;
    const int most = resident(kernel, threads_of(TPR), smem);
    if (most < 1) return cudaErrorInvalidConfiguration;
    const int64_t need = (p.t_max * p.H + R - 1) / R;
    *blocks = (int)(need < most ? need : most);
    kernel<<<*blocks, threads_of(TPR), smem, s>>>(p);
    return cudaGetLastError();
}

// Threads of a row by its width: at most two vectors a thread up to 8,192 values, four beyond.
template <typename T, typename S, bool BWD>
cudaError_t launch_ts(const Params &p, int *blocks, cudaStream_t s) {
    if (p.D <= 64) return launch_kernel<T, S, 8, 1, BWD>(p, blocks, s);
    if (p.D <= 128) return launch_kernel<T, S, 16, 1, BWD>(p, blocks, s);
    if (p.D <= 256) return launch_kernel<T, S, 32, 1, BWD>(p, blocks, s);
    if (p.D <= 1024) return launch_kernel<T, S, 128, 1, BWD>(p, blocks, s);
    if (p.D <= 2048) return launch_kernel<T, S, 256, 1, BWD>(p, blocks, s);
    if (p.D <= 4096) return launch_kernel<T, S, 256, 2, BWD>(p, blocks, s);
    if (p.D <= 8192) return launch_kernel<T, S, 512, 2, BWD>(p, blocks, s);
    return launch_kernel<T, S, 512, 4, BWD>(p, blocks, s);
}

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
