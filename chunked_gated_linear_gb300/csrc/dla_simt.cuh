// dla_simt.cuh -- decayed linear attention on the CUDA cores, all arithmetic in fp32: the engine of
// dla.cuh for fp32 and fp16 inputs.  (One 16-bit operand a value holds neither: fp32 results leave no room for its
// rounding, and states and scores can pass fp16's largest value.  Sums of bf16 terms would, two for an fp16 value and
// three for an fp32 one, at as many more products on the tensor cores; that form is not built.)
//
// One CTA of 256 threads owns one segment of one (sequence, head) in one role and walks its chunks
// of C = 64 tokens with the state M [NA x NV] in shared memory.  Per chunk:
//   X = a b^T             16 x 16 threads, 4 x 4 values each, decayed and masked into shared memory
//   out = X c + gamma^e a M   rows 4 ty .., columns 4 tx + 64 jj ..: per inner index one scalar of X
//                         (or a) per row and one float4 of c (or M) per column block
//   M = gamma^len M + (gamma^e b)^T c   (NA / 16) x (NV / 16) values per thread
// Bound by shared memory: a 16-byte load takes its port four cycles, and the tiles give one per 8 to 16
// FMAs (2 (64 NA + 64 NV + 2 NA NV) FLOPs a token in all).  Twice the threads with half the tile each were a
// quarter slower.  4,096 tokens, 8 heads, 64 x 64: 67 us with the own states and the scan.
#pragma once

#include "dla.cuh"

namespace gcl {
namespace dla {

constexpr int kSimtThreads = 256;
constexpr int kSimtC = 64;

template <int NA, int NV>
struct SimtLayout {
    static constexpr int LA = NA + 4, LV = NV + 4, LX = kSimtC + 4;
    static constexpr int oA = 0;                       // a                 [C][LA]
    static constexpr int oB = oA + kSimtC * LA;        // b, later decayed  [C][LA]
    static constexpr int oC = oB + kSimtC * LA;        // c                 [C][LV]
    static constexpr int oX = oC + kSimtC * LV;        // X                 [C][LX]
    static constexpr int oM = oX + kSimtC * LX;        // M                 [NA][LV]
    static constexpr int oP = oM + NA * LV;            // gamma^0 .. gamma^C
    static constexpr int total = oP + kSimtC + 4;
    static constexpr size_t bytes = sizeof(float) * total;
};

// Eight consecutive values of a row as floats (16-byte aligned).
__device__ __forceinline__ void load8f(const float *p, float *v) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8f(const __nv_bfloat16 *p, float *v) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = __bfloat1622float2(h[e]);
        v[2 * e] = f.x;
        v[2 * e + 1] = f.y;
    }
}
__device__ __forceinline__ void load8f(const __half *p, float *v) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const __half2 *h = reinterpret_cast<const __half2 *>(&u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(h[e]);
        v[2 * e] = f.x;
        v[2 * e + 1] = f.y;
    }
}
// Four values into consecutive elements of a row (8-byte aligned, fp32: 16).
__device__ __forceinline__ void store4f(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4f(__nv_bfloat16 *p, const float *v) {
    __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(h);
}
__device__ __forceinline__ void store4f(__half *p, const float *v) {
    __half2 h[2] = {__floats2half2_rn(v[0], v[1]), __floats2half2_rn(v[2], v[3])};
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(h);
}

template <typename T, int NA, int NV, bool OWN>
__global__ void __launch_bounds__(kSimtThreads, simt_ctas(NA, NV)) dla_simt_kernel(const Params p) {
    using Lay = SimtLayout<NA, NV>;
    constexpr int C = kSimtC, LA = Lay::LA, LV = Lay::LV, LX = Lay::LX;
    constexpr int RM = NA / 16, JV = NV / 64;             // state rows and output column blocks per thread
    extern __shared__ __align__(16) float sm[];
    float *sA = sm + Lay::oA, *sB = sm + Lay::oB, *sC = sm + Lay::oC, *sX = sm + Lay::oX, *sM = sm + Lay::oM,
          *sP = sm + Lay::oP;
    if (OWN) launch_dependents();                          // (the scan waits for this grid's end)
    else if (blockIdx.x / p.n_roles / p.H >= p.n_max) grid_dependency_wait();    // (not a first segment: after the scan)
    if (status_blocks_cta(p.status)) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int unit = blockIdx.x / p.n_roles, h = unit % p.H;
    const int role = (p.roles >> (2 * (blockIdx.x % p.n_roles))) & 3;
    const bool rev = role >= kDv, trans = role == kDq || role == kDk;
    Item it;
    if (!find_item<kSimtThreads, OWN>(p, unit / p.H, rev, it)) return;
    const Rows ra = role == kFwd ? p.q : role == kDq ? p.d_o : role == kDv ? p.k : p.v;
    const Rows rb = role == kFwd ? p.k : role == kDq ? p.v : role == kDv ? p.q : p.d_o;
    const Rows rc = role == kFwd ? p.v : role == kDq ? p.k : role == kDv ? p.d_o : p.q;
    const Rows ro = role == kFwd ? p.o : role == kDq ? p.dq : role == kDv ? p.dv : p.dk;
    const float g = p.g[h];
    // scale: of the scores (every role), of the state's part (it holds scale q do^T backwards), of
    // the increments
    const float s_inner = p.scale, s_state = rev ? 1.f : p.scale, s_inc = rev ? p.scale : 1.f;
    const int64_t KV = (int64_t)NA * NV;
    const int64_t seq_state = ((int64_t)it.n * p.H + h) * KV, row_state = (it.row * p.H + h) * KV;
    const int64_t n_seq = (int64_t)p.n_max * p.H * KV, n_row = p.n_rows * p.H * KV;

    for (int e = tid; e <= C; e += kSimtThreads) sP[e] = decay_pow(g, e);
    {   // the entering state; element (r, c) of M is at r * NV + c, transposed roles: c * NA + r
        const float *seg = it.row < 0 ? nullptr : rev ? p.seg_rev : p.seg_fwd;
        const float *src = OWN ? nullptr : seg ? seg + row_state : rev ? p.dht : p.h0;
        if (!OWN && !seg && src) src += seq_state;
        if (src && !GCL_RANGE_IN_BOUNDS(seg ? row_state : seq_state, (seg ? row_state : seq_state) + KV - 1,
                                        seg ? n_row : n_seq, p.status))
            src = nullptr;
        // sixteen bytes at a time, every load in flight before the first store
        constexpr int N4 = NA * NV / 4 / kSimtThreads;
#pragma unroll 1
        for (int b0 = 0; b0 < N4; b0 += 8) {
            constexpr int PT = N4 < 8 ? N4 : 8;
            float4 v[PT];
#pragma unroll
            for (int i = 0; i < PT; ++i)
                v[i] = src ? reinterpret_cast<const float4 *>(src)[(b0 + i) * kSimtThreads + tid] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                const int e = ((b0 + i) * kSimtThreads + tid) * 4;
                if (!trans) {
                    *reinterpret_cast<float4 *>(sM + (e / NV) * LV + e % NV) = v[i];
                } else {
                    float *m = sM + (e % NA) * LV + e / NA;
                    m[0] = v[i].x; m[LV] = v[i].y; m[2 * LV] = v[i].z; m[3 * LV] = v[i].w;
                }
            }
        }
    }
    const int nch = (int)((it.s1 - it.s0 + C - 1) / C);
    for (int ic = 0; ic < nch; ++ic) {
        const int64_t t0 = it.s0 + (int64_t)(rev ? nch - 1 - ic : ic) * C;
        const int len = (int)(it.s1 - t0 < C ? it.s1 - t0 : C);
        __syncthreads();                                  // the previous chunk's tiles are read
        // rows past the end are zeros
        for (int e = tid; e < C * NA / 8; e += kSimtThreads) {
            const int r = e / (NA / 8), c = (e % (NA / 8)) * 8;
            float a[8] = {}, b[8] = {};
            if (r < len && GCL_IN_BOUNDS(t0 + r, p.t_max, p.status)) {
                if (!OWN) load8f(row_ptr<const T>(ra, t0 + r, h) + c, a);
                load8f(row_ptr<const T>(rb, t0 + r, h) + c, b);
            }
            if (!OWN) {
                store4f(sA + r * LA + c, a);
                store4f(sA + r * LA + c + 4, a + 4);
            }
            store4f(sB + r * LA + c, b);
            store4f(sB + r * LA + c + 4, b + 4);
        }
        for (int e = tid; e < C * NV / 8; e += kSimtThreads) {
            const int r = e / (NV / 8), c = (e % (NV / 8)) * 8;
            float v[8] = {};
            if (r < len && GCL_IN_BOUNDS(t0 + r, p.t_max, p.status)) load8f(row_ptr<const T>(rc, t0 + r, h) + c, v);
            store4f(sC + r * LV + c, v);
            store4f(sC + r * LV + c + 4, v + 4);
        }
        __syncthreads();
        if (!OWN) {
            // ---- X = a b^T, decayed and masked
            float x[4][4] = {};
#pragma unroll 4
            for (int kk = 0; kk < NA; kk += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = *reinterpret_cast<const float4 *>(sA + (ty + 16 * i) * LA + kk);
                    b[i] = *reinterpret_cast<const float4 *>(sB + (tx + 16 * i) * LA + kk);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[i][j] = fmaf(a[i].x, b[j].x, x[i][j]);
                        x[i][j] = fmaf(a[i].y, b[j].y, x[i][j]);
                        x[i][j] = fmaf(a[i].z, b[j].z, x[i][j]);
                        x[i][j] = fmaf(a[i].w, b[j].w, x[i][j]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // (zeros past the end as well: gamma^d may be infinite there if g > 0)
                    const int r = ty + 16 * i, c = tx + 16 * j, d = rev ? c - r : r - c;
                    sX[r * LX + c] = d >= 0 && (rev ? c : r) < len ? s_inner * sP[d] * x[i][j] : 0.f;
                }
            __syncthreads();
            // ---- out = X c + gamma^e a M
            float oin[4][4 * JV] = {}, ost[4][4 * JV] = {};
#pragma unroll 2
            for (int j = 0; j < C; j += 4) {
                float4 xr[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) xr[i] = *reinterpret_cast<const float4 *>(sX + (ty * 4 + i) * LX + j);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int b = 0; b < JV; ++b) {
                        const float4 c4 = *reinterpret_cast<const float4 *>(sC + (j + e) * LV + tx * 4 + 64 * b);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float xv = e == 0 ? xr[i].x : e == 1 ? xr[i].y : e == 2 ? xr[i].z : xr[i].w;
                            oin[i][4 * b] = fmaf(xv, c4.x, oin[i][4 * b]);
                            oin[i][4 * b + 1] = fmaf(xv, c4.y, oin[i][4 * b + 1]);
                            oin[i][4 * b + 2] = fmaf(xv, c4.z, oin[i][4 * b + 2]);
                            oin[i][4 * b + 3] = fmaf(xv, c4.w, oin[i][4 * b + 3]);
                        }
                    }
            }
#pragma unroll 2
            for (int k = 0; k < NA; k += 4) {
                float4 ar[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) ar[i] = *reinterpret_cast<const float4 *>(sA + (ty * 4 + i) * LA + k);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int b = 0; b < JV; ++b) {
                        const float4 m4 = *reinterpret_cast<const float4 *>(sM + (k + e) * LV + tx * 4 + 64 * b);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float av = e == 0 ? ar[i].x : e == 1 ? ar[i].y : e == 2 ? ar[i].z : ar[i].w;
                            ost[i][4 * b] = fmaf(av, m4.x, ost[i][4 * b]);
                            ost[i][4 * b + 1] = fmaf(av, m4.y, ost[i][4 * b + 1]);
                            ost[i][4 * b + 2] = fmaf(av, m4.z, ost[i][4 * b + 2]);
                            ost[i][4 * b + 3] = fmaf(av, m4.w, ost[i][4 * b + 3]);
                        }
                    }
            }
            if (ro.p) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = ty * 4 + i;
                    if (r >= len || !GCL_IN_BOUNDS(t0 + r, p.t_max, p.status)) continue;
                    const float f = s_state * sP[rev ? len - 1 - r : r + 1];
                    T *dst = row_ptr<T>(ro, t0 + r, h);
#pragma unroll
                    for (int b = 0; b < JV; ++b) {
                        float y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = fmaf(f, ost[i][4 * b + e], oin[i][4 * b + e]);
                        store4f(dst + tx * 4 + 64 * b, y);
                    }
                }
            }
        }
        // ---- M = gamma^len M + (gamma^e b)^T c
        __syncthreads();                                  // M and the raw b are read
        for (int e = tid; e < len * (NA / 4); e += kSimtThreads) {
            const int r = e / (NA / 4), c = (e % (NA / 4)) * 4;
            const float w = s_inc * sP[rev ? r + 1 : len - 1 - r];
            float4 *b = reinterpret_cast<float4 *>(sB + r * LA + c);
            float4 v = *b;
            v.x *= w; v.y *= w; v.z *= w; v.w *= w;
            *b = v;
        }
        __syncthreads();
        {
            float acc[RM][4 * JV];
            const float gl = sP[len];
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int b = 0; b < JV; ++b) {
                    const float4 m4 = *reinterpret_cast<const float4 *>(sM + (ty * RM + i) * LV + tx * 4 + 64 * b);
                    acc[i][4 * b] = gl * m4.x;
                    acc[i][4 * b + 1] = gl * m4.y;
                    acc[i][4 * b + 2] = gl * m4.z;
                    acc[i][4 * b + 3] = gl * m4.w;
                }
            for (int j = 0; j < len; ++j) {
                float bv[RM];
#pragma unroll
                for (int i = 0; i < RM; i += 4) {
                    const float4 b4 = *reinterpret_cast<const float4 *>(sB + j * LA + ty * RM + i);
                    bv[i] = b4.x; bv[i + 1] = b4.y; bv[i + 2] = b4.z; bv[i + 3] = b4.w;
                }
#pragma unroll
                for (int b = 0; b < JV; ++b) {
                    const float4 c4 = *reinterpret_cast<const float4 *>(sC + j * LV + tx * 4 + 64 * b);
#pragma unroll
                    for (int i = 0; i < RM; ++i) {
                        acc[i][4 * b] = fmaf(bv[i], c4.x, acc[i][4 * b]);
                        acc[i][4 * b + 1] = fmaf(bv[i], c4.y, acc[i][4 * b + 1]);
                        acc[i][4 * b + 2] = fmaf(bv[i], c4.z, acc[i][4 * b + 2]);
                        acc[i][4 * b + 3] = fmaf(bv[i], c4.w, acc[i][4 * b + 3]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int b = 0; b < JV; ++b) store4f(sM + (ty * RM + i) * LV + tx * 4 + 64 * b, acc[i] + 4 * b);
        }
    }
    __syncthreads();
    // ---- the leaving state: the segment's own, or ht (dh0) from the sequence's last segment in time
    float *dst = nullptr;
    int64_t at = 0, n_dst = n_seq;
    if (OWN) {
        dst = rev ? p.seg_rev : p.seg_fwd;
        at = row_state;
        n_dst = n_row;
    } else if (role == kFwd && it.last) {
        dst = p.ht;
        at = seq_state;
    } else if (role == kDv && it.i == 0) {
        dst = p.dh0;
        at = seq_state;
    }
    if (dst && GCL_RANGE_IN_BOUNDS(at, at + KV - 1, n_dst, p.status))
        for (int e = tid * 4; e < NA * NV; e += kSimtThreads * 4)
            *reinterpret_cast<float4 *>(dst + at + e) = *reinterpret_cast<const float4 *>(sM + (e / NV) * LV + e % NV);
}

template <typename T, int NA, int NV, bool OWN>
cudaError_t launch_simt_one(const Params &p, cudaStream_t s) {
    auto kern = dla_simt_kernel<T, NA, NV, OWN>;
    constexpr size_t smem = SimtLayout<NA, NV>::bytes;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)(((OWN ? 0 : p.n_max) + p.n_rows) * p.H * p.n_roles);
    if (!OWN && (p.seg_fwd || p.seg_rev)) return launch_dependent(kern, dim3(grid), dim3(kSimtThreads), smem, s, p);
    kern<<<grid, kSimtThreads, smem, s>>>(p);
    return cudaGetLastError();
}

// Roles kFwd and kDv run on [K, V] states, kDq and kDk on [V, K]: one launch for each shape.
template <typename T>
cudaError_t launch_simt_t(const Params &p0, bool own_states, int n_roles, const int *roles, cudaStream_t s) {
    for (int shape = 0; shape < 2; ++shape) {
        Params p = p0;
        if (!take_roles(p, n_roles, roles, shape)) continue;
        const int na = shape == 0 ? p.K : p.V, nv = shape == 0 ? p.V : p.K;
        cudaError_t e = cudaErrorInvalidValue;
        if (own_states) {
            if (na == 64 && nv == 64) e = launch_simt_one<T, 64, 64, true>(p, s);
            if (na == 64 && nv == 128) e = launch_simt_one<T, 64, 128, true>(p, s);
            if (na == 128 && nv == 64) e = launch_simt_one<T, 128, 64, true>(p, s);
            if (na == 128 && nv == 128) e = launch_simt_one<T, 128, 128, true>(p, s);
        } else {
            if (na == 64 && nv == 64) e = launch_simt_one<T, 64, 64, false>(p, s);
            if (na == 64 && nv == 128) e = launch_simt_one<T, 64, 128, false>(p, s);
            if (na == 128 && nv == 64) e = launch_simt_one<T, 128, 64, false>(p, s);
            if (na == 128 && nv == 128) e = launch_simt_one<T, 128, 128, false>(p, s);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace dla
}  // namespace gcl
