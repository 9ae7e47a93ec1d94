// qk_norm_rope.cu -- norm of the queries and keys of each head and the position rotation in one pass,
// forward and backward, and the table of angles.
//
// For a row x of D values: n = r x with r = 1 / sqrt(sum(x^2) / D + eps) (RMS), without the / D (L2)
// or 1; z = n w; y = rotation of z.  The rotation's transpose turns by the opposite angle, so with
// dz = rotation^T dy and u = dz w:
//   dx = r (u - x r^2 sum(u x) / D)   (RMS; L2 without / D),   dw = sum over rows of dz n.
// HBM-bound: rows are read and written once (the backward reads x and dy, writes dx).  D / 8 lanes
// hold one row, 16 bytes (fp32: 32) each; sums over a row are shuffles inside those lanes, and the
// partner of a half-split pair sits R / 16 lanes away.  Lanes keep one token for up to four heads: its
// cos and sin rows and the weights are loaded once for them, and the rows of all four are in flight
// together (one row at a time left HBM at half its rate).
#include "dla.cuh"
#include "dla_simt.cuh"

namespace gcl {
namespace qk {
namespace {

using dla::Rows;
using dla::row_ptr;
constexpr int kThreads = 256;

struct Side {                      // q or k
    Rows x, dy, y;                 // y: the forward's output, or dx
    const void *w;
    float *partial;                // [blocks, D] sums of the weight's gradient, or NULL
    float *dw;
    int32_t H;
};
struct QkParams {
    Side side[2];
    const float *cos_t, *sin_t;
    const int32_t *pos;
    int32_t *status;
    int64_t t_max, n_pos;
    int32_t R, norm, pair;
    float eps;
    int32_t groups[2];             // head groups of q and of k for each token
};

__device__ __forceinline__ void store8f(float *p, const float *v) {
    dla::store4f(p, v);
    dla::store4f(p + 4, v + 4);
}
template <typename T>
__device__ __forceinline__ void store8f(T *p, const float *v) {
    uint4 u;
    dla::store4f(reinterpret_cast<T *>(&u), v);
    dla::store4f(reinterpret_cast<T *>(&u) + 4, v + 4);
    *reinterpret_cast<uint4 *>(p) = u;
}

// Sum over the D / 8 lanes of a row.
template <int L>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int d = L / 2; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// Turns the eight channels 8 l .. 8 l + 7 of a row by the token's angles (sign -1: back).  c, s: the
// lane's cosines and sines.  Every lane of the warp calls it.
template <int L>
__device__ __forceinline__ void rotate(float *z, const float *c, const float *s, int l, int R, int pair, float sign) {
    if (R == 0) return;
    const bool in = l < R / 8;
    if (pair == GCL_PAIR_ADJACENT) {
        if (in) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = z[2 * e], b = z[2 * e + 1], sn = sign * s[e];
                z[2 * e] = a * c[e] - b * sn;
                z[2 * e + 1] = fmaf(a, sn, b * c[e]);
            }
        }
        return;
    }
    const int half = R / 16;                               // lanes of half the rotated channels
    const bool first = l < half;
    const int lane = threadIdx.x & 31;
    const int src = in ? (first ? lane + half : lane - half) : lane;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float o = __shfl_sync(0xffffffffu, z[e], src);
        const float sn = sign * s[e];
        if (in) z[e] = first ? z[e] * c[e] - o * sn : fmaf(o, sn, z[e] * c[e]);
    }
}

// The lane's cosines and sines of position `pos`.
__device__ __forceinline__ void angles(const QkParams &p, int64_t pos, int l, float *c, float *s) {
    if (l >= p.R / 8) return;
    const int64_t row = pos * (p.R / 2);
    if (p.pair == GCL_PAIR_ADJACENT) {
        const float4 a = *reinterpret_cast<const float4 *>(p.cos_t + row + l * 4);
        const float4 b = *reinterpret_cast<const float4 *>(p.sin_t + row + l * 4);
        c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
        s[0] = b.x; s[1] = b.y; s[2] = b.z; s[3] = b.w;
    } else {
        const int at = (l % (p.R / 16)) * 8;
        dla::load8f(p.cos_t + row + at, c);
        dla::load8f(p.sin_t + row + at, s);
    }
}

// Eight consecutive values of a row as loaded.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int e = 0; e < (int)sizeof(T) / 2; ++e) v[e] = reinterpret_cast<const uint4 *>(p)[e];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < (int)sizeof(T) / 2; ++e) v[e] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float *x) const { dla::load8f(reinterpret_cast<const T *>(v), x); }
};

// One lane group (D / 8 lanes) takes PER heads of one token of q or k at a time; groups walk the (token,
// head group) pairs with the grid's stride.  Lanes without work stay for the shuffles.  BWD: y gets
// dx, and the weights' gradients are summed per block.
template <typename T, int D, bool BWD, int PER>
__global__ void __launch_bounds__(kThreads) qk_kernel(const QkParams p) {
    constexpr int L = D / 8, G = kThreads / L;             // lanes per row, lane groups per block
    __shared__ float s_dw[BWD ? 2 : 1][BWD ? G : 1][BWD ? D : 1];
    if (status_blocks_cta(p.status)) return;
    const int tid = threadIdx.x, l = tid % L, grp = tid / L;
    const uint32_t per_token = p.groups[0] + p.groups[1];
    const int64_t work = p.t_max * per_token;
    float dw[BWD ? 2 : 1][8] = {};
    for (int64_t i0 = (int64_t)blockIdx.x * G; i0 < work; i0 += (int64_t)gridDim.x * G) {
        const int64_t i = i0 + grp;
        bool live = i < work;
        int64_t t = 0;
        int hg = 0;
        if (live) {
            t = i >> 32 ? i / per_token : (uint32_t)i / per_token;
            hg = (int)(i - t * per_token);
        }
        const int which = hg < p.groups[0] ? 0 : 1;
        const Side &sd = p.side[which];
        const int h0 = (hg - (which ? p.groups[0] : 0)) * PER;
        float c[8] = {}, s[8] = {};
        int64_t pos = 0;
        if (live && p.pos) {
            pos = p.pos[t];
            live = pos >= 0;
            if (p.R > 0 && pos >= p.n_pos) {
                live = false;
                status_set(p.status, GCL_DEV_BAD_RANGE);
            }
        }
        Raw<T> xr[PER], dr[BWD ? PER : 1];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const bool on = live && h0 + j < sd.H;
            if (on) xr[j].load(row_ptr<const T>(sd.x, t, h0 + j) + l * 8);
            else xr[j].zero();
            if (BWD) {
                if (on) dr[j].load(row_ptr<const T>(sd.dy, t, h0 + j) + l * 8);
                else dr[j].zero();
            }
        }
        if (live && p.R > 0) angles(p, pos, l, c, s);
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
        if (sd.w) dla::load8f(static_cast<const T *>(sd.w) + l * 8, w);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int h = h0 + j;
            const bool on = live && h < sd.H;
            float x[8], y[8];
            xr[j].get(x);
            if (BWD) dr[j].get(y);
            float r = 1.f;
            if (p.norm != GCL_NORM_NONE) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
                ss = row_sum<L>(ss);
                r = rsqrtf((p.norm == GCL_NORM_RMS ? ss * (1.f / D) : ss) + p.eps);
            }
            if (!BWD) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = x[e] * r * w[e];
                rotate<L>(y, c, s, l, p.R, p.pair, 1.f);
                if (on) store8f(row_ptr<T>(sd.y, t, h) + l * 8, y);
            } else {
                rotate<L>(y, c, s, l, p.R, p.pair, -1.f);  // dz
                float ux = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = x[e] * r;
                    if (on) {                              // (constant indexes: dw stays in registers)
                        if (which == 0) dw[0][e] = fmaf(y[e], n, dw[0][e]);
                        else dw[BWD][e] = fmaf(y[e], n, dw[BWD][e]);
                    }
                    y[e] *= w[e];                          // u
                    ux = fmaf(y[e], n, ux);
                    x[e] = n;
                }
                if (p.norm != GCL_NORM_NONE) {
                    ux = row_sum<L>(ux) * (p.norm == GCL_NORM_RMS ? 1.f / D : 1.f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = r * fmaf(-x[e], ux, y[e]);
                }
                if (on) store8f(row_ptr<T>(sd.y, t, h) + l * 8, y);
            }
        }
    }
    if (BWD && (p.side[0].partial || p.side[1].partial)) {
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
            for (int e = 0; e < 8; ++e) s_dw[which][grp][l * 8 + e] = dw[which][e];
        __syncthreads();
        for (int e = tid; e < 2 * D; e += kThreads) {
            const int which = e / D, ch = e % D;
            float sum = 0.f;
            for (int g = 0; g < G; ++g) sum += s_dw[which][g][ch];
            if (p.side[which].partial) p.side[which].partial[(int64_t)blockIdx.x * D + ch] = sum;
        }
    }
}

// The weights' gradients from the blocks' sums, in a fixed order: one block per 32 channels, eight
// rows of threads over the sums.
__global__ void __launch_bounds__(256) qk_dw_kernel(const QkParams p, int blocks, int D) {
    __shared__ float s[8][32];
    if (status_blocks_cta(p.status)) return;
    const Side &sd = p.side[blockIdx.y];
    if (!sd.partial) return;
    const int ch = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
    float sum = 0.f;
    for (int b = r; b < blocks; b += 8) sum += sd.partial[(int64_t)b * D + ch];
    s[r][threadIdx.x & 31] = sum;
    __syncthreads();
    if (r == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i) sum += s[i][threadIdx.x];
        sd.dw[ch] = sum;
    }
}

__global__ void rope_table_kernel(float *cos_t, float *sin_t, int64_t n, int half, double base) {
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= n * half) return;
    const double a = (double)(e / half) * pow(base, -(double)(e % half) / half);
    double sn, cs;
    sincos(a, &sn, &cs);
    cos_t[e] = (float)cs;
    sin_t[e] = (float)sn;
}

// Blocks of the backward: a fixed number per SM, each walking many tokens, so that the partial
// sums of the weights' gradients stay few.
int bwd_blocks(int64_t t_max, int32_t HQ, int32_t HK, int D) {
    const int64_t groups = kThreads / (D / 8);
    const int64_t most = (t_max * ((int64_t)HQ + HK) + groups - 1) / groups;
    const int64_t want = 4 * (int64_t)num_sms();
    return (int)(most < want ? most : want);
}

template <typename T, int D, int PER>
cudaError_t launch_qk_per(QkParams &p, bool backward, cudaStream_t s) {
    const int64_t G = kThreads / (D / 8), sms = num_sms();
    for (int i = 0; i < 2; ++i) p.groups[i] = (p.side[i].H + PER - 1) / PER;
    const int64_t work = p.t_max * (p.groups[0] + p.groups[1]);
    const int64_t most = (work + G - 1) / G;
    if (!backward) {
        qk_kernel<T, D, false, PER><<<(unsigned)(most < 16 * sms ? most : 16 * sms), kThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    const int cap = bwd_blocks(p.t_max, p.side[0].H, p.side[1].H, D);
    const int blocks = (int)(most < cap ? most : cap);
    qk_kernel<T, D, true, PER><<<blocks, kThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && (p.side[0].partial || p.side[1].partial)) {
        qk_dw_kernel<<<dim3(D / 32, 2), 256, 0, s>>>(p, blocks, D);
        e = cudaGetLastError();
    }
    return e;
}

template <typename T, int D>
cudaError_t launch_qk(QkParams &p, bool backward, cudaStream_t s) {
    // four heads per lane group once there are rows for two full waves; few rows are spread one by one,
    // for latency
    const int64_t G = kThreads / (D / 8), rows = p.t_max * ((int64_t)p.side[0].H + p.side[1].H);
    return rows >= 4 * 16 * (int64_t)num_sms() * G ? launch_qk_per<T, D, 4>(p, backward, s) : launch_qk_per<T, D, 1>(p, backward, s);
}

template <typename T>
cudaError_t launch_qk_t(QkParams &p, int D, bool backward, cudaStream_t s) {
    if (D == 64) return launch_qk<T, 64>(p, backward, s);
    if (D == 128) return launch_qk<T, 128>(p, backward, s);
    return launch_qk<T, 256>(p, backward, s);
}

size_t bwd_workspace(const gcl_qk_args *a) {
    if (!a || a->t_max < 1 || a->t_max >= (int64_t(1) << 31) || a->HQ < 1 || a->HK < 0 ||
        (a->D != 64 && a->D != 128 && a->D != 256) || (int64_t)a->HQ + a->HK > 65535)
        return 0;
    return (size_t)bwd_blocks(a->t_max, a->HQ, a->HK, a->D) * 2 * a->D * sizeof(float);
}

gcl_status_t run(const char *fn, const gcl_qk_args *a, bool backward, cudaStream_t s) {
    fail(GCL_OK, "%s", "");                                // clears gcl_last_error()
    if (!a) return fail(GCL_ERR_INVALID_ARG, "%s: args is NULL", fn);
    if (a->t_max < 1 || a->t_max >= (int64_t(1) << 31) || a->HQ < 1 || a->HK < 0 || (int64_t)a->HQ + a->HK > 65535)
        return fail(GCL_ERR_INVALID_ARG, "%s: need 1 <= t_max < 2^31, HQ >= 1, HK >= 0, HQ + HK <= 65535", fn);
    if (a->D != 64 && a->D != 128 && a->D != 256)
        return fail(GCL_ERR_UNSUPPORTED, "%s: D=%d (supported: 64, 128, 256)", fn, a->D);
    if (a->R < 0 || a->R > a->D || a->R % 16)
        return fail(GCL_ERR_UNSUPPORTED, "%s: R=%d (a multiple of 16 from 0 to D=%d)", fn, a->R, a->D);
    if (a->dtype != GCL_F32 && a->dtype != GCL_BF16 && a->dtype != GCL_F16)
        return fail(GCL_ERR_UNSUPPORTED, "%s: dtype %d (supported: GCL_F32, GCL_BF16, GCL_F16)", fn, a->dtype);
    if (a->norm < GCL_NORM_NONE || a->norm > GCL_NORM_L2)
        return fail(GCL_ERR_UNSUPPORTED, "%s: norm %d (supported: none, RMS, L2)", fn, a->norm);
    if (a->pair != GCL_PAIR_HALF && a->pair != GCL_PAIR_ADJACENT)
        return fail(GCL_ERR_UNSUPPORTED, "%s: pair %d (supported: half, adjacent)", fn, a->pair);
    if (!(a->eps >= 0.f)) return fail(GCL_ERR_INVALID_ARG, "%s: eps must not be negative", fn);
    if (a->R > 0 && (!a->cos_table || !a->sin_table || !a->positions || a->n_positions < 1))
        return fail(GCL_ERR_INVALID_ARG, "%s: R=%d needs cos_table, sin_table, positions and n_positions >= 1", fn, a->R);
    const int es = a->dtype == GCL_F32 ? 4 : 2;
    struct { const char *name; const gcl_rows *r; int32_t H; bool in, out; } need[] = {
        {"q", &a->q, a->HQ, true, false}, {"k", &a->k, a->HK, a->HK > 0, false},
        {"yq", &a->yq, a->HQ, false, !backward}, {"yk", &a->yk, a->HK, false, !backward && a->HK > 0},
        {"dyq", &a->dyq, a->HQ, backward, false}, {"dyk", &a->dyk, a->HK, backward && a->HK > 0, false},
        {"dq", &a->dq, a->HQ, false, backward}, {"dk", &a->dk, a->HK, false, backward && a->HK > 0}};
    gcl_status_t st;
    for (const auto &x : need)
        if ((x.in || x.out) && (st = dla::check_rows(fn, x.name, *x.r, a->t_max, x.H, a->D, es, x.out)) != GCL_OK) return st;
    for (const void *x : {a->q_weight, a->k_weight, (const void *)a->cos_table, (const void *)a->sin_table,
                          (const void *)a->workspace})
        if (!dla::aligned(x, 16))
            return fail(GCL_ERR_INVALID_ARG, "%s: weights, tables and the workspace must be 16-byte aligned", fn);
    QkParams p{};
    p.side[0].x = dla::rows(a->q);
    p.side[1].x = dla::rows(a->k);
    p.side[0].w = a->q_weight;
    p.side[1].w = a->k_weight;
    p.side[0].H = a->HQ;
    p.side[1].H = a->HK;
    if (!backward) {
        p.side[0].y = dla::rows(a->yq);
        p.side[1].y = dla::rows(a->yk);
    } else {
        if ((a->dq_weight && !a->q_weight) || (a->dk_weight && (!a->k_weight || a->HK == 0)))
            return fail(GCL_ERR_INVALID_ARG, "%s: a weight's gradient needs the weight", fn);
        p.side[0].dy = dla::rows(a->dyq);
        p.side[1].dy = dla::rows(a->dyk);
        p.side[0].y = dla::rows(a->dq);
        p.side[1].y = dla::rows(a->dk);
        if (a->dq_weight || a->dk_weight) {
            const size_t bytes = bwd_workspace(a);
            if (!a->workspace || a->workspace_bytes < bytes)
                return fail(GCL_ERR_CAPACITY, "%s: workspace of %zu bytes needed, %zu given", fn, bytes,
                            a->workspace ? a->workspace_bytes : (size_t)0);
            float *ws = static_cast<float *>(a->workspace);
            p.side[0].dw = a->dq_weight;
            p.side[1].dw = a->dk_weight;
            p.side[0].partial = a->dq_weight ? ws : nullptr;
            p.side[1].partial = a->dk_weight ? ws + bytes / 2 / sizeof(float) : nullptr;
        }
    }
    p.cos_t = a->cos_table; p.sin_t = a->sin_table; p.pos = a->positions; p.status = a->dev_status;
    p.t_max = a->t_max; p.n_pos = a->n_positions; p.R = a->R; p.norm = a->norm; p.pair = a->pair; p.eps = a->eps;
    const cudaError_t e = a->dtype == GCL_BF16 ? launch_qk_t<__nv_bfloat16>(p, a->D, backward, s)
                          : a->dtype == GCL_F16 ? launch_qk_t<__half>(p, a->D, backward, s)
                                                : launch_qk_t<float>(p, a->D, backward, s);
    return cuda_check(e, fn);
}

}  // namespace
}  // namespace qk
}  // namespace gcl

using namespace gcl;

extern "C" {

gcl_status_t qk_norm_rope_fwd(const gcl_qk_args *a, gcl_stream_t stream) {
    return qk::run("qk_norm_rope_fwd", a, false, static_cast<cudaStream_t>(stream));
}
size_t gcl_qk_norm_rope_bwd_workspace_bytes(const gcl_qk_args *a) { return qk::bwd_workspace(a); }
gcl_status_t qk_norm_rope_bwd(const gcl_qk_args *a, gcl_stream_t stream) {
    return qk::run("qk_norm_rope_bwd", a, true, static_cast<cudaStream_t>(stream));
}

gcl_status_t rope_table_build(float *cos_table, float *sin_table, int64_t n_positions, int32_t R, double base,
                              gcl_stream_t stream) {
    const char *fn = "rope_table_build";
    fail(GCL_OK, "%s", "");                                // clears gcl_last_error()
    if (!cos_table || !sin_table) return fail(GCL_ERR_INVALID_ARG, "%s: cos_table and sin_table are required", fn);
    if (n_positions < 1 || R < 2 || R % 2 || !(base > 0.0) || n_positions * (int64_t)(R / 2) >= (int64_t(1) << 38))
        return fail(GCL_ERR_INVALID_ARG, "%s: need n_positions >= 1, R even and positive, base > 0", fn);
    const int64_t n = n_positions * (R / 2);
    qk::rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        cos_table, sin_table, n_positions, R / 2, base);
    return cuda_check(cudaGetLastError(), fn);
}

}  // extern "C"
