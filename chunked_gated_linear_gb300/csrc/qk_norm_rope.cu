// qk_norm_rope.cu -- norm of the queries and keys of each head and the position rotation in one pass,
// forward and backward, and the table of angles.
//
// For a row x of D values: n = r x with r = 1 / sqrt(sum(x^2) / D + eps) (RMS), without the / D (L2)
// or 1; z = n w; y = rotation of z.  The rotation's transpose turns by the opposite angle, so with
// dz = rotation^T dy and u = dz w:
//   dx = r (u - x r^2 sum(u x) / D)   (RMS; L2 without / D),   dw = sum over rows of dz n.
// (Neither sum(x^2) nor sum(u x) waits for the other: they cross the row's lanes together.)
// HBM-bound: rows are read and written once (the backward reads x and dy, writes dx).  D / 8 lanes
// hold one row, 16 bytes (fp32: 32) each; sums over a row are shuffles inside those lanes, and the
// partner of a half-split pair sits R / 16 lanes away (shuffled as loaded, two values to a word).  A lane
// group keeps a token for its heads: the cos and sin rows are loaded once and joined with the weights
// (forward: y = r (x c w + x' s w'), four fp32 pairs of products a lane), and the rows of four heads are in
// flight together.  32,768 tokens of 16 + 16 heads of 128, bf16: 97 us, 5.5 TB/s; backward, 16,384
// tokens of 16 + 2 heads: 60 us, 3.8 TB/s (bound by issue and the shuffles' latency: two blocks of 126 registers
// an SM; three spill, 79 us, and rows brought ahead through shared memory take as long, 60).  The shuffles are this
// layout's, twelve for a lane's eight values: lanes that held both halves of a pair would need none for the partners and
// half of those for the sums (not tried).  fp32 rows, twice the registers, spill 156 bytes a thread with four in flight
// (204 backwards at D = 256); they were not timed at a size that fills the GPU.
#include "dla.cuh"
#include "dla_simt.cuh"
#include "f32x2.cuh"

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
    int32_t heads[2], groups[2];   // heads per item (a multiple of PER) and items per token, of q and of k
    int32_t blocks_q;              // blocks of q; the others take k
};

// Sum over the D / 8 lanes of a row.
template <int L>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int d = L / 2; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// Two sums over the row's lanes at once.
template <int L>
__device__ __forceinline__ void row_sums(float &a, float &b) {
#pragma unroll
    for (int d = L / 2; d; d >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, a, d), v = __shfl_xor_sync(0xffffffffu, b, d);
        a += u;
        b += v;
    }
}

// The lane's factors of the rotation of one token, y_e = z_e c_e + z_partner(e) s_e: with the signs of the two
// halves of a pair in s (turned back: `sign` -1), and c = 1, s = 0 past the rotated channels.
__device__ __forceinline__ void angles(const QkParams &p, int64_t pos, int l, float sign, float *c, float *s) {
    if (l >= p.R / 8) return;
    const int64_t row = pos * (p.R / 2);
    if (p.pair == GCL_PAIR_ADJACENT) {
        const float4 a = *reinterpret_cast<const float4 *>(p.cos_t + row + l * 4);
        const float4 b = *reinterpret_cast<const float4 *>(p.sin_t + row + l * 4);
        c[0] = c[1] = a.x; c[2] = c[3] = a.y; c[4] = c[5] = a.z; c[6] = c[7] = a.w;
        s[1] = sign * b.x; s[3] = sign * b.y; s[5] = sign * b.z; s[7] = sign * b.w;
#pragma unroll
        for (int e = 0; e < 8; e += 2) s[e] = -s[e + 1];
    } else {
        const int half = p.R / 16, at = (l % half) * 8;
        dla::load8f(p.cos_t + row + at, c);
        dla::load8f(p.sin_t + row + at, s);
        const float sg = l < half ? -sign : sign;
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] *= sg;
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
    __device__ __forceinline__ void get(uint64_t *x) const {
        float f[8];
        dla::load8f(reinterpret_cast<const T *>(v), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = pair(f[2 * e], f[2 * e + 1]);
    }
    // The values' partners: another lane's eight (lane src; zeros where `in` is false), or the neighbours
    // within the lane's pairs.
    __device__ __forceinline__ void partners(uint64_t *x, bool adjacent, int src, bool in) const {
        Raw o;
        if (adjacent) {
            get(x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = unpair(x[e]);
                x[e] = in ? pair(f.y, f.x) : 0;
            }
            return;
        }
        const uint32_t *a = reinterpret_cast<const uint32_t *>(v);
        uint32_t *b = reinterpret_cast<uint32_t *>(o.v);
#pragma unroll
        for (int e = 0; e < 2 * (int)sizeof(T); ++e) {
            const uint32_t y = __shfl_sync(0xffffffffu, a[e], src);
            b[e] = in ? y : 0;
        }
        o.get(x);
    }
    __device__ __forceinline__ void put(const uint64_t *x) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 t = unpair(x[e]);
            f[2 * e] = t.x;
            f[2 * e + 1] = t.y;
        }
        dla::store4f(reinterpret_cast<T *>(v), f);
        dla::store4f(reinterpret_cast<T *>(v) + 4, f + 4);
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int e = 0; e < (int)sizeof(T) / 2; ++e) reinterpret_cast<uint4 *>(p)[e] = v[e];
    }
};

constexpr int qk_ctas(bool bwd) { return bwd ? 2 : 3; }    // resident blocks per SM

// The call does nothing.  (A position of its own past the tables leaves that token's rows alone, not the others.)
__device__ __forceinline__ bool blocked(const QkParams &p) {
    return dla::call_blocked(p.status, p.R > 0 ? p.t_max : 0, [&](int64_t t) { return p.pos[t] >= p.n_pos; });
}

// An item is some of the heads of one token, of q or of k by the block; a lane group (D / 8 lanes) takes its
// heads PER at a time, with their rows in flight together, and keeps the token's rotation factors.  Lane
// groups walk the items with the stride of the side's blocks.  Lanes without work stay for the
// shuffles.  BWD: y gets dx, and the weight's gradient is summed per block.
template <typename T, int D, bool BWD, int PER>
__global__ void __launch_bounds__(kThreads, qk_ctas(BWD)) qk_kernel(const QkParams p) {
    constexpr int L = D / 8, G = kThreads / L;             // lanes per row, lane groups per block
    __shared__ __align__(8) float s_dw[BWD ? G : 1][BWD ? D : 1];
    if (BWD) launch_dependents();                          // (the sums of the weights' gradients wait for this grid's end)
    if (blocked(p)) return;
    const int tid = threadIdx.x, l = tid % L, grp = tid / L;
    const int which = blockIdx.x < p.blocks_q ? 0 : 1;
    const int block = which ? blockIdx.x - p.blocks_q : blockIdx.x, blocks = which ? gridDim.x - p.blocks_q : p.blocks_q;
    const Side &sd = p.side[which];
    const uint32_t per_token = p.groups[which];
    const int64_t work = p.t_max * per_token;
    uint64_t dw[4] = {};
    const bool adjacent = p.pair == GCL_PAIR_ADJACENT, rot = p.R > 0;
    const bool in = l < p.R / 8;                           // the lane's channels are rotated
    const int lane = tid & 31, half = p.R / 16;
    const int src = !in ? lane : l < half ? lane + half : lane - half;
    uint64_t w2[4];
    if (sd.w) {
        Raw<T> w;
        w.load(static_cast<const T *>(sd.w) + l * 8);
        w.get(w2);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w2[e] = pair(1.f, 1.f);
    }
    const int heads = p.heads[which];
    // item i: heads h0 .. of token t
    auto item = [&](int64_t i, int64_t &t, int &h0) {
        t = i >> 32 ? i / per_token : (uint32_t)i / per_token;
        h0 = (int)(i - t * per_token) * heads;
    };
    const int64_t step = (int64_t)blocks * G;
    int64_t i = (int64_t)block * G + grp, t_next = 0, pos_next = 0;
    int h_next = 0;
    if (i < work) {
        item(i, t_next, h_next);
        if (p.pos) pos_next = p.pos[t_next];
    }
    for (int64_t i0 = (int64_t)block * G; i0 < work; i0 += step, i += step) {
        const bool exists = i < work;
        bool live = exists;
        const int64_t pos = pos_next, t = t_next;
        const int h0 = h_next, h1 = h0 + heads < sd.H ? h0 + heads : sd.H;
        // the first rows (of padding too: its values are not used), before anything that waits for the position
        Raw<T> xr[PER], dr[BWD ? PER : 1];
        const T *px = row_ptr<const T>(sd.x, t, h0) + l * 8, *pd = BWD ? row_ptr<const T>(sd.dy, t, h0) + l * 8 : nullptr;
        T *py = row_ptr<T>(sd.y, t, h0) + l * 8;
        int left = exists ? h1 - h0 : 0;                   // heads of the item not yet loaded
        auto load = [&]() {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (j < left) xr[j].load(px);
                else xr[j].zero();
                px += sd.x.sh;
                if (BWD) {
                    if (j < left) dr[j].load(pd);
                    else dr[j].zero();
                    pd += sd.dy.sh;
                }
            }
        };
        load();
        if (live && p.pos) {
            live = pos >= 0;
            if (rot && pos >= p.n_pos) {
                live = false;
                status_set(p.status, GCL_DEV_BAD_RANGE);
            }
        }
        float c[8], s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) { c[e] = 1.f; s[e] = 0.f; }
        if (live && rot) angles(p, pos, l, BWD ? -1.f : 1.f, c, s);
        if (i + step < work) {                             // the next item's position is under way meanwhile
            item(i + step, t_next, h_next);
            if (p.pos) pos_next = p.pos[t_next];
        }
        uint64_t c2[4], s2[4];
        // forward: y = r (x c w + x' s w') with ' the partner; the weights join the factors once per token.
        // Backward: dz = dy c + dy' s.
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            c2[e] = pair(c[2 * e], c[2 * e + 1]);
            s2[e] = pair(s[2 * e], s[2 * e + 1]);
            if (!BWD) c2[e] = mul2(c2[e], w2[e]);
        }
        if (!BWD && rot) {
            uint64_t wp[4];
            if (adjacent) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpair(w2[e]);
                    wp[e] = pair(f.y, f.x);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpair(w2[e]);
                    wp[e] = pair(__shfl_sync(0xffffffffu, f.x, src), __shfl_sync(0xffffffffu, f.y, src));
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s2[e] = in ? mul2(s2[e], wp[e]) : 0;
        }
        for (int hb = 0; hb < heads; hb += PER, left -= PER) {     // (the same count for every lane of the warp)
            if (hb > 0) load();
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const bool on = live && j < left;
                uint64_t x[4], y[4];
                xr[j].get(x);
                Raw<T> out;
                if (!BWD) {
                    float r = 1.f;
                    if (p.norm != GCL_NORM_NONE) {
                        uint64_t q = mul2(x[0], x[0]);
#pragma unroll
                        for (int e = 1; e < 4; ++e) q = fma2(x[e], x[e], q);
                        const float2 f = unpair(q);
                        const float ss = row_sum<L>(f.x + f.y);
                        r = rsqrtf((p.norm == GCL_NORM_RMS ? ss * (1.f / D) : ss) + p.eps);
                    }
                    const uint64_t r2 = pair(r, r);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = mul2(x[e], c2[e]);
                    if (rot) {
                        uint64_t xp[4];
                        xr[j].partners(xp, adjacent, src, in);
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = fma2(xp[e], s2[e], y[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], r2);
                } else {
                    uint64_t z[4];
                    dr[j].get(z);
                    if (rot) {
                        uint64_t zp[4];
                        dr[j].partners(zp, adjacent, src, in);
#pragma unroll
                        for (int e = 0; e < 4; ++e) z[e] = fma2(zp[e], s2[e], mul2(z[e], c2[e]));
                    }
                    // u = z w; the sums of x^2 and of u x together
                    uint64_t q = mul2(x[0], x[0]), m2;
#pragma unroll
                    for (int e = 1; e < 4; ++e) q = fma2(x[e], x[e], q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = mul2(z[e], w2[e]);
                    m2 = mul2(y[0], x[0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e) m2 = fma2(y[e], x[e], m2);
                    const float2 fq = unpair(q), fm = unpair(m2);
                    float ss = fq.x + fq.y, su = fm.x + fm.y;
                    float r = 1.f, m = 0.f;
                    if (p.norm != GCL_NORM_NONE) {
                        row_sums<L>(ss, su);
                        r = rsqrtf((p.norm == GCL_NORM_RMS ? ss * (1.f / D) : ss) + p.eps);
                        m = su * r * r * (p.norm == GCL_NORM_RMS ? -1.f / D : -1.f);
                    }
                    const uint64_t r2 = pair(r, r), mm = pair(m, m);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (on) dw[e] = fma2(mul2(z[e], x[e]), r2, dw[e]);
                        y[e] = mul2(fma2(x[e], mm, y[e]), r2);
                    }
                }
                out.put(y);
                if (on) out.store(py);
                py += sd.y.sh;
            }
        }
    }
    if (BWD && sd.partial) {
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<float2 *>(&s_dw[grp][l * 8 + 2 * e]) = unpair(dw[e]);
        __syncthreads();
        for (int ch = tid; ch < D; ch += kThreads) {
            float sum = 0.f;
            for (int g = 0; g < G; ++g) sum += s_dw[g][ch];
            sd.partial[(int64_t)block * D + ch] = sum;
        }
    }
}

// The weights' gradients from the blocks' sums, in a fixed order: one block per 32 channels, 32 rows of
// threads over the sums, eight loads of each in flight.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const QkParams p, int blocks_k, int D) {
    __shared__ float s[32][33];
    grid_dependency_wait();
    if (blocked(p)) return;
    const Side &sd = p.side[blockIdx.y];
    if (!sd.partial) return;
    const int lane = threadIdx.x & 31, ch = blockIdx.x * 32 + lane, r = threadIdx.x >> 5;
    const int blocks = blockIdx.y ? blocks_k : p.blocks_q;
    float sum = 0.f;
    for (int b0 = r; b0 < blocks; b0 += 8 * 32) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = b0 + i * 32 < blocks ? sd.partial[(int64_t)(b0 + i * 32) * D + ch] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[i];
    }
    s[r][lane] = sum;
    __syncthreads();
    // thread (r, lane): the sum over the rows of channel r of the block's 32
    float t = s[lane][r];
#pragma unroll
    for (int d = 16; d; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    if (lane == 0) sd.dw[blockIdx.x * 32 + r] = t;
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

// Most blocks of the backward: those that are resident, each walking many tokens, so that the partial sums of
// the weights' gradients stay few.
int bwd_blocks() { return qk_ctas(true) * num_sms(); }

template <typename T, int D, bool BWD, int PER>
cudaError_t launch_qk_per(QkParams &p, cudaStream_t s) {
    const int64_t G = kThreads / (D / 8);
    int64_t need[2];                                       // blocks that give every lane group one item
    for (int i = 0; i < 2; ++i) {
        // a whole token per item while that gives every lane group of the GPU two; else fewer heads
        int32_t heads = (p.side[i].H + PER - 1) / PER * PER;
        const int64_t fill = 2 * (int64_t)num_sms() * qk_ctas(BWD) * G;
        while (heads > PER && p.t_max * ((p.side[i].H + heads - 1) / heads) < fill) heads = (heads / PER + 1) / 2 * PER;
        p.heads[i] = heads > 0 ? heads : PER;
        p.groups[i] = (p.side[i].H + p.heads[i] - 1) / p.heads[i];
        need[i] = (p.t_max * p.groups[i] + G - 1) / G;
    }
    // at most one wave (32,768 tokens of 16 + 16 heads forwards: 97 us, two waves 99; backwards a
    // tenth less), shared by the sides' rows, and by their items for the angles (16 + 2 heads forwards: 64 us; by
    // rows alone 72)
    const int64_t most = qk_ctas(BWD) * (int64_t)num_sms();
    if (need[0] + need[1] > most) {
        double w[2];
        for (int i = 0; i < 2; ++i) w[i] = p.side[i].H > 0 ? (double)p.groups[i] * (p.heads[i] + 1) : 0.;
        for (int i = 0; i < 2; ++i)
            if (need[i] > 0) {
                const int64_t part = (int64_t)(w[i] / (w[0] + w[1]) * most + 0.5);
                need[i] = part < 1 ? 1 : part < need[i] ? part : need[i];
            }
    }
    p.blocks_q = (int32_t)need[0];
    qk_kernel<T, D, BWD, PER><<<(unsigned)(need[0] + need[1]), kThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (BWD && e == cudaSuccess && (p.side[0].partial || p.side[1].partial)) {
        e = launch_dependent(qk_dw_kernel, dim3(D / 32, 2), dim3(1024), 0, s, p, (int)need[1], D);
    }
    return e;
}

template <typename T, int D>
cudaError_t launch_qk(QkParams &p, bool backward, cudaStream_t s) {
    // four heads per lane group and step once there are rows for two full waves (32,768 tokens of 16 + 16
    // heads of 128, bf16: 97 us with four, 131 with two, 168 with one; the other types follow bf16); few rows are
    // spread one by one, for latency
    const int64_t G = kThreads / (D / 8), rows = p.t_max * ((int64_t)p.side[0].H + p.side[1].H);
    const bool many = rows >= 4 * 16 * (int64_t)num_sms() * G;
    if (backward) return many ? launch_qk_per<T, D, true, 4>(p, s) : launch_qk_per<T, D, true, 1>(p, s);
    return many ? launch_qk_per<T, D, false, 4>(p, s) : launch_qk_per<T, D, false, 1>(p, s);
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
    return (size_t)(bwd_blocks() + 2) * 2 * a->D * sizeof(float);
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
