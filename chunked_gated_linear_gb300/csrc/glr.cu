// glr.cu -- gated linear recurrence over packed sequences: forward and backward.
//
// A tile is kTile tokens of the packed axis by one warp's width of channels; a warp of it walks kRun tokens.  The
// sequences need no plan of their own: a token that starts one takes its state from h0, whatever was before.
// Three launches: each tile's product of decays and own state; the states that enter the tiles, along the packed
// axis; the outputs.  Backwards likewise, from the states before each 64 tokens (saved by the forward, or formed
// again): with c_t = a_t G_t the gradient that token t passes on,
//   G_t = d_o_t + c_{t+1},   c_t = a_t G_t,
// the same recurrence with the same decays, cut where a sequence ends.
#include "glr.cuh"

namespace gcl {
namespace glr {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRunF = 16, kRunB = 8;                   // tokens of a warp
constexpr int kTileF = kWarps * kRunF, kTileB = kWarps * kRunB;

// ---- set-up: checks cu_seqlens, finds each tile's first sequence, passes states of empty sequences through ----
__global__ void __launch_bounds__(1024) glr_setup_kernel(const Params p, const float *in_state, float *out_state, int tile) {
    const int tid = threadIdx.x;
    int bad = 0;
    for (int n = tid; n < p.n_max; n += blockDim.x) {
        const int b = p.cu[n], e = p.cu[n + 1];
        bad |= b < 0 || e < b || e > p.t_max || (n == 0 && b != 0);
    }
    const bool blocked = status_blocks_cta(p.status);
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && tid == 0) {
        p.head->blocked = blocked || bad;
        p.head->live = blocked || bad ? 0 : p.cu[p.n_max];
        if (bad) status_set(p.status, GCL_DEV_BAD_RANGE);
    }
    if (blocked || bad) return;
    for (int64_t j = blockIdx.x * (int64_t)blockDim.x + tid; j <= p.tiles; j += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t0 = j * tile;
        int lo = 0, hi = p.n_max;                          // first n with cu[n] >= t0 (n_max + 1 if none)
        if (p.cu[p.n_max] < t0) lo = p.n_max + 1;
        else while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p.cu[mid] >= t0) hi = mid;
            else lo = mid + 1;
        }
        p.first[j] = lo;
    }
    if (!out_state) return;
    for (int n = blockIdx.x; n < p.n_max; n += gridDim.x) {
        if (p.cu[n + 1] != p.cu[n]) continue;
        for (int d = tid; d < p.D; d += blockDim.x) {
            const int64_t at = (int64_t)n * p.D + d;
            out_state[at] = in_state ? in_state[at] : 0.f;
        }
    }
}

// Sequences that start and end within the tile's tokens, by token; -1: none.  (Block barriers.)
template <int TILE>
__device__ __forceinline__ void borders(const Params &p, int64_t j, int64_t t0, int *s_start, int *s_end) {
    for (int k = threadIdx.x; k < TILE; k += kThreads) s_start[k] = s_end[k] = -1;
    __syncthreads();
    const int f = p.first[j];
    for (int n = (f > 0 ? f - 1 : 0) + (int)threadIdx.x; n < p.n_max; n += kThreads) {
        const int64_t b = p.cu[n] - t0, e = p.cu[n + 1] - t0;
        if (b >= TILE) break;
        if (e <= b) continue;
        if (b >= 0) s_start[b] = n;
        if (e >= 1 && e <= TILE) s_end[e - 1] = n;
    }
    __syncthreads();
}

template <typename T>
__device__ __forceinline__ const uint32_t *word(const Rows &r, int64_t t, int ch) {
    return reinterpret_cast<const uint32_t *>(static_cast<const T *>(r.p) + t * r.st + ch);
}

// The lane's values of N / V tokens from t on; zeros past `live`.
template <typename T, int RUN>
__device__ __forceinline__ void load_run(const Params &p, const Rows &r, int64_t t, int64_t live, int ch, bool on, float *v) {
    constexpr int V = Lane<T>::V;
    uint32_t w[RUN];
#pragma unroll
    for (int k = 0; k < RUN; ++k)
        w[k] = on && t + k < live && GCL_IN_BOUNDS(t + k, p.t_max, p.status) ? *word<T>(r, t + k, ch) : 0;
#pragma unroll
    for (int k = 0; k < RUN; ++k) Lane<T>::get(w[k], v + k * V);
}

// states [n, D]
template <int V>
__device__ __forceinline__ void load_state(const float *s, int64_t n, int D, int ch, bool on, float *h) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = s && on ? s[n * D + ch + v] : 0.f;
}
template <int V>
__device__ __forceinline__ void store_state(float *s, int64_t n, int D, int ch, bool on, const float *h) {
    if (!s || !on) return;
#pragma unroll
    for (int v = 0; v < V; ++v) s[n * D + ch + v] = h[v];
}

// ---- forward -------------------------------------------------------------
template <typename T, bool OUT>
__global__ void __launch_bounds__(kThreads, 2) glr_fwd_kernel(const Params p) {
    constexpr int V = Lane<T>::V, CB = Lane<T>::CB, RUN = kRunF, N = RUN * V;
    __shared__ float s_a[kWarps][CB], s_b[kWarps][CB];
    __shared__ int s_start[kTileF], s_end[kTileF], s_cut[kWarps];
    if (p.head->blocked) return;
    const int64_t live = p.head->live, j = blockIdx.x / p.n_cb, t0 = j * kTileF;
    if (t0 >= live) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ch = (blockIdx.x % p.n_cb) * CB + lane * V;
    const bool on = ch < p.D;
    const int64_t t = t0 + warp * RUN;
    float rate[V];
    load_state<V>(p.kind.rate, 0, p.D, ch, on && p.kind.decay == GCL_DECAY_POWER, rate);
    float a[N], b[N];
    {
        float r[N];
        load_run<T, RUN>(p, p.r, t, live, ch, on, r);
        decays<T, N>(p.kind, rate, r, a, b);
        mixes<T, N>(p.kind, a, b);
        load_run<T, RUN>(p, p.x, t, live, ch, on, r);
#pragma unroll
        for (int e = 0; e < N; ++e) b[e] *= r[e];
        if (p.i.p) {
            load_run<T, RUN>(p, p.i, t, live, ch, on, r);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float s, c;
                sigmoids<T>(r[e], s, c);
                b[e] *= s;
            }
        }
#pragma unroll
        for (int k = 0; k < RUN; ++k)
            if (t + k >= live)
#pragma unroll
                for (int v = 0; v < V; ++v) { a[k * V + v] = 1.f; b[k * V + v] = 0.f; }
    }
    borders<kTileF>(p, j, t0, s_start, s_end);
    const uint32_t starts = __ballot_sync(0xffffffffu, lane < RUN && s_start[(warp * RUN + lane) % kTileF] >= 0);
    const uint32_t ends = __ballot_sync(0xffffffffu, lane < RUN && s_end[(warp * RUN + lane) % kTileF] >= 0);
    // the warp's own state and product of decays (from its last start on, if it has one)
    {
        float A[V], h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) { A[v] = 1.f; h[v] = 0.f; }
#pragma unroll
        for (int k = 0; k < RUN; ++k) {
            if (starts >> k & 1) load_state<V>(p.h0, s_start[warp * RUN + k], p.D, ch, on, h);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[v] = fmaf(a[k * V + v], h[v], b[k * V + v]);
                A[v] *= a[k * V + v];
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) { s_a[warp][lane * V + v] = A[v]; s_b[warp][lane * V + v] = h[v]; }
        if (lane == 0) s_cut[warp] = starts != 0;
    }
    __syncthreads();
    if (!OUT) {
        if (warp == 0 && on) {
            float A[V], h[V];
            bool cut = false;
#pragma unroll
            for (int v = 0; v < V; ++v) { A[v] = 1.f; h[v] = 0.f; }
            for (int w = 0; w < kWarps; ++w) {
                cut |= s_cut[w] != 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    h[v] = s_cut[w] ? s_b[w][lane * V + v] : fmaf(s_a[w][lane * V + v], h[v], s_b[w][lane * V + v]);
                    A[v] *= s_a[w][lane * V + v];
                }
            }
            store_state<V>(p.agg_a, j, p.D, ch, on, A);
            store_state<V>(p.agg_b, j, p.D, ch, on, h);
            if (lane == 0) p.cut[j] = cut;                 // (every block of channels writes the same)
        }
        return;
    }
    float h[V];
    load_state<V>(p.agg_b, j, p.D, ch, on, h);
    for (int w = 0; w < warp; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = s_cut[w] ? s_b[w][lane * V + v] : fmaf(s_a[w][lane * V + v], h[v], s_b[w][lane * V + v]);
#pragma unroll
    for (int k = 0; k < RUN; ++k) {
        if (starts >> k & 1) load_state<V>(p.h0, s_start[warp * RUN + k], p.D, ch, on, h);
        if ((warp * RUN + k) % kSave == 0 && t + k < live) store_state<V>(p.h_save, (t + k) / kSave, p.D, ch, on, h);
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(a[k * V + v], h[v], b[k * V + v]);
        if (p.o.p && on && t + k < live && GCL_IN_BOUNDS(t + k, p.t_max, p.status))
            *const_cast<uint32_t *>(word<T>(p.o, t + k, ch)) = Lane<T>::put(h);
        if (ends >> k & 1) store_state<V>(p.ht, s_end[warp * RUN + k], p.D, ch, on, h);
    }
}

// The states that enter the tiles, in place of their own states; REV: from the last tile to the first.
template <bool REV>
__global__ void glr_scan_kernel(const Params p, int tile) {
    if (p.head->blocked) return;
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= p.D) return;
    const int64_t n = (p.head->live + tile - 1) / tile;
    float h = 0.f;
    for (int64_t i = 0; i < n; ++i) {
        const int64_t j = REV ? n - 1 - i : i, at = j * p.D + d;
        const float a = p.agg_a[at], b = p.agg_b[at];
        p.agg_b[at] = h;
        h = p.cut[j] ? b : fmaf(a, h, b);
    }
}

// ---- backward ------------------------------------------------------------
template <typename T, bool OUT>
__global__ void __launch_bounds__(kThreads, 2) glr_bwd_kernel(const Params p) {
    constexpr int V = Lane<T>::V, CB = Lane<T>::CB, RUN = kRunB, N = RUN * V;
    static_assert(kTileB == kSave, "one saved state a tile");
    __shared__ float s_a[kWarps][CB], s_b[kWarps][CB], s_c[kWarps][CB];
    __shared__ int s_start[kTileB], s_end[kTileB], s_cut[kWarps], s_cute[kWarps];
    if (p.head->blocked) return;
    const int64_t live = p.head->live, j = blockIdx.x / p.n_cb, t0 = j * kTileB;
    if (t0 >= live) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ch = (blockIdx.x % p.n_cb) * CB + lane * V;
    const bool on = ch < p.D;
    const int64_t t = t0 + warp * RUN;
    float rate[V];
    load_state<V>(p.kind.rate, 0, p.D, ch, on && p.kind.decay == GCL_DECAY_POWER, rate);
    float r[N], a[N], m[N], x[N], g[N], go[N];
    load_run<T, RUN>(p, p.r, t, live, ch, on, r);
    load_run<T, RUN>(p, p.d_o, t, live, ch, on, go);
    decays<T, N>(p.kind, rate, r, a, m);
    if (OUT) {
        mixes<T, N>(p.kind, a, m);
        load_run<T, RUN>(p, p.x, t, live, ch, on, x);
        if (p.i.p) load_run<T, RUN>(p, p.i, t, live, ch, on, g);
    }
#pragma unroll
    for (int k = 0; k < RUN; ++k)
        if (t + k >= live)
#pragma unroll
            for (int v = 0; v < V; ++v) { a[k * V + v] = 1.f; m[k * V + v] = 0.f; go[k * V + v] = 0.f; }
    borders<kTileB>(p, j, t0, s_start, s_end);
    const uint32_t starts = __ballot_sync(0xffffffffu, lane < RUN && s_start[(warp * RUN + lane) % kTileB] >= 0);
    const uint32_t ends = __ballot_sync(0xffffffffu, lane < RUN && s_end[(warp * RUN + lane) % kTileB] >= 0);
    float A[V], h[V], c[V], u[OUT ? N : 1];
#pragma unroll
    for (int v = 0; v < V; ++v) { A[v] = 1.f; h[v] = c[v] = 0.f; }
    if (OUT) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float s = 1.f, q;
            if (p.i.p) sigmoids<T>(g[e], s, q);
            u[e] = x[e] * s;
        }
#pragma unroll
        for (int k = 0; k < RUN; ++k) {
            if (starts >> k & 1) load_state<V>(p.h0, s_start[warp * RUN + k], p.D, ch, on, h);
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(a[k * V + v], h[v], m[k * V + v] * u[k * V + v]);
        }
    }
#pragma unroll
    for (int k = RUN - 1; k >= 0; --k) {
        if (ends >> k & 1) load_state<V>(p.dht, s_end[warp * RUN + k], p.D, ch, on, c);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            c[v] = a[k * V + v] * (go[k * V + v] + c[v]);
            A[v] *= a[k * V + v];
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s_a[warp][lane * V + v] = A[v];
        s_b[warp][lane * V + v] = h[v];
        s_c[warp][lane * V + v] = c[v];
    }
    if (lane == 0) { s_cut[warp] = starts != 0; s_cute[warp] = ends != 0; }
    __syncthreads();
    if (!OUT) {
        if (warp == 0 && on) {
            bool cut = false;
#pragma unroll
            for (int v = 0; v < V; ++v) { A[v] = 1.f; c[v] = 0.f; }
            for (int w = kWarps - 1; w >= 0; --w) {
                cut |= s_cute[w] != 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    c[v] = s_cute[w] ? s_c[w][lane * V + v] : fmaf(s_a[w][lane * V + v], c[v], s_c[w][lane * V + v]);
                    A[v] *= s_a[w][lane * V + v];
                }
            }
            store_state<V>(p.agg_a, j, p.D, ch, on, A);
            store_state<V>(p.agg_b, j, p.D, ch, on, c);
            if (lane == 0) p.cut[j] = cut;
        }
        return;
    }
    load_state<V>(p.h_save, j, p.D, ch, on, h);
    for (int w = 0; w < warp; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = s_cut[w] ? s_b[w][lane * V + v] : fmaf(s_a[w][lane * V + v], h[v], s_b[w][lane * V + v]);
    load_state<V>(p.agg_b, j, p.D, ch, on, c);
    for (int w = kWarps - 1; w > warp; --w)
#pragma unroll
        for (int v = 0; v < V; ++v)
            c[v] = s_cute[w] ? s_c[w][lane * V + v] : fmaf(s_a[w][lane * V + v], c[v], s_c[w][lane * V + v]);
    float prev[N];                                         // the state before each token
#pragma unroll
    for (int k = 0; k < RUN; ++k) {
        if (starts >> k & 1) load_state<V>(p.h0, s_start[warp * RUN + k], p.D, ch, on, h);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            prev[k * V + v] = h[v];
            h[v] = fmaf(a[k * V + v], h[v], m[k * V + v] * u[k * V + v]);
        }
    }
    float dsum[V];
#pragma unroll
    for (int v = 0; v < V; ++v) dsum[v] = 0.f;
#pragma unroll
    for (int k = RUN - 1; k >= 0; --k) {
        if (ends >> k & 1) load_state<V>(p.dht, s_end[warp * RUN + k], p.D, ch, on, c);
        float dx[V], dr[V], di[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = k * V + v;
            const float G = go[e] + c[v];
            c[v] = a[e] * G;
            float dl = c[v] * prev[e];
            if (p.kind.mix == GCL_MIX_COMPLEMENT) dl = fmaf(-a[e] * G, u[e], dl);
            else if (p.kind.mix == GCL_MIX_ROOT && m[e] > 0.f) dl = fmaf(-a[e] * a[e] * frcp<T>(m[e]) * G, u[e], dl);
            float s = 1.f, q = 0.f;
            if (p.i.p) sigmoids<T>(g[e], s, q);
            dx[v] = G * m[e] * s;
            di[v] = dx[v] * x[e] * q;
            if (p.kind.decay != GCL_DECAY_LOG) {
                sigmoids<T>(r[e], s, q);
                if (p.kind.decay == GCL_DECAY_SIGMOID) dl *= q;
                else {
                    if (t + k < live) dsum[v] = fmaf(-dl, s, dsum[v]);
                    dl *= -rate[v] * s * q;
                }
            }
            dr[v] = dl;
        }
        if (on && t + k < live && GCL_IN_BOUNDS(t + k, p.t_max, p.status)) {
            *const_cast<uint32_t *>(word<T>(p.dx, t + k, ch)) = Lane<T>::put(dx);
            *const_cast<uint32_t *>(word<T>(p.dr, t + k, ch)) = Lane<T>::put(dr);
            if (p.i.p) *const_cast<uint32_t *>(word<T>(p.di, t + k, ch)) = Lane<T>::put(di);
        }
        if (starts >> k & 1) store_state<V>(p.dh0, s_start[warp * RUN + k], p.D, ch, on, c);
    }
    if (p.drate_part) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) s_a[warp][lane * V + v] = dsum[v];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float sum = 0.f;
                for (int w = 0; w < kWarps; ++w) sum += s_a[w][lane * V + v];
                dsum[v] = sum;
            }
            store_state<V>(p.drate_part, j, p.D, ch, on, dsum);
        }
    }
}

// drate from the tiles' sums, in a fixed order: 32 channels a block, 32 rows of threads over the tiles.
__global__ void __launch_bounds__(1024) glr_drate_kernel(const Params p, int tile) {
    __shared__ float s[32][33];
    if (p.head->blocked) return;
    const int64_t n = (p.head->live + tile - 1) / tile;
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (d < p.D)
        for (int64_t j = r; j < n; j += 32) sum += p.drate_part[j * p.D + d];
    s[r][lane] = sum;
    __syncthreads();
    float t = s[lane][r];
#pragma unroll
    for (int k = 16; k; k >>= 1) t += __shfl_xor_sync(0xffffffffu, t, k);
    if (lane == 0 && blockIdx.x * 32 + r < p.D) p.drate[blockIdx.x * 32 + r] = t;
}

// ---- host ----------------------------------------------------------------
size_t up16(size_t n) { return (n + 15) / 16 * 16; }

bool sizes_ok(const gcl_glr_args *a) {
    return a && a->t_max >= 1 && a->t_max < (int64_t(1) << 31) && a->n_max >= 1 && a->D >= 8 && a->D % 8 == 0 &&
           a->D <= (1 << 20) && (a->dtype == GCL_F32 || a->dtype == GCL_BF16 || a->dtype == GCL_F16);
}

// The workspace's parts, in order; `base` may be NULL (for the size alone).
size_t layout(const gcl_glr_args *a, bool backward, Params *p) {
    uint8_t *base = static_cast<uint8_t *>(a->workspace);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        uint8_t *q = base ? base + at : nullptr;
        at += up16(bytes);
        return q;
    };
    auto set = [&](auto *&field, size_t bytes) { field = reinterpret_cast<std::remove_reference_t<decltype(field)>>(take(bytes)); };
    Params dummy{};
    Params &o = p ? *p : dummy;
    const int64_t tf = (a->t_max + kTileF - 1) / kTileF, tb = (a->t_max + kTileB - 1) / kTileB;
    const int64_t tiles = backward ? tb : tf;
    const size_t row = sizeof(float) * (size_t)a->D;
    set(o.head, sizeof(Header));
    set(o.first, sizeof(int32_t) * (size_t)(tiles + 1));
    set(o.cut, sizeof(int32_t) * (size_t)tiles);
    set(o.agg_a, row * tiles);
    set(o.agg_b, row * tiles);
    if (backward) {
        if (a->drate) set(o.drate_part, row * tiles);
        if (!a->h_save) set(o.h_save, row * tb);
    }
    return at;
}

template <typename T>
cudaError_t launch_fwd(Params p, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.tiles * p.n_cb);
    const int64_t setup = (p.tiles + 1024) / 1024 > p.n_max ? (p.tiles + 1024) / 1024 : p.n_max;
    glr_setup_kernel<<<(unsigned)(setup < 2 * num_sms() ? setup : 2 * num_sms()), 1024, 0, s>>>(p, p.h0, p.ht, kTileF);
    glr_fwd_kernel<T, false><<<grid, kThreads, 0, s>>>(p);
    glr_scan_kernel<false><<<(p.D + 63) / 64, 64, 0, s>>>(p, kTileF);
    glr_fwd_kernel<T, true><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(Params p, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.tiles * p.n_cb);
    const int64_t setup = (p.tiles + 1024) / 1024 > p.n_max ? (p.tiles + 1024) / 1024 : p.n_max;
    glr_setup_kernel<<<(unsigned)(setup < 2 * num_sms() ? setup : 2 * num_sms()), 1024, 0, s>>>(p, p.dht, p.dh0, kTileB);
    glr_bwd_kernel<T, false><<<grid, kThreads, 0, s>>>(p);
    glr_scan_kernel<true><<<(p.D + 63) / 64, 64, 0, s>>>(p, kTileB);
    glr_bwd_kernel<T, true><<<grid, kThreads, 0, s>>>(p);
    if (p.drate) glr_drate_kernel<<<(p.D + 31) / 32, 1024, 0, s>>>(p, kTileB);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const gcl_glr_args *a, Params p, bool backward, cudaStream_t s) {
    p.n_cb = (p.D + Lane<T>::CB - 1) / Lane<T>::CB;
    if (!backward) return launch_fwd<T>(p, s);
    if (!a->h_save) {                                      // the states before each 64 tokens, by the forward without o and ht
        Params f = p;
        layout(a, true, &f);
        f.tiles = (p.t_max + kTileF - 1) / kTileF;
        f.ht = nullptr;
        f.o.p = nullptr;
        const cudaError_t e = launch_fwd<T>(f, s);
        if (e != cudaSuccess) return e;
    }
    return launch_bwd<T>(p, s);
}

}  // namespace

gcl_status_t check_kind(const char *fn, const float *rate, int32_t D, int32_t decay, int32_t mix, int32_t dtype) {
    if (D < 8 || D % 8 || D > (1 << 20)) return fail(GCL_ERR_UNSUPPORTED, "%s: D=%d (a multiple of 8, at most 2^20)", fn, D);
    if (dtype != GCL_F32 && dtype != GCL_BF16 && dtype != GCL_F16)
        return fail(GCL_ERR_UNSUPPORTED, "%s: dtype %d (supported: GCL_F32, GCL_BF16, GCL_F16)", fn, dtype);
    if (decay < GCL_DECAY_LOG || decay > GCL_DECAY_POWER)
        return fail(GCL_ERR_UNSUPPORTED, "%s: decay %d (supported: log, sigmoid, power)", fn, decay);
    if (mix < GCL_MIX_ONE || mix > GCL_MIX_ROOT)
        return fail(GCL_ERR_UNSUPPORTED, "%s: mix %d (supported: one, complement, root)", fn, mix);
    if (decay == GCL_DECAY_POWER && !rate) return fail(GCL_ERR_INVALID_ARG, "%s: the power decay needs rate", fn);
    return GCL_OK;
}

namespace {

gcl_status_t run(const char *fn, const gcl_glr_args *a, bool backward, cudaStream_t s) {
    fail(GCL_OK, "%s", "");                                // clears gcl_last_error()
    if (!a) return fail(GCL_ERR_INVALID_ARG, "%s: args is NULL", fn);
    if (!a->cu_seqlens) return fail(GCL_ERR_INVALID_ARG, "%s: cu_seqlens is required", fn);
    if (a->t_max < 1 || a->t_max >= (int64_t(1) << 31) || a->n_max < 1)
        return fail(GCL_ERR_INVALID_ARG, "%s: need 1 <= t_max < 2^31 and n_max >= 1", fn);
    gcl_status_t st = check_kind(fn, a->rate, a->D, a->decay, a->mix, a->dtype);
    if (st != GCL_OK) return st;
    const int es = a->dtype == GCL_F32 ? 4 : 2;
    if ((a->t_max + kTileB - 1) / kTileB * (int64_t)((a->D * es + 127) / 128) >= (int64_t(1) << 31))
        return fail(GCL_ERR_UNSUPPORTED, "%s: t_max / 64 * D is too large", fn);
    const bool gate = a->i.ptr != nullptr;
    struct { const char *name; const gcl_rows *r; bool in, out; } need[] = {
        {"x", &a->x, true, false}, {"r", &a->r, true, false}, {"i", &a->i, gate, false},
        {"o", &a->o, false, !backward && a->o.ptr}, {"d_o", &a->d_o, backward, false}, {"dx", &a->dx, false, backward},
        {"dr", &a->dr, false, backward}, {"di", &a->di, false, backward && gate}};
    for (const auto &x : need) {
        if (!x.in && !x.out) continue;
        gcl_rows r = *x.r;
        r.head_stride = a->D;
        if ((st = dla::check_rows(fn, x.name, r, a->t_max, 1, a->D, es, x.out)) != GCL_OK) return st;
    }
    if (backward && a->drate && a->decay != GCL_DECAY_POWER)
        return fail(GCL_ERR_INVALID_ARG, "%s: drate is for the power decay", fn);
    for (const void *x : {(const void *)a->rate, (const void *)a->h0, (const void *)a->ht, (const void *)a->dht, (const void *)a->dh0,
                          (const void *)a->drate, (const void *)a->h_save, (const void *)a->workspace})
        if (!dla::aligned(x, 16))
            return fail(GCL_ERR_INVALID_ARG, "%s: rate, states, their gradients and the workspace must be 16-byte aligned", fn);
    const float *out_state = backward ? a->dh0 : a->ht;
    const uintptr_t state_bytes = sizeof(float) * (uintptr_t)a->n_max * a->D;
    struct { const char *name; const float *p; } in_state[] = {{"h0", a->h0}, {"dht", backward ? a->dht : nullptr}};
    for (const auto &x : in_state) {
        const uintptr_t i = reinterpret_cast<uintptr_t>(x.p), o = reinterpret_cast<uintptr_t>(out_state);
        if (i && o && (i < o ? o - i : i - o) < state_bytes)
            return fail(GCL_ERR_INVALID_ARG, "%s: %s must not be %s (their states overlap)", fn, backward ? "dh0" : "ht", x.name);
    }
    Params p{};
    const size_t bytes = layout(a, backward, &p);
    if (!a->workspace || a->workspace_bytes < bytes)
        return fail(GCL_ERR_CAPACITY, "%s: workspace of %zu bytes needed, %zu given", fn, bytes, a->workspace ? a->workspace_bytes : (size_t)0);
    p.x = dla::rows(a->x); p.r = dla::rows(a->r); p.i = dla::rows(a->i);
    if (backward) {
        p.d_o = dla::rows(a->d_o); p.dx = dla::rows(a->dx); p.dr = dla::rows(a->dr); p.di = dla::rows(a->di);
        p.dht = a->dht; p.dh0 = a->dh0; p.drate = a->drate;
    } else {
        p.o = dla::rows(a->o);
        p.ht = a->ht;
    }
    if (a->h_save) p.h_save = a->h_save;
    p.kind = Kind{a->rate, a->decay, a->mix};
    p.h0 = a->h0; p.cu = a->cu_seqlens; p.status = a->dev_status;
    p.t_max = a->t_max; p.n_max = a->n_max; p.D = a->D;
    p.tiles = (a->t_max + (backward ? kTileB : kTileF) - 1) / (backward ? kTileB : kTileF);
    const cudaError_t e = a->dtype == GCL_BF16 ? launch<__nv_bfloat16>(a, p, backward, s)
                          : a->dtype == GCL_F16 ? launch<__half>(a, p, backward, s)
                                                : launch<float>(a, p, backward, s);
    return cuda_check(e, fn);
}

}  // namespace
}  // namespace glr
}  // namespace gcl

using namespace gcl;

extern "C" {

size_t gcl_glr_fwd_workspace_bytes(const gcl_glr_args *a) { return glr::sizes_ok(a) ? glr::layout(a, false, nullptr) : 0; }
size_t gcl_glr_bwd_workspace_bytes(const gcl_glr_args *a) { return glr::sizes_ok(a) ? glr::layout(a, true, nullptr) : 0; }
gcl_status_t glr_fwd(const gcl_glr_args *a, gcl_stream_t stream) { return glr::run("glr_fwd", a, false, static_cast<cudaStream_t>(stream)); }
gcl_status_t glr_bwd(const gcl_glr_args *a, gcl_stream_t stream) { return glr::run("glr_bwd", a, true, static_cast<cudaStream_t>(stream)); }

}  // extern "C"
