// glr.cu -- gated linear recurrence over packed sequences: forward and backward.
//
// A tile is kTile tokens of the packed axis by the 128 bytes of a warp's width of channels; each of its warps walks kRun
// tokens.  The sequences need no plan of their own: a token that starts one takes its state from h0, whatever
// was before.  One pass: blocks take tiles in the order of the recurrence (a counter), form a tile's product of decays and its
// state from zero, publish both, and take the state that enters from the tile before, or from an earlier one and the products and
// own states between; the sum is folded from the oldest on, so the result is the same whichever tile had its state
// ready.  A block waits for tiles with lower tickets alone, whose blocks run already, so the first of them
// never waits: the launch ends whatever else runs on the GPU.  (Three launches -- own states, their scan, outputs -- read
// x, r and i twice: 65,536 tokens of 2,048 channels 1,424 us.)
// Backwards from the states before each 64 tokens (saved by the forward, or formed again): with c_t = a_t G_t the gradient that
// token t passes on,
//   G_t = d_o_t + c_{t+1},   c_t = a_t G_t,
// the same recurrence with the same decays, cut where a sequence ends, over the tiles from last to first.
#include <type_traits>

#include "glr.cuh"
#include "tc_ptx.cuh"

namespace gcl {
namespace glr {
namespace {

// Forward: 128 tokens, 16 warps of 8.  Backward: 64 tokens, 8 warps of 8.
constexpr int kRun = 8;
constexpr int kWarpsF = 16, kWarpsB = 8, kTileF = kWarpsF * kRun, kTileB = kWarpsB * kRun;
constexpr int kCtasF = 2, kCtasB = 3;                  // resident blocks an SM

// ---- set-up: checks cu_seqlens, finds each tile's first sequence, passes states of empty sequences through, clears the
// flags between tiles ----
__global__ void __launch_bounds__(1024) glr_setup_kernel(const Params p, const float *in_state, float *out_state, int tile) {
    launch_dependents();
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
        p.head->ticket = 0;
        if (bad) status_set(p.status, GCL_DEV_BAD_RANGE);
    }
    if (blocked || bad) return;
    const int64_t at = blockIdx.x * (int64_t)blockDim.x + tid, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t e = at; e < p.tiles * p.n_cb; e += step) p.chain.flag[e] = 0;
    for (int64_t j = at; j < p.tiles; j += step) {
        const int64_t t0 = j * tile;
        int lo = 0, hi = p.n_max;                          // first n with cu[n] >= t0 (n_max if none)
        while (lo < hi) {
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
            const int64_t e = (int64_t)n * p.D + d;
            out_state[e] = in_state ? in_state[e] : 0.f;
        }
    }
}

// Sequences that start and end within the tile's tokens, by token; -1: none.  One warp.
template <int TILE>
__device__ __forceinline__ void borders(const Params &p, int64_t j, int *s_start, int *s_end) {
    const int lane = threadIdx.x & 31;
    const int64_t t0 = j * TILE;
    const int f = p.first[j];
#pragma unroll
    for (int k = lane; k < TILE; k += 32) s_start[k] = s_end[k] = -1;
    __syncwarp();
    for (int n = (f > 0 ? f - 1 : 0) + lane; n < p.n_max; n += 32) {
        const int64_t b = p.cu[n] - t0, e = p.cu[n + 1] - t0;
        if (b >= TILE) break;
        if (e <= b) continue;
        if (b >= 0) s_start[b] = n;
        if (e >= 1 && e <= TILE) s_end[e - 1] = n;
    }
}

template <typename T>
__device__ __forceinline__ uint32_t *word(const Rows &r, int64_t t, int ch) {
    return reinterpret_cast<uint32_t *>(static_cast<T *>(r.p) + t * r.st + ch);
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

// The tile's rows (n_live tokens from t0 on, channels of block cb) into shared memory, asynchronously; zeros elsewhere.
template <typename T, int TILE, int THREADS>
__device__ __forceinline__ void stage_rows(const Params &p, const Rows &r, int64_t t0, int n_live, int cb, uint8_t *dst) {
    constexpr int E = 16 / sizeof(T), ROWS = THREADS / 8;
    const int row = threadIdx.x >> 3, ch = cb * Lane<T>::CB + (threadIdx.x & 7) * E;
    const int n = ch < p.D ? n_live : 0;
    const T *src = static_cast<const T *>(r.p) + (t0 + row) * r.st + ch;
    const uint32_t to = tc::smem_u32(dst) + threadIdx.x * 16;
#pragma unroll
    for (int i = 0; i < TILE / ROWS; ++i) {
        const bool on = row + i * ROWS < n && GCL_IN_BOUNDS(t0 + row + i * ROWS, p.t_max, p.status);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * THREADS * 16),
                     "l"(on ? src + i * ROWS * r.st : static_cast<const T *>(r.p)), "r"(on ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void stage_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ int32_t load_flag(const int32_t *f) {
    int32_t v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(f) : "memory");
    return v;
}
__device__ __forceinline__ void store_flag(int32_t *f, int32_t v) {
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(f), "r"(v) : "memory");
}

// One warp: the warp's states of row `at` of a chain array, past the L1.
template <int V>
__device__ __forceinline__ void chain_load(const float *s, int64_t at, bool on, float *h) {
    if (V == 2) {
        const float2 f = on ? __ldcg(reinterpret_cast<const float2 *>(s + at)) : make_float2(0.f, 0.f);
        h[0] = f.x;
        h[V - 1] = f.y;
    } else {
        h[0] = on ? __ldcg(s + at) : 0.f;
    }
}

// One warp: the state that enters tile `seq` (its number in the order of the recurrence, > 0), from the nearest tile
// before it whose state is out and the own states between, folded from the oldest on.
template <int V>
__device__ __forceinline__ void chain_enter(const Params &p, int64_t seq, int cb, int ch, bool on, float *h) {
    const int lane = threadIdx.x & 31;
    const int32_t *flag = p.chain.flag + (int64_t)cb * p.tiles;
    const int64_t mine = seq - 1 - lane;
    const uint64_t t0 = tc::globaltimer();
    int near;
    while (true) {
        const int32_t f = mine >= 0 ? load_flag(flag + mine) : 0;
        const uint32_t done = __ballot_sync(0xffffffffu, f == kDone), own = __ballot_sync(0xffffffffu, f != 0);
        near = __ffs(done) - 1;
        if (near >= 0 && !(~own & ((1u << near) - 1))) break;
        if (__shfl_sync(0xffffffffu, tc::globaltimer() - t0 > tc::kWaitLimitNs, 0)) {
            if (lane == 0) status_set(p.status, GCL_DEV_WAIT_TIMEOUT);
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = 0.f;
            return;
        }
    }
    __syncwarp();
    int64_t at = (seq - 1 - near) * p.D + ch;
    chain_load<V>(p.chain.out, at, on, h);
    for (int m = near; m > 0; m -= 4) {                    // four tiles' loads in flight
        float a[4][V], b[4][V];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            chain_load<V>(p.chain.a, at + (u + 1) * (int64_t)p.D, on && u < m, a[u]);
            chain_load<V>(p.chain.own, at + (u + 1) * (int64_t)p.D, on && u < m, b[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (u < m)
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = fmaf(a[u][v], h[v], b[u][v]);
        at += 4 * (int64_t)p.D;
    }
}

// One warp: publishes its channels of a tile: own states (kOwn) or the state that leaves (kDone).
template <int V>
__device__ __forceinline__ void chain_publish(const Params &p, int64_t seq, int cb, int ch, bool on, const float *a, const float *h, int32_t what) {
    const int64_t at = seq * p.D + ch;
    if (on) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (what == kOwn) {
                __stcg(p.chain.a + at + v, a[v]);
                __stcg(p.chain.own + at + v, h[v]);
            } else {
                __stcg(p.chain.out + at + v, h[v]);
            }
        }
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        __threadfence();
        store_flag(p.chain.flag + (int64_t)cb * p.tiles + seq, what);
    }
}

// One warp: from the warps' products and own states (rows of s_a and s_b, in the order of the recurrence where REV is
// false, from last to first else; s_cut: the row does not depend on the one before), publishes the tile and puts the
// state that enters each row into s_b.
template <int V, int WARPS, int CB, bool REV>
__device__ __forceinline__ void chain_tile(const Params &p, int64_t seq, int cb, int ch, bool on, float (*s_a)[CB], float (*s_b)[CB], const int *s_cut) {
    const int l = (threadIdx.x & 31) * V;
    float A[V], h[V], c[V];
    bool cut = false;
#pragma unroll
    for (int v = 0; v < V; ++v) { A[v] = 1.f; h[v] = 0.f; c[v] = 0.f; }
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        const int w = REV ? WARPS - 1 - i : i;
        const bool k = s_cut[w] != 0;
        cut |= k;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = k ? s_b[w][l + v] : fmaf(s_a[w][l + v], h[v], s_b[w][l + v]);
            A[v] *= s_a[w][l + v];
        }
    }
    chain_publish<V>(p, seq, cb, ch, on, A, h, cut ? kDone : kOwn);
    if (seq > 0) chain_enter<V>(p, seq, cb, ch, on, c);    // (the first tile is cut at its first token)
    if (!cut) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(A[v], c[v], h[v]);
        chain_publish<V>(p, seq, cb, ch, on, A, h, kDone);
    }
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        const int w = REV ? WARPS - 1 - i : i;
        const bool k = s_cut[w] != 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float b = s_b[w][l + v], a = s_a[w][l + v];
            s_b[w][l + v] = c[v];
            c[v] = k ? b : fmaf(a, c[v], b);
        }
    }
}

template <int CB, int WARPS>
struct Shared {
    float a[WARPS][CB], b[WARPS][CB];
    int start[2][WARPS * kRun], end[2][WARPS * kRun];
    int cut[WARPS];
    uint32_t ticket[2];
};

// ---- forward -------------------------------------------------------------
// Per block: two tiles staged, so that the next one's rows are under way while this one is computed.  Bound by HBM and issue together.
template <typename T>
__global__ void __launch_bounds__(32 * kWarpsF, kCtasF) glr_fwd_kernel(const Params p) {
    constexpr int V = Lane<T>::V, CB = Lane<T>::CB, RUN = kRun, N = RUN * V, THREADS = 32 * kWarpsF, BYTES = kTileF * 128;
    __shared__ Shared<CB, kWarpsF> s;
    extern __shared__ __align__(16) uint8_t s_rows[];      // [2][r, x, i][kTileF][128]
    grid_dependency_wait();
    if (p.head->blocked) return;
    const int64_t live = p.head->live;
    const uint32_t units = (uint32_t)((live + kTileF - 1) / kTileF * p.n_cb);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, narr = p.i.p ? 3 : 2;
    auto stage = [&](uint32_t unit, int buf) {
        if (unit < units) {
            const uint32_t j = unit / p.n_cb;
            const int64_t t0 = (int64_t)j * kTileF;
            const int cb = unit - j * p.n_cb, n = live - t0 < kTileF ? (int)(live - t0) : kTileF;
            uint8_t *dst = s_rows + buf * narr * BYTES;
            stage_rows<T, kTileF, THREADS>(p, p.r, t0, n, cb, dst);
            stage_rows<T, kTileF, THREADS>(p, p.x, t0, n, cb, dst + BYTES);
            if (narr == 3) stage_rows<T, kTileF, THREADS>(p, p.i, t0, n, cb, dst + 2 * BYTES);
        }
        stage_commit();
    };
    if (threadIdx.x == 0) s.ticket[0] = atomicAdd(&p.head->ticket, 1u);
    __syncthreads();
    uint32_t unit = s.ticket[0], next = 0;
    if (unit >= units) return;
    stage(unit, 0);
    if (warp == 1) borders<kTileF>(p, unit / p.n_cb, s.start[0], s.end[0]);
    bool first = true;
    for (int buf = 0; unit < units; buf ^= 1) {
        if (first) stage_wait<0>();
        else stage_wait<1>();
        __syncthreads();
        // (a second tile is taken only when the first has arrived, so that few tiles spread over all blocks)
        uint32_t taken = 0;
        if (threadIdx.x == 32) taken = atomicAdd(&p.head->ticket, first ? 2u : 1u);
        const uint32_t j = unit / p.n_cb;
        const int64_t t = (int64_t)j * kTileF + warp * RUN;
        const int cb = unit - j * p.n_cb, ch = cb * CB + lane * V;
        const int n = live - t < RUN ? (int)(live - t) : RUN;            // live tokens of the warp (none: <= 0)
        const bool on = ch < p.D;
        const uint8_t *rows = s_rows + buf * narr * BYTES + warp * RUN * 128 + lane * 4;
        float a[N], b[N];
        {
            float rate[V];
            load_state<V>(p.kind.rate, 0, p.D, ch, on && p.kind.decay == GCL_DECAY_POWER, rate);
            float r[N];
#pragma unroll
            for (int k = 0; k < RUN; ++k) Lane<T>::get(*reinterpret_cast<const uint32_t *>(rows + k * 128), r + k * V);
            decays<T, N>(p.kind, rate, r, a, b);
            mixes<T, N>(p.kind, a, b);
#pragma unroll
            for (int k = 0; k < RUN; ++k) {
                float x[V];
                Lane<T>::get(*reinterpret_cast<const uint32_t *>(rows + BYTES + k * 128), x);
#pragma unroll
                for (int v = 0; v < V; ++v) b[k * V + v] *= x[v];
            }
            if (narr == 3) {
#pragma unroll
                for (int k = 0; k < RUN; ++k) {
                    float g[V];
                    Lane<T>::get(*reinterpret_cast<const uint32_t *>(rows + 2 * BYTES + k * 128), g);
#pragma unroll
                    for (int v = 0; v < V; ++v) b[k * V + v] *= sigmoid<T>(g[v]);
                }
            }
        }
        if (n < RUN)
#pragma unroll
            for (int k = 0; k < RUN; ++k)
                if (k >= n)
#pragma unroll
                    for (int v = 0; v < V; ++v) { a[k * V + v] = 1.f; b[k * V + v] = 0.f; }
        const int *start = s.start[buf] + warp * RUN, *end = s.end[buf] + warp * RUN;
        const uint32_t starts = __ballot_sync(0xffffffffu, lane < RUN && start[lane % RUN] >= 0);
        const uint32_t ends = __ballot_sync(0xffffffffu, lane < RUN && end[lane % RUN] >= 0);
        {
            float A[V], h[V];
#pragma unroll
            for (int v = 0; v < V; ++v) { A[v] = 1.f; h[v] = 0.f; }
            auto walk = [&](auto cut) {
#pragma unroll
                for (int k = 0; k < RUN; ++k) {
                    if (decltype(cut)::value && (starts >> k & 1)) load_state<V>(p.h0, start[k], p.D, ch, on, h);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        h[v] = fmaf(a[k * V + v], h[v], b[k * V + v]);
                        A[v] *= a[k * V + v];
                    }
                }
            };
            if (starts) walk(std::true_type());
            else walk(std::false_type());
#pragma unroll
            for (int v = 0; v < V; ++v) { s.a[warp][lane * V + v] = A[v]; s.b[warp][lane * V + v] = h[v]; }
            if (lane == 0) s.cut[warp] = starts != 0;
        }
        if (threadIdx.x == 32) {
            s.ticket[0] = first ? taken : next;
            s.ticket[1] = first ? taken + 1 : taken;
        }
        __syncthreads();                                   // the rows are read, the warps' own states there
        if (first) stage(s.ticket[0], buf ^ 1);
        stage(s.ticket[1], buf);
        const uint32_t unit1 = s.ticket[0];
        next = s.ticket[1];
        if (warp == 0) chain_tile<V, kWarpsF, CB, false>(p, j, cb, ch, on, s.a, s.b, s.cut);
        if (warp == 1 && unit1 < units) borders<kTileF>(p, unit1 / p.n_cb, s.start[buf ^ 1], s.end[buf ^ 1]);
        __syncthreads();
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = s.b[warp][lane * V + v];
        if (warp * RUN % kSave == 0 && p.h_save && n > 0) {
            if (starts & 1) load_state<V>(p.h0, start[0], p.D, ch, on, h);
            store_state<V>(p.h_save, t / kSave, p.D, ch, on, h);
        }
        uint32_t *to = word<T>(p.o, t, ch);
        const int n_out = p.o.p && on && n > 0 && GCL_RANGE_IN_BOUNDS(t, t + n - 1, p.t_max, p.status) ? n : 0;
        auto walk = [&](auto plain) {                      // plain: no borders, all tokens live
#pragma unroll
            for (int k = 0; k < RUN; ++k) {
                if (!decltype(plain)::value && (starts >> k & 1)) load_state<V>(p.h0, start[k], p.D, ch, on, h);
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = fmaf(a[k * V + v], h[v], b[k * V + v]);
                if (decltype(plain)::value ? n_out > 0 : k < n_out) *to = Lane<T>::put(h);
                to += p.o.st / V;
                if (!decltype(plain)::value && (ends >> k & 1)) store_state<V>(p.ht, end[k], p.D, ch, on, h);
            }
        };
        if (!(starts | ends) && n == RUN) walk(std::true_type());
        else walk(std::false_type());
        unit = unit1;
        first = false;
    }
    stage_wait<0>();
}

// ---- backward ------------------------------------------------------------
// As the forward, over the tiles from last to first; a tile's rows stay staged until its gradients are out, and sigmoids are
// formed again for them (registers).  The states inside the tile come from the one saved before it.
template <typename T>
__global__ void __launch_bounds__(32 * kWarpsB, kCtasB) glr_bwd_kernel(const Params p) {
    constexpr int V = Lane<T>::V, CB = Lane<T>::CB, RUN = kRun, N = RUN * V, THREADS = 32 * kWarpsB, BYTES = kTileB * 128;
    static_assert(kTileB == kSave, "one saved state a tile");
    __shared__ Shared<CB, kWarpsB> s;
    __shared__ float s_h[kWarpsB][CB], s_d[kWarpsB][CB];
    __shared__ int s_cuth[kWarpsB];
    extern __shared__ __align__(16) uint8_t s_rows[];      // [2][r, x, d_o, i][kTileB][128]
    launch_dependents();                                   // (the sum of the rates' gradients waits for this grid's end)
    grid_dependency_wait();
    if (p.head->blocked) return;
    const int64_t live = p.head->live, n_live = (live + kTileB - 1) / kTileB;
    const uint32_t units = (uint32_t)(n_live * p.n_cb);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, narr = p.i.p ? 4 : 3;
    auto stage = [&](uint32_t unit, int buf) {
        if (unit < units) {
            const uint32_t seq = unit / p.n_cb;
            const int64_t t0 = (n_live - 1 - seq) * kTileB;
            const int cb = unit - seq * p.n_cb, n = live - t0 < kTileB ? (int)(live - t0) : kTileB;
            uint8_t *dst = s_rows + buf * narr * BYTES;
            stage_rows<T, kTileB, THREADS>(p, p.r, t0, n, cb, dst);
            stage_rows<T, kTileB, THREADS>(p, p.x, t0, n, cb, dst + BYTES);
            stage_rows<T, kTileB, THREADS>(p, p.d_o, t0, n, cb, dst + 2 * BYTES);
            if (narr == 4) stage_rows<T, kTileB, THREADS>(p, p.i, t0, n, cb, dst + 3 * BYTES);
        }
        stage_commit();
    };
    if (threadIdx.x == 0) s.ticket[0] = atomicAdd(&p.head->ticket, 1u);
    __syncthreads();
    uint32_t unit = s.ticket[0];
    if (unit >= units) return;
    stage(unit, 0);
    if (warp == 1) borders<kTileB>(p, n_live - 1 - unit / p.n_cb, s.start[0], s.end[0]);
    for (int buf = 0; unit < units; buf ^= 1) {
        stage_wait<0>();
        __syncthreads();
        uint32_t taken = 0;
        if (threadIdx.x == 32) taken = atomicAdd(&p.head->ticket, 1u);
        const uint32_t seq = unit / p.n_cb;
        const int64_t j = n_live - 1 - seq, t = j * kTileB + warp * RUN;
        const int cb = unit - seq * p.n_cb, ch = cb * CB + lane * V;
        const int n = live - t < RUN ? (int)(live - t) : RUN;            // live tokens of the warp (none: <= 0)
        const bool on = ch < p.D;
        const uint8_t *rows = s_rows + buf * narr * BYTES + warp * RUN * 128 + lane * 4;
        auto row = [&](int arr, int k, float *v) { Lane<T>::get(*reinterpret_cast<const uint32_t *>(rows + arr * BYTES + k * 128), v); };
        float rate[V], a[N], m[N], before[V];
        load_state<V>(p.kind.rate, 0, p.D, ch, on && p.kind.decay == GCL_DECAY_POWER, rate);
        if (warp == 1) load_state<V>(p.h_save, j, p.D, ch, on, before);
        {
            float r[N];
#pragma unroll
            for (int k = 0; k < RUN; ++k) row(0, k, r + k * V);
            decays<T, N>(p.kind, rate, r, a, m);
            mixes<T, N>(p.kind, a, m);
        }
        if (n < RUN)
#pragma unroll
            for (int k = 0; k < RUN; ++k)
                if (k >= n)
#pragma unroll
                    for (int v = 0; v < V; ++v) { a[k * V + v] = 1.f; m[k * V + v] = 0.f; }
        const int *start = s.start[buf] + warp * RUN, *end = s.end[buf] + warp * RUN;
        const uint32_t starts = __ballot_sync(0xffffffffu, lane < RUN && start[lane % RUN] >= 0);
        const uint32_t ends = __ballot_sync(0xffffffffu, lane < RUN && end[lane % RUN] >= 0);
        float prev[N];                                     // b = m u, then the state before each token
        {
            float A[V], h[V], c[V];
#pragma unroll
            for (int v = 0; v < V; ++v) { A[v] = 1.f; h[v] = c[v] = 0.f; }
            auto walk = [&](auto cut) {
#pragma unroll
                for (int k = 0; k < RUN; ++k) {
                    float x[V], g[V];
                    row(1, k, x);
                    if (narr == 4) row(3, k, g);
                    if (decltype(cut)::value && (starts >> k & 1)) load_state<V>(p.h0, start[k], p.D, ch, on, h);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        prev[k * V + v] = m[k * V + v] * (narr == 4 ? x[v] * sigmoid<T>(g[v]) : x[v]);
                        h[v] = fmaf(a[k * V + v], h[v], prev[k * V + v]);
                        A[v] *= a[k * V + v];
                    }
                }
#pragma unroll
                for (int k = RUN - 1; k >= 0; --k) {
                    float go[V];
                    row(2, k, go);
                    if (decltype(cut)::value && (ends >> k & 1)) load_state<V>(p.dht, end[k], p.D, ch, on, c);
#pragma unroll
                    for (int v = 0; v < V; ++v) c[v] = a[k * V + v] * (go[v] + c[v]);
                }
            };
            if (starts | ends) walk(std::true_type());
            else walk(std::false_type());
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s.a[warp][lane * V + v] = A[v];
                s.b[warp][lane * V + v] = c[v];
                s_h[warp][lane * V + v] = h[v];
            }
            if (lane == 0) { s.cut[warp] = ends != 0; s_cuth[warp] = starts != 0; }
        }
        if (threadIdx.x == 32) s.ticket[0] = taken;
        __syncthreads();
        const uint32_t unit1 = s.ticket[0];
        stage(unit1, buf ^ 1);
        if (warp == 0) {
            chain_tile<V, kWarpsB, CB, true>(p, seq, cb, ch, on, s.a, s.b, s.cut);
        } else if (warp == 1) {                            // the states that enter the warps' tokens
#pragma unroll
            for (int w = 0; w < kWarpsB; ++w)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float b = s_h[w][lane * V + v], A = s.a[w][lane * V + v];
                    s_h[w][lane * V + v] = before[v];
                    before[v] = s_cuth[w] ? b : fmaf(A, before[v], b);
                }
            if (unit1 < units) borders<kTileB>(p, n_live - 1 - unit1 / p.n_cb, s.start[buf ^ 1], s.end[buf ^ 1]);
        }
        __syncthreads();
        float h[V], c[V], dsum[V];
#pragma unroll
        for (int v = 0; v < V; ++v) { h[v] = s_h[warp][lane * V + v]; c[v] = s.b[warp][lane * V + v]; dsum[v] = 0.f; }
        const int64_t last = t + RUN - 1;
        uint32_t *to_x = word<T>(p.dx, last, ch), *to_r = word<T>(p.dr, last, ch), *to_i = word<T>(p.di, last, ch);
        const int n_out = on && n > 0 && GCL_RANGE_IN_BOUNDS(t, t + n - 1, p.t_max, p.status) ? n : 0;
        auto walk = [&](auto plain) {                      // plain: no borders, all tokens live
            constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
            for (int k = 0; k < RUN; ++k) {
                if (!PLAIN && (starts >> k & 1)) load_state<V>(p.h0, start[k], p.D, ch, on, h);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float b = prev[k * V + v];
                    prev[k * V + v] = h[v];
                    h[v] = fmaf(a[k * V + v], h[v], b);
                }
            }
#pragma unroll
            for (int k = RUN - 1; k >= 0; --k) {
                if (!PLAIN && (ends >> k & 1)) load_state<V>(p.dht, end[k], p.D, ch, on, c);
                float dx[V], dr[V], di[V], x[V], g[V], go[V], r[V];
                row(0, k, r);
                row(1, k, x);
                row(2, k, go);
                if (narr == 4) row(3, k, g);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int e = k * V + v;
                    const float G = go[v] + c[v];
                    c[v] = a[e] * G;
                    float sg = 1.f, ng = 0.f;
                    if (narr == 4) sigmoids<T>(g[v], sg, ng);
                    const float u = x[v] * sg;
                    dx[v] = G * m[e] * sg;
                    di[v] = dx[v] * x[v] * ng;
                    float dl = c[v] * prev[e];
                    if (p.kind.mix == GCL_MIX_COMPLEMENT) dl = fmaf(-c[v], u, dl);
                    else if (p.kind.mix == GCL_MIX_ROOT) dl = fmaf(m[e] > 0.f ? -a[e] * frcp<T>(m[e]) * c[v] : 0.f, u, dl);
                    if (p.kind.decay != GCL_DECAY_LOG) {
                        float sr, nr;
                        sigmoids<T>(r[v], sr, nr);
                        if (p.kind.decay == GCL_DECAY_SIGMOID) {
                            dl *= nr;
                        } else {
                            if (PLAIN || k < n) dsum[v] = fmaf(-dl, sr, dsum[v]);
                            dl *= -rate[v] * sr * nr;
                        }
                    }
                    dr[v] = dl;
                }
                if (PLAIN ? n_out > 0 : k < n_out) {
                    *to_x = Lane<T>::put(dx);
                    *to_r = Lane<T>::put(dr);
                    if (narr == 4) *to_i = Lane<T>::put(di);
                }
                to_x -= p.dx.st / V;
                to_r -= p.dr.st / V;
                to_i -= p.di.st / V;
                if (!PLAIN && (starts >> k & 1)) store_state<V>(p.dh0, start[k], p.D, ch, on, c);
            }
        };
        if (!(starts | ends) && n == RUN) walk(std::true_type());
        else walk(std::false_type());
        if (p.drate_part) {
#pragma unroll
            for (int v = 0; v < V; ++v) s_d[warp][lane * V + v] = dsum[v];
            __syncthreads();
            if (warp == 2) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarpsB; ++w) sum += s_d[w][lane * V + v];
                    dsum[v] = sum;
                }
                store_state<V>(p.drate_part, j, p.D, ch, on, dsum);
            }
        }
        unit = unit1;
    }
    stage_wait<0>();
}

// drate from the tiles' sums, in a fixed order: 32 channels a block, 32 rows of threads over the tiles, eight loads of
// each in flight.
__global__ void __launch_bounds__(1024) glr_drate_kernel(const Params p, int tile) {
    __shared__ float s[32][33];
    grid_dependency_wait();
    if (p.head->blocked) return;
    const int64_t n = (p.head->live + tile - 1) / tile;
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (d < p.D)
        for (int64_t j0 = r; j0 < n; j0 += 8 * 32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = j0 + i * 32 < n ? p.drate_part[(j0 + i * 32) * p.D + d] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i];
        }
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
    const int64_t n_cb = (a->D * (a->dtype == GCL_F32 ? 4 : 2) + 127) / 128;
    set(o.first, sizeof(int32_t) * (size_t)tiles);
    set(o.chain.flag, sizeof(int32_t) * (size_t)(tiles * n_cb));
    set(o.chain.a, row * tiles);
    set(o.chain.own, row * tiles);
    set(o.chain.out, row * tiles);
    if (backward) {
        if (a->drate) set(o.drate_part, row * tiles);
        if (!a->h_save) set(o.h_save, row * tb);
    }
    return at;
}

// Launches the set-up and, as its dependent, `kernel` with at most `ctas` blocks an SM.
template <typename K>
cudaError_t launch_tiles(K kernel, const Params &p, const float *in_state, float *out_state, int tile, int threads, int ctas, size_t smem,
                         cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t units = p.tiles * p.n_cb, most = (int64_t)ctas * num_sms();
    int64_t setup = (units + 4095) / 4096;
    if (out_state && setup < (p.n_max + 7) / 8) setup = (p.n_max + 7) / 8;
    if (setup > num_sms()) setup = num_sms();
    glr_setup_kernel<<<(unsigned)setup, 1024, 0, s>>>(p, in_state, out_state, tile);
    return launch_dependent(kernel, dim3((unsigned)(units < most ? units : most)), dim3(threads), smem, s, p);
}

template <typename T>
cudaError_t launch_fwd(const Params &p, cudaStream_t s) {
    return launch_tiles(glr_fwd_kernel<T>, p, p.h0, p.ht, kTileF, 32 * kWarpsF, kCtasF, (size_t)2 * (p.i.p ? 3 : 2) * kTileF * 128, s);
}

template <typename T>
cudaError_t launch_bwd(const Params &p, cudaStream_t s) {
    const cudaError_t e = launch_tiles(glr_bwd_kernel<T>, p, p.dht, p.dh0, kTileB, 32 * kWarpsB, kCtasB, (size_t)2 * (p.i.p ? 4 : 3) * kTileB * 128, s);
    if (e != cudaSuccess || !p.drate) return e;
    return launch_dependent(glr_drate_kernel, dim3((p.D + 31) / 32), dim3(1024), 0, s, p, kTileB);
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
