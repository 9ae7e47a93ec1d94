// glr.cu -- gated linear recurrence over packed sequences: forward and backward.
//
// The packed axis is cut into tiles of some tokens by the 128 bytes of a warp's width of channels; each warp of a block walks
// kRun tokens of a tile.  The sequences need no plan of their own: a token that starts one takes its state from h0,
// whatever was before.  One pass: a cluster of kRanks blocks takes kRanks consecutive tiles of the same channels (a span), in the
// order of the recurrence (a counter).  Its blocks form their tiles' products of decays and states from zero, exchange them
// through shared memory, and take the state that enters the span from the span before, or from an earlier one and the products and
// own states between; the sum is folded from the oldest on, so the result is the same whichever span had its state ready.
// A cluster waits for spans with lower numbers alone, whose clusters run already, so the first of them never waits: the
// launch ends whatever else runs on the GPU.
// The wait for the state before is what a tile spends longest on: spans meet in packets of 16 bytes, values and tag in one access
// (XCHAIN).
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

constexpr int kRun = 8;                                // tokens of a warp
constexpr int kRanks = 4;                              // blocks of a cluster
constexpr int kWarpsF = 16, kWarpsB = 8;               // warps of a block; a tile has kRun tokens for each
constexpr int kTileF = kWarpsF * kRun, kTileB = kWarpsB * kRun;
constexpr int kCtasF = 2, kCtasB = 3;                  // resident blocks an SM
static_assert(kWarpsB * kRun == kSave && kWarpsF * kRun % kSave == 0, "saved states lie at tiles' starts");

// ---- set-up: checks cu_seqlens, finds each tile's first sequence, passes states of empty sequences through, clears the
// packets of the spans that will be taken ----
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
    const int64_t spans = (p.cu[p.n_max] + (int64_t)kRanks * tile - 1) / (kRanks * tile);
    for (int64_t e = at; e < spans * p.D; e += step) reinterpret_cast<uint4 *>(p.chain)[e] = make_uint4(0, 0, 0, 0);
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

// ---- clusters ----
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
    return a;
}
// Stores that count their bytes on the peer's barrier when they have landed there.
__device__ __forceinline__ void peer_send(void *p, uint64_t *bar, uint32_t rank, uint32_t v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(peer_addr(p, rank)), "r"(v),
                 "r"(peer_addr(bar, rank))
                 : "memory");
}
__device__ __forceinline__ void peer_send(void *p, uint64_t *bar, uint32_t rank, uint32_t v, uint32_t w) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.u32 [%0], {%1, %2}, [%3];" ::"r"(peer_addr(p, rank)), "r"(v),
                 "r"(w), "r"(peer_addr(bar, rank))
                 : "memory");
}
__device__ __forceinline__ uint32_t peer_load(const void *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
// (orders no memory: a release waits for the outputs' stores of the tile before)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// ---- what a block holds of a tile beside its rows ----
template <int TILE>
struct Tile {
    int32_t seq, cb;               // its span's place in the order of the recurrence, its block of channels
    int32_t t0, n;                 // its first token, its live tokens (0: none)
    uint32_t starts[TILE / 32], ends[TILE / 32];       // tokens that start and end a sequence, a bit each
    int32_t start[TILE], end[TILE];                    // which (where the bit is set)
};

// One warp: the sequences that start and end among the tile's tokens.
template <int TILE>
__device__ __forceinline__ void borders(const Params &p, Tile<TILE> &t) {
    const int lane = threadIdx.x & 31;
    uint32_t starts[TILE / 32] = {}, ends[TILE / 32] = {};
    if (t.n > 0) {
        const int f = p.first[t.t0 / TILE];
        for (int n = (f > 0 ? f - 1 : 0) + lane; n < p.n_max; n += 32) {
            const int b = p.cu[n] - t.t0, e = p.cu[n + 1] - t.t0;          // (both lie in [0, 2^31))
            if (b >= TILE) break;
            if (e <= b) continue;
#pragma unroll
            for (int k = 0; k < TILE / 32; ++k) {
                if (b >> 5 == k) starts[k] |= 1u << (b & 31);
                if ((e - 1) >> 5 == k) ends[k] |= 1u << ((e - 1) & 31);
            }
            if (b >= 0) t.start[b] = n;
            if (e >= 1 && e <= TILE) t.end[e - 1] = n;
        }
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < TILE / 32; ++k) {
        const uint32_t u = __reduce_or_sync(0xffffffffu, starts[k]), v = __reduce_or_sync(0xffffffffu, ends[k]);
        if (lane == 0) { t.starts[k] = u; t.ends[k] = v; }
    }
}
// The bits of warp w's tokens; whether there are any in the tile.
__device__ __forceinline__ uint32_t bits_of(const uint32_t *words, int w) { return words[w / 4] >> (w % 4 * 8) & 0xffu; }
template <int N>
__device__ __forceinline__ bool any_of(const uint32_t *words) {
    uint32_t a = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) a |= words[k];
    return a != 0;
}

template <typename T>
__device__ __forceinline__ uint32_t *word(const Rows &r, int64_t t, int ch) {
    return reinterpret_cast<uint32_t *>(static_cast<T *>(r.p) + t * r.st + ch);
}

// A lane's values of row n of [n, D]; zeros without the array or past the channels.
template <typename T>
__device__ __forceinline__ typename Lane<T>::P load_state(const float *s, int64_t n, int D, int ch) {
    return s && ch < D ? Lane<T>::load(s + n * D + ch) : Lane<T>::all(0.f);
}
template <typename T>
__device__ __forceinline__ void store_state(float *s, int64_t n, int D, int ch, typename Lane<T>::P h) {
    if (s && ch < D) Lane<T>::store(s + n * D + ch, h);
}

// ---- what spans leave each other ----
__device__ __forceinline__ Packet load_packet(const Packet *p) {
    unsigned __int128 v;
    asm volatile("ld.relaxed.gpu.global.b128 %0, [%1];" : "=q"(v) : "l"(p) : "memory");
    Packet k;
    k.a = __uint_as_float((uint32_t)v);
    k.own = __uint_as_float((uint32_t)(v >> 32));
    k.out = __uint_as_float((uint32_t)(v >> 64));
    k.tag = (uint32_t)(v >> 96);
    return k;
}
__device__ __forceinline__ void store_packet(Packet *p, float a, float own, float out, uint32_t tag) {
    const unsigned __int128 v = (unsigned __int128)__float_as_uint(a) | (unsigned __int128)__float_as_uint(own) << 32 |
                                (unsigned __int128)__float_as_uint(out) << 64 | (unsigned __int128)tag << 96;
    asm volatile("st.relaxed.gpu.global.b128 [%0], %1;" ::"l"(p), "q"(v) : "memory");
}

// One warp, a channel a lane: the state that enters span `seq` (> 0): from the nearest span before it whose state is out for all
// the warp's channels, and the own states of the spans between, folded from the oldest on.  False: it did not come in time.
__device__ __forceinline__ bool chain_enter(const Params &p, int64_t seq, int ch, bool on, float &h) {
    constexpr int W = 2;                                   // packets in flight
    const int64_t base = seq - 1;
    int depth = 0;
    uint64_t t0 = 0;
    while (true) {
        Packet k[W];
#pragma unroll
        for (int u = 0; u < W; ++u) {
            const int64_t at = base - depth - u;
            k[u].a = k[u].own = k[u].out = 0.f;
            k[u].tag = on ? 0 : kDone;
            if (on && at >= 0) k[u] = load_packet(p.chain + at * p.D + ch);
        }
        int found = W;
        bool gap = false;
#pragma unroll
        for (int u = 0; u < W; ++u)
            if (found == W && !gap) {
                if (__all_sync(0xffffffffu, k[u].tag == kDone)) found = u;
                else gap = !__all_sync(0xffffffffu, k[u].tag != 0);
            }
        if (found < W) {
#pragma unroll
            for (int u = W - 1; u >= 0; --u) h = u == found ? k[u].out : u < found ? fmaf(k[u].a, h, k[u].own) : h;
            for (int d = depth - 1; d >= 0; d -= W) {      // the spans nearer than these (a multiple of W)
                Packet n[W];
#pragma unroll
                for (int u = 0; u < W; ++u) {
                    n[u].a = n[u].own = 0.f;
                    if (on) n[u] = load_packet(p.chain + (base - d + u) * p.D + ch);
                }
#pragma unroll
                for (int u = 0; u < W; ++u) h = fmaf(n[u].a, h, n[u].own);
            }
            return true;
        }
        depth = gap || depth >= 15 * W ? 0 : depth + W;
        if (t0 == 0) t0 = tc::globaltimer();
        if (__shfl_sync(0xffffffffu, tc::globaltimer() - t0 > tc::kWaitLimitNs, 0)) return false;
    }
}

template <int CB, int WARPS>
struct Shared {
    float a[WARPS][CB], b[WARPS][CB];
    float2 tot[2][kRanks - 1][CB]; // products and own states of the blocks before, by parity of the tile
    uint32_t tot_cut[2][kRanks - 1];
    uint32_t next[2];              // the next span, by parity; next[1] at first: the cluster's first
    uint64_t sent[2];              // these have come
    Tile<WARPS * kRun> tile[2];
    int err;
    uint64_t full[2];
};

// One warp, a channel a lane (column c of s.a, s.b): from the warps' products and own states (in the order of the recurrence: from
// the first row, REV from the last) the block's, exchanged with the cluster's blocks; then the state that enters each row into s.b.
// `cuts`: a bit a token; a warp with one does not depend on the state before.  False: the state before did not
// come in time (s.err is set; then nothing is waited for any more).
template <bool REV, int CB, int WARPS>
__device__ __forceinline__ bool chain_tile(const Params &p, int64_t seq, int ch, int c, uint32_t rank, int par, const uint32_t *cuts,
                                           Shared<CB, WARPS> &s, uint32_t phase) {
    const bool on = ch < p.D, cut = any_of<WARPS * kRun / 32>(cuts);
    float A = 1.f, h = 0.f;
    if (!cut) {
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            const int w = REV ? WARPS - 1 - i : i;
            const float a = s.a[w][c];
            h = fmaf(a, h, s.b[w][c]);
            A *= a;
        }
    } else {
        A = 0.f;
        for (int i = 0; i < WARPS; ++i) {
            const int w = REV ? WARPS - 1 - i : i;
            h = bits_of(cuts, w) ? s.b[w][c] : fmaf(s.a[w][c], h, s.b[w][c]);
        }
    }
    for (uint32_t r = rank + 1; r < kRanks; ++r) {
        peer_send(&s.tot[par][rank][c], &s.sent[par], r, __float_as_uint(A), __float_as_uint(h));
        if (c == 0) peer_send(&s.tot_cut[par][rank], &s.sent[par], r, cut);
    }
    tc::mbar_wait(&s.sent[par], phase, &s.err, GCL_DEV_WAIT_TIMEOUT);
    const bool wait = *reinterpret_cast<volatile int *>(&s.err) == 0;
    Packet *mine = p.chain + seq * p.D + ch;
    bool ok = true, span_cut = cut;
    if (rank == kRanks - 1) {                              // the last block speaks for the span
        float before = 0.f, product = 1.f;
#pragma unroll
        for (int r = 0; r < kRanks - 1; ++r) {
            const bool k = s.tot_cut[par][r] != 0;
            span_cut |= k;
            const float2 t = s.tot[par][r][c];
            before = k ? t.y : fmaf(t.x, before, t.y);
            product *= t.x;
        }
        if (!cut) h = fmaf(A, before, h);
        A *= product;
        if (on) store_packet(mine, A, h, h, span_cut ? kDone : kOwn);
    }
    float in = 0.f;
    if (seq > 0 && wait) ok = chain_enter(p, seq, ch, on, in);             // (the first span is cut at its first token)
    if (rank == kRanks - 1 && on && !span_cut) store_packet(mine, A, h, fmaf(A, in, h), kDone);
    for (uint32_t r = 0; r < rank; ++r) {
        const float2 t = s.tot[par][r][c];
        in = s.tot_cut[par][r] ? t.y : fmaf(t.x, in, t.y);
    }
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        const int w = REV ? WARPS - 1 - i : i;
        const float a = s.a[w][c], b = s.b[w][c];
        s.b[w][c] = in;
        in = cut && bits_of(cuts, w) ? b : fmaf(a, in, b);
    }
    return ok;
}

struct Maps {                      // the staged rows: r, x, d_o (backward), i
    CUtensorMap m[4];
};

constexpr int kIssuer = 96;        // the thread that takes spans and issues the copies

// A block's walk over its tiles, which both directions share.  Its next tile's rows are staged while one is computed.
template <bool REV, int CB, int WARPS>
struct Walk {
    static constexpr int TILE = WARPS * kRun, BYTES = TILE * 128;
    const Params &p;
    Shared<CB, WARPS> &s;
    const Maps &maps;
    uint8_t *rows;                 // [2][narr][TILE][128]
    int narr;
    int64_t live, tiles;           // live tokens; tiles that have some
    uint32_t units, rank;
    uint32_t phase;                // parity of the barriers of what the peers send: bit by buffer
    uint32_t parity, issued;       // of the copies into the two buffers: the next wait's; the last issued one's, inverted, and
                                   // whether any was (issuer)

    // The issuer: this block's tile in span `unit`, and its copies.
    __device__ __forceinline__ void issue(uint32_t unit, int buf) {
        Tile<TILE> &t = s.tile[buf];
        t.seq = unit / p.n_cb;
        t.cb = unit - t.seq * p.n_cb;
        const int64_t k = (int64_t)t.seq * kRanks + rank, j = REV ? tiles - 1 - k : k;
        t.n = 0;
        if (j < 0 || j >= tiles || *reinterpret_cast<volatile int *>(&s.err) != 0) return;
        t.t0 = (int)(j * TILE);
        t.n = live - t.t0 < TILE ? (int)(live - t.t0) : TILE;
        issued = (issued ^ 1u << buf) | 4u << buf;
        tc::mbar_arrive_expect_tx(&s.full[buf], narr * BYTES);
        for (int a = 0; a < narr; ++a)
            tc::tma_load_2d(rows + (buf * narr + a) * BYTES, &maps.m[!REV && a == 2 ? 3 : a], t.cb * CB, t.t0, &s.full[buf]);
    }
    // Sets up the barriers and takes the cluster's first span; false: there is none.  Every thread of the cluster.
    __device__ __forceinline__ bool start() {
        const int tid = threadIdx.x;
        if (tid == kIssuer) {
            tc::mbar_init(&s.full[0], 1);
            tc::mbar_init(&s.full[1], 1);
            tc::mbar_init(&s.sent[0], 1);
            tc::mbar_init(&s.sent[1], 1);
            tc::fence_barrier_init();
            s.err = 0;
            if (rank == 0) s.next[1] = atomicAdd(&p.head->ticket, 1u);
        }
        cluster_arrive();
        cluster_wait();
        const uint32_t unit = peer_load(&s.next[1], 0);
        if (unit >= units) {
            cluster_arrive();                              // (the first block stays until all have read)
            cluster_wait();
            return false;
        }
        if (tid / 32 == kIssuer / 32) {
            if (tid == kIssuer) issue(unit, 0);
            __syncwarp();
            borders(p, s.tile[0]);
        }
        cluster_arrive_relaxed();
        __syncthreads();
        return true;
    }
    // The staged rows have landed.
    __device__ __forceinline__ void landed(int buf) {
        if (s.tile[buf].n == 0) return;
        tc::mbar_wait(&s.full[buf], parity >> buf & 1, &s.err, GCL_DEV_WAIT_TIMEOUT);
        parity ^= 1u << buf;
    }
    // Takes the cluster's next span (its number reaches the blocks by the exchange).
    __device__ __forceinline__ uint32_t take() { return rank == 0 && threadIdx.x == kIssuer ? atomicAdd(&p.head->ticket, 1u) : 0; }
    // Between a tile's halves: the warps' own states are in s.a, s.b; afterwards the states that enter them in s.b.
    // What a block receives at parity `buf` it has used when it arrives on the cluster's barrier, and the peers send there again
    // two tiles later, after they have waited on that barrier.
    template <typename Side>
    __device__ __forceinline__ void exchange(int buf, uint32_t taken, const uint32_t *cuts, Side side) {
        const int tid = threadIdx.x, warp = tid >> 5;
        const Tile<TILE> &t = s.tile[buf];
        const uint32_t ph = phase >> buf & 1;
        phase ^= 1u << buf;
        cluster_wait();
        if (tid == kIssuer) {
            tc::mbar_arrive_expect_tx(&s.sent[buf], 4 + rank * (CB * 8 + 4));
            if (rank == 0)
                for (int r = 0; r < kRanks; ++r) peer_send(&s.next[buf], &s.sent[buf], r, taken);
        }
        __syncthreads();
        if (warp < CB / 32) {
            if (!chain_tile<REV>(p, t.seq, t.cb * CB + tid, tid, rank, buf, cuts, s, ph)) atomicCAS(&s.err, 0, GCL_DEV_WAIT_TIMEOUT);
        } else if (warp == 2) {
            side();
        } else if (warp == kIssuer / 32) {
            tc::mbar_wait(&s.sent[buf], ph, &s.err, GCL_DEV_WAIT_TIMEOUT);
            const uint32_t unit = s.next[buf];
            if (unit < units) {
                if (tid == kIssuer) issue(unit, buf ^ 1);
                __syncwarp();
                borders(p, s.tile[buf ^ 1]);
            }
        }
        __syncthreads();
        cluster_arrive_relaxed();
    }
    __device__ __forceinline__ bool more(int buf) const { return s.next[buf] < units; }
    // After the last tile: a wait that ran out is reported, and copies still under way are waited for (with a limit).
    __device__ __forceinline__ void finish() {
        cluster_wait();
        cluster_arrive();                                  // (no block leaves while another may send to it)
        cluster_wait();
        if (s.err == 0 || threadIdx.x != kIssuer) return;
        status_set(p.status, GCL_DEV_WAIT_TIMEOUT);
        const uint64_t t0 = tc::globaltimer();
        for (int b = 0; b < 2; ++b)
            while ((issued >> (2 + b) & 1) && !tc::mbar_try_wait(&s.full[b], (issued >> b & 1) ^ 1) && tc::globaltimer() - t0 < tc::kWaitLimitNs) {}
    }
};

// ---- forward -------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(32 * kWarpsF, kCtasF) glr_fwd_kernel(const __grid_constant__ Maps maps, const Params p) {
    using L = Lane<T>;
    using P = typename L::P;
    using W = Walk<false, L::CB, kWarpsF>;
    constexpr int V = L::V, CB = L::CB, RUN = kRun, BYTES = W::BYTES;
    __shared__ Shared<CB, kWarpsF> s;
    extern __shared__ __align__(128) uint8_t s_rows[];     // [2][r, x, i][tile][128]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, narr = p.i.p ? 3 : 2;
    grid_dependency_wait();
    if (p.head->blocked) return;
    const int64_t live = p.head->live, tiles = (live + W::TILE - 1) / W::TILE;
    W walk{p, s, maps, s_rows, narr, live, tiles, (uint32_t)((tiles + kRanks - 1) / kRanks * p.n_cb), cluster_rank(), 0, 0, 0};
    if (!walk.start()) return;
    for (int buf = 0;; buf ^= 1) {
        const Tile<W::TILE> &tile = s.tile[buf];
        const int64_t t = tile.t0 + warp * RUN;
        const int ch = tile.cb * CB + lane * V, n = tile.n - warp * RUN;          // n: live tokens from the warp's first on
        const uint8_t *rows = s_rows + buf * narr * BYTES + warp * RUN * 128 + lane * 4;
        auto row = [&](int arr, int k) { return L::get(*reinterpret_cast<const uint32_t *>(rows + arr * BYTES + k * 128)); };
        const P rate = load_state<T>(p.kind.decay == GCL_DECAY_POWER ? p.kind.rate : nullptr, 0, p.D, ch);
        const bool near = __all_sync(0xffffffffu, L::every(rate, [](float v) { return v >= 0.f && v <= kNear; }));
        walk.landed(buf);
        // (the next span is taken only when this one's rows are here: few spans go to all clusters, and none is held back for long)
        const uint32_t taken = walk.take();
        P a[RUN], b[RUN];
        if (sizeof(T) == 2 && p.kind.decay == GCL_DECAY_POWER && narr == 3) {
            constexpr int H = RUN / 2;                     // (four tokens at a time: registers)
#pragma unroll
            for (int k0 = 0; k0 < RUN; k0 += H) {
                P g[H];
#pragma unroll
                for (int k = 0; k < H; ++k) two_sigmoids<T>(row(0, k0 + k), row(2, k0 + k), b[k0 + k], g[k]);
#pragma unroll
                for (int k = 0; k < H; ++k) g[k] = L::mul(g[k], row(1, k0 + k));
                decays<T, H>(p.kind, rate, near, a + k0, b + k0, true);
#pragma unroll
                for (int k = 0; k < H; ++k) b[k0 + k] = L::mul(b[k0 + k], g[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < RUN; ++k) b[k] = row(0, k);
            decays<T, RUN>(p.kind, rate, near, a, b);
#pragma unroll
            for (int k = 0; k < RUN; ++k) b[k] = L::mul(b[k], row(1, k));
            if (narr == 3)
#pragma unroll
                for (int k = 0; k < RUN; ++k) b[k] = L::mul(b[k], sigmoid<T>(row(2, k)));
        }
        if (n < RUN)
#pragma unroll
            for (int k = 0; k < RUN; ++k)
                if (k >= n) { a[k] = L::all(1.f); b[k] = L::all(0.f); }
        const int32_t *start = tile.start + warp * RUN, *end = tile.end + warp * RUN;
        const uint32_t starts = bits_of(tile.starts, warp), ends = bits_of(tile.ends, warp);
        {
            P A = L::all(1.f), h = L::all(0.f);
            auto run = [&](auto cut) {
#pragma unroll
                for (int k = 0; k < RUN; ++k) {
                    if (decltype(cut)::value && (starts >> k & 1)) h = load_state<T>(p.h0, start[k], p.D, ch);
                    h = L::fma(a[k], h, b[k]);
                    A = L::mul(A, a[k]);
                }
            };
            if (starts) run(std::true_type());
            else run(std::false_type());
            L::store(&s.a[warp][lane * V], A);
            L::store(&s.b[warp][lane * V], h);
        }
        walk.exchange(buf, taken, tile.starts, [] {});
        P h = L::load(&s.b[warp][lane * V]);
        if (warp * RUN % kSave == 0 && p.h_save && n > 0) {
            if (starts & 1) h = load_state<T>(p.h0, start[0], p.D, ch);
            store_state<T>(p.h_save, t / kSave, p.D, ch, h);
        }
        uint32_t *to = word<T>(p.o, t, ch);
        const int n_out = p.o.p && ch < p.D && n > 0 && GCL_RANGE_IN_BOUNDS(t, t + (n < RUN ? n : RUN) - 1, p.t_max, p.status) ? n : 0;
        auto run = [&](auto plain) {                       // plain: no borders, all tokens live
            constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
            for (int k = 0; k < RUN; ++k) {
                if (!PLAIN && (starts >> k & 1)) h = load_state<T>(p.h0, start[k], p.D, ch);
                h = L::fma(a[k], h, b[k]);
                if (PLAIN ? n_out > 0 : k < n_out) *to = L::put(h);
                to += p.o.st / V;
                if (!PLAIN && (ends >> k & 1)) store_state<T>(p.ht, end[k], p.D, ch, h);
            }
        };
        if (!(starts | ends) && n >= RUN) run(std::true_type());
        else run(std::false_type());
        if (!walk.more(buf)) break;
    }
    walk.finish();
}

// ---- backward ------------------------------------------------------------
// As the forward, over the tiles from last to first; a tile's rows stay staged until its gradients are out, and sigmoids are
// formed again for them (registers).  The states inside the tile come from the one saved before it.
template <typename T>
__global__ void __launch_bounds__(32 * kWarpsB, kCtasB) glr_bwd_kernel(const __grid_constant__ Maps maps, const Params p) {
    using L = Lane<T>;
    using P = typename L::P;
    using W = Walk<true, L::CB, kWarpsB>;
    constexpr int V = L::V, CB = L::CB, RUN = kRun, BYTES = W::BYTES;
    __shared__ Shared<CB, kWarpsB> s;
    __shared__ float s_h[kWarpsB][CB];
    extern __shared__ __align__(128) uint8_t s_rows[];     // [2][r, x, d_o, i][tile][128]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, narr = p.i.p ? 4 : 3;
    launch_dependents();                                   // (the sum of the rates' gradients waits for this grid's end)
    grid_dependency_wait();
    if (p.head->blocked) return;
    const int64_t live = p.head->live, tiles = (live + W::TILE - 1) / W::TILE;
    W walk{p, s, maps, s_rows, narr, live, tiles, (uint32_t)((tiles + kRanks - 1) / kRanks * p.n_cb), cluster_rank(), 0, 0, 0};
    if (!walk.start()) return;
    for (int buf = 0;; buf ^= 1) {
        const Tile<W::TILE> &tile = s.tile[buf];
        const int64_t t = tile.t0 + warp * RUN;
        const int ch = tile.cb * CB + lane * V, n = tile.n - warp * RUN;
        const uint8_t *rows = s_rows + buf * narr * BYTES + warp * RUN * 128 + lane * 4;
        auto row = [&](int arr, int k) { return L::get(*reinterpret_cast<const uint32_t *>(rows + arr * BYTES + k * 128)); };
        const P rate = load_state<T>(p.kind.decay == GCL_DECAY_POWER ? p.kind.rate : nullptr, 0, p.D, ch);
        const bool near = __all_sync(0xffffffffu, L::every(rate, [](float v) { return v >= 0.f && v <= kNear; }));
        P before = L::all(0.f);
        if (warp == 2 && tile.n > 0) before = load_state<T>(p.h_save, tile.t0 / kSave, p.D, ch);
        walk.landed(buf);
        const uint32_t taken = walk.take();
        P a[RUN], m[RUN], prev[RUN];                       // prev: b = m u, later the state before each token
#pragma unroll
        for (int k = 0; k < RUN; ++k) m[k] = row(0, k);
        decays<T, RUN>(p.kind, rate, near, a, m);
        if (n < RUN)
#pragma unroll
            for (int k = 0; k < RUN; ++k)
                if (k >= n) { a[k] = L::all(1.f); m[k] = L::all(0.f); }
        const int32_t *start = tile.start + warp * RUN, *end = tile.end + warp * RUN;
        const uint32_t starts = bits_of(tile.starts, warp), ends = bits_of(tile.ends, warp);
        const bool edge = (starts | ends) || n < RUN;
        {
            P A = L::all(1.f), h = L::all(0.f), c = L::all(0.f);
            auto run = [&](auto cut) {
                constexpr bool CUT = decltype(cut)::value;
#pragma unroll
                for (int k = 0; k < RUN; ++k) {
                    if (CUT && (starts >> k & 1)) h = load_state<T>(p.h0, start[k], p.D, ch);
                    prev[k] = L::mul(m[k], row(1, k));
                    if (narr == 4) prev[k] = L::mul(prev[k], sigmoid<T>(row(3, k)));
                    if (CUT && k >= n) prev[k] = L::all(0.f);
                    h = L::fma(a[k], h, prev[k]);
                    A = L::mul(A, a[k]);
                }
#pragma unroll
                for (int k = RUN - 1; k >= 0; --k) {
                    if (CUT && (ends >> k & 1)) c = load_state<T>(p.dht, end[k], p.D, ch);
                    c = L::mul(a[k], L::add(CUT && k >= n ? L::all(0.f) : row(2, k), c));
                }
            };
            if (edge) run(std::true_type());
            else run(std::false_type());
            L::store(&s.a[warp][lane * V], A);
            L::store(&s.b[warp][lane * V], c);
            L::store(&s_h[warp][lane * V], h);
        }
        walk.exchange(buf, taken, tile.ends, [&] {         // (a warp at leisure: the states that enter the warps' tokens)
#pragma unroll
            for (int w = 0; w < kWarpsB; ++w) {
                const P b = L::load(&s_h[w][lane * V]), A = L::load(&s.a[w][lane * V]);
                L::store(&s_h[w][lane * V], before);
                before = bits_of(tile.starts, w) ? b : L::fma(A, before, b);
            }
        });
        P h = L::load(&s_h[warp][lane * V]), c = L::load(&s.b[warp][lane * V]), dsum = L::all(0.f);
        const int64_t last = t + RUN - 1;
        uint32_t *to_x = word<T>(p.dx, last, ch), *to_r = word<T>(p.dr, last, ch), *to_i = word<T>(p.di, last, ch);
        const int n_out = ch < p.D && n > 0 && GCL_RANGE_IN_BOUNDS(t, t + (n < RUN ? n : RUN) - 1, p.t_max, p.status) ? n : 0;
        auto run = [&](auto plain) {                       // plain: no borders, all tokens live
            constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
            for (int k = 0; k < RUN; ++k) {
                if (!PLAIN && (starts >> k & 1)) h = load_state<T>(p.h0, start[k], p.D, ch);
                const P b = prev[k];
                prev[k] = h;
                h = L::fma(a[k], h, b);
            }
#pragma unroll
            for (int k = RUN - 1; k >= 0; --k) {
                if (!PLAIN && (ends >> k & 1)) c = load_state<T>(p.dht, end[k], p.D, ch);
                const P x = row(1, k), G = L::add(row(2, k), c), Gm = L::mul(G, m[k]);
                c = L::mul(a[k], !PLAIN && k >= n ? c : G);
                P dx = Gm, di = L::all(0.f), u = x, sg, ng;
                if (narr == 4) {
                    sigmoids<T>(row(3, k), sg, ng);
                    dx = L::mul(Gm, sg);
                    di = L::mul(L::mul(dx, x), ng);
                    u = L::mul(x, sg);
                }
                P dl = L::mul(c, prev[k]);
                if (p.kind.mix == GCL_MIX_COMPLEMENT) {
                    dl = L::fma(L::mul(c, L::all(-1.f)), u, dl);
                } else if (p.kind.mix == GCL_MIX_ROOT) {   // c (prev - u a / m), the second term 0 where m is
                    const P q = L::map(L::mul(a[k], L::all(-1.f)), m[k], [](float a, float m) { return m > 0.f ? a * frcp<T>(m) : 0.f; });
                    dl = L::mul(c, L::fma(q, u, prev[k]));
                }
                P dr = dl;
                if (p.kind.decay != GCL_DECAY_LOG) {
                    P sr, nr;
                    sigmoids<T>(row(0, k), sr, nr);
                    if (p.kind.decay == GCL_DECAY_SIGMOID) {
                        dr = L::mul(dl, nr);
                    } else {
                        const P part = L::mul(L::mul(dl, L::all(-1.f)), sr);
                        if (PLAIN || k < n) dsum = L::add(dsum, part);
                        dr = L::mul(L::mul(part, rate), nr);
                    }
                }
                if (PLAIN ? n_out > 0 : k < n_out) {
                    *to_x = L::put(dx);
                    *to_r = L::put(dr);
                    if (narr == 4) *to_i = L::put(di);
                }
                to_x -= p.dx.st / V;
                to_r -= p.dr.st / V;
                to_i -= p.di.st / V;
                if (!PLAIN && (starts >> k & 1)) store_state<T>(p.dh0, start[k], p.D, ch, c);
            }
        };
        if (!edge) run(std::true_type());
        else run(std::false_type());
        if (p.drate_part) {
            // (through the staged rows of r, which are read; the copies into them come after the next barrier)
            float (*s_d)[kRun * 32] = reinterpret_cast<float (*)[kRun * 32]>(s_rows + buf * narr * BYTES);
            __syncwarp();
            L::store(&s_d[warp][lane * V], dsum);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
            if (warp == 4 && tile.n > 0) {
                P sum = L::all(0.f);
#pragma unroll
                for (int w = 0; w < kWarpsB; ++w) sum = L::add(sum, L::load(&s_d[w][lane * V]));
                store_state<T>(p.drate_part, tile.t0 / W::TILE, p.D, ch, sum);
            }
        }
        if (!walk.more(buf)) break;
    }
    walk.finish();
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
    const int64_t tf = (a->t_max + kTileF - 1) / kTileF, tb = (a->t_max + kTileB - 1) / kTileB, tiles = backward ? tb : tf;
    const size_t row = sizeof(float) * (size_t)a->D;
    set(o.head, sizeof(Header));
    set(o.first, sizeof(int32_t) * (size_t)tiles);
    set(o.chain, sizeof(Packet) * (size_t)a->D * ((tiles + kRanks - 1) / kRanks));
    if (backward) {
        if (a->drate) set(o.drate_part, row * tiles);
        if (!a->h_save) set(o.h_save, row * tb);
    }
    return at;
}

// Tensor map of rows [t_max, D]: a tile by a warp's width of channels.
template <typename T>
bool rows_map(CUtensorMap *m, const Params &p, const Rows &r, int tile) {
    const cuuint64_t dims[2] = {(cuuint64_t)p.D, (cuuint64_t)p.t_max}, strides[1] = {(cuuint64_t)r.st * sizeof(T)};
    const cuuint32_t box[2] = {(cuuint32_t)Lane<T>::CB, (cuuint32_t)tile};
    const CUtensorMapDataType dt = sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return make_tensor_map(m, r.p, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE, dt);
}

// Launches the set-up and, as its dependent, `kernel` in clusters, at most `ctas` blocks an SM.
template <typename T, typename K>
cudaError_t launch_tiles(K kernel, const Params &p, const float *in_state, float *out_state, int warps, int ctas, cudaStream_t s) {
    const int tile = warps * kRun;
    Maps maps;
    const Rows *rows[4] = {&p.r, &p.x, &p.d_o, &p.i};
    int n = 0;
    for (int k = 0; k < 4; ++k)
        if (rows[k]->p) {
            if (!rows_map<T>(&maps.m[k], p, *rows[k], tile)) return cudaErrorInvalidValue;
            ++n;
        }
    const size_t smem = (size_t)2 * n * tile * 128;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t spans = (p.tiles + kRanks - 1) / kRanks, units = spans * p.n_cb, most = (int64_t)ctas * num_sms() / kRanks;
    int64_t setup = (spans * p.D + 4095) / 4096;
    if (out_state && setup < (p.n_max + 7) / 8) setup = (p.n_max + 7) / 8;
    if (setup > num_sms()) setup = num_sms();
    glr_setup_kernel<<<(unsigned)setup, 1024, 0, s>>>(p, in_state, out_state, tile);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((units < most ? units : most) * kRanks));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kRanks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t l = cudaLaunchKernelEx(&cfg, kernel, maps, p);
    return l != cudaSuccess ? l : cudaGetLastError();
}

template <typename T>
cudaError_t launch_fwd(const Params &p, cudaStream_t s) {
    return launch_tiles<T>(glr_fwd_kernel<T>, p, p.h0, p.ht, kWarpsF, kCtasF, s);
}

template <typename T>
cudaError_t launch_bwd(const Params &p, cudaStream_t s) {
    const cudaError_t e = launch_tiles<T>(glr_bwd_kernel<T>, p, p.dht, p.dh0, kWarpsB, kCtasB, s);
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
        f.o.p = f.d_o.p = nullptr;
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
