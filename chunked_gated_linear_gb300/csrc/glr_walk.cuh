// glr_walk.cuh -- gated linear recurrence over packed sequences: how blocks walk the tiles, and the launch.
//
// The packed axis is cut into tiles of some tokens by the 128 bytes of a warp's width of channels; each warp of a block walks
// an eighth of a tile's tokens.  The sequences need no plan of their own: a token that starts one takes its state from h0,
// whatever was before.  One pass: a cluster of kRanks blocks takes kRanks consecutive tiles of the same channels (a span), in the
// order of the recurrence (a counter).  Its blocks form their tiles' products of decays and states from zero, exchange them
// through shared memory, and take the state that enters the span from the span before, or from an earlier one and the products and
// own states between; the sum is folded from the oldest on, so the result is the same whichever span had its state ready.
// A cluster waits for spans with lower numbers alone, whose clusters run already, so the first of them never waits: the
// launch ends whatever else runs on the GPU.
// The wait for the state before is what a tile spends longest on: spans meet in packets of 16 bytes, values and tag in one access
// (one sequence of 65,536 tokens of 2,048 channels: three launches, states from zero, their scan and the outputs, 1,424 us; one pass
// with a flag beside each state 655; packets, TMA copies of the rows and fp32 pairs 396; clusters of four, exchanging by shared memory, 342;
// sends that count on the receiver's barrier 312; kernels for each kind and 16 tokens a warp 251; clusters of two 246).
// Backwards from the states before each 64 tokens (saved by the forward, or formed again): with c_t = a_t G_t the gradient that
// token t passes on,
//   G_t = d_o_t + c_{t+1},   c_t = a_t G_t,
// the same recurrence with the same decays, cut where a sequence ends, over the tiles from last to first.
#pragma once

#include <atomic>

#include "glr.cuh"
#include "tc_ptx.cuh"

namespace gcl {
namespace glr {
namespace {

constexpr int kWarps = 8;                              // warps of a block; each walks tile / kWarps tokens
constexpr int kEnd = -1;

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
__device__ __forceinline__ void peer_store(void *p, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_addr(p, rank)), "r"(v) : "memory");
}
// Stores that count their bytes on the peer's barrier when they have landed there.
__device__ __forceinline__ void peer_send(void *p, uint64_t *bar, uint32_t rank, uint32_t v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(peer_addr(p, rank)), "r"(v),
                 "r"(peer_addr(bar, rank))
                 : "memory");
}
__device__ __forceinline__ void peer_send(void *p, uint64_t *bar, uint32_t rank, float a, float b, uint32_t c) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %3}, [%4];" ::"r"(peer_addr(p, rank)),
                 "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(c), "r"(peer_addr(bar, rank))
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
__device__ __forceinline__ void cluster_fence() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// ---- what a block holds of a tile beside its rows ----
template <int TILE>
struct Tile {
    int32_t seq, cb;               // its span's place in the order of the recurrence, its block of channels (kEnd: no tile, the walk is over)
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
        int f;
        if (p.first) {
            f = GCL_IN_BOUNDS(t.t0 / TILE, p.tiles, p.status) ? p.first[t.t0 / TILE] : 0;
        } else {                                           // first n with cu[n] >= t0 (n_max if none)
            int hi = p.n_max;
            f = 0;
            while (f < hi) {
                const int mid = (f + hi) >> 1;
                if (p.cu[mid] >= t.t0) hi = mid;
                else f = mid + 1;
            }
        }
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
// The bits of warp w's RUN tokens; whether there are any in the tile.
template <int RUN>
__device__ __forceinline__ uint32_t bits_of(const uint32_t *words, int w) {
    constexpr int PER = 32 / RUN;
    return words[w / PER] >> (w % PER * RUN) & ((1u << RUN) - 1);
}
template <int RUN>
__device__ __forceinline__ bool any_of(const uint32_t *words) {
    uint32_t a = 0;
#pragma unroll
    for (int k = 0; k < kWarps * RUN / 32; ++k) a |= words[k];
    return a != 0;
}

template <typename T>
__device__ __forceinline__ uint32_t *word(const Rows &r, int64_t t, int ch) {
    return reinterpret_cast<uint32_t *>(static_cast<T *>(r.p) + t * r.st + ch);
}

// A lane's values of row n of [rows, D]; zeros without the array or past the channels.
template <typename T>
__device__ __forceinline__ typename Lane<T>::P load_state(const Params &p, const float *s, int64_t n, int64_t rows, int ch) {
    return s && ch < p.D && GCL_IN_BOUNDS(n, rows, p.status) ? Lane<T>::load(s + n * p.D + ch) : Lane<T>::all(0.f);
}
template <typename T>
__device__ __forceinline__ void store_state(const Params &p, float *s, int64_t n, int64_t rows, int ch, typename Lane<T>::P h) {
    if (s && ch < p.D && GCL_IN_BOUNDS(n, rows, p.status)) Lane<T>::store(s + n * p.D + ch, h);
}
__device__ __forceinline__ int64_t save_rows(const Params &p) { return (p.t_max + kSave - 1) / kSave; }

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

// One warp, a channel a lane: packets of the spans before span `seq`, `depth` and depth + 1 back.
constexpr int kWindow = 2;                             // (65,536 tokens of 2,048 channels: 246 us; one 250, three 248, four 283)
__device__ __forceinline__ void load_window(const Params &p, int64_t seq, int depth, int ch, bool on, Packet *k) {
#pragma unroll
    for (int u = 0; u < kWindow; ++u) {
        const int64_t at = seq - 1 - depth - u;
        k[u].a = k[u].own = k[u].out = 0.f;
        k[u].tag = on ? 0 : kDone;
        if (on && at >= 0 && GCL_IN_BOUNDS(at, (p.tiles + kRanks - 1) / kRanks, p.status)) k[u] = load_packet(p.chain + at * p.D + ch);
    }
}
// The state that enters span `seq` (> 0): from the nearest span before it whose state is out for all the warp's channels, and the
// own states of the spans between, folded from the oldest on.  k: the first window.  False: it did not come in time, or another wait of
// the block's had run out (*err).
__device__ __forceinline__ bool chain_enter(const Params &p, int64_t seq, int ch, bool on, Packet *k, float &h, const int *err) {
    constexpr int W = kWindow;
    int depth = 0;
    uint64_t t0 = 0;
    while (true) {
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
            for (int d = depth - W; d >= 0; d -= W) {      // the spans nearer than these
                load_window(p, seq, d, ch, on, k);
#pragma unroll
                for (int u = W - 1; u >= 0; --u) h = fmaf(k[u].a, h, k[u].own);
            }
            return true;
        }
        depth = gap || depth >= 15 * W ? 0 : depth + W;
        if (t0 == 0) t0 = tc::globaltimer();
        // (lane 0's answer for all: they may see the error at different times)
        if (__shfl_sync(0xffffffffu, tc::globaltimer() - t0 > tc::kWaitLimitNs || *reinterpret_cast<const volatile int *>(err) != 0, 0)) return false;
        load_window(p, seq, depth, ch, on, k);
    }
}

template <int CB, int RUN>
struct Shared {
    float a[kWarps][CB], b[kWarps][CB];
    float4 sent_own[2][kRanks - 1][CB];    // product and own state of the blocks before (z: whether one is cut), by parity of the tile
    uint32_t next[2];              // the next span, by parity, from the first block; next[1] at first: the cluster's first
    uint64_t sent[2];              // these have come
    int lost;                      // exchanges since (and with) the one that the next span's number did not come in time for; 0: none
    Tile<kWarps * RUN> tile[2];
    int err;
    uint64_t full[2];
};

// One warp, a channel a lane (column c of s.a, s.b): from the warps' products and own states (in the order of the recurrence: from
// the first row, REV from the last) the block's, exchanged with the cluster's blocks; then the state that enters each row into s.b.
// `cuts`: a bit a token; a warp with one does not depend on the state before.  False: the state before did not
// come in time (s.err is set; then nothing is waited for any more).
template <bool REV, int CB, int RUN>
__device__ __forceinline__ bool chain_tile(const Params &p, int64_t seq, int ch, int c, uint32_t rank, int par, const uint32_t *cuts,
                                           Shared<CB, RUN> &s, uint32_t phase) {
    const bool on = ch < p.D, cut = any_of<RUN>(cuts);
    float a[kWarps], b[kWarps], A = 1.f, h = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const int w = REV ? kWarps - 1 - i : i;
        a[i] = s.a[w][c];
        b[i] = s.b[w][c];
    }
    if (!cut) {
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            h = fmaf(a[i], h, b[i]);
            A *= a[i];
        }
    } else {
        A = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) h = bits_of<RUN>(cuts, REV ? kWarps - 1 - i : i) ? b[i] : fmaf(a[i], h, b[i]);
    }
    for (uint32_t r = rank + 1; r < kRanks; ++r) peer_send(&s.sent_own[par][rank][c], &s.sent[par], r, A, h, cut);
    Packet k[kWindow];
    if (seq > 0) load_window(p, seq, 0, ch, on, k);        // (under way while the peers' states come)
    tc::mbar_wait(&s.sent[par], phase, &s.err, GCL_DEV_WAIT_TIMEOUT);
    Packet *mine = p.chain + seq * p.D + ch;
    // the blocks before this one, composed
    float A0 = 1.f, h0 = 0.f;
    bool ok = true, cut0 = false;
#pragma unroll
    for (int r = 0; r < kRanks - 1; ++r)
        if (r < rank) {
            const float4 t = s.sent_own[par][r][c];
            const bool q = __float_as_uint(t.z) != 0;
            cut0 |= q;
            h0 = q ? t.y : fmaf(t.x, h0, t.y);
            A0 *= t.x;
        }
    const bool speaks = rank == kRanks - 1 && on && p.first && GCL_IN_BOUNDS(seq, (p.tiles + kRanks - 1) / kRanks, p.status);
    const bool span_cut = cut || cut0;                     // (the last block speaks for the span)
    if (!cut) h = fmaf(A, h0, h);
    A *= A0;
    if (speaks) store_packet(mine, A, h, h, span_cut ? kDone : kOwn);
    float in = 0.f;
    if (seq > 0) ok = chain_enter(p, seq, ch, on, k, in, &s.err);          // (the first span is cut at its first token)
    if (speaks && !span_cut) store_packet(mine, A, h, fmaf(A, in, h), kDone);
    in = cut0 ? h0 : fmaf(A0, in, h0);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const int w = REV ? kWarps - 1 - i : i;
        s.b[w][c] = in;
        in = cut && bits_of<RUN>(cuts, w) ? b[i] : fmaf(a[i], in, b[i]);
    }
    return ok;
}

struct Maps {                      // the staged rows: r, x, d_o (backward), i
    CUtensorMap m[4];
};

constexpr uint32_t kStopped = 0xffffffffu;             // no span: the call does nothing, or the end
constexpr int kLeave = 3;                              // exchanges after which a block that lost the number leaves
constexpr int kIssuer = 96;        // the thread that takes spans and issues the copies

// Live tokens, once the set-up is done; -1: the call does nothing.  A solo call's blocks check cu_seqlens themselves; the status word
// is read by each cluster's first block alone (`stop`, in one thread: `start` tells the others), since it may change between two reads
// and a block that left alone would be sent to.  Every thread of the block (block barriers).
__device__ __forceinline__ int64_t live_tokens(const Params &p, bool &stop) {
    stop = false;
    grid_dependency_wait();
    if (p.first) return p.head->blocked ? -1 : p.head->live;
    int bad = 0;
    for (int n = threadIdx.x; n < p.n_max; n += blockDim.x) {
        const int b = p.cu[n], e = p.cu[n + 1];
        bad |= b < 0 || e < b || e > p.t_max || (n == 0 && b != 0);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == kIssuer && cluster_rank() == 0) {
        stop = p.status && *reinterpret_cast<volatile int32_t *>(p.status) != 0;
        if (bad && !stop) status_set(p.status, GCL_DEV_BAD_RANGE);
        if (blockIdx.x == 0) {                             // (for the sum of the rates' gradients)
            p.head->blocked = stop || bad;
            p.head->live = stop || bad ? 0 : p.cu[p.n_max];
        }
    }
    return bad ? -1 : p.cu[p.n_max];
}
// The states of empty sequences, of the block's channels (a solo call).
template <typename T>
__device__ __forceinline__ void pass_empty(const Params &p, const float *in_state, float *out_state) {
    if (!out_state) return;
    const int ch = (blockIdx.x / kRanks) * Lane<T>::CB + (threadIdx.x & 31) * Lane<T>::V;
    for (int n = blockIdx.x % kRanks * kWarps + (threadIdx.x >> 5); n < p.n_max; n += kRanks * kWarps)
        if (p.cu[n + 1] == p.cu[n]) store_state<T>(p, out_state, n, p.n_max, ch, load_state<T>(p, in_state, n, p.n_max, ch));
}

// A block's walk over its tiles, which both directions share.  Its next tile's rows are staged while one is computed.
template <bool REV, int CB, int RUN>
struct Walk {
    static constexpr int TILE = kWarps * RUN, BYTES = TILE * 128;
    const Params &p;
    Shared<CB, RUN> &s;
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
    // Sets up the barriers and takes the cluster's first span; false: there is none, or a solo call is to do nothing (`stop`, the first
    // block's issuer's).  Every thread of the cluster.
    template <typename T>
    __device__ __forceinline__ bool start(bool stop, const float *in_state, float *out_state) {
        const int tid = threadIdx.x;
        if (tid == kIssuer) {
            tc::mbar_init(&s.full[0], 1);
            tc::mbar_init(&s.full[1], 1);
            tc::mbar_init(&s.sent[0], 1);
            tc::mbar_init(&s.sent[1], 1);
            tc::fence_barrier_init();
            s.err = s.lost = 0;
            if (rank == 0) s.next[1] = p.first ? atomicAdd(&p.head->ticket, 1u) : stop ? kStopped : blockIdx.x / kRanks;
        }
        cluster_arrive();
        cluster_wait();
        const uint32_t unit = peer_load(&s.next[1], 0);
        if (!p.first && unit != kStopped) pass_empty<T>(p, in_state, out_state);
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
    // The first block takes the cluster's next span (its number reaches the others by the exchange); none after an error.
    __device__ __forceinline__ uint32_t take() {
        if (rank != 0 || threadIdx.x != kIssuer) return 0;
        return p.first && *reinterpret_cast<volatile int *>(&s.err) == 0 ? atomicAdd(&p.head->ticket, 1u) : units;
    }
    // Between a tile's halves: the warps' own states are in s.a, s.b; afterwards the states that enter them in s.b.
    // What a block receives at parity `buf` it has used when it arrives on the cluster's barrier, and the peers send there again
    // two tiles later, after they have waited on that barrier.
    // A block that the next span's number does not reach in time cannot know whether the first block goes on.  It sets that block's error,
    // before it arrives on the barrier behind which the exchange after this one lies, and takes part in two more with empty tiles, so that it
    // is still there to be sent to: the first block sees the error when it takes a span after the first of them, and ends with the
    // second (or did before).
    template <typename Side>
    __device__ __forceinline__ void exchange(int buf, uint32_t taken, const uint32_t *cuts, Side side) {
        static_assert(kRanks == 2, "a block that lost the number sends to no other");
        const int tid = threadIdx.x, warp = tid >> 5;
        const Tile<TILE> &t = s.tile[buf];
        const uint32_t ph = phase >> buf & 1;
        phase ^= 1u << buf;
        cluster_wait();
        if (tid == kIssuer) {
            if (rank == 0) s.next[buf] = taken;
            tc::mbar_arrive_expect_tx(&s.sent[buf], rank == 0 ? 0 : 4 + rank * CB * 16);
            if (rank == 0)
                for (int r = 1; r < kRanks; ++r) peer_send(&s.next[buf], &s.sent[buf], r, taken);
        }
        __syncthreads();
        if (warp < CB / 32) {
            if (!chain_tile<REV>(p, t.seq, t.cb * CB + tid, tid, rank, buf, cuts, s, ph)) atomicCAS(&s.err, 0, GCL_DEV_WAIT_TIMEOUT);
        } else if (warp == 2) {
            side();
        } else if (warp == kIssuer / 32) {
            const int before = *reinterpret_cast<volatile int *>(&s.lost);
            __syncwarp();
            // (by its own limit: an error elsewhere in the block does not cut it short)
            const bool come = __all_sync(0xffffffffu, tc::mbar_wait(&s.sent[buf], ph, &s.lost, 1)) && before == 0;
            if (!come || s.next[buf] < units) {
                if (tid == kIssuer) {
                    if (come) issue(s.next[buf], buf ^ 1);
                    else lose(before + 1, buf ^ 1);
                }
                __syncwarp();
                borders(p, s.tile[buf ^ 1]);
            } else if (tid == kIssuer) {
                s.tile[buf ^ 1].cb = kEnd;
            }
        }
        __syncthreads();
        cluster_arrive_relaxed();
    }
    // The issuer of a block that the number did not reach; exchanges: since then.
    __device__ __forceinline__ void lose(int exchanges, int buf) {
        atomicCAS(&s.err, 0, GCL_DEV_WAIT_TIMEOUT);
        s.lost = exchanges;
        if (exchanges == 1) {                              // (later the first block may have left)
            peer_store(&s.err, 0, GCL_DEV_WAIT_TIMEOUT);
            cluster_fence();                               // (the barrier is arrived on without one)
        }
        Tile<TILE> &t = s.tile[buf];
        t.seq = t.t0 = t.n = 0;
        t.cb = exchanges < kLeave ? p.n_cb : kEnd;         // (past the channels: nothing is read, written or waited for)
    }
    __device__ __forceinline__ bool more(int buf) const { return s.tile[buf ^ 1].cb != kEnd; }
    // After the last tile: a wait that ran out is reported; copies and what the peers sent are waited for (with a limit).
    __device__ __forceinline__ void finish() {
        cluster_wait();
        cluster_arrive();                                  // (no block leaves while another may send to it)
        cluster_wait();
        if (s.err == 0 || threadIdx.x != kIssuer) return;
        status_set(p.status, GCL_DEV_WAIT_TIMEOUT);
        const uint64_t t0 = tc::globaltimer();
        for (int b = 0; b < 2; ++b) {
            while ((issued >> (2 + b) & 1) && !tc::mbar_try_wait(&s.full[b], (issued >> b & 1) ^ 1) && tc::globaltimer() - t0 < tc::kWaitLimitNs) {}
            while (!tc::mbar_try_wait(&s.sent[b], (phase >> b & 1) ^ 1) && tc::globaltimer() - t0 < tc::kWaitLimitNs) {}
        }
    }
};

// Tensor map of rows [t_max, D]: a tile by a warp's width of channels.
template <typename T>
bool rows_map(CUtensorMap *m, const Params &p, const Rows &r, int tile) {
    const cuuint64_t dims[2] = {(cuuint64_t)p.D, (cuuint64_t)p.t_max}, strides[1] = {(cuuint64_t)r.st * sizeof(T)};
    const cuuint32_t box[2] = {(cuuint32_t)Lane<T>::CB, (cuuint32_t)tile};
    const CUtensorMapDataType dt = sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return make_tensor_map(m, r.p, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE, dt);
}

// Launches `kernel` in clusters, at most `ctas` blocks an SM, as the dependent of the launch before (the set-up, or the walk that
// forms the states).
template <typename T, auto kernel>
cudaError_t launch_tiles(const Params &p, int ctas, cudaStream_t s) {
    const int tile = p.tile;
    Maps maps;
    const Rows *rows[4] = {&p.r, &p.x, &p.d_o, &p.i};
    int n = 0;
    for (int k = 0; k < 4; ++k)
        if (rows[k]->p) {
            if (!rows_map<T>(&maps.m[k], p, *rows[k], tile)) return cudaErrorInvalidValue;
            ++n;
        }
    const size_t smem = (size_t)2 * n * tile * 128;
    static std::atomic<bool> allowed[64];                  // by device; zero-initialised (static storage)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !allowed[dev].load(std::memory_order_relaxed)) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) allowed[dev].store(true, std::memory_order_relaxed);
    }
    const int64_t spans = (p.tiles + kRanks - 1) / kRanks, units = spans * p.n_cb, most = (int64_t)ctas * num_sms() / kRanks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((units < most || !p.first ? units : most) * kRanks));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kRanks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.first ? 2 : 1;                        // (a solo call waits for whatever was before)
    e = cudaLaunchKernelEx(&cfg, kernel, maps, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace
}  // namespace glr
}  // namespace gcl
