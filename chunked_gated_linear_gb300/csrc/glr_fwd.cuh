// glr_fwd.cuh -- gated linear recurrence, forward.
//
// XFWD
#pragma once

#include "glr_walk.cuh"

namespace gcl {
namespace glr {
namespace {

constexpr int kCtas = 3;                               // resident blocks an SM
static_assert(kTileF % kSave == 0, "saved states lie at tiles' starts");

template <typename T, int DECAY, int MIX, bool GATE>
__global__ void __launch_bounds__(32 * kWarps, kCtas) glr_fwd_kernel(const __grid_constant__ Maps maps, const Params p) {
    using L = Lane<T>;
    using P = typename L::P;
    using W = Walk<false, L::CB, kTileF / kWarps>;
    constexpr int V = L::V, CB = L::CB, RUN = kTileF / kWarps, BYTES = W::BYTES;
    __shared__ Shared<CB, RUN> s;
    __shared__ uint32_t s_tmem;
    extern __shared__ __align__(128) uint8_t s_rows[];     // [r, x, i][tile][128]
    constexpr int G = 8 / V, WORDS = RUN / G * 16, COLS = WORDS * kWarps / 4;        // words of a lane; columns of a block
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int narr = GATE ? 3 : 2;
    bool stop;
    const int64_t live = live_tokens(p, stop);
    if (live < 0) return;
    const int64_t tiles = (live + W::TILE - 1) / W::TILE;
    W walk{p, s, maps, s_rows, narr, live, tiles, (uint32_t)((tiles + kRanks - 1) / kRanks * p.n_cb), cluster_rank(), 0, 0, 0};
    if (warp == 0) {
        tc::tmem_alloc(&s_tmem, COLS);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    const bool some = walk.template start<T>(stop, p.h0, p.ht);
    tc::tc_fence_after();
    if (!some) {
        if (warp == 0) tc::tmem_dealloc(s_tmem, COLS);
        return;
    }
    const uint32_t words = s_tmem + ((warp & 3) << 21) + (warp >> 2) * WORDS;
    for (int buf = 0;; buf ^= 1) {
        const Tile<W::TILE> &tile = s.tile[buf];
        const int64_t t = tile.t0 + warp * RUN;
        const int ch = tile.cb * CB + lane * V, n = tile.n - warp * RUN;          // n: live tokens from the warp's first on
        const uint8_t *rows = s_rows + warp * RUN * 128 + lane * 4;
        auto row = [&](int arr, int k) { return L::get(*reinterpret_cast<const uint32_t *>(rows + arr * BYTES + k * 128)); };
        const P rate = load_state<T>(DECAY == GCL_DECAY_POWER ? p.kind.rate : nullptr, 0, p.D, ch);
        const bool near = __all_sync(0xffffffffu, L::every(rate, [](float v) { return v >= 0.f && v <= kNear; }));
        walk.landed(buf);
        // (the next span is taken only when this one's rows are here: few spans go to all clusters, and none is held back for long)
        const uint32_t taken = walk.take();
        const int32_t *start = tile.start + warp * RUN, *end = tile.end + warp * RUN;
        const uint32_t starts = bits_of<RUN>(tile.starts, warp), ends = bits_of<RUN>(tile.ends, warp);
        {
            P A = L::all(1.f), h = L::all(0.f);
#pragma unroll
            for (int k0 = 0; k0 < RUN; k0 += G) {
                P r[G], g[G], sg[G], a[G], b[G];
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    r[k] = row(0, k0 + k);
                    if (GATE) g[k] = row(2, k0 + k);
                }
                gates<T, DECAY, MIX, GATE, G>(rate, near, r, g, a, b, sg);
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    const P x = row(1, k0 + k);
                    b[k] = L::mul(b[k], GATE ? L::mul(x, sg[k]) : x);
                }
                if (n < k0 + G)
#pragma unroll
                    for (int k = 0; k < G; ++k)
                        if (k0 + k >= n) { a[k] = L::all(1.f); b[k] = L::all(0.f); }
                tmem_put<T>(words + k0 / G * 16, a, b);
                auto run = [&](auto cut) {
#pragma unroll
                    for (int k = 0; k < G; ++k) {
                        if (decltype(cut)::value && (starts >> (k0 + k) & 1)) h = load_state<T>(p.h0, start[k0 + k], p.D, ch);
                        h = L::fma(a[k], h, b[k]);
                        A = L::mul(A, a[k]);
                    }
                };
                if (starts >> k0 & ((1u << G) - 1)) run(std::true_type());
                else run(std::false_type());
            }
            L::store(&s.a[warp][lane * V], A);
            L::store(&s.b[warp][lane * V], h);
            tc::tmem_st_wait();
        }
        walk.exchange(buf, taken, tile.starts, [] {});
        P h = L::load(&s.b[warp][lane * V]);
        if (warp * RUN % kSave == 0 && p.h_save && n > 0) {
            if (starts & 1) h = load_state<T>(p.h0, start[0], p.D, ch);
            store_state<T>(p.h_save, t / kSave, p.D, ch, h);
        }
        uint32_t *to = word<T>(p.o, t, ch);
        const int n_out = p.o.p && ch < p.D && n > 0 && GCL_RANGE_IN_BOUNDS(t, t + (n < RUN ? n : RUN) - 1, p.t_max, p.status) ? n : 0;
        __align__(8) float v[2][16];
        tc::tmem_ld16(words, v[0]);
        auto run = [&](auto plain) {                       // plain: no borders, all tokens live
            constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
            for (int k0 = 0; k0 < RUN; k0 += G) {
                float *c = v[k0 / G % 2];
                tmem_wait<16>(c);
                if (k0 + G < RUN) tc::tmem_ld16(words + (k0 / G + 1) * 16, v[(k0 / G + 1) % 2]);
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    if (!PLAIN && (starts >> (k0 + k) & 1)) h = load_state<T>(p.h0, start[k0 + k], p.D, ch);
                    h = L::fma(L::load(c + k * V), h, L::load(c + 8 + k * V));
                    if (PLAIN ? n_out > 0 : k0 + k < n_out) *to = L::put(h);
                    to += p.o.st / V;
                    if (!PLAIN && (ends >> (k0 + k) & 1)) store_state<T>(p.ht, end[k0 + k], p.D, ch, h);
                }
            }
        };
        if (!(starts | ends) && n >= RUN) run(std::true_type());
        else run(std::false_type());
        if (!walk.more(buf)) break;
    }
    walk.finish();
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(s_tmem, COLS);
}

}  // namespace

template <typename T>
cudaError_t launch_fwd(const Params &p, cudaStream_t s) {
    return for_kind(p.kind.decay, p.kind.mix, p.i.p != nullptr, [&](auto d, auto m, auto g) {
        return launch_tiles<T, glr_fwd_kernel<T, decltype(d)::value, decltype(m)::value, decltype(g)::value>>(p, kCtas, 1, s);
    });
}

}  // namespace glr
}  // namespace gcl
