// glr_fwd.cuh -- gated linear recurrence, forward.
//
// A warp's 16 tokens: gates (three special-function results and about 30 other instructions a value), their product of decays and
// state from zero; the state that enters from the walk's exchange; then the states, rounded, out.  Each row is read once
// and written once; a and b of the tokens stay in registers (64 of 128 a thread), which leaves two blocks an SM.  Bound by the exchange
// between spans beside the issue of 35 instructions a value (45% of slots): one sequence of 65,536 tokens of 2,048 channels, bf16, power
// decay, root mix, input gate 247 us, 64% of copy bandwidth; fp32, 32,768 tokens, 348 us, 45%.  Not kept: tiles of 64 tokens 333 to 375; a and b in tensor memory, three
// blocks an SM, 230 us, because a cluster whose blocks wait for each other's tensor memory can meet another stream's cluster that does the
// same, each holding what the other waits for; without clusters (16 warps a block) 239 us, but a call of 256 tokens 10.0 us instead of 8.0
// and short ones 16% longer.
#pragma once

#include "glr_walk.cuh"

namespace gcl {
namespace glr {
namespace {

constexpr int kCtas = 2;                               // resident blocks an SM (a and b of a tile are 64 registers a thread)
static_assert(kTileF % kSave == 0, "saved states lie at tiles' starts");

template <typename T, int DECAY, int MIX, bool GATE>
__global__ void __launch_bounds__(32 * kWarps, kCtas) glr_fwd_kernel(const __grid_constant__ Maps maps, const Params p) {
    using L = Lane<T>;
    using P = typename L::P;
    using W = Walk<false, L::CB, kTileF / kWarps>;
    constexpr int V = L::V, CB = L::CB, RUN = kTileF / kWarps, BYTES = W::BYTES;
    __shared__ Shared<CB, RUN> s;
    extern __shared__ __align__(128) uint8_t s_rows[];     // [2][r, x, i][tile][128]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int narr = GATE ? 3 : 2;
    bool stop;
    const int64_t live = live_tokens(p, stop);
    if (live < 0) return;
    const int64_t tiles = (live + W::TILE - 1) / W::TILE;
    W walk{p, s, maps, s_rows, narr, live, tiles, (uint32_t)((tiles + kRanks - 1) / kRanks * p.n_cb), cluster_rank(), 0, 0, 0};
    if (!walk.template start<T>(stop, p.h0, p.ht)) return;
    for (int buf = 0;; buf ^= 1) {
        const Tile<W::TILE> &tile = s.tile[buf];
        const int64_t t = tile.t0 + warp * RUN;
        const int ch = tile.cb * CB + lane * V, n = tile.n - warp * RUN;          // n: live tokens from the warp's first on
        const uint8_t *rows = s_rows + buf * narr * BYTES + warp * RUN * 128 + lane * 4;
        auto row = [&](int arr, int k) { return L::get(*reinterpret_cast<const uint32_t *>(rows + arr * BYTES + k * 128)); };
        const P rate = load_state<T>(p, DECAY == GCL_DECAY_POWER ? p.kind.rate : nullptr, 0, 1, ch);
        const bool near = __all_sync(0xffffffffu, L::every(rate, [](float v) { return v >= 0.f && v <= kNear; }));
        walk.landed(buf);
        // (the next span is taken only when this one's rows are here: few spans go to all clusters, and none is held back for long)
        const uint32_t taken = walk.take();
        P a[RUN], b[RUN];
        constexpr int H = 4;                               // tokens at a time (registers)
#pragma unroll
        for (int k0 = 0; k0 < RUN; k0 += H) {
            P r[H], g[H], sg[H];
#pragma unroll
            for (int k = 0; k < H; ++k) {
                r[k] = row(0, k0 + k);
                if (GATE) g[k] = row(2, k0 + k);
            }
            gates<T, DECAY, MIX, GATE, H>(rate, near, r, g, a + k0, b + k0, sg);
#pragma unroll
            for (int k = 0; k < H; ++k) {
                const P x = row(1, k0 + k);
                b[k0 + k] = L::mul(b[k0 + k], GATE ? L::mul(x, sg[k]) : x);
            }
        }
        if (n < RUN)
#pragma unroll
            for (int k = 0; k < RUN; ++k)
                if (k >= n) { a[k] = L::all(1.f); b[k] = L::all(0.f); }
        const int32_t *start = tile.start + warp * RUN, *end = tile.end + warp * RUN;
        const uint32_t starts = bits_of<RUN>(tile.starts, warp), ends = bits_of<RUN>(tile.ends, warp);
        {
            P A = L::all(1.f), h = L::all(0.f);
            auto run = [&](auto cut) {
#pragma unroll
                for (int k = 0; k < RUN; ++k) {
                    if (decltype(cut)::value && (starts >> k & 1)) h = load_state<T>(p, p.h0, start[k], p.n_max, ch);
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
            if (starts & 1) h = load_state<T>(p, p.h0, start[0], p.n_max, ch);
            store_state<T>(p, p.h_save, t / kSave, save_rows(p), ch, h);
        }
        uint32_t *to = word<T>(p.o, t, ch);
        const int n_out = p.o.p && ch < p.D && n > 0 && GCL_RANGE_IN_BOUNDS(t, t + (n < RUN ? n : RUN) - 1, p.t_max, p.status) ? n : 0;
        auto run = [&](auto plain) {                       // plain: no borders, all tokens live
            constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
            for (int k = 0; k < RUN; ++k) {
                if (!PLAIN && (starts >> k & 1)) h = load_state<T>(p, p.h0, start[k], p.n_max, ch);
                h = L::fma(a[k], h, b[k]);
                if (PLAIN ? n_out > 0 : k < n_out) *to = L::put(h);
                to += p.o.st / V;
                if (!PLAIN && (ends >> k & 1)) store_state<T>(p, p.ht, end[k], p.n_max, ch, h);
            }
        };
        if (!(starts | ends) && n >= RUN) run(std::true_type());
        else run(std::false_type());
        if (!walk.more(buf)) break;
    }
    walk.finish();
}

}  // namespace

template <typename T>
cudaError_t launch_fwd(const Params &p, cudaStream_t s) {
    return for_kind(p.kind.decay, p.kind.mix, p.i.p != nullptr, [&](auto d, auto m, auto g) {
        return launch_tiles<T, glr_fwd_kernel<T, decltype(d)::value, decltype(m)::value, decltype(g)::value>>(p, kCtas, s);
    });
}

}  // namespace glr
}  // namespace gcl
