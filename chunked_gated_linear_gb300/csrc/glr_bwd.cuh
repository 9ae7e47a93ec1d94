// glr_bwd.cuh -- gated linear recurrence, backward.
//
// Gradients of G_t = d_o_t + c_{t+1}, c_t = a_t G_t, over the tiles from last to first, together with the states again: a tile's come
// from the one saved before it.  The walk's exchange passes c.  A tile's rows stay staged until its gradients are out, and sigmoids are
// formed again for them; a, m and b (later the states) of a warp's eight tokens are 48 registers a thread.  Bound by issue (87
// instructions a value, 48% of slots) and the special-function unit, then by the exchange between spans: 32,768 tokens of 2,048 channels,
// bf16, with drate 277 us, 50% of copy bandwidth; fp32, 16,384 tokens, 348 us, 40%.  Not kept (beside 272 at that time): three blocks an SM (80 registers spill, 374 us); clusters of four (295); a, m,
// b and the sigmoids in tensor memory (261; the forward says why).
#pragma once

#include "glr_walk.cuh"

namespace gcl {
namespace glr {
namespace {

constexpr int kCtas = 2;                               // resident blocks an SM
static_assert(kTileB == kSave, "one saved state a tile");

template <typename T, int DECAY, int MIX, bool GATE>
__global__ void __launch_bounds__(32 * kWarps, kCtas) glr_bwd_kernel(const __grid_constant__ Maps maps, const Params p) {
    using L = Lane<T>;
    using P = typename L::P;
    using W = Walk<true, L::CB, kTileB / kWarps>;
    constexpr int V = L::V, CB = L::CB, RUN = kTileB / kWarps, BYTES = W::BYTES;
    __shared__ Shared<CB, RUN> s;
    __shared__ float s_h[kWarps][CB];
    extern __shared__ __align__(128) uint8_t s_rows[];     // [2][r, x, d_o, i][tile][128]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int narr = GATE ? 4 : 3;
    launch_dependents();                                   // (the sum of the rates' gradients waits for this grid's end)
    bool stop;
    const int64_t live = live_tokens(p, stop);
    if (live < 0) return;
    const int64_t tiles = (live + W::TILE - 1) / W::TILE;
    W walk{p, s, maps, s_rows, narr, live, tiles, (uint32_t)((tiles + kRanks - 1) / kRanks * p.n_cb), cluster_rank(), 0, 0, 0};
    if (!walk.template start<T>(stop, p.dht, p.dh0)) return;
    for (int buf = 0;; buf ^= 1) {
        const Tile<W::TILE> &tile = s.tile[buf];
        const int64_t t = tile.t0 + warp * RUN;
        const int ch = tile.cb * CB + lane * V, n = tile.n - warp * RUN;
        const uint8_t *rows = s_rows + buf * narr * BYTES + warp * RUN * 128 + lane * 4;
        auto row = [&](int arr, int k) { return L::get(*reinterpret_cast<const uint32_t *>(rows + arr * BYTES + k * 128)); };
        const P rate = load_state<T>(p, DECAY == GCL_DECAY_POWER ? p.kind.rate : nullptr, 0, 1, ch);
        const bool near = __all_sync(0xffffffffu, L::every(rate, [](float v) { return v >= 0.f && v <= kNear; }));
        P before = L::all(0.f);
        if (warp == 2 && tile.n > 0) before = load_state<T>(p, p.h_save, tile.t0 / kSave, save_rows(p), ch);
        walk.landed(buf);
        const uint32_t taken = walk.take();
        P a[RUN], m[RUN], prev[RUN];                       // prev: b = m u, later the state before each token
        constexpr int H = 4;                               // tokens at a time (registers)
#pragma unroll
        for (int k0 = 0; k0 < RUN; k0 += H) {
            P r[H], g[H], sg[H];
#pragma unroll
            for (int k = 0; k < H; ++k) {
                r[k] = row(0, k0 + k);
                if (GATE) g[k] = row(3, k0 + k);
            }
            gates<T, DECAY, MIX, GATE, H, true>(rate, near, r, g, a + k0, m + k0, sg);
#pragma unroll
            for (int k = 0; k < H; ++k) {
                const P x = row(1, k0 + k);
                prev[k0 + k] = L::mul(m[k0 + k], GATE ? L::mul(x, sg[k]) : x);
            }
        }
        if (n < RUN)
#pragma unroll
            for (int k = 0; k < RUN; ++k)
                if (k >= n) { a[k] = L::all(1.f); m[k] = prev[k] = L::all(0.f); }
        const int32_t *start = tile.start + warp * RUN, *end = tile.end + warp * RUN;
        const uint32_t starts = bits_of<RUN>(tile.starts, warp), ends = bits_of<RUN>(tile.ends, warp);
        const bool edge = (starts | ends) || n < RUN;
        {
            P A = L::all(1.f), h = L::all(0.f), c = L::all(0.f);
            auto run = [&](auto cut) {
                constexpr bool CUT = decltype(cut)::value;
#pragma unroll
                for (int k = 0; k < RUN; ++k) {
                    if (CUT && (starts >> k & 1)) h = load_state<T>(p, p.h0, start[k], p.n_max, ch);
                    h = L::fma(a[k], h, prev[k]);
                    A = L::mul(A, a[k]);
                }
#pragma unroll
                for (int k = RUN - 1; k >= 0; --k) {
                    if (CUT && (ends >> k & 1)) c = load_state<T>(p, p.dht, end[k], p.n_max, ch);
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
            for (int w = 0; w < kWarps; ++w) {
                const P b = L::load(&s_h[w][lane * V]), A = L::load(&s.a[w][lane * V]);
                L::store(&s_h[w][lane * V], before);
                before = bits_of<RUN>(tile.starts, w) ? b : L::fma(A, before, b);
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
                if (!PLAIN && (starts >> k & 1)) h = load_state<T>(p, p.h0, start[k], p.n_max, ch);
                const P b = prev[k];
                prev[k] = h;
                h = L::fma(a[k], h, b);
            }
#pragma unroll
            for (int k = RUN - 1; k >= 0; --k) {
                if (!PLAIN && (ends >> k & 1)) c = load_state<T>(p, p.dht, end[k], p.n_max, ch);
                const P x = row(1, k), G = L::add(row(2, k), c), Gm = L::mul(G, m[k]);
                c = L::mul(a[k], !PLAIN && k >= n ? c : G);
                P sr, nr, sg, ng;
                if (DECAY != GCL_DECAY_LOG && GATE && MIX == GCL_MIX_ONE) {           // (here dx does not depend on r's)
                    sigmoids<T>(row(0, k), sr, nr);
                    sigmoids<T>(row(3, k), sg, ng);
                } else if (DECAY != GCL_DECAY_LOG && GATE) sigmoids<T>(row(0, k), row(3, k), sr, nr, sg, ng);
                else if (DECAY != GCL_DECAY_LOG) sigmoids<T>(row(0, k), sr, nr);
                else if (GATE) sigmoids<T>(row(3, k), sg, ng);
                const P u = GATE ? L::mul(x, sg) : x, dx = GATE ? L::mul(Gm, sg) : Gm;
                P dl;
                if (MIX == GCL_MIX_ROOT) {                 // c (prev - u a / m), the second term 0 where m is
                    const P q = L::map(L::mul(a[k], L::all(-1.f)), m[k], [](float a, float m) { return m > 0.f ? a * frcp<T>(m) : 0.f; });
                    dl = L::mul(c, L::fma(q, u, prev[k]));
                } else {
                    dl = L::mul(c, MIX == GCL_MIX_COMPLEMENT ? L::fma(u, L::all(-1.f), prev[k]) : prev[k]);
                }
                P dr = dl;
                if (DECAY == GCL_DECAY_SIGMOID) dr = L::mul(dl, nr);
                if (DECAY == GCL_DECAY_POWER) {
                    const P part = L::mul(L::mul(dl, L::all(-1.f)), sr);
                    if (PLAIN || k < n) dsum = L::add(dsum, part);
                    dr = L::mul(L::mul(part, rate), nr);
                }
                if (PLAIN ? n_out > 0 : k < n_out) {
                    *to_x = L::put(dx);
                    *to_r = L::put(dr);
                    if (GATE) *to_i = L::put(L::mul(L::mul(dx, x), ng));
                }
                to_x -= p.dx.st / V;
                to_r -= p.dr.st / V;
                to_i -= p.di.st / V;
                if (!PLAIN && (starts >> k & 1)) store_state<T>(p, p.dh0, start[k], p.n_max, ch, c);
            }
        };
        if (!edge) run(std::true_type());
        else run(std::false_type());
        if (p.drate_part) {
            // (through the staged rows of r, which are read; the copies into them come after the next barrier)
            float (*s_d)[RUN * 32] = reinterpret_cast<float (*)[RUN * 32]>(s_rows + buf * narr * BYTES);
            __syncwarp();
            L::store(&s_d[warp][lane * V], dsum);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
            if (warp == 4 && tile.n > 0) {
                P sum = L::all(0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) sum = L::add(sum, L::load(&s_d[w][lane * V]));
                store_state<T>(p, p.drate_part, tile.t0 / W::TILE, p.tiles, ch, sum);
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
    // (the clusters of a call of one span look at the status word each for itself: one that stopped leaves no sums)
    if (p.head->blocked || (!p.first && status_blocks_cta(p.status))) return;
    const int64_t n = (p.head->live + tile - 1) / tile;
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (d < p.D)
        for (int64_t j0 = r; j0 < n; j0 += 8 * 32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = j0 + i * 32 < n && GCL_IN_BOUNDS(j0 + i * 32, p.tiles, p.status) ? p.drate_part[(j0 + i * 32) * p.D + d] : 0.f;
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

}  // namespace

template <typename T>
cudaError_t launch_bwd(const Params &p, cudaStream_t s) {
    const cudaError_t e = for_kind(p.kind.decay, p.kind.mix, p.i.p != nullptr, [&](auto d, auto m, auto g) {
        return launch_tiles<T, glr_bwd_kernel<T, decltype(d)::value, decltype(m)::value, decltype(g)::value>>(p, kCtas, s);
    });
    if (e != cudaSuccess || !p.drate) return e;
    return launch_dependent(glr_drate_kernel, dim3((p.D + 31) / 32), dim3(1024), 0, s, p, kTileB);
}

}  // namespace glr
}  // namespace gcl
