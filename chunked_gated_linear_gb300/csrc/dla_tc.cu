// dla_tc.cu -- decayed linear attention on the tensor cores: the engine of dla.cuh for bf16 rows.
//
// One CTA owns one segment of one (sequence, head) in one role and walks its chunks of C = 128 tokens.
// Per chunk, on tcgen05 with the 128 tokens (or the state's NA rows) on the MMA rows:
//   MMA1  X   = a b^T                       [C x C]   -> TMEM, decayed and masked to bf16 in place
//   MMA2  Oc  = a M                         [C x NV]  (M: the entering state in bf16)
//   MMA3  Oi  = X~ c                        [C x NV]  (A operand X~ from TMEM)
//   MMA4  D   = (w o b)^T c                 [NA x NV] w the decay to the chunk's far end
//   out = Oi + gamma^e Oc,   M <- gamma^len M + D     (fp32, M in registers)
// Precision.  X~, M and the result are rounded to bf16: X~ and M are MMA operands, and each output
// then carries about one operand rounding beside its own.  The state itself leaves the call in
// fp32, so its increments are formed to fp32: w o b is split into three bf16 terms (8 + 8 + 8 bits;
// two terms leave 2.6e-6 in the root mean square, three 1e-8), b's own bits are exact and c needs no
// rounding, so D is the fp32 sum of exact products.
//
// Bounds: per token and head with K = V = 128, 1 KiB of HBM traffic forwards and 2 C (NA + 2 NV) +
// 6 NA NV FLOPs (192 per byte, below the 281 of the measured peaks): HBM-bound, with the tensor
// pipe at two thirds of the time, so both have to run without a pause.  Hence one CTA per SM with
// every stage on warps of its own, joined by mbarriers only:
//   warps 0-7    score and output epilogues (a token per lane, half of the columns per warp)
//   warps 8-15   the split of b, the state (a state row per lane, half of the columns per warp)
//   warp 16      TMA loads, one chunk ahead: five tiles, three of the chunk and two of the next;
//                the third of the next goes where a was once MMA2 has read it
//   warp 17      MMA issue
// Shared memory at NA = NV = 128: 5 tiles of 32 KiB, two 64-token split terms of 16 KiB (the third
// overwrites b in place once MMA1 has read it), M 32 KiB.  TMEM: X, Oi, Oc, D, 128 columns each.
// Rows past the end are selected to zero in w o b and zeroed in c, so no other sequence's rows
// (or NaN padding) reach a sum.
#include <cudaTypedefs.h>

#include "dla.cuh"
#include "op16.cuh"
#include "tc_ptx.cuh"

namespace gcl {
namespace dla {
namespace {

using namespace tc;
using BF = __nv_bfloat16;
constexpr int C = 128;
constexpr int kWarpsA = 8, kWarpsB = 8;
constexpr int kTmaWarp = 16, kMmaWarp = 17;
constexpr int kEngineThreads = 18 * 32;
constexpr uint32_t cX = 0, cOi = 128, cOc = 256, cD = 384, kTmemCols = 512;

struct Maps {                      // q, k, v, d_o: boxes of 128 tokens x 64 channels of one head
    CUtensorMap m[4];
};

template <int NA, int NV>
struct TcLayout {
    static constexpr uint32_t slot = C * (NA > NV ? NA : NV) * 2;
    static constexpr uint32_t oMid = 5 * slot;             // [NA / 64][64 rows][128 B]
    static constexpr uint32_t oLo = oMid + 64 * NA * 2;
    static constexpr uint32_t oM = oLo + 64 * NA * 2;      // [NV / 64][NA rows][128 B]
    static constexpr uint32_t oP = oM + NA * NV * 2;       // gamma^0 .. gamma^C; then scaled
    static constexpr uint32_t total = oP + 2 * 132 * 4;
    static constexpr uint32_t bytes = total + 1024;        // + alignment slack
};

// Five tile slots in rotation: chunk c has b, a, c in (s[0], s[1], s[2]); the next chunk's b and a go
// to s[3], s[4] and its c to this chunk's a.
struct Slots {
    int s[5] = {0, 1, 2, 3, 4};
    __device__ __forceinline__ void next() {
        const int b = s[0], a = s[1], c = s[2];
        s[0] = s[3];
        s[1] = s[4];
        s[2] = a;
        s[3] = b;
        s[4] = c;
    }
};

// Bounded wait that does not look at the error word: for a copy or MMA still in flight after another
// wait gave up.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity) && globaltimer() - t0 < kWaitLimitNs) {}
}

struct Ctx {                       // what every warp of a CTA needs
    Item it;
    int h, role, nch;
    bool rev, trans, leaves;       // leaves: the last chunk's state is wanted
    __device__ __forceinline__ int64_t t0(int ic) const { return it.s0 + (int64_t)(rev ? nch - 1 - ic : ic) * C; }
    __device__ __forceinline__ int len(int ic) const {
        const int64_t n = it.s1 - t0(ic);
        return (int)(n < C ? n : C);
    }
};

// Splits rows [r0, r0 + 64) of the b tile: w_r b = hi + mid + lo, hi in place, mid and lo into 64-row
// buffers.  weight(r): the row's factor, selected to zero past the end.
template <int NA, int kThreads, typename F>
__device__ __forceinline__ void split_rows(uint8_t *b, uint8_t *mid, uint8_t *lo, int r0, int len, int tid, F weight) {
    constexpr int VR = NA / 8;
#pragma unroll
    for (int e0 = 0; e0 < 64 * VR; e0 += kThreads) {
        const int e = e0 + tid;
        if (64 * VR % kThreads != 0 && e >= 64 * VR) break;
        const int rr = e / VR, cv = e % VR, r = r0 + rr;
        const uint32_t sw = ((cv & 7) ^ (r & 7)) << 4;
        uint4 *hp = reinterpret_cast<uint4 *>(b + (cv >> 3) * (C * 128) + r * 128 + sw);
        const uint32_t off = (cv >> 3) * (64 * 128) + rr * 128 + sw;
        uint4 hi = make_uint4(0, 0, 0, 0), md = hi, lw = hi;
        if (r < len) {
            const float w = weight(r);
            float x[8], y[8];
            unpack8_as<BF>(*hp, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= w;
            hi = pack8_as<BF>(x);
            unpack8_as<BF>(hi, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] -= y[i];
            md = pack8_as<BF>(x);
            unpack8_as<BF>(md, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] -= y[i];
            lw = pack8_as<BF>(x);
        }
        *hp = hi;
        *reinterpret_cast<uint4 *>(mid + off) = md;
        *reinterpret_cast<uint4 *>(lo + off) = lw;
    }
}

// Rows [len, C) of the c tile to zero.
template <int NV, int kThreads>
__device__ __forceinline__ void zero_tail(uint8_t *c, int len, int tid) {
    for (int e = tid; e < C * (NV / 8); e += kThreads) {
        const int r = e / (NV / 8), cv = e % (NV / 8);
        if (r >= len) *reinterpret_cast<uint4 *>(c + (cv >> 3) * (C * 128) + r * 128 + (cv & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
}

// Half of MMA4: D (+)= (hi + mid + lo)^T c over 64 tokens.
template <int NV>
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t b, uint32_t mid, uint32_t lo, uint32_t c, int half, bool first) {
    constexpr uint32_t id = idesc_bf16(128, NV, 1, 1);
    const uint64_t dc = smem_desc(c + half * 8192, C * 128, 1024, kSwizzle128B);
    const uint64_t dh = smem_desc(b + half * 8192, C * 128, 1024, kSwizzle128B);
    const uint64_t dm = smem_desc(mid, 8192, 1024, kSwizzle128B), dl = smem_desc(lo, 8192, 1024, kSwizzle128B);
#pragma unroll
    for (int s = 0; s < 4; ++s) mma_bf16(d, dh + s * 128, dc + s * 128, id, !(first && s == 0));
#pragma unroll
    for (int s = 0; s < 4; ++s) mma_bf16(d, dm + s * 128, dc + s * 128, id, 1);
#pragma unroll
    for (int s = 0; s < 4; ++s) mma_bf16(d, dl + s * 128, dc + s * 128, id, 1);
}

__device__ __forceinline__ int map_of(int role, int operand) {   // operand 0: a, 1: b, 2: c -> q, k, v, d_o
    const uint32_t t = role == kFwd ? 0x210u : role == kDq ? 0x123u : role == kDv ? 0x301u : 0x032u;
    return (t >> (4 * operand)) & 15;
}

template <int NA, int NV>
__global__ void __launch_bounds__(kEngineThreads, 1) dla_tc_kernel(const __grid_constant__ Maps maps, const Params p) {
    using Lay = TcLayout<NA, NV>;
    constexpr int HV = NV / 2;                             // columns per warp of a pair
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ uint64_t full_b[2], full_a[2], full_c[2], bar_m1, bar_m2, bar_split[2], bar_m4[2], bar_p, bar_o, bar_ofree,
        bar_s, bar_end;
    __shared__ uint32_t s_tmem;
    __shared__ int s_err;
    if (status_blocks_cta(p.status)) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Ctx x;
    int bx = blockIdx.x;
    x.role = (p.roles >> (2 * (bx % p.n_roles))) & 3;
    bx /= p.n_roles;
    x.h = bx % p.H;
    const int64_t row = bx / p.H;
    if (!find_item<kEngineThreads>(p, row, x.it)) return;
    x.rev = x.role >= kDv;
    x.trans = x.role == kDq || x.role == kDk;
    x.nch = (int)((x.it.s1 - x.it.s0 + C - 1) / C);
    const bool rev = x.rev;
    const int nch = x.nch, h = x.h;
    const float g = p.g[h];
    const float s_state = rev ? 1.f : p.scale, s_inc = rev ? p.scale : 1.f;
    const int64_t KV = (int64_t)NA * NV, seq_state = ((int64_t)x.it.n * p.H + h) * KV;
    float *dst = x.role == kFwd && x.it.last ? p.ht : x.role == kDv && x.it.i == 0 ? p.dh0 : nullptr;
    if (dst) dst += seq_state;
    x.leaves = dst != nullptr;
    const float *src = rev ? p.seg_rev : p.seg_fwd;
    if (src) src += (row * p.H + h) * KV;
    else if ((src = rev ? p.dht : p.h0) != nullptr) src += seq_state;
    if (nch == 0) {                                        // an empty sequence passes its state on
        if (dst)
            for (int e = tid; e < NA * NV; e += kEngineThreads) dst[e] = src ? src[e] : 0.f;
        return;
    }

    float *sP = reinterpret_cast<float *>(smem + Lay::oP), *sPs = sP + 132;
    for (int e = tid; e <= C; e += kEngineThreads) {
        const float w = decay_pow(g, e);
        sP[e] = w;
        sPs[e] = p.scale * w;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full_b[i], 1);
            mbar_init(&full_a[i], 1);
            mbar_init(&full_c[i], 1);
            mbar_init(&bar_split[i], kWarpsB);
            mbar_init(&bar_m4[i], 1);
        }
        mbar_init(&bar_m1, 1);
        mbar_init(&bar_m2, 1);
        mbar_init(&bar_p, kWarpsA);
        mbar_init(&bar_o, 1);
        mbar_init(&bar_ofree, kWarpsA);
        mbar_init(&bar_s, kWarpsB);
        mbar_init(&bar_end, 1);
        s_err = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem, sbase = smem_u32(smem);
    // whether chunk ic's state is needed: by the next chunk or as the leaving state
    auto updates = [&](int ic) { return ic + 1 < nch || x.leaves; };

    if (warp == kTmaWarp) {
        if (lane == 0) {
            const CUtensorMap *ma = &maps.m[map_of(x.role, 0)], *mb = &maps.m[map_of(x.role, 1)], *mc = &maps.m[map_of(x.role, 2)];
            auto load = [&](const CUtensorMap *m, int slot, int D, int ic, uint64_t *bar) {
                mbar_arrive_expect_tx(bar, C * D * 2);
                for (int cb = 0; cb < D / 64; ++cb)
                    tma_load_3d(smem + slot * Lay::slot + cb * C * 128, m, cb * 64, h, (int)x.t0(ic), bar);
            };
            Slots sl;
            load(mb, sl.s[0], NA, 0, &full_b[0]);
            load(ma, sl.s[1], NA, 0, &full_a[0]);
            load(mc, sl.s[2], NV, 0, &full_c[0]);
            bool ok = true;
            int ic = 0;
            for (; ic + 1 < nch; ++ic) {                   // the next chunk's tiles
                const int b = (ic + 1) & 1;
                if (ic > 0) ok = mbar_wait(&bar_m4[1], (ic - 1) & 1, &s_err, 1);   // b and c of chunk ic - 1 are read
                if (!ok) break;
                load(mb, sl.s[3], NA, ic + 1, &full_b[b]);
                load(ma, sl.s[4], NA, ic + 1, &full_a[b]);
                ok = mbar_wait(&bar_m2, ic & 1, &s_err, 2);                        // a of chunk ic is read
                if (!ok) break;
                load(mc, sl.s[1], NV, ic + 1, &full_c[b]);
                sl.next();
            }
            if (!ok) {                                     // no copy may land after the CTA is gone
                for (int c = ic > 0 ? ic - 1 : 0; c <= ic; ++c) {
                    drain(&full_b[c & 1], (c >> 1) & 1);
                    drain(&full_a[c & 1], (c >> 1) & 1);
                    drain(&full_c[c & 1], (c >> 1) & 1);
                }
                drain(&full_b[(ic + 1) & 1], ((ic + 1) >> 1) & 1);
                drain(&full_a[(ic + 1) & 1], ((ic + 1) >> 1) & 1);
            }
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            Slots sl;
            for (int ic = 0; ic < nch; ++ic, sl.next()) {
                const uint32_t ph = ic & 1, fp = (ic >> 1) & 1, pv = (ic - 1) & 1;
                const uint32_t tb = sbase + sl.s[0] * Lay::slot, ta = sbase + sl.s[1] * Lay::slot, tcc = sbase + sl.s[2] * Lay::slot;
                const bool upd = updates(ic);
                if (!mbar_wait(&full_b[ph], fp, &s_err, 3) || !mbar_wait(&full_a[ph], fp, &s_err, 4)) break;
                if (ic > 0 && !mbar_wait(&bar_o, pv, &s_err, 5)) break;            // X~ is read
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < NA / 16; ++s) {
                    const uint32_t off = (s >> 2) * (C * 128) + (s & 3) * 32;
                    mma_bf16(tmem + cX, smem_desc(ta + off, 16, 1024, kSwizzle128B), smem_desc(tb + off, 16, 1024, kSwizzle128B),
                             idesc_bf16(128, 128), s > 0);
                }
                mma_commit(&bar_m1);
                if (!mbar_wait(&bar_s, ph, &s_err, 6)) break;                      // M in shared memory, D read
                if (ic > 0 && !mbar_wait(&bar_ofree, pv, &s_err, 7)) break;        // Oi, Oc read
                tc_fence_after();
                const uint64_t dm = smem_desc(sbase + Lay::oM, NA * 128, 1024, kSwizzle128B);
#pragma unroll
                for (int s = 0; s < NA / 16; ++s)
                    mma_bf16(tmem + cOc, smem_desc(ta + (s >> 2) * (C * 128) + (s & 3) * 32, 16, 1024, kSwizzle128B), dm + s * 128,
                             idesc_bf16(128, NV, 0, 1), s > 0);
                mma_commit(&bar_m2);
                if (!mbar_wait(&full_c[ph], fp, &s_err, 8) || !mbar_wait(&bar_split[0], ph, &s_err, 9)) break;
                tc_fence_after();
                if (upd) {
                    mma_state<NV>(tmem + cD, tb, sbase + Lay::oMid, sbase + Lay::oLo, tcc, 0, true);
                    mma_commit(&bar_m4[0]);
                }
                if (!mbar_wait(&bar_p, ph, &s_err, 10)) break;
                tc_fence_after();
                const uint64_t dc = smem_desc(tcc, C * 128, 1024, kSwizzle128B);
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_bf16_ta(tmem + cOi, tmem + cX + (s >> 2) * 64 + (s & 3) * 8, dc + s * 128, idesc_bf16(128, NV, 0, 1), s > 0);
                mma_commit(&bar_o);
                if (upd) {
                    if (!mbar_wait(&bar_split[1], ph, &s_err, 11)) break;
                    tc_fence_after();
                    mma_state<NV>(tmem + cD, tb, sbase + Lay::oMid, sbase + Lay::oLo, tcc, 1, false);
                    mma_commit(&bar_m4[1]);
                }
            }
            mma_commit(&bar_end);                          // every MMA issued has finished
            drain(&bar_end, 0);
        }
    } else if (warp < kWarpsA) {
        // ---- scores and outputs: token i of the chunk, columns half * 64 .. (scores), half * HV .. (out)
        const int quarter = warp & 3, half = warp >> 2, i = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const Rows ro = x.role == kFwd ? p.o : x.role == kDq ? p.dq : x.role == kDv ? p.dv : p.dk;
        for (int ic = 0; ic < nch; ++ic) {
            const uint32_t ph = ic & 1;
            const int len = x.len(ic);
            if (!mbar_wait(&bar_m1, ph, &s_err, 12)) break;
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j0 = half * 64 + u * 16;
                uint32_t pk[8];
                // (a block of 16 columns that the mask leaves empty for the warp's 32 rows is zeros)
                if (rev ? j0 + 15 < quarter * 32 || j0 >= len : j0 > quarter * 32 + 31) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) pk[e] = 0;
                } else {
                    float d[16];
                    tmem_ld16(tmem + lane_off + cX + j0, d);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int j = j0 + e, n = rev ? j - i : i - j;
                        d[e] = n >= 0 && (!rev || j < len) ? d[e] * sPs[n] : 0.f;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) pk[e] = Op16<BF>::pack2(d[2 * e], d[2 * e + 1]);
                }
                tmem_st8_b32(tmem + lane_off + cX + half * 64 + u * 8, pk);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_p);
            if (!mbar_wait(&bar_o, ph, &s_err, 13)) break;
            tc_fence_after();
            uint32_t out[HV / 2];
            const float f = s_state * sP[i < len ? (rev ? len - 1 - i : i + 1) : 0];
#pragma unroll
            for (int u = 0; u < HV / 16; ++u) {
                float a[16], b[16];
                tmem_ld16(tmem + lane_off + cOi + half * HV + u * 16, a);
                tmem_ld16(tmem + lane_off + cOc + half * HV + u * 16, b);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    out[u * 8 + e] = Op16<BF>::pack2(fmaf(f, b[2 * e], a[2 * e]), fmaf(f, b[2 * e + 1], a[2 * e + 1]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_ofree);
            const int64_t t = x.t0(ic) + i;
            if (ro.p && i < len && GCL_IN_BOUNDS(t, p.t_max, p.status)) {
                uint4 *o = reinterpret_cast<uint4 *>(row_ptr<BF>(ro, t, h) + half * HV);
#pragma unroll
                for (int u = 0; u < HV / 8; ++u) o[u] = make_uint4(out[4 * u], out[4 * u + 1], out[4 * u + 2], out[4 * u + 3]);
            }
        }
    } else {
        // ---- the state: row m, columns half * HV ..; the split of b
        const int bt = tid - kWarpsA * 32, quarter = warp & 3, half = (warp - kWarpsA) >> 2, m = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const bool mine = m < NA;
        float S[HV];
        if (src && mine) {
            if (x.trans) {                                 // element (r, c) at c * NA + r
#pragma unroll
                for (int j = 0; j < HV; ++j) S[j] = src[(int64_t)(half * HV + j) * NA + m];
            } else {
#pragma unroll
                for (int j = 0; j < HV; j += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(src + (int64_t)m * NV + half * HV + j);
                    S[j] = v.x; S[j + 1] = v.y; S[j + 2] = v.z; S[j + 3] = v.w;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < HV; ++j) S[j] = 0.f;
        }
        // M in bf16 for MMA2: rows m, 64-column blocks
        auto publish = [&]() {
            if (mine) {
#pragma unroll
                for (int j = 0; j < HV; j += 8) {
                    const int c = half * HV + j;
                    *reinterpret_cast<uint4 *>(smem + Lay::oM + (c >> 6) * (NA * 128) + m * 128 + ((((c & 63) >> 3) ^ (m & 7)) << 4)) =
                        pack8_as<BF>(S + j);
                }
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_s);
        };
        publish();
        Slots sl;
        for (int ic = 0; ic < nch; ++ic, sl.next()) {
            const uint32_t ph = ic & 1, fp = (ic >> 1) & 1;
            const int len = x.len(ic);
            const bool upd = updates(ic);
            uint8_t *tb = smem + sl.s[0] * Lay::slot, *tcc = smem + sl.s[2] * Lay::slot;
            if (len < C) {
                if (!mbar_wait(&full_c[ph], fp, &s_err, 14)) break;
                zero_tail<NV, kWarpsB * 32>(tcc, len, bt);
            }
            auto weight = [&](int r) { return s_inc * sP[rev ? r + 1 : len - 1 - r]; };
            if (upd) {
                if (!mbar_wait(&full_b[ph], fp, &s_err, 15) || !mbar_wait(&bar_m1, ph, &s_err, 16)) break;
                split_rows<NA, kWarpsB * 32>(tb, smem + Lay::oMid, smem + Lay::oLo, 0, len, bt, weight);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_split[0]);
            if (!upd) break;
            if (!mbar_wait(&bar_m4[0], ph, &s_err, 17)) break;                     // mid and lo are read
            split_rows<NA, kWarpsB * 32>(tb, smem + Lay::oMid, smem + Lay::oLo, 64, len, bt, weight);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_split[1]);
            if (!mbar_wait(&bar_m4[1], ph, &s_err, 18)) break;
            tc_fence_after();
            const float gl = sP[len];
#pragma unroll
            for (int u = 0; u < HV / 16; ++u) {
                float d[16];
                tmem_ld16(tmem + lane_off + cD + half * HV + u * 16, d);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) S[u * 16 + e] = fmaf(gl, S[u * 16 + e], d[e]);
            }
            if (ic + 1 < nch) {
                publish();
            } else if (dst && mine) {
#pragma unroll
                for (int j = 0; j < HV; j += 4)
                    *reinterpret_cast<float4 *>(dst + (int64_t)m * NV + half * HV + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
    if (tid == 0 && s_err != 0) status_set(p.status, GCL_DEV_WAIT_TIMEOUT);
}

// ---------------------------------------------------------------- the segments' own states
// sum_j gamma^(distance to the segment's end) b_j c_j^T over one segment: MMA4 alone, with the decay
// taken to the segment's end, so that the sum stays in TMEM until the last chunk.  Warps 0-15 split b
// (64 tokens at a time, two buffers), warp 16 loads, warp 17 issues.  b, c: two tiles each.
constexpr int kOwnWarps = 16;

template <int NA, int NV>
struct OwnLayout {
    static constexpr uint32_t sb = C * NA * 2, sc = C * NV * 2;
    static constexpr uint32_t oB = 0, oC = 2 * sb, oMid = oC + 2 * sc;             // mid[2], lo[2]
    static constexpr uint32_t part = 64 * NA * 2;
    static constexpr uint32_t total = oMid + 4 * part + (NA == 64 ? 8192 : 0);     // (MMA4 reads 128 rows)
    static constexpr uint32_t bytes = total + 1024;
};

template <int NA, int NV>
__global__ void __launch_bounds__(kEngineThreads, 1) dla_own_kernel(const __grid_constant__ Maps maps, const Params p) {
    using Lay = OwnLayout<NA, NV>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ uint64_t full[2], bar_split[2], bar_m4[2], bar_end;
    __shared__ uint32_t s_tmem;
    __shared__ int s_err;
    if (status_blocks_cta(p.status)) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Ctx x;
    int bx = blockIdx.x;
    x.role = (p.roles >> (2 * (bx % p.n_roles))) & 3;
    bx /= p.n_roles;
    x.h = bx % p.H;
    const int64_t row = bx / p.H;
    if (!find_item<kEngineThreads>(p, row, x.it)) return;
    x.rev = x.role >= kDv;
    if (x.rev ? x.it.i == 0 : x.it.last) return;           // no later (earlier) segment reads it
    const bool rev = x.rev;
    const int h = x.h, nch = x.nch = (int)((x.it.s1 - x.it.s0 + C - 1) / C);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&bar_split[i], kOwnWarps);
            mbar_init(&bar_m4[i], 1);
        }
        mbar_init(&bar_end, 1);
        s_err = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem, sbase = smem_u32(smem);
    if (warp == kTmaWarp) {
        if (lane == 0) {
            const CUtensorMap *mb = &maps.m[map_of(x.role, 1)], *mc = &maps.m[map_of(x.role, 2)];
            int ic = 0;
            for (; ic < nch; ++ic) {
                const int s = ic & 1;
                if (ic >= 2 && !mbar_wait(&bar_m4[1], ic & 1, &s_err, 1)) break;   // chunk ic - 2 is read
                mbar_arrive_expect_tx(&full[s], C * (NA + NV) * 2);
                for (int cb = 0; cb < NA / 64; ++cb)
                    tma_load_3d(smem + Lay::oB + s * Lay::sb + cb * C * 128, mb, cb * 64, h, (int)x.t0(ic), &full[s]);
                for (int cb = 0; cb < NV / 64; ++cb)
                    tma_load_3d(smem + Lay::oC + s * Lay::sc + cb * C * 128, mc, cb * 64, h, (int)x.t0(ic), &full[s]);
            }
            if (ic < nch)                                  // no copy may land after the CTA is gone
                for (int c = ic >= 2 ? ic - 2 : 0; c < ic; ++c) drain(&full[c & 1], (c >> 1) & 1);
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int ic = 0; ic < nch; ++ic) {
                const int s = ic & 1;
                bool ok = mbar_wait(&full[s], (ic >> 1) & 1, &s_err, 2);
                for (int hf = 0; hf < 2 && ok; ++hf) {
                    ok = mbar_wait(&bar_split[hf], ic & 1, &s_err, 3);
                    if (!ok) break;
                    tc_fence_after();
                    mma_state<NV>(tmem, sbase + Lay::oB + s * Lay::sb, sbase + Lay::oMid + hf * Lay::part,
                                  sbase + Lay::oMid + (2 + hf) * Lay::part, sbase + Lay::oC + s * Lay::sc, hf, ic == 0 && hf == 0);
                    mma_commit(&bar_m4[hf]);
                }
                if (!ok) break;
            }
            mma_commit(&bar_end);
            drain(&bar_end, 0);
        }
    } else {
        const float g = p.g[h], s_inc = rev ? p.scale : 1.f;
        bool ok = true;
        for (int ic = 0; ic < nch && ok; ++ic) {
            const int s = ic & 1, len = x.len(ic);
            const int64_t t0 = x.t0(ic);
            ok = mbar_wait(&full[s], (ic >> 1) & 1, &s_err, 4);
            if (!ok) break;
            if (len < C) zero_tail<NV, kOwnWarps * 32>(smem + Lay::oC + s * Lay::sc, len, tid);
            auto weight = [&](int r) { return s_inc * decay_pow(g, rev ? t0 + r - x.it.s0 + 1 : x.it.s1 - 1 - t0 - r); };
            for (int hf = 0; hf < 2; ++hf) {
                if (ic > 0 && !(ok = mbar_wait(&bar_m4[hf], (ic - 1) & 1, &s_err, 5))) break;
                split_rows<NA, kOwnWarps * 32>(smem + Lay::oB + s * Lay::sb, smem + Lay::oMid + hf * Lay::part,
                                               smem + Lay::oMid + (2 + hf) * Lay::part, hf * 64, len, tid, weight);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_split[hf]);
            }
        }
        if (ok && mbar_wait(&bar_m4[1], (nch - 1) & 1, &s_err, 6)) {
            tc_fence_after();
            const int quarter = warp & 3, q4 = warp >> 2, m = quarter * 32 + lane;
            float *dst = (rev ? p.seg_rev : p.seg_fwd) + (row * p.H + h) * (int64_t)(NA * NV) + (int64_t)m * NV + q4 * (NV / 4);
#pragma unroll
            for (int u = 0; u < NV / 4; u += 16) {
                float d[16];
                tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + q4 * (NV / 4) + u, d);
                tmem_ld_wait();
                if (m < NA) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4 *>(dst + u + j) = make_float4(d[j], d[j + 1], d[j + 2], d[j + 3]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 128);
    if (tid == 0 && s_err != 0) status_set(p.status, GCL_DEV_WAIT_TIMEOUT);
}

bool make_map(CUtensorMap *m, const Rows &r, int D, int H, int64_t t_max) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)t_max};
    const cuuint64_t strides[2] = {(cuuint64_t)r.sh * 2, (cuuint64_t)r.st * 2};
    const cuuint32_t box[3] = {64, 1, C};
    return make_tensor_map(m, r.p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int NA, int NV>
cudaError_t launch_one(const Maps &maps, const Params &p, bool own_states, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.n_rows * p.H * p.n_roles);
    if (own_states) {
        cudaError_t e = cudaFuncSetAttribute(dla_own_kernel<NA, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)OwnLayout<NA, NV>::bytes);
        if (e != cudaSuccess) return e;
        dla_own_kernel<NA, NV><<<grid, kEngineThreads, OwnLayout<NA, NV>::bytes, s>>>(maps, p);
    } else {
        cudaError_t e = cudaFuncSetAttribute(dla_tc_kernel<NA, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)TcLayout<NA, NV>::bytes);
        if (e != cudaSuccess) return e;
        dla_tc_kernel<NA, NV><<<grid, kEngineThreads, TcLayout<NA, NV>::bytes, s>>>(maps, p);
    }
    return cudaGetLastError();
}

}  // namespace

// Roles kFwd and kDv run on [K, V] states, kDq and kDk on [V, K]: one launch for each shape.
cudaError_t launch_tc(const Params &p0, bool own_states, int n_roles, const int *roles, cudaStream_t s) {
    Maps maps;
    bool ok = make_map(&maps.m[0], p0.q, p0.K, p0.H, p0.t_max) && make_map(&maps.m[1], p0.k, p0.K, p0.H, p0.t_max) &&
              make_map(&maps.m[2], p0.v, p0.V, p0.H, p0.t_max);
    if (p0.d_o.p) ok = ok && make_map(&maps.m[3], p0.d_o, p0.V, p0.H, p0.t_max);
    else maps.m[3] = maps.m[2];
    if (!ok) return cudaErrorInvalidValue;
    for (int shape = 0; shape < 2; ++shape) {
        Params p = p0;
        if (!take_roles(p, n_roles, roles, shape)) continue;
        const int na = shape == 0 ? p.K : p.V, nv = shape == 0 ? p.V : p.K;
        const cudaError_t e = na == 64 ? (nv == 64 ? launch_one<64, 64>(maps, p, own_states, s) : launch_one<64, 128>(maps, p, own_states, s))
                                       : (nv == 64 ? launch_one<128, 64>(maps, p, own_states, s) : launch_one<128, 128>(maps, p, own_states, s));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace dla
}  // namespace gcl
