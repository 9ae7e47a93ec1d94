// dla_tc.cu -- decayed linear attention on the tensor cores: the engine of dla.cuh for bf16 rows.
//
// One CTA owns one segment of one (sequence, head) in one role and walks its chunks of C = 128 tokens.
// Per chunk, on tcgen05 with the 128 tokens (or the state's NA rows) on the MMA rows:
//   MMA1  X  = a b^T                        [C x C]   -> TMEM, decayed and masked to bf16 in place
//   MMA2  O  = a M                          [C x NV]  M: the entering state in bf16; then rows times gamma^e
//   MMA3  O += X~ c                         [C x NV]  (A operand X~ from TMEM)
//   MMA4  D  = (w o b)^T c                  [NA x NV] w the decay to the chunk's far end (A from TMEM)
//   out = O,   M <- gamma^len M + D         (fp32, M in registers)
// Precision.  X~, M and the result are rounded to bf16: X~ and M are MMA operands, and each output
// then carries about one operand rounding beside its own.  A state that leaves the call does so in
// fp32, so its increments are formed to fp32: w o b is split into three bf16 terms (8 + 8 + 8 bits;
// two terms leave 2.6e-6 in the root mean square, three 1e-8), b's own bits are exact and c needs no
// rounding, so D is the fp32 sum of exact products.  In the roles whose state never leaves (DQ, DK)
// it only feeds MMA2, which rounds it to 8 bits, and two terms do.
//
// Bounds: per token and head with K = V = 128, 1 KiB of HBM traffic forwards and 2 C (NA + NV) +
// (2 + 2 terms) NA NV FLOPs (192 per byte, below the 281 of the measured peaks): HBM-bound, with the
// tensor pipe at two thirds of the time, so both have to run without a pause.  Hence one CTA per SM
// with every stage on warps of its own, joined by mbarriers only:
//   warps 0-3    score and output epilogues (a token per lane)
//   warps 4-11   the split of b, 32 tokens at a time into two TMEM buffers, and the state (a row per
//                lane, half of the columns per warp)
//   warp 12      MMA issue: MMA2, three quarters of MMA4, MMA3, the last quarter, the next chunk's MMA1
//   warp 13      TMA loads, one chunk ahead: five tiles, three of the chunk and two of the next;
//                the third of the next goes where a was once MMA2 has read it
// (128 registers a thread: what spills misses the little L1 that 224 KiB of shared memory leave, and
// with 96 registers those misses took more time than the arithmetic.  At NV = 128 12 registers a thread still
// spill, 48 to 52 bytes; at NV = 64 none.)
// What an MMA of this shape reads from shared memory (A and B, 8 KiB in 64 cycles) fills its port, so
// everything else that goes through it waits: the split terms therefore go to TMEM, and outputs and
// states cross a staging tile to leave and enter in whole lines (a lane per row touches 32 lines with
// every 16-byte access: 2,048 cycles of the load-store pipe a chunk).
// Measured: 33,000 tokens in 32 sequences of 16 heads, 146 us, 4.6 TB/s; a chunk takes 6,600 to 6,800 cycles, of which
// HBM alone would need 5,570 and the 48 MMAs 3,200.  The issuing warp sets that pace: beside the epilogues' TMEM
// and shared-memory traffic an MMA takes about 100 cycles, alone 66.  (Two issuing warps, one of them for
// MMA4: the same time.)
// Shared memory at NA = NV = 128: 5 tiles, the staging tile and M, 32 KiB each.  TMEM: X, O, D and
// the two split buffers, 128 columns each.
// Rows past the end are selected to zero in w o b and zeroed in c, so no other sequence's rows
// (or NaN padding) reach a sum.  Within a sequence masked scores are zeros, which a row of c that is not finite
// turns into NaN for its whole chunk; an infinite b gives NaN in the state (its terms are inf and inf - inf).
#include <cudaTypedefs.h>

#include "dla.cuh"
#include "f32x2.cuh"
#include "op16.cuh"
#include "tc_ptx.cuh"

namespace gcl {
namespace dla {
namespace {

using namespace tc;
using BF = __nv_bfloat16;
constexpr int C = 128;
constexpr int kWarpsA = 4, kWarpsB = 8;
constexpr int kMmaWarp = kWarpsA + kWarpsB, kTmaWarp = kMmaWarp + 1;
constexpr int kEngineThreads = 14 * 32;

constexpr int kRows = 32;                                  // tokens per step of the split
constexpr uint32_t cX = 0, cO = 128, cD = 256, cSplit = 384, kTmemCols = 512;
constexpr uint32_t kTermCols = kRows / 2;                  // columns of a split term (two tokens each)

struct Maps {                      // q, k, v, d_o: boxes of 128 tokens x 64 channels of one head;
    CUtensorMap m[4], out[3];      // the outputs of the roles: boxes of 32 tokens x 64 channels
};

template <int NA, int NV>
struct TcLayout {
    static constexpr uint32_t slot = C * (NA > NV ? NA : NV) * 2;
    static constexpr uint32_t oStage = 5 * slot;           // outputs on their way out: [4 warps][NV / 64][32 rows][128 B]
    static constexpr uint32_t oM = oStage + C * NV * 2;    // [NV / 64][NA rows][128 B]
    static constexpr uint32_t oP = oM + NA * NV * 2;       // gamma^0 .. gamma^C; over a block of 32; MMA4's w,
                                                           // in a whole chunk and in the segment's short one
    static constexpr uint32_t total = oP + (132 + 32 + 2 * C) * 4;
    static constexpr uint32_t bytes = total + 1024;        // + alignment slack
    static_assert(NA * NV * 4 <= C * NV * 2 + NA * NV * 2, "an fp32 state fits the staging tile and M");
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

// Bounded wait with a suspend time, so that waiting warps stay off the issue slots and the
// shared-memory pipe that the working warps need.
__device__ __forceinline__ bool try_bar(uint32_t at, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(at), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint32_t timer_lo() {            // nanoseconds, modulo 4.3 s
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
__device__ __forceinline__ bool wait_more(uint32_t at, uint32_t parity, int *err, int code) {
    const uint32_t t0 = timer_lo();
    while (true) {
        if (try_bar(at, parity)) return true;
        if (*reinterpret_cast<volatile int *>(err) != 0) return false;
        if (timer_lo() - t0 > (uint32_t)kWaitLimitNs) {
            atomicCAS(err, 0, code);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, int *err, int code) {
    const uint32_t at = smem_u32(bar);
    return mbar_test(bar, parity) || wait_more(at, parity, err, code);
}
// The same for a whole warp, which then takes one way: a wait that gave up in some lanes only would
// leave the others at the warp's next barrier.  (A phase that is complete already costs one probe and one
// vote; the polling loop is out of the way of the code that follows.)
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, int *err, int code) {
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_test(bar, parity)), 1)) return true;
    return __all_sync(0xffffffffu, wait_more(smem_u32(bar), parity, err, code));
}

// Barrier N of the block over `threads` threads.
template <int N>
__device__ __forceinline__ void named_sync(int threads) { asm volatile("bar.sync %0, %1;" ::"n"(N), "r"(threads) : "memory"); }

// Bounded wait that does not look at the error word: for a copy or MMA still in flight after another
// wait gave up.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity) && globaltimer() - t0 < kWaitLimitNs) {}
}

// Lane 0's value, known to be the same in every lane.
template <typename T>
__device__ __forceinline__ T uniform(T v) { return __shfl_sync(0xffffffffu, v, 0); }

struct Ctx {                       // what every warp of a CTA needs of its work (32 bits: few registers)
    int n, i, s0, s1, h, role, nch;
    bool rev, leaves;              // leaves: the last chunk's state is wanted
    __device__ __forceinline__ int t0(int ic) const { return s0 + (rev ? nch - 1 - ic : ic) * C; }
    __device__ __forceinline__ int len(int ic) const {
        const int n = s1 - t0(ic);
        return n < C ? n : C;
    }
    // Three split terms in the roles whose state can leave; two in the others.  (By the role alone: o has
    // the same bits whether ht is asked for or not.)
    __device__ __forceinline__ bool three() const { return role == kFwd || role == kDv; }
    // The role, head and segment of block b; false: nothing to do.
    // (Its values are made uniform, so that code on them stays convergent.)
    template <int kBlock, bool kOwn>
    __device__ __forceinline__ bool find(const Params &p, int b, int &row, bool &last) {
        role = (p.roles >> (2 * (b % p.n_roles))) & 3;
        b /= p.n_roles;
        h = b % p.H;
        rev = role >= kDv;
        Item it = {};
        const bool ok = find_item<kBlock, kOwn>(p, b / p.H, rev, it);
        row = uniform((int)it.row);
        n = uniform(it.n);
        i = uniform(it.i);
        s0 = uniform((int)it.s0);
        s1 = uniform((int)it.s1);
        last = uniform((int)it.last) != 0;
        nch = (s1 - s0 + C - 1) / C;
        return ok;
    }
};

// Two fp32 values (f32x2.cuh) to and from two bf16 ones.
__device__ __forceinline__ uint32_t pack(uint64_t a) {
    const float2 f = unpair(a);
    return Op16<BF>::pack2(f.x, f.y);
}
__device__ __forceinline__ uint64_t unpack(uint32_t w) {
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// 16 lanes x 8 columns: registers 0, 1 hold columns 0-3 of lanes 0-7 and 8-15 (thread t: lane t / 4, column
// t % 4), registers 2, 3 columns 4-7.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]) : "memory");
}

// Splits tokens [r0, r0 + 16) of channels [m0, m0 + 32) of the b tile (one warp): w_r b = hi + mid + lo, two
// tokens to a 32-bit column, each term's 8 columns at taddr + term * kTermCols (the caller waits for
// the stores).  w: the weights of the 16 tokens.  Tokens past the end are selected to zero.
// Transposed matrix loads give each thread token pairs of one channel, in the fragments that the
// 16 x 128-bit TMEM store takes (lane = channel).
template <int NA>
__device__ __forceinline__ void split16(uint32_t b, int m0, int r0, int len, const float *w, uint32_t taddr, bool three) {
    const int lane = threadIdx.x & 31, ch = ((m0 & 63) >> 3) + (lane >> 3);
    const uint32_t row = b + (m0 >> 6) * (C * 128) + (r0 + (lane & 7)) * 128 + ((ch ^ (lane & 7)) << 4);
    const uint64_t minus = pair(-1.f, -1.f);
    uint32_t x8[2][4];                                     // [8 tokens][8 channels]
    uint64_t w2[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x8[t][0]), "=r"(x8[t][1]), "=r"(x8[t][2]), "=r"(x8[t][3]) : "r"(row + t * 1024) : "memory");
        const int r = t * 8 + (lane & 3) * 2;
        const float2 wv = *reinterpret_cast<const float2 *>(w + r);
        w2[t] = pair(wv.x, wv.y);
        if (r0 + 16 > len) {
            const uint32_t keep = (r0 + r < len ? 0xffffu : 0u) | (r0 + r + 1 < len ? 0xffff0000u : 0u);
#pragma unroll
            for (int c = 0; c < 4; ++c) x8[t][c] &= keep;
        }
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {                          // channels 0-15, 16-31
        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {                      // (token group e / 2, channels 8 (2 g + e % 2) ..)
            uint64_t x = mul2(unpack(x8[e >> 1][2 * g + (e & 1)]), w2[e >> 1]);
            hi[e] = pack(x);
            x = fma2(unpack(hi[e]), minus, x);
            mid[e] = pack(x);
            x = fma2(unpack(mid[e]), minus, x);
            lo[e] = pack(x);
        }
        const uint32_t at = taddr + (uint32_t)(g * 16 << 16);
        tmem_st_frag(at, hi);
        tmem_st_frag(at + kTermCols, mid);
        if (three) tmem_st_frag(at + 2 * kTermCols, lo);
    }
}

// MMA issue by a whole, converged warp: one elected lane issues, and because nothing diverges the
// descriptors stay in uniform registers (issued from one lane's branch, each MMA spent 110 to 180 cycles
// moving its operands there, against the 66 that it takes).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit_warp(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
// Rows [len, C) of the c tile to zero.
template <int NV, int kThreads>
__device__ __forceinline__ void zero_tail(uint8_t *c, int len, int tid) {
    for (int e = tid; e < C * (NV / 8); e += kThreads) {
        const int r = e / (NV / 8), cv = e % (NV / 8);
        if (r >= len) *reinterpret_cast<uint4 *>(c + (cv >> 3) * (C * 128) + r * 128 + (cv & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
}

// One step of MMA4: D (+)= (hi + mid + lo)^T c over kRows tokens, the step-th of the chunk.
template <int NV>
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t terms, uint32_t c, int step, uint32_t accumulate, bool three) {
    constexpr uint32_t id = idesc_bf16(128, NV, 0, 1);
    const uint64_t dc = smem_desc(c + step * (kRows * 128), C * 128, 1024, kSwizzle128B);
    mma_ts(d, terms, dc, id, accumulate);
    mma_ts(d, terms + 8, dc + 128, id, 1);
    mma_ts(d, terms + kTermCols, dc, id, 1);
    mma_ts(d, terms + kTermCols + 8, dc + 128, id, 1);
    if (three) {
        mma_ts(d, terms + 2 * kTermCols, dc, id, 1);
        mma_ts(d, terms + 2 * kTermCols + 8, dc + 128, id, 1);
    }
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
    __shared__ uint64_t full_ab[2], full_c[2], bar_m1, bar_m2, bar_split[2], bar_free[2], bar_d[2], bar_p, bar_o,
        bar_go, bar_end;
    __shared__ uint32_t s_tmem, s_rows[2];
    __shared__ int s_err;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    // a row past the sequences' first segments needs the scan's states; the others start before it
    if (blockIdx.x / p.n_roles / p.H >= p.n_max) grid_dependency_wait();
    // the status word is loaded beside the item, not before it: each is a chain of loads, and what needs neither
    // is done meanwhile
    const bool blocked = status_blocks(p.status);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full_ab[i], 1);
            mbar_init(&full_c[i], 1);
            mbar_init(&bar_split[i], kWarpsB);
            mbar_init(&bar_free[i], 1);
            mbar_init(&bar_d[i], 1);
        }
        mbar_init(&bar_m1, 1);
        mbar_init(&bar_m2, 1);
        mbar_init(&bar_p, kWarpsA);
        mbar_init(&bar_o, 1);
        mbar_init(&bar_go, kWarpsA + kWarpsB);
        mbar_init(&bar_end, 1);
        s_err = 0;
        fence_barrier_init();
    }
    if (warp == kTmaWarp && lane < (p.d_o.p ? 4 : 3)) prefetch_tmap(&maps.m[lane]);
    Ctx x;
    int row;
    bool last;
    const bool found = x.find<kEngineThreads, false>(p, blockIdx.x, row, last);
    if (__syncthreads_or(blocked) || !found) return;
    const bool rev = x.rev;
    const int nch = x.nch, h = x.h;
    // the entering state (NULL: zeros) and where the leaving one goes (NULL: nowhere)
    auto entering = [&]() -> const float * {
        const int64_t KV = (int64_t)NA * NV;
        const float *seg = row < 0 ? nullptr : rev ? p.seg_rev : p.seg_fwd, *first = rev ? p.dht : p.h0;
        return seg ? seg + ((int64_t)row * p.H + h) * KV : first ? first + ((int64_t)x.n * p.H + h) * KV : nullptr;
    };
    auto leaving = [&]() -> float * {
        float *d = x.role == kFwd && last ? p.ht : x.role == kDv && x.i == 0 ? p.dh0 : nullptr;
        return d ? d + ((int64_t)x.n * p.H + h) * (NA * NV) : nullptr;
    };
    x.leaves = leaving() != nullptr;
    if (nch == 0) {                                        // an empty sequence passes its state on
        const float4 *src = reinterpret_cast<const float4 *>(entering());
        float4 *dst = reinterpret_cast<float4 *>(leaving());
        if (dst) {
            constexpr int N4 = NA * NV / 4, PT = (N4 + kEngineThreads - 1) / kEngineThreads;
            float4 v[PT];                                  // (all in flight: one at a time took 20 us a state)
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                const int e = tid + i * kEngineThreads;
                v[i] = src && e < N4 ? src[e] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < PT; ++i)
                if (tid + i * kEngineThreads < N4) dst[tid + i * kEngineThreads] = v[i];
        }
        return;
    }

    // tile loads (one thread); those of the first chunk go out at once
    auto load = [&](int operand, int slot, int D, int ic, uint64_t *bar) {
        const CUtensorMap *m = &maps.m[map_of(x.role, operand)];
        for (int cb = 0; cb < D / 64; ++cb)
            tma_load_3d(smem + slot * Lay::slot + cb * C * 128, m, cb * 64, h, x.t0(ic), bar);
    };
    auto load_ab = [&](int slot_b, int slot_a, int ic) {
        mbar_arrive_expect_tx(&full_ab[ic & 1], 2 * C * NA * 2);
        load(1, slot_b, NA, ic, &full_ab[ic & 1]);
        load(0, slot_a, NA, ic, &full_ab[ic & 1]);
    };
    auto load_c = [&](int slot, int ic) {
        mbar_arrive_expect_tx(&full_c[ic & 1], C * NV * 2);
        load(2, slot, NV, ic, &full_c[ic & 1]);
    };
    if (warp == kTmaWarp && lane == 0) {
        load_ab(0, 1, 0);
        load_c(2, 0);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, kTmemCols);
        tmem_relinquish();
    }
    const float g = p.g[h], s_inc = rev ? p.scale : 1.f;   // (s_inc: of the increments, s_state: of a M)
    float *sP = reinterpret_cast<float *>(smem + Lay::oP), *sNear = sP + 132, *sW = sNear + 32;
    for (int e = tid; e <= C; e += kEngineThreads) {
        const float w = decay_pow(g, e);
        sP[e] = w;
        if (e < 32) sNear[rev ? e : 31 - e] = w;           // gamma^(block's near end to column)
        // w of a whole chunk's tokens, and of the short chunk at the segment's end (zero past it, where w may be
        // infinite if g > 0 and the split has zeros for b)
        if (rev ? e > 0 : e < C) sW[rev ? e - 1 : C - 1 - e] = s_inc * w;
        const int tail = (x.s1 - x.s0) % C;
        if (rev ? e > 0 && e <= tail : e < tail) sW[C + (rev ? e - 1 : tail - 1 - e)] = s_inc * w;
        if (e >= tail && e < C) sW[C + e] = 0.f;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(s_tmem);
    // whether chunk ic's state is needed: by the next chunk or as the leaving state
    auto updates = [&](int ic) { return ic + 1 < nch || x.leaves; };

    if (warp >= kMmaWarp) {
        if (warp == kTmaWarp && lane == 0) {
            Slots sl;
            bool ok = true, half = false;                  // half: b and a of chunk ic + 1 are under way
            int ic = 0;
            for (; ic + 1 < nch; ++ic) {                   // the next chunk's tiles
                half = false;
                // b and c of chunk ic - 1 are read.  (A barrier for odd and one for even chunks: neither can pass its
                // next phase before these loads, so a wait that comes late does not miss one.)
                if (ic > 0) ok = wait_bar(&bar_d[(ic - 1) & 1], ((ic - 1) >> 1) & 1, &s_err, 1);
                if (!ok) break;
                load_ab(sl.s[3], sl.s[4], ic + 1);
                half = true;
                ok = wait_bar(&bar_m2, ic & 1, &s_err, 2);                         // a of chunk ic is read
                if (!ok) break;
                load_c(sl.s[1], ic + 1);
                sl.next();
            }
            if (!ok) {                                     // no copy may land after the CTA is gone
                for (int c = ic > 0 ? ic - 1 : 0; c <= ic; ++c) {
                    drain(&full_ab[c & 1], (c >> 1) & 1);
                    drain(&full_c[c & 1], (c >> 1) & 1);
                }
                if (half) drain(&full_ab[(ic + 1) & 1], ((ic + 1) >> 1) & 1);
            }
        } else if (warp == kMmaWarp) {
            const uint32_t sbase = smem_u32(smem);
            Slots sl;
            // (descriptor addresses count 16 bytes: 2 per 16 channels, C * 8 per 64-channel block, 128 per
            // 16 rows)
            auto scores = [&](int ic, int slot_b, int slot_a) {                    // MMA1 of chunk ic
                if (!wait_warp(&full_ab[ic & 1], (ic >> 1) & 1, &s_err, 3)) return false;
                if (ic > 0 && !wait_warp(&bar_o, (ic - 1) & 1, &s_err, 5)) return false;    // X~ is read
                tc_fence_after();
                const uint64_t da = smem_desc(sbase + slot_a * Lay::slot, 16, 1024, kSwizzle128B);
                const uint64_t db = smem_desc(sbase + slot_b * Lay::slot, 16, 1024, kSwizzle128B);
#pragma unroll
                for (int s = 0; s < NA / 16; ++s) {
                    const uint32_t off = (s >> 2) * (C * 8) + (s & 3) * 2;
                    mma_ss(tmem + cX, da + off, db + off, idesc_bf16(128, 128), s > 0);
                }
                commit_warp(&bar_m1);
                return true;
            };
            bool ok = true;
            for (int ic = -1; ic < nch && ok; ++ic) {
                if (ic >= 0) {
                    const uint32_t ph = ic & 1, tcc = sbase + sl.s[2] * Lay::slot;
                    // (what is ready before M is waited for first, while MMA1 runs: the MMAs then follow each other)
                    const bool upd = updates(ic);
                    ok = wait_warp(&full_c[ph], (ic >> 1) & 1, &s_err, 8) && (!upd || wait_warp(&bar_split[0], 0, &s_err, 9)) &&
                         wait_warp(&bar_go, ph, &s_err, 6);                        // M in shared memory; D and O read
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = smem_desc(sbase + sl.s[1] * Lay::slot, 16, 1024, kSwizzle128B);
                    const uint64_t dm = smem_desc(sbase + Lay::oM, NA * 128, 1024, kSwizzle128B);
#pragma unroll
                    for (int s = 0; s < NA / 16; ++s)
                        mma_ss(tmem + cO, da + (s >> 2) * (C * 8) + (s & 3) * 2, dm + s * 128, idesc_bf16(128, NV, 0, 1), s > 0);
                    commit_warp(&bar_m2);
                    // MMA3 goes before the last quarter of MMA4: its scores are ready by then, and the outputs and
                    // the next chunk's scores no longer wait for the state's chain
#pragma unroll 1
                    for (int q = 0; q < C / kRows; ++q) {  // (step 4 ic + q: buffer q & 1, its use 2 ic + (q >> 1))
                        if (q == C / kRows - 1) {
                            ok = wait_warp(&bar_p, ph, &s_err, 10);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t dc = smem_desc(tcc, C * 128, 1024, kSwizzle128B);
#pragma unroll
                            for (int s = 0; s < 8; ++s)
                                mma_ts(tmem + cO, tmem + cX + s * 8, dc + s * 128, idesc_bf16(128, NV, 0, 1), 1);
                            commit_warp(&bar_o);
                        }
                        if (!upd) continue;
                        if (q > 0) {
                            ok = wait_warp(&bar_split[q & 1], q >> 1, &s_err, 20);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        mma_state<NV>(tmem + cD, tmem + cSplit + (q & 1) * 64, tcc, q, q, x.three());
                        commit_warp(&bar_free[q & 1]);
                    }
                    if (!ok) break;
                    if (upd) commit_warp(&bar_d[ph]);
                    if (ic + 1 == nch) break;
                    sl.next();
                }
                ok = scores(ic + 1, sl.s[0], sl.s[1]);
            }
            commit_warp(&bar_end);                          // every MMA issued has finished
            if (lane == 0) drain(&bar_end, 0);
            __syncwarp();
        }
    } else if (warp < kWarpsA) {
        // ---- scores and outputs: token i of the chunk
        const int quarter = warp, i = quarter * 32 + lane, r0 = quarter * 32;
        const uint32_t tm = tmem + ((uint32_t)r0 << 16);
        uint8_t *stage = smem + Lay::oStage + quarter * (32 * NV * 2);
        if (lane == 0) mbar_arrive(&bar_go);               // O may be written
        for (int ic = 0; ic < nch; ++ic) {
            const uint32_t ph = ic & 1;
            const int len = x.len(ic);
            if (!wait_warp(&bar_m1, ph, &s_err, 12)) break;
            tc_fence_after();
            // 32 columns at a time; the warp's rows are r0 ..  Columns that the mask leaves empty for all of
            // them are zeros.  Whole blocks: gamma^|i - j| as gamma^(distance of row i to the block's near
            // end) gamma^(that end to j), both at most 1; the diagonal block: the table.
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
                uint32_t pk[16];
                if (rev ? u < quarter : u > quarter) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[e] = 0;
                } else {
                    float d[32];
                    tmem_ld16(tm + cX + u * 32, d);
                    tmem_ld16(tm + cX + u * 32 + 16, d + 16);
                    tmem_ld_wait();
                    if (u != quarter && (!rev || u * 32 + 32 <= len)) {
                        const float f = p.scale * sP[rev ? u * 32 - i : i - u * 32 - 31];
                        const uint64_t f2 = pair(f, f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 c = *reinterpret_cast<const float4 *>(sNear + 4 * e);
                            pk[2 * e] = pack(mul2(mul2(pair(d[4 * e], d[4 * e + 1]), f2), pair(c.x, c.y)));
                            pk[2 * e + 1] = pack(mul2(mul2(pair(d[4 * e + 2], d[4 * e + 3]), f2), pair(c.z, c.w)));
                        }
                    } else {
                        const int lim = rev ? len : C;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int j = u * 32 + e, n = rev ? j - i : i - j;
                            d[e] = n >= 0 && j < lim ? d[e] * (p.scale * sP[n]) : 0.f;
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) pk[e] = Op16<BF>::pack2(d[2 * e], d[2 * e + 1]);
                    }
                }
                tmem_st16_b32(tm + cX + u * 16, pk);
            }
            // rows of a M times gamma^e; MMA3 adds to them
            if (!wait_warp(&bar_m2, ph, &s_err, 11)) break;
            tc_fence_after();
            {
                const float s_state = rev ? 1.f : p.scale, f = s_state * sP[i < len ? (rev ? len - 1 - i : i + 1) : 0];
                const uint64_t f2 = pair(f, f);
#pragma unroll 1
                for (int u = 0; u < NV / 32; ++u) {
                    float d[32];
                    tmem_ld16(tm + cO + u * 32, d);
                    tmem_ld16(tm + cO + u * 32 + 16, d + 16);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 y = unpair(mul2(pair(d[e], d[e + 1]), f2));
                        d[e] = y.x;
                        d[e + 1] = y.y;
                    }
                    tmem_st16(tm + cO + u * 32, d);
                    tmem_st16(tm + cO + u * 32 + 16, d + 16);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar_p);
                bulk_wait_read();                          // the previous outputs have left the staging tile
            }
            __syncwarp();
            if (!wait_warp(&bar_o, ph, &s_err, 13)) break;
            tc_fence_after();
            // the warp's 32 rows through its part of the staging tile and a TMA store per 64 channels; rows of
            // a partial block one by one, so that the next sequence's rows stay untouched
            const Rows &ro = x.role == kFwd ? p.o : x.role == kDq ? p.dq : x.role == kDv ? p.dv : p.dk;
            const int t0 = x.t0(ic);
            const bool whole = r0 + 32 <= len && ro.p != nullptr, some = !whole && i < len && ro.p != nullptr;
#pragma unroll 1
            for (int cb = 0; cb < NV / 64; ++cb) {
                uint4 w[8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float d[32];
                    tmem_ld16(tm + cO + cb * 64 + u * 32, d);
                    tmem_ld16(tm + cO + cb * 64 + u * 32 + 16, d + 16);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[u * 4 + e] = pack8_as<BF>(d + 8 * e);
                }
                if (cb == NV / 64 - 1) {                   // O is read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar_go);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (whole) *reinterpret_cast<uint4 *>(stage + cb * 4096 + lane * 128 + ((e ^ (lane & 7)) << 4)) = w[e];
                    else if (some && GCL_IN_BOUNDS(t0 + i, p.t_max, p.status))
                        *reinterpret_cast<uint4 *>(row_ptr<BF>(ro, t0 + i, h) + cb * 64 + e * 8) = w[e];
                }
            }
            if (whole) {
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    const CUtensorMap *mo = &maps.out[x.role == kFwd ? 0 : x.role - kDq];
                    for (int cb = 0; cb < NV / 64; ++cb) tma_store_3d(mo, stage + cb * 4096, cb * 64, h, t0 + r0);
                    bulk_commit();
                }
            }
        }
        if (lane == 0) bulk_wait_read();
    } else {
        // ---- the split (16 of each step's 32 tokens per warp) and the state: row m, columns half * HV ..;
        // rows of c past the end to zero
        const int quarter = warp & 3, half = (warp - kWarpsA) >> 2, m = quarter * 32 + lane;
        const bool mine = m < NA;
        float S[HV];
        {
            const float *src = entering();
            const int bt = tid - kWarpsA * 32;
            // the entering fp32 rows cross the staging tile and M (16-byte pieces, exclusive or of the row against
            // bank conflicts), so that global accesses are whole lines
            float4 *rows = reinterpret_cast<float4 *>(smem + Lay::oStage);
            constexpr int RC = NV / 4;                     // pieces of a row
            if (src && (x.role == kDq || x.role == kDk)) { // element (r, c) at c * NA + r: lanes are contiguous
#pragma unroll
                for (int j = 0; j < HV; ++j) S[j] = mine ? src[(int64_t)(half * HV + j) * NA + m] : 0.f;
            } else if (src) {
                // (every load before the first store: one after the other they took 10,000 cycles)
                constexpr int PT = NA * RC / (kWarpsB * 32);
                float4 v[PT];
#pragma unroll
                for (int i = 0; i < PT; ++i) v[i] = reinterpret_cast<const float4 *>(src)[bt + i * (kWarpsB * 32)];
#pragma unroll
                for (int i = 0; i < PT; ++i) {
                    const int e = bt + i * (kWarpsB * 32);
                    rows[(e / RC) * RC + ((e % RC) ^ ((e / RC) & (RC - 1)))] = v[i];
                }
                named_sync<1>(kWarpsB * 32);
#pragma unroll
                for (int j = 0; j < HV; j += 4) {
                    const float4 v = mine ? rows[m * RC + (((half * HV + j) / 4) ^ (m & (RC - 1)))] : make_float4(0.f, 0.f, 0.f, 0.f);
                    S[j] = v.x; S[j + 1] = v.y; S[j + 2] = v.z; S[j + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < HV; ++j) S[j] = 0.f;
            }
            named_sync<1>(kWarpsB * 32);                   // M may be written
        }
        const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16), td = tq + cD + half * HV;
        const uint32_t tsp = tq + cSplit + half * 8;
        uint8_t *mrow = smem + Lay::oM + m * 128;
        const uint32_t sbase = smem_u32(smem);
        Slots sl;
        // (One copy of each stage in a rolled loop: the warps' code has to stay in the instruction cache.)
        bool ok = true;
        for (int ic = 0; ok; ++ic) {
            const bool more = ic < nch, upd = more && updates(ic);
            const int len = more ? x.len(ic) : C;
            if (more && len < C) {
                ok = wait_warp(&full_c[ic & 1], (ic >> 1) & 1, &s_err, 14);
                if (!ok) break;
                zero_tail<NV, kWarpsB * 32>(smem + sl.s[2] * Lay::slot, len, tid - kWarpsA * 32);
                fence_async_smem();
            }
            if (upd && !(ok = wait_warp(&full_ab[ic & 1], (ic >> 1) & 1, &s_err, 15))) break;
#pragma unroll 1
            for (int q = 0; q < C / kRows; ++q) {
                // step q of chunk ic: buffer q & 1, its use 2 ic + (q >> 1)
                if (upd) {
                    if ((ic > 0 || q > 1) && !(ok = wait_warp(&bar_free[q & 1], (q >> 1) ^ 1, &s_err, 17))) break;
                    tc_fence_after();
                    const int r0 = q * kRows + half * 16;
                    if (NA == 128 || quarter * 32 < NA)
                        split16<NA>(sbase + sl.s[0] * Lay::slot, quarter * 32, r0, len, sW + (len < C ? C : 0) + r0, tsp + (q & 1) * 64,
                                    x.three());
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (upd && lane == 0) mbar_arrive(&bar_split[q & 1]);
                if (q > 0) continue;
                // the state that enters chunk ic (after the chunk's first step, which needs no state and fills the
                // time until MMA4 of the last chunk is done)
                if (ic > 0) {
                    if (!(ok = wait_warp(&bar_d[(ic - 1) & 1], ((ic - 1) >> 1) & 1, &s_err, 18))) break;
                    tc_fence_after();
                    const float gl = sP[x.len(ic - 1)];
#pragma unroll
                    for (int u = 0; u < HV / 16; ++u) {
                        float d[16];
                        tmem_ld16(td + u * 16, d);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) S[u * 16 + e] = fmaf(gl, S[u * 16 + e], d[e]);
                    }
                }
                if (!more) break;
                if (mine) {                                // in bf16 for MMA2: rows m, 64-column blocks
#pragma unroll
                    for (int j = 0; j < HV; j += 8) {
                        const int c = half * HV + j;
                        *reinterpret_cast<uint4 *>(mrow + (c >> 6) * (NA * 128) + ((((c & 63) >> 3) ^ (m & 7)) << 4)) = pack8_as<BF>(S + j);
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_go);
                if (!upd) break;
            }
            if (!upd) break;
            sl.next();
        }
        if (ok && x.leaves) {
            // the leaving state, stored below: through the tiles of the chunk that does not follow
            const int slot = half ? sl.s[1] : sl.s[0];
            if (mine) {
                float4 *out = reinterpret_cast<float4 *>(smem + slot * Lay::slot);
                constexpr int HC = HV / 4;
#pragma unroll
                for (int j = 0; j < HC; ++j)
                    out[m * HC + (j ^ (m & (HC - 1)))] = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
                if (m == 0) s_rows[half] = slot;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
    if (tid == 0 && s_err != 0) status_set(p.status, GCL_DEV_WAIT_TIMEOUT);
    if (x.leaves && s_err == 0) {
        float4 *dst = reinterpret_cast<float4 *>(leaving());
        constexpr int RC = NV / 4, HC = HV / 4;
        for (int e = tid; e < NA * RC; e += kEngineThreads) {
            const int r = e / RC, c = e % RC;
            dst[e] = reinterpret_cast<const float4 *>(smem + s_rows[c / HC] * Lay::slot)[r * HC + ((c % HC) ^ (r & (HC - 1)))];
        }
    }
}

// ---------------------------------------------------------------- the segments' own states
// sum_j gamma^(distance to the segment's end) b_j c_j^T over one segment: MMA4 alone, with the decay
// taken to the segment's end, so that the sum stays in TMEM until the last chunk.  Warps 0-15 split b
// (eight take 32 tokens at a time, four TMEM buffers), warp 16 loads, warp 17 issues.  b, c: three tiles each.
// Every wait is for a barrier whose next phase its waiter has to allow first (a parity says nothing about the phase
// after): a buffer's by the warps that fill it next, a tile's by the loader, the sum's by a barrier that completes once.
// 65,536 tokens of 4 heads, 128 x 128: 32 us, 4.1 TB/s, with the split's instructions (52% of issue) before HBM.
constexpr int kOwnWarps = 16, kOwnTma = 16, kOwnMma = 17, kOwnThreads = 18 * 32, kBufs = C / kRows, kOwnTiles = 3;

template <int NA, int NV>
struct OwnLayout {
    static constexpr uint32_t sb = C * NA * 2, sc = C * NV * 2;
    static constexpr uint32_t oB = 0, oC = kOwnTiles * sb, oW = oC + kOwnTiles * sc;
    static constexpr uint32_t total = oW + kOwnWarps * 16 * 4;                     // weights of each warp's tokens
    static constexpr uint32_t bytes = total + 1024;
};

template <int NA, int NV>
__global__ void __launch_bounds__(kOwnThreads, 1) dla_own_kernel(const __grid_constant__ Maps maps, const Params p) {
    using Lay = OwnLayout<NA, NV>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ uint64_t full[kOwnTiles], empty[kOwnTiles], bar_split[kBufs], bar_free[kBufs], bar_end;
    __shared__ uint32_t s_tmem;
    __shared__ int s_err;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    launch_dependents();                                   // (the scan waits for this grid's end)
    const bool blocked = status_blocks(p.status);
    Ctx x;
    int row;
    bool last;
    const bool found = x.find<kOwnThreads, true>(p, blockIdx.x, row, last);
    if (__syncthreads_or(blocked) || !found) return;
    const bool rev = x.rev;
    const int h = x.h, nch = x.nch;
    if (tid == 0) {
        for (int i = 0; i < kOwnTiles; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&bar_split[i], kOwnWarps / 2);
            mbar_init(&bar_free[i], 1);
        }
        mbar_init(&bar_end, 1);
        s_err = 0;
        fence_barrier_init();
    }
    if (warp == kOwnMma) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(s_tmem);
    if (warp == kOwnTma) {
        if (lane == 0) {
            const CUtensorMap *mb = &maps.m[map_of(x.role, 1)], *mc = &maps.m[map_of(x.role, 2)];
            int ic = 0;
            for (; ic < nch; ++ic) {
                const int s = ic % kOwnTiles;
                // (MMA4 of chunk ic - kOwnTiles has read c; its split has read b before)
                if (ic >= kOwnTiles && !wait_bar(&empty[s], (ic / kOwnTiles - 1) & 1, &s_err, 1)) break;
                mbar_arrive_expect_tx(&full[s], C * (NA + NV) * 2);
                for (int cb = 0; cb < NA / 64; ++cb)
                    tma_load_3d(smem + Lay::oB + s * Lay::sb + cb * C * 128, mb, cb * 64, h, x.t0(ic), &full[s]);
                for (int cb = 0; cb < NV / 64; ++cb)
                    tma_load_3d(smem + Lay::oC + s * Lay::sc + cb * C * 128, mc, cb * 64, h, x.t0(ic), &full[s]);
            }
            if (ic < nch)                                  // no copy may land after the CTA is gone
                for (int c = ic >= kOwnTiles ? ic - kOwnTiles : 0; c < ic; ++c) drain(&full[c % kOwnTiles], (c / kOwnTiles) & 1);
        }
    } else if (warp == kOwnMma) {
        const uint32_t sbase = smem_u32(smem);
        bool ok = true;
        for (int ic = 0; ic < nch && ok; ++ic) {
            const int s = ic % kOwnTiles;
            ok = wait_warp(&full[s], (ic / kOwnTiles) & 1, &s_err, 2);
#pragma unroll 1
            for (int q = 0; q < kBufs && ok; ++q) {
                ok = wait_warp(&bar_split[q], ic & 1, &s_err, 3);
                if (!ok) break;
                tc_fence_after();
                mma_state<NV>(tmem, tmem + 128 + q * 64, sbase + Lay::oC + s * Lay::sc, q, ic + q, true);
                commit_warp(&bar_free[q]);
            }
            if (ok) commit_warp(&empty[s]);
        }
        commit_warp(&bar_end);                              // every MMA issued has finished
        if (lane == 0) drain(&bar_end, 0);
        __syncwarp();
    } else {
        const float g = p.g[h], s_inc = rev ? p.scale : 1.f;
        const int m = (warp & 3) * 32 + lane, half = (warp >> 2) & 1, odd = warp >> 3;   // odd: takes steps 1, 3
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        float *w = reinterpret_cast<float *>(smem + Lay::oW) + warp * 16;
        bool ok = true;
        for (int ic = 0; ic < nch && ok; ++ic) {
            const int s = ic % kOwnTiles, len = x.len(ic), t0 = x.t0(ic);
            ok = wait_warp(&full[s], (ic / kOwnTiles) & 1, &s_err, 4);
            if (ok && len < C) {                           // (each group of eight the whole tail, before its first step)
                zero_tail<NV, kOwnWarps / 2 * 32>(smem + Lay::oC + s * Lay::sc, len, tid & (kOwnWarps / 2 * 32 - 1));
                fence_async_smem();
            }
#pragma unroll 1
            for (int q = odd; q < kBufs && ok; q += 2) {
                if (ic > 0 && !(ok = wait_warp(&bar_free[q], (ic - 1) & 1, &s_err, 5))) break;
                tc_fence_after();
                const int r0 = q * kRows + half * 16, t = t0 + r0 + lane;          // the warp's 16 weights
                if (lane < 16) w[lane] = t < x.s1 ? s_inc * decay_pow(g, rev ? t - x.s0 + 1 : x.s1 - 1 - t) : 0.f;
                __syncwarp();
                if (NA == 128 || m < NA)
                    split16<NA>(smem_u32(smem) + Lay::oB + s * Lay::sb, (warp & 3) * 32, r0, len, w,
                                tmem + lane_off + 128 + q * 64 + half * 8, true);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_split[q]);
            }
        }
        // (Not bar_free of the last step: the warps that take the even steps have not waited for it before, so that
        // its phase may still be the one before the last chunk's, whose parity passes.)
        if (ok && wait_warp(&bar_end, 0, &s_err, 6)) {
            tc_fence_after();
            float4 *rows = reinterpret_cast<float4 *>(smem);       // through the tiles, to whole lines
            constexpr int RC = NV / 4;
            if (NA == 128 || m < NA) {
#pragma unroll 1
                for (int u = (warp >> 2) * 16; u < NV; u += 64) {
                    float d[16];
                    tmem_ld16(tmem + lane_off + u, d);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        rows[m * RC + ((u / 4 + j) ^ (m & (RC - 1)))] = make_float4(d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kOwnMma) tmem_dealloc(tmem, 512);
    if (tid == 0 && s_err != 0) status_set(p.status, GCL_DEV_WAIT_TIMEOUT);
    if (s_err == 0) {
        const float4 *rows = reinterpret_cast<const float4 *>(smem);
        float4 *dst = reinterpret_cast<float4 *>((rev ? p.seg_rev : p.seg_fwd) + ((int64_t)row * p.H + h) * (NA * NV));
        constexpr int RC = NV / 4;
        for (int e = tid; e < NA * RC; e += kOwnThreads) dst[e] = rows[(e / RC) * RC + ((e % RC) ^ ((e / RC) & (RC - 1)))];
    }
}

bool make_map(CUtensorMap *m, const Rows &r, int D, int H, int64_t t_max, int box_t) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)t_max};
    const cuuint64_t strides[2] = {(cuuint64_t)r.sh * 2, (cuuint64_t)r.st * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_t};
    return make_tensor_map(m, r.p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int NA, int NV>
cudaError_t launch_one(const Maps &maps, const Params &p, bool own_states, cudaStream_t s) {
    const unsigned grid = (unsigned)(((own_states ? 0 : p.n_max) + p.n_rows) * p.H * p.n_roles);
    if (own_states) {
        cudaError_t e = cudaFuncSetAttribute(dla_own_kernel<NA, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)OwnLayout<NA, NV>::bytes);
        if (e != cudaSuccess) return e;
        dla_own_kernel<NA, NV><<<grid, kOwnThreads, OwnLayout<NA, NV>::bytes, s>>>(maps, p);
    } else {
        cudaError_t e = cudaFuncSetAttribute(dla_tc_kernel<NA, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)TcLayout<NA, NV>::bytes);
        if (e != cudaSuccess) return e;
        if (p.seg_fwd || p.seg_rev)                        // (first segments run beside the launches before)
            return launch_dependent(dla_tc_kernel<NA, NV>, dim3(grid), dim3(kEngineThreads), TcLayout<NA, NV>::bytes, s, maps, p);
        dla_tc_kernel<NA, NV><<<grid, kEngineThreads, TcLayout<NA, NV>::bytes, s>>>(maps, p);
    }
    return cudaGetLastError();
}

}  // namespace

// Roles kFwd and kDv run on [K, V] states, kDq and kDk on [V, K]: one launch for each shape.
cudaError_t launch_tc(const Params &p0, bool own_states, int n_roles, const int *roles, cudaStream_t s) {
    Maps maps;
    const Rows *in[4] = {&p0.q, &p0.k, &p0.v, &p0.d_o}, *out[3] = {p0.dq.p ? &p0.dq : &p0.o, &p0.dv, &p0.dk};
    const int din[4] = {p0.K, p0.K, p0.V, p0.V}, dout[3] = {p0.dq.p ? p0.K : p0.V, p0.V, p0.K};
    for (int i = 0; i < 4; ++i) {
        maps.m[i] = CUtensorMap{};
        if (in[i]->p && !make_map(&maps.m[i], *in[i], din[i], p0.H, p0.t_max, C)) return cudaErrorInvalidValue;
    }
    for (int i = 0; i < 3; ++i) {                          // (forward: the first; backward: dq, dv, dk)
        maps.out[i] = CUtensorMap{};
        if (out[i]->p && !make_map(&maps.out[i], *out[i], dout[i], p0.H, p0.t_max, 32)) return cudaErrorInvalidValue;
    }
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
