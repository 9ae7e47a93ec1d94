// glr.cu -- gated linear recurrence over packed sequences: the C entry points, the workspace and the set-up launch.
#include "glr.cuh"

namespace gcl {
namespace glr {
namespace {

// ---- set-up: checks cu_seqlens, finds each tile's first sequence, passes states of empty sequences through, clears the
// packets of the spans that will be taken ----
__device__ __forceinline__ void set_up(const Params &p, bool blocked, bool bad, int64_t at, int64_t step) {
    if (at == 0) {                                         // (this thread's block decides for the call)
        p.head->blocked = blocked || bad;
        p.head->live = blocked || bad ? 0 : p.cu[p.n_max];
        p.head->ticket = 0;
    }
    if (bad) return;
    const int64_t spans = (p.cu[p.n_max] + (int64_t)kRanks * p.tile - 1) / (kRanks * p.tile);
    for (int64_t e = at; e < spans * p.D; e += step) reinterpret_cast<uint4 *>(p.chain)[e] = make_uint4(0, 0, 0, 0);
    for (int64_t j = at; j < p.tiles; j += step) {
        const int64_t t0 = j * p.tile;
        int lo = 0, hi = p.n_max;                          // first n with cu[n] >= t0 (n_max if none)
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p.cu[mid] >= t0) hi = mid;
            else lo = mid + 1;
        }
        p.first[j] = lo;
    }
}

// before: the walk that forms the states for p's, or one without tiles.
__global__ void __launch_bounds__(1024) glr_setup_kernel(const Params p, const Params before, const float *in_state, float *out_state) {
    launch_dependents();
    const int tid = threadIdx.x;
    int bad = 0;
    for (int n = tid; n < p.n_max; n += blockDim.x) {
        const int b = p.cu[n], e = p.cu[n + 1];
        bad |= b < 0 || e < b || e > p.t_max || (n == 0 && b != 0);
    }
    const bool blocked = status_blocks_cta(p.status);
    bad = __syncthreads_or(bad);
    const int64_t at = blockIdx.x * (int64_t)blockDim.x + tid, step = (int64_t)gridDim.x * blockDim.x;
    if (at == 0 && bad) status_set(p.status, GCL_DEV_BAD_RANGE);
    set_up(p, blocked, bad, at, step);
    if (before.tiles > 0) set_up(before, blocked, bad, at, step);
    if (blocked || bad || !out_state) return;
    for (int n = blockIdx.x; n < p.n_max; n += gridDim.x) {
        if (p.cu[n + 1] != p.cu[n]) continue;
        for (int d = tid; d < p.D; d += blockDim.x) {
            const int64_t e = (int64_t)n * p.D + d;
            out_state[e] = in_state ? in_state[e] : 0.f;
        }
    }
}

}  // namespace

// (The blocks' looks at the status word may differ, where another call sets it in the meantime: the first block's decides, and what the walks
// read is set up by every block whatever it saw; a block that saw the word set leaves its empty sequences' states unwritten.)
cudaError_t launch_setup(const Params &p, const Params &before, const float *in_state, float *out_state, cudaStream_t s) {
    int64_t blocks = ((p.tiles + before.tiles + kRanks - 1) / kRanks * p.D + 4095) / 4096;
    if (out_state && blocks < (p.n_max + 7) / 8) blocks = (p.n_max + 7) / 8;
    if (blocks > num_sms()) blocks = num_sms();
    glr_setup_kernel<<<(unsigned)blocks, 1024, 0, s>>>(p, before, in_state, out_state);
    return cudaGetLastError();
}

extern template cudaError_t launch_fwd<float>(const Params &, cudaStream_t);
extern template cudaError_t launch_fwd<__half>(const Params &, cudaStream_t);
extern template cudaError_t launch_fwd<__nv_bfloat16>(const Params &, cudaStream_t);
extern template cudaError_t launch_bwd<float>(const Params &, cudaStream_t);
extern template cudaError_t launch_bwd<__half>(const Params &, cudaStream_t);
extern template cudaError_t launch_bwd<__nv_bfloat16>(const Params &, cudaStream_t);

namespace {

// ---- host ----------------------------------------------------------------
size_t up16(size_t n) { return (n + 15) / 16 * 16; }

bool sizes_ok(const gcl_glr_args *a) {
    return a && a->t_max >= 1 && a->t_max < (int64_t(1) << 31) && a->n_max >= 1 && a->D >= 8 && a->D % 8 == 0 &&
           a->D <= (1 << 20) && (a->dtype == GCL_F32 || a->dtype == GCL_BF16 || a->dtype == GCL_F16);
}

// A call of one span needs no meeting of spans and no launch before it (256 tokens of 512 channels, fp16: 10.0 -> 8.0 us captured;
// backward of 100 tokens 12.4 -> 9.3).
bool solo(const Params &p) { return p.tiles <= kRanks; }

// The workspace's parts, in order; its base may be NULL (for the size alone).  before: the walk that forms the states which a
// backward without h_save needs.
size_t layout(const gcl_glr_args *a, bool backward, Params *p, Params *before) {
    uint8_t *base = static_cast<uint8_t *>(a->workspace);
    size_t at = 0;
    const size_t row = sizeof(float) * (size_t)a->D;
    auto set = [&](auto *&field, size_t bytes) {
        field = base ? reinterpret_cast<std::remove_reference_t<decltype(field)>>(base + at) : nullptr;
        at += up16(bytes);
    };
    auto walk = [&](Params &w, int tile) {
        w.tile = tile;
        w.tiles = (a->t_max + tile - 1) / tile;
        set(w.head, sizeof(Header));
        set(w.first, sizeof(int32_t) * (size_t)w.tiles);
        set(w.chain, sizeof(Packet) * (size_t)a->D * ((w.tiles + kRanks - 1) / kRanks));
    };
    walk(*p, backward ? kTileB : kTileF);
    p->h_save = a->h_save;
    if (backward && a->drate) set(p->drate_part, row * p->tiles);
    if (backward && !a->h_save) {
        set(p->h_save, row * p->tiles);
        walk(*before, kTileF);
    }
    return at;
}

template <typename T>
cudaError_t launch(Params p, Params before, bool backward, cudaStream_t s) {
    p.n_cb = before.n_cb = (p.D + Lane<T>::CB - 1) / Lane<T>::CB;
    const bool states = before.tiles > 0;
    cudaError_t e = cudaSuccess;
    if (solo(p)) {
        p.first = before.first = nullptr;
    } else {                                               // (then the states' walk goes by the set-up's look at the status word too)
        e = launch_setup(p, before, backward ? p.dht : p.h0, backward ? p.dh0 : p.ht, s);
    }
    if (e == cudaSuccess && states) e = launch_fwd<T>(before, s);
    if (e != cudaSuccess) return e;
    return backward ? launch_bwd<T>(p, s) : launch_fwd<T>(p, s);
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

size_t workspace(const gcl_glr_args *a, bool backward) {
    Params p{}, before{};
    return sizes_ok(a) ? layout(a, backward, &p, &before) : 0;
}

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
    Params p{}, before{};
    const size_t bytes = layout(a, backward, &p, &before);
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
    p.kind = Kind{a->rate, a->decay, a->mix};
    p.h0 = a->h0; p.cu = a->cu_seqlens; p.status = a->dev_status;
    p.t_max = a->t_max; p.n_max = a->n_max; p.D = a->D;
    if (before.tiles > 0) {                                // the states before each 64 tokens, by a forward without o and ht
        const Params w = before;
        before = p;
        before.head = w.head; before.first = w.first; before.chain = w.chain;
        before.tile = w.tile; before.tiles = w.tiles;
        before.d_o.p = nullptr;
    }
    const cudaError_t e = a->dtype == GCL_BF16 ? launch<__nv_bfloat16>(p, before, backward, s)
                          : a->dtype == GCL_F16 ? launch<__half>(p, before, backward, s)
                                                : launch<float>(p, before, backward, s);
    return cuda_check(e, fn);
}

}  // namespace
}  // namespace glr
}  // namespace gcl

using namespace gcl;

extern "C" {

size_t gcl_glr_fwd_workspace_bytes(const gcl_glr_args *a) { return glr::workspace(a, false); }
size_t gcl_glr_bwd_workspace_bytes(const gcl_glr_args *a) { return glr::workspace(a, true); }
gcl_status_t glr_fwd(const gcl_glr_args *a, gcl_stream_t stream) { return glr::run("glr_fwd", a, false, static_cast<cudaStream_t>(stream)); }
gcl_status_t glr_bwd(const gcl_glr_args *a, gcl_stream_t stream) { return glr::run("glr_bwd", a, true, static_cast<cudaStream_t>(stream)); }

}  // extern "C"
