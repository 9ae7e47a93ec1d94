// glr_step.cu -- gated linear recurrence for single tokens: h <- a h + m(a) u for one token of each
// request, on a pool of fp32 states updated in place.
//
// A lane takes eight channels: a 16-byte load of each row (fp32: two), two of the state, all before the first use.  Bound by the latency of
// one pass of loads: one request of 512 channels takes 2.0 to 2.4 us in a captured graph; a call from Python
// 8, as 256 requests of 2,048 channels do (8 MB moved, floor 1.2).
#include "dla_simt.cuh"
#include "glr.cuh"

namespace gcl {
namespace glr {

gcl_status_t check_kind(const char *fn, const float *rate, int32_t D, int32_t decay, int32_t mix, int32_t dtype);

namespace {

constexpr int kStepThreads = 128;

struct StepParams {
    Rows x, r, i, o;
    Kind kind;
    float *state;
    const int32_t *slots;
    int32_t *status;
    int32_t batch, n_slots, D;
};

template <typename T, int DECAY, int MIX, bool GATE>
__global__ void __launch_bounds__(kStepThreads) glr_step_kernel(const StepParams p) {
    constexpr int V = Lane<T>::V;
    if (dla::call_blocked(p.status, p.slots ? p.batch : 0, [&](int64_t i) { return p.slots[i] >= p.n_slots; })) return;
    const int per = p.D / 8;
    const int64_t e = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
    const int64_t b = e / per;
    if (b >= p.batch) return;
    const int ch = (int)(e % per) * 8;
    const int64_t slot = p.slots ? p.slots[b] : b;
    T *o = dla::row_ptr<T>(p.o, b, 0) + ch;
    if (slot < 0 || slot >= p.n_slots) {
        if (slot >= p.n_slots) status_set(p.status, GCL_DEV_BAD_RANGE);
        const float z[4] = {0.f, 0.f, 0.f, 0.f};
        dla::store4f(o, z);
        dla::store4f(o + 4, z);
        return;
    }
    if (!GCL_RANGE_IN_BOUNDS(slot * p.D + ch, slot * p.D + ch + 7, (int64_t)p.n_slots * p.D, p.status)) return;
    float *st = p.state + slot * p.D + ch;
    using L = Lane<T>;
    constexpr int N = 8 / V;                               // words of eight channels
    __align__(8) float h[8];
    typename L::P x[N], m[N], g[N], rate[N], a[N];
    auto load = [&](const Rows &r, typename L::P *v) {
        const T *q = dla::row_ptr<const T>(r, b, 0) + ch;
        uint4 w[sizeof(T) / 2];
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) w[k] = reinterpret_cast<const uint4 *>(q)[k];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = L::get(reinterpret_cast<const uint32_t *>(w)[k]);
    };
    dla::load8f(st, h);
    load(p.x, x);
    load(p.r, m);
    if (GATE) load(p.i, g);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        rate[k] = L::all(0.f);
        if (DECAY == GCL_DECAY_POWER) rate[k] = L::load(p.kind.rate + ch + k * V);
    }
    typename L::P sg[N];
#pragma unroll
    for (int k = 0; k < N; ++k) gates<T, DECAY, MIX, GATE, 1>(rate[k], false, m + k, g + k, a + k, m + k, sg + k);
#pragma unroll
    for (int k = 0; k < N; ++k) L::store(h + k * V, L::fma(a[k], L::load(h + k * V), L::mul(m[k], GATE ? L::mul(x[k], sg[k]) : x[k])));
    dla::store4f(st, h);
    dla::store4f(st + 4, h + 4);
    dla::store4f(o, h);
    dla::store4f(o + 4, h + 4);
}

template <typename T>
cudaError_t launch_step(const StepParams &p, cudaStream_t s) {
    const int64_t n = (int64_t)p.batch * (p.D / 8);
    for_kind(p.kind.decay, p.kind.mix, p.i.p != nullptr, [&](auto d, auto m, auto g) {
        glr_step_kernel<T, decltype(d)::value, decltype(m)::value, decltype(g)::value>
            <<<(unsigned)((n + kStepThreads - 1) / kStepThreads), kStepThreads, 0, s>>>(p);
    });
    return cudaGetLastError();
}

}  // namespace
}  // namespace glr
}  // namespace gcl

using namespace gcl;

extern "C" gcl_status_t glr_step(const gcl_glr_step_args *a, gcl_stream_t stream) {
    const char *fn = "glr_step";
    fail(GCL_OK, "%s", "");                                // clears gcl_last_error()
    if (!a) return fail(GCL_ERR_INVALID_ARG, "%s: args is NULL", fn);
    if (!a->state) return fail(GCL_ERR_INVALID_ARG, "%s: state is required", fn);
    if (a->batch < 1 || a->n_slots < 1) return fail(GCL_ERR_INVALID_ARG, "%s: need batch >= 1 and n_slots >= 1", fn);
    gcl_status_t st = glr::check_kind(fn, a->rate, a->D, a->decay, a->mix, a->dtype);
    if (st != GCL_OK) return st;
    if (!a->slots && a->batch > a->n_slots)
        return fail(GCL_ERR_INVALID_ARG, "%s: %d requests without slots need as many states (%d given)", fn, a->batch, a->n_slots);
    if ((int64_t)a->batch * a->D >= (int64_t(1) << 38))
        return fail(GCL_ERR_UNSUPPORTED, "%s: batch * D must be below 2^38", fn);
    const int es = a->dtype == GCL_F32 ? 4 : 2;
    struct { const char *name; const gcl_rows *r; bool in, out; } need[] = {
        {"x", &a->x, true, false}, {"r", &a->r, true, false}, {"i", &a->i, a->i.ptr != nullptr, false}, {"o", &a->o, false, true}};
    for (const auto &x : need) {
        if (!x.in && !x.out) continue;
        gcl_rows r = *x.r;
        r.head_stride = a->D;
        if ((st = dla::check_rows(fn, x.name, r, a->batch, 1, a->D, es, x.out)) != GCL_OK) return st;
    }
    if (!dla::aligned(a->state, 16) || !dla::aligned(a->rate, 16))
        return fail(GCL_ERR_INVALID_ARG, "%s: state and rate must be 16-byte aligned", fn);
    glr::StepParams p{};
    p.x = dla::rows(a->x); p.r = dla::rows(a->r); p.i = dla::rows(a->i); p.o = dla::rows(a->o);
    p.kind = glr::Kind{a->rate, a->decay, a->mix};
    p.state = a->state; p.slots = a->slots; p.status = a->dev_status;
    p.batch = a->batch; p.n_slots = a->n_slots; p.D = a->D;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->dtype == GCL_BF16 ? glr::launch_step<__nv_bfloat16>(p, s)
                          : a->dtype == GCL_F16 ? glr::launch_step<__half>(p, s)
                                                : glr::launch_step<float>(p, s);
    return cuda_check(e, fn);
}
