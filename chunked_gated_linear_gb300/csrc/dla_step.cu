// dla_step.cu -- decayed linear attention for single tokens: S <- gamma S + k v^T, o = scale S^T q,
// for one token of each request of a batch, on a pool of fp32 states updated in place.
//
// HBM-bound: a state is read and written once (2 x 4 K V bytes), everything else is 1/100 of that.
// A CTA takes VS value columns of one (request, head) state; each of its 256 threads holds float4
// columns of K / (1024 / VS) key rows, all loaded before the first use, so a CTA has its whole tile
// in flight.  The partial sums of o over the key rows are added through shared memory in a fixed
// order.  VS = V (whole rows, contiguous 4 K V bytes per CTA) for batches that fill the GPU; VS = 32
// (one 128-byte line per row) for the few states of a small batch, whose latency is what counts.
// 256 requests of 16 heads of 128 x 128: 83 us, 6.5 TB/s.
#include "dla.cuh"

namespace gcl {
namespace dla {
namespace {

constexpr int kStepThreads = 256;

struct StepParams {
    Rows q, k, v, o;
    const float *g;
    float *state;
    const int32_t *slots;
    int32_t *status;
    int32_t batch, n_slots, H;
    float scale;
};

template <typename T, int K, int V, int VS>
__global__ void __launch_bounds__(kStepThreads) dla_step_kernel(const StepParams p) {
    constexpr int CG = VS / 4, RG = kStepThreads / CG;     // column groups of a row, row groups
    constexpr int RPT = K / RG > 0 ? K / RG : 1;           // key rows per thread
    __shared__ float sq[K], sk[K];
    __shared__ __align__(16) float so[RG][VS];
    if (call_blocked(p.status, p.slots ? p.batch : 0, [&](int64_t i) { return p.slots[i] >= p.n_slots; })) return;
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
    const int h = (blockIdx.x / (V / VS)) % p.H, v0 = (blockIdx.x % (V / VS)) * VS;
    const int b = blockIdx.x / (V / VS) / p.H;
    const int64_t slot = p.slots ? p.slots[b] : b;
    const bool idle = slot < 0 || slot >= p.n_slots;
    if (idle) {
        if (slot >= p.n_slots && tid == 0) status_set(p.status, GCL_DEV_BAD_RANGE);
        for (int c = tid; c < VS; c += kStepThreads) st_out(row_ptr<T>(p.o, b, h) + v0, c, 0.f);
        return;
    }
    const int64_t at = (slot * p.H + h) * (int64_t)(K * V) + v0 + cg * 4;
    float *S = p.state + at;
    const bool ok = rg * RPT < K && GCL_RANGE_IN_BOUNDS(at + (int64_t)rg * RPT * V, at + (int64_t)(rg * RPT + RPT - 1) * V + 3,
                                                        (int64_t)p.n_slots * p.H * K * V, p.status);
    float4 s[RPT];
    if (ok) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) s[i] = *reinterpret_cast<const float4 *>(S + (int64_t)(rg * RPT + i) * V);
    }
    for (int e = tid; e < K; e += kStepThreads) {
        sq[e] = ld_in(row_ptr<const T>(p.q, b, h), e);
        sk[e] = ld_in(row_ptr<const T>(p.k, b, h), e);
    }
    float v[4];
    {
        const T *vp = row_ptr<const T>(p.v, b, h) + v0 + cg * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = ld_in(vp, e);
    }
    const float gam = expf(p.g[h]);
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ok) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float kk = sk[rg * RPT + i], qq = sq[rg * RPT + i];
            s[i].x = fmaf(gam, s[i].x, kk * v[0]);
            s[i].y = fmaf(gam, s[i].y, kk * v[1]);
            s[i].z = fmaf(gam, s[i].z, kk * v[2]);
            s[i].w = fmaf(gam, s[i].w, kk * v[3]);
            *reinterpret_cast<float4 *>(S + (int64_t)(rg * RPT + i) * V) = s[i];
            acc.x = fmaf(qq, s[i].x, acc.x);
            acc.y = fmaf(qq, s[i].y, acc.y);
            acc.z = fmaf(qq, s[i].z, acc.z);
            acc.w = fmaf(qq, s[i].w, acc.w);
        }
    }
    *reinterpret_cast<float4 *>(&so[rg][cg * 4]) = acc;
    __syncthreads();
    for (int c = tid; c < VS; c += kStepThreads) {
        float o = 0.f;
#pragma unroll
        for (int r = 0; r < RG; ++r) o += so[r][c];
        st_out(row_ptr<T>(p.o, b, h) + v0, c, p.scale * o);
    }
}

template <typename T, int K, int V>
cudaError_t launch_step(const StepParams &p, cudaStream_t s) {
    const int64_t units = (int64_t)p.batch * p.H;
    if (units >= 2 * (int64_t)num_sms()) dla_step_kernel<T, K, V, V><<<(unsigned)units, kStepThreads, 0, s>>>(p);
    else dla_step_kernel<T, K, V, 32><<<(unsigned)(units * (V / 32)), kStepThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step_t(const StepParams &p, int K, int V, cudaStream_t s) {
    if (K == 64) return V == 64 ? launch_step<T, 64, 64>(p, s) : launch_step<T, 64, 128>(p, s);
    return V == 64 ? launch_step<T, 128, 64>(p, s) : launch_step<T, 128, 128>(p, s);
}

}  // namespace
}  // namespace dla
}  // namespace gcl

using namespace gcl;
using namespace gcl::dla;

extern "C" gcl_status_t dla_step(const gcl_dla_step_args *a, gcl_stream_t stream) {
    const char *fn = "dla_step";
    fail(GCL_OK, "%s", "");                                // clears gcl_last_error()
    if (!a) return fail(GCL_ERR_INVALID_ARG, "%s: args is NULL", fn);
    if (!a->g || !a->state) return fail(GCL_ERR_INVALID_ARG, "%s: g and state are required", fn);
    if (a->batch < 1 || a->n_slots < 1) return fail(GCL_ERR_INVALID_ARG, "%s: need batch >= 1 and n_slots >= 1", fn);
    gcl_status_t st = check_sizes(fn, a->H, a->K, a->V, a->dtype);
    if (st != GCL_OK) return st;
    if (!a->slots && a->batch > a->n_slots)
        return fail(GCL_ERR_INVALID_ARG, "%s: %d requests without slots need as many states (%d given)", fn, a->batch, a->n_slots);
    if ((int64_t)a->batch * a->H * 4 >= (int64_t(1) << 31))
        return fail(GCL_ERR_UNSUPPORTED, "%s: batch * H must be below 2^29", fn);
    const int es = a->dtype == GCL_F32 ? 4 : 2;
    struct { const char *name; const gcl_rows *r; int32_t D; bool out; } need[] = {
        {"q", &a->q, a->K, false}, {"k", &a->k, a->K, false}, {"v", &a->v, a->V, false}, {"o", &a->o, a->V, true}};
    for (const auto &x : need)
        if ((st = check_rows(fn, x.name, *x.r, a->batch, a->H, x.D, es, x.out)) != GCL_OK) return st;
    if (!aligned(a->state, 16)) return fail(GCL_ERR_INVALID_ARG, "%s: state must be 16-byte aligned", fn);
    StepParams p{};
    p.q = rows(a->q); p.k = rows(a->k); p.v = rows(a->v); p.o = rows(a->o);
    p.g = a->g; p.state = a->state; p.slots = a->slots; p.status = a->dev_status;
    p.batch = a->batch; p.n_slots = a->n_slots; p.H = a->H; p.scale = a->scale;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->dtype == GCL_BF16 ? launch_step_t<__nv_bfloat16>(p, a->K, a->V, s)
                          : a->dtype == GCL_F16 ? launch_step_t<__half>(p, a->K, a->V, s)
                                                : launch_step_t<float>(p, a->K, a->V, s);
    return cuda_check(e, fn);
}
