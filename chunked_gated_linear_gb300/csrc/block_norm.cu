// block_norm.cu -- the norms around a block: the C entry points and the sums of the weights' gradients.
#include "block_norm.cuh"

namespace gcl {
namespace blk {

template <> cudaError_t launch_fwd<float, float>(const Params &, cudaStream_t);
template <> cudaError_t launch_fwd<__nv_bfloat16, __nv_bfloat16>(const Params &, cudaStream_t);
template <> cudaError_t launch_fwd<__half, __half>(const Params &, cudaStream_t);
template <> cudaError_t launch_fwd<__nv_bfloat16, float>(const Params &, cudaStream_t);
template <> cudaError_t launch_fwd<__half, float>(const Params &, cudaStream_t);
template <> cudaError_t launch_bwd<float, float>(const Params &, int *, cudaStream_t);
template <> cudaError_t launch_bwd<__nv_bfloat16, __nv_bfloat16>(const Params &, int *, cudaStream_t);
template <> cudaError_t launch_bwd<__half, __half>(const Params &, int *, cudaStream_t);
template <> cudaError_t launch_bwd<__nv_bfloat16, float>(const Params &, int *, cudaStream_t);
template <> cudaError_t launch_bwd<__half, float>(const Params &, int *, cudaStream_t);

namespace {

// The weights' gradients from the blocks' sums, in a fixed order: 32 channels a block, 32 rows of threads over the
// sums, eight loads of each in flight.  blockIdx.y: w_post, w_pre.
__global__ void __launch_bounds__(1024) block_dw_kernel(const Params p, int blocks) {
    __shared__ float s[32][33];
    grid_dependency_wait();
    int64_t rows;
    if (!live_rows(p, rows)) return;
    const float *part = blockIdx.y ? p.part_pre : p.part_post;
    if (!part) return;
    const int lane = threadIdx.x & 31, ch = blockIdx.x * 32 + lane, r = threadIdx.x >> 5;
    float sum = 0.f;
    if (ch < p.D)
        for (int b0 = r; b0 < blocks; b0 += 8 * 32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = b0 + i * 32 < blocks ? part[(int64_t)(b0 + i * 32) * p.D + ch] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i];
        }
    s[r][lane] = sum;
    __syncthreads();
    float t = s[lane][r];                                  // thread (r, lane): a part of channel r of the block's 32
#pragma unroll
    for (int d = 16; d; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    if (lane == 0 && blockIdx.x * 32 + r < p.D) (blockIdx.y ? p.dw_pre : p.dw_post)[blockIdx.x * 32 + r] = t;
}

bool sizes_ok(const gcl_block_args *a) {
    return a && a->t_max >= 1 && a->t_max < (int64_t(1) << 31) && a->H >= 1 && a->H <= 65535 && a->D >= 8 && a->D % 8 == 0 && a->D <= 16384;
}

size_t bwd_workspace(const gcl_block_args *a) {
    if (!sizes_ok(a)) return 0;
    const int64_t rows = a->t_max * a->H, most = (int64_t)kBwdBlocks * num_sms();
    return (size_t)(rows < most ? rows : most) * 2 * a->D * sizeof(float);
}

gcl_status_t run(const char *fn, const gcl_block_args *a, bool backward, cudaStream_t s) {
    fail(GCL_OK, "%s", "");                                // clears gcl_last_error()
    if (!a) return fail(GCL_ERR_INVALID_ARG, "%s: args is NULL", fn);
    if (a->t_max < 1 || a->t_max >= (int64_t(1) << 31) || a->H < 1 || a->H > 65535)
        return fail(GCL_ERR_INVALID_ARG, "%s: need 1 <= t_max < 2^31 and 1 <= H <= 65535", fn);
    if (!sizes_ok(a)) return fail(GCL_ERR_UNSUPPORTED, "%s: D=%d (a multiple of 8, at most 16384)", fn, a->D);
    if (a->dtype != GCL_F32 && a->dtype != GCL_BF16 && a->dtype != GCL_F16)
        return fail(GCL_ERR_UNSUPPORTED, "%s: dtype %d (supported: GCL_F32, GCL_BF16, GCL_F16)", fn, a->dtype);
    if (a->stream_dtype != a->dtype && a->stream_dtype != GCL_F32)
        return fail(GCL_ERR_UNSUPPORTED, "%s: stream_dtype %d (supported: dtype's, GCL_F32)", fn, a->stream_dtype);
    for (int32_t n : {a->post_norm, a->pre_norm})
        if (n < GCL_NORM_NONE || n > GCL_NORM_L2) return fail(GCL_ERR_UNSUPPORTED, "%s: norm %d (supported: none, RMS, L2)", fn, n);
    if (a->activation < GCL_ACT_NONE || a->activation > GCL_ACT_SIGMOID)
        return fail(GCL_ERR_UNSUPPORTED, "%s: activation %d (supported: none, SiLU, sigmoid)", fn, a->activation);
    if (!(a->eps >= 0.f)) return fail(GCL_ERR_INVALID_ARG, "%s: eps must not be negative", fn);
    const int32_t cut = a->dropout >= 0.f && a->dropout < 1.f ? (int32_t)((double)a->dropout * 65536. + 0.5) : -1;
    if (cut < 0 || cut > 65535) return fail(GCL_ERR_INVALID_ARG, "%s: dropout must be at least 0 and round below 1 in steps of 1/65536", fn);
    if (cut && !a->rng) return fail(GCL_ERR_INVALID_ARG, "%s: dropout needs rng", fn);
    if (a->cu_seqlens && a->n_max < 1) return fail(GCL_ERR_INVALID_ARG, "%s: cu_seqlens needs n_max >= 1", fn);
    const bool gate = a->gate.ptr != nullptr, x = a->x.ptr != nullptr;
    if (!backward && !a->xo.ptr && !a->z.ptr) return fail(GCL_ERR_INVALID_ARG, "%s: xo or z is required", fn);
    if (backward && !a->dxo.ptr && !a->dz.ptr) return fail(GCL_ERR_INVALID_ARG, "%s: dxo or dz is required", fn);
    if (backward && a->dx.ptr && !x) return fail(GCL_ERR_INVALID_ARG, "%s: dx needs x", fn);
    const int es = a->dtype == GCL_F32 ? 4 : 2, ss = a->stream_dtype == GCL_F32 ? 4 : 2;
    struct { const char *name; const gcl_rows *r; int esize; bool in, out; } need[] = {
        {"y", &a->y, es, true, false}, {"gate", &a->gate, es, gate, false}, {"x", &a->x, ss, x, false},
        {"xo", &a->xo, ss, false, !backward && a->xo.ptr}, {"z", &a->z, es, false, !backward && a->z.ptr},
        {"dxo", &a->dxo, ss, backward && a->dxo.ptr, false}, {"dz", &a->dz, es, backward && a->dz.ptr, false},
        {"dy", &a->dy, es, false, backward}, {"dgate", &a->dgate, es, false, backward && gate},
        {"dx", &a->dx, ss, false, backward && a->dx.ptr}};
    gcl_status_t st;
    for (const auto &n : need)
        if ((n.in || n.out) && (st = dla::check_rows(fn, n.name, *n.r, a->t_max, a->H, a->D, n.esize, n.out)) != GCL_OK) return st;
    for (const void *w : {a->post_weight, a->pre_weight, (const void *)a->workspace})
        if (!dla::aligned(w, 16)) return fail(GCL_ERR_INVALID_ARG, "%s: weights and the workspace must be 16-byte aligned", fn);
    Params p{};
    p.y = Rows(a->y); p.gate = Rows(a->gate); p.x = Rows(a->x);
    if (!backward) {
        p.xo = Rows(a->xo);
        p.z = Rows(a->z);
    } else {
        if ((a->dpost_weight && !a->post_weight) || (a->dpre_weight && (!a->pre_weight || !a->dz.ptr)))
            return fail(GCL_ERR_INVALID_ARG, "%s: a weight's gradient needs the weight (and dpre_weight dz)", fn);
        p.dxo = Rows(a->dxo); p.dz = Rows(a->dz);
        p.dy = Rows(a->dy); p.dgate = Rows(a->dgate); p.dx = Rows(a->dx);
        if (a->dpost_weight || a->dpre_weight) {
            const size_t bytes = bwd_workspace(a);
            if (!a->workspace || a->workspace_bytes < bytes)
                return fail(GCL_ERR_CAPACITY, "%s: workspace of %zu bytes needed, %zu given", fn, bytes,
                            a->workspace ? a->workspace_bytes : (size_t)0);
            float *ws = static_cast<float *>(a->workspace);
            p.dw_post = a->dpost_weight; p.dw_pre = a->dpre_weight;
            p.part_post = a->dpost_weight ? ws : nullptr;
            p.part_pre = a->dpre_weight ? ws + bytes / 2 / sizeof(float) : nullptr;
        }
    }
    p.w_post = a->post_weight; p.w_pre = a->pre_weight; p.rng = a->rng; p.cu = a->cu_seqlens; p.status = a->dev_status;
    p.t_max = a->t_max; p.n_max = a->n_max; p.H = a->H; p.D = a->D; p.scale = a->scale; p.eps = a->eps; p.cut = cut;
    p.post = a->post_norm; p.pre = a->pre_norm; p.act = a->activation;
    const bool wide = a->stream_dtype != a->dtype;
    using bf = __nv_bfloat16;
    if (!backward) {
        const cudaError_t e = a->dtype == GCL_F32 ? launch_fwd<float, float>(p, s)
                              : a->dtype == GCL_BF16 ? (wide ? launch_fwd<bf, float> : launch_fwd<bf, bf>)(p, s)
                                                     : (wide ? launch_fwd<__half, float> : launch_fwd<__half, __half>)(p, s);
        return cuda_check(e, fn);
    }
    int blocks = 0;
    cudaError_t e = a->dtype == GCL_F32 ? launch_bwd<float, float>(p, &blocks, s)
                    : a->dtype == GCL_BF16 ? (wide ? launch_bwd<bf, float> : launch_bwd<bf, bf>)(p, &blocks, s)
                                           : (wide ? launch_bwd<__half, float> : launch_bwd<__half, __half>)(p, &blocks, s);
    if (e == cudaSuccess && (p.part_post || p.part_pre))
        e = launch_dependent(block_dw_kernel, dim3((a->D + 31) / 32, 2), dim3(1024), 0, s, p, blocks);
    return cuda_check(e, fn);
}

}  // namespace
}  // namespace blk
}  // namespace gcl

using namespace gcl;

extern "C" {

gcl_status_t block_norm_fwd(const gcl_block_args *a, gcl_stream_t stream) {
    return blk::run("block_norm_fwd", a, false, static_cast<cudaStream_t>(stream));
}
size_t gcl_block_norm_bwd_workspace_bytes(const gcl_block_args *a) { return blk::bwd_workspace(a); }
gcl_status_t block_norm_bwd(const gcl_block_args *a, gcl_stream_t stream) {
    return blk::run("block_norm_bwd", a, true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
