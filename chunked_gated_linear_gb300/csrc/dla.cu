// dla.cu -- decayed linear attention: the C entry points, the segment plan and the scan of the
// segments' states.
//
// Plans.  Where whole sequences keep the SMs evenly busy one CTA walks each: every input is read once.  Else
// sequences are cut into segments: the segments' own states (a launch that reads k and v once more), their
// scan, then the outputs from the entering states; a sequence's first segment (in the role's time) waits for
// neither and runs beside them.  The scan is elementwise over a [K, V] state: S(i + 1) = gamma^seg S(i) + own(i).
#include "dla.cuh"

namespace gcl {
namespace dla {
namespace {

constexpr int kScanThreads = 256;

// Threads take four state values of one (sequence, head) each, over the borders of the sequence's segments in
// time order; blockIdx.z: 0 forwards, 1 backwards.  The sequence's first row is the number of borders
// before it, summed by the block.
__global__ void __launch_bounds__(kScanThreads) dla_scan_kernel(const Params p) {
    launch_dependents();                                   // (the outputs' launch waits for this grid's end)
    grid_dependency_wait();                                // the segments' own states
    if (status_blocks_cta(p.status)) return;
    const int h = blockIdx.y % p.H, n = blockIdx.y / p.H, tid = threadIdx.x;
    const bool rev = blockIdx.z != 0;
    __shared__ int s_sum[kScanThreads / 32];
    int sum = 0, bad = 0;
    for (int m = tid; m <= n; m += kScanThreads) {
        const int64_t b = p.cu[m], e = p.cu[m + 1];
        if (b < 0 || e < b || e > p.t_max) bad = 1;
        else if (m < n) sum += borders(e - b, p.seg);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if ((tid & 31) == 0) s_sum[tid >> 5] = sum;
    if (__syncthreads_or(bad)) {
        if (tid == 0) status_set(p.status, GCL_DEV_BAD_RANGE);
        return;
    }
    int64_t row0 = 0;
    for (int w = 0; w < kScanThreads / 32; ++w) row0 += s_sum[w];
    const int64_t len = (int64_t)p.cu[n + 1] - p.cu[n];
    const int count = borders(len, p.seg);
    if (row0 + count > p.n_rows) {
        if (tid == 0) status_set(p.status, GCL_DEV_BAD_RANGE);
        return;
    }
    if (count == 0) return;
    const int64_t KV = (int64_t)p.K * p.V, n_state = (int64_t)p.n_max * p.H * KV, base = ((int64_t)n * p.H + h) * KV;
    const float g = p.g[h], gs = decay_pow(g, p.seg);
    const float *first = rev ? p.dht : p.h0;
    float *seg = rev ? p.seg_rev : p.seg_fwd;
    const int64_t step = (int64_t)p.H * KV;
    for (int64_t e = ((int64_t)blockIdx.x * kScanThreads + tid) * 4; e < KV; e += (int64_t)gridDim.x * kScanThreads * 4) {
        const int64_t at = base + e;
        (void)n_state;                                     // (checked in the debug build)
        float4 cur = first && GCL_RANGE_IN_BOUNDS(at, at + 3, n_state, p.status) ? *reinterpret_cast<const float4 *>(first + at)
                                                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
        float *at_row = seg + row0 * step + h * KV + e;
        for (int j0 = 0; j0 < count; j0 += 16) {           // sixteen loads in flight
            float4 own[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const int j = j0 + u;
                own[u] = j < count ? *reinterpret_cast<const float4 *>(at_row + (rev ? count - 1 - j : j) * step)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const int j = j0 + u;
                if (j >= count) break;
                // backwards the first segment met is the sequence's last, possibly a short one
                const float f = rev && j == 0 ? decay_pow(g, len - (int64_t)count * p.seg) : gs;
                cur.x = fmaf(f, cur.x, own[u].x);
                cur.y = fmaf(f, cur.y, own[u].y);
                cur.z = fmaf(f, cur.z, own[u].z);
                cur.w = fmaf(f, cur.w, own[u].w);
                *reinterpret_cast<float4 *>(at_row + (rev ? count - 1 - j : j) * step) = cur;
            }
        }
    }
}

}  // namespace

cudaError_t launch_scan(const Params &p, bool backward, cudaStream_t s) {
    // blocks per state: as many as fill the GPU twice, at most one per 1,024 values
    const int64_t most = (int64_t)p.K * p.V / 4 / kScanThreads, units = (int64_t)p.n_max * p.H;
    int64_t per = 4 * (int64_t)num_sms() / units;
    per = per < 1 ? 1 : per > most ? most : per;
    return launch_dependent(dla_scan_kernel, dim3((unsigned)per, (unsigned)units, backward ? 2 : 1), dim3(kScanThreads), 0, s, p);
}

cudaError_t launch(const Params &p, int dtype, bool own_states, int n_roles, const int *roles, cudaStream_t s) {
    if (dtype == GCL_BF16) return launch_tc(p, own_states, n_roles, roles, s);
    if (dtype == GCL_F16) return launch_simt_t<__half>(p, own_states, n_roles, roles, s);
    return launch_simt_t<float>(p, own_states, n_roles, roles, s);
}

namespace {

// Tokens per segment, from the capacities.  Time is counted in chunks (128 tokens on the tensor cores, 64 on
// the CUDA cores) of one CTA: an output CTA takes its chunks and kStart, an own-state CTA kOwn of its
// chunks and kStart, the scan and the two further launches kLaunch.
//  - Candidate lengths, every one up to 128 chunks and then a 64th apart (a plan is made on every call; a million
//    tokens are 8,192 chunks, 400 candidates), are costed for n_max sequences of t_max / n_max tokens.  (One sequence of
//    65,536 tokens, 4 heads: whole 1,540 us, segments of 1,792 or 1,920 101 to 104, of 4,096 163.  4 sequences of
//    8,192, 16 heads, backward: whole 454 us, segments of 2,816 or 4,096 413 to 422, of 1,792 452.  fp32, 2 sequences,
//    4,096 tokens, 8 heads of 64: whole 659 us, segments of 64 74, of 128 68, of 256 107.)
//  - With several sequences their lengths differ, and where units are few (less than two per SM) the
//    longest one's CTA would be the last to finish: no segment is longer than half of each SM's share of
//    all tokens, but four chunks (two on the CUDA cores) are allowed (7 ragged sequences of 5,003 tokens in
//    all, 6 heads, backward: 62 us, without this 105).
//    More units are balanced by their order instead (32 prompts of 73 to 4,716 tokens in 64 slots, 16 heads:
//    whole in seq_order 147 us, cut at 1,792 tokens 225, at 2,432 to 4,096 190 to 203: own states and scan come
//    first).  The price: one prompt of 33,000 tokens alone in the 64 slots takes 806 us, in one slot 161.
//  - Sequences of one or two chunks on average, and units that fill every SM eight times, stay whole.
int64_t segment_tokens(int64_t t_max, int32_t n_max, int32_t H, bool backward, int32_t dtype, int32_t K, int32_t V) {
    const bool tc = dtype == GCL_BF16;
    const int64_t unit = tc ? 128 : 64, sms = num_sms() * (tc ? 1 : simt_ctas(K, V)), roles = backward ? 3 : 1;
    const int64_t units = (int64_t)n_max * H * roles, chunks = (t_max / n_max + unit - 1) / unit;
    const int64_t whole = (t_max + unit - 1) / unit * unit;
    if (units >= 8 * sms || chunks <= (tc ? 2 : 1) || units > 65535) return whole;
    const double kStart = tc ? 2.2 : 0.3, kOwn = tc ? 0.58 : 0.4, kLaunch = tc ? 4.0 : 0.6;
    int64_t most = chunks;                                 // longest candidate, in chunks
    if (n_max > 1 && units < 2 * sms) {
        const int64_t half = (t_max * H * roles / (2 * sms) + unit - 1) / unit;
        const int64_t least = tc ? 4 : 2;
        most = half < least ? least : half;
    }
    double best = 1e300;
    int64_t seg = whole;
    if (most > chunks) most = chunks;
    for (int64_t c = 1, next; c <= most; c = next) {
        next = c < 128 ? c + 1 : c + c / 64;
        if (next > most && c < most) next = most;          // (the longest, for a whole sequence, always)
        const int64_t full = chunks / c, rest = chunks % c, parts = full + (rest > 0);
        const double item = c + kStart, work = (double)units * (chunks + parts * kStart) / sms;
        const double waves = (double)((units * full + sms - 1) / sms) * item;
        const double spread = work + (rest > 0 ? 0.5 * (rest + kStart) : 0.0);
        double cost = waves > spread ? waves : spread;
        if (parts > 1) {
            const int64_t own = (int64_t)n_max * H * (backward ? 2 : 1) * (parts - 1);
            cost += (double)((own + sms - 1) / sms) * (kOwn * c + kStart) + kLaunch;
        }
        if (cost < best) {
            best = cost;
            seg = c * unit;
        }
    }
    return seg >= chunks * unit ? whole : seg;
}

// Borders between segments, at most: a sequence has (length - 1) / seg of them.
int64_t border_rows(int64_t t_max, int64_t seg) { return seg >= t_max ? 0 : (t_max - 1) / seg; }

// The plan of a call, 0 for sizes that have none.
int64_t plan(const gcl_dla_args *a, bool backward) {
    if (a->t_max < 1 || a->t_max >= (int64_t(1) << 31) || a->n_max < 1 || a->H < 1 || a->K < 1 || a->V < 1) return 0;
    return segment_tokens(a->t_max, a->n_max, a->H, backward, a->dtype, a->K, a->V);
}

// Workspace of the plan with segments of seg tokens.
size_t segment_bytes(const gcl_dla_args *a, bool backward, int64_t seg) {
    if (seg < 1 || seg >= a->t_max) return 0;
    // a state per segment (a border's states need one less a sequence)
    return (size_t)gcl_nt_max(a->t_max, a->n_max, (int32_t)seg) * a->H * a->K * a->V * sizeof(float) * (backward ? 2 : 1);
}

}  // namespace

gcl_status_t check_rows(const char *fn, const char *name, const gcl_rows &r, int64_t tokens, int64_t heads, int32_t D,
                        int32_t esize, bool output) {
    if (!r.ptr) return fail(GCL_ERR_INVALID_ARG, "%s: %s is required", fn, name);
    const int64_t unit = 16 / esize;
    if (!aligned(r.ptr, 16)) return fail(GCL_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", fn, name);
    if (r.token_stride < D || r.head_stride < D || r.token_stride % unit || r.head_stride % unit ||
        r.token_stride >= (int64_t(1) << 36) || r.head_stride >= (int64_t(1) << 36))
        return fail(GCL_ERR_INVALID_ARG, "%s: %s strides (%lld, %lld) must be at least the row's %d values and multiples of 16 bytes",
                    fn, name, (long long)r.token_stride, (long long)r.head_stride, D);
    if (output && r.token_stride < (heads - 1) * r.head_stride + D && r.head_stride < (tokens - 1) * r.token_stride + D)
        return fail(GCL_ERR_INVALID_ARG, "%s: rows of %s overlap", fn, name);
    return GCL_OK;
}

gcl_status_t check_sizes(const char *fn, int32_t H, int32_t K, int32_t V, int32_t dtype) {
    if (H < 1 || H > 65535) return fail(GCL_ERR_INVALID_ARG, "%s: H=%d (1 to 65535)", fn, H);
    if ((K != 64 && K != 128) || (V != 64 && V != 128))
        return fail(GCL_ERR_UNSUPPORTED, "%s: K=%d V=%d (supported: 64 or 128 each)", fn, K, V);
    if (dtype != GCL_F32 && dtype != GCL_BF16 && dtype != GCL_F16)
        return fail(GCL_ERR_UNSUPPORTED, "%s: dtype %d (supported: GCL_F32, GCL_BF16, GCL_F16)", fn, dtype);
    return GCL_OK;
}

namespace {

gcl_status_t run_chunk(const char *fn, const gcl_dla_args *a, bool backward, cudaStream_t s) {
    fail(GCL_OK, "%s", "");                                // clears gcl_last_error()
    if (!a) return fail(GCL_ERR_INVALID_ARG, "%s: args is NULL", fn);
    if (!a->g || !a->cu_seqlens) return fail(GCL_ERR_INVALID_ARG, "%s: g and cu_seqlens are required", fn);
    if (a->t_max < 1 || a->t_max >= (int64_t(1) << 31) || a->n_max < 1)
        return fail(GCL_ERR_INVALID_ARG, "%s: need 1 <= t_max < 2^31 and n_max >= 1", fn);
    gcl_status_t st = check_sizes(fn, a->H, a->K, a->V, a->dtype);
    if (st != GCL_OK) return st;
    if ((int64_t)a->n_max * a->H >= (int64_t(1) << 29))
        return fail(GCL_ERR_UNSUPPORTED, "%s: n_max * H must be below 2^29", fn);
    const int es = a->dtype == GCL_F32 ? 4 : 2;
    struct { const char *name; const gcl_rows *r; int32_t D; bool in, out; } need[] = {
        {"q", &a->q, a->K, true, false}, {"k", &a->k, a->K, true, false}, {"v", &a->v, a->V, true, false},
        {"o", &a->o, a->V, false, !backward && a->o.ptr}, {"d_o", &a->d_o, a->V, backward, false},
        {"dq", &a->dq, a->K, false, backward}, {"dk", &a->dk, a->K, false, backward},
        {"dv", &a->dv, a->V, false, backward}};
    for (const auto &x : need)
        if ((x.in || x.out) && (st = check_rows(fn, x.name, *x.r, a->t_max, a->H, x.D, es, x.out)) != GCL_OK) return st;
    for (const void *x : {(const void *)a->h0, (const void *)a->ht, (const void *)a->dht, (const void *)a->dh0})
        if (!aligned(x, 16)) return fail(GCL_ERR_INVALID_ARG, "%s: states must be 16-byte aligned", fn);
    // (a sequence's segments run side by side: one may write the state before another has read it)
    const float *out_state = backward ? a->dh0 : a->ht;
    const uintptr_t state_bytes = sizeof(float) * (uintptr_t)a->n_max * a->H * a->K * a->V;
    struct { const char *name; const float *p; } in_state[] = {{"h0", a->h0}, {"dht", backward ? a->dht : nullptr}};
    for (const auto &x : in_state) {
        const uintptr_t i = reinterpret_cast<uintptr_t>(x.p), o = reinterpret_cast<uintptr_t>(out_state);
        if (i && o && (i < o ? o - i : i - o) < state_bytes)
            return fail(GCL_ERR_INVALID_ARG, "%s: %s must not be %s (their states overlap)", fn, backward ? "dh0" : "ht", x.name);
    }
    const int64_t seg = plan(a, backward);
    const size_t bytes = segment_bytes(a, backward, seg);
    if (bytes && (!a->workspace || a->workspace_bytes < bytes))
        return fail(GCL_ERR_CAPACITY, "%s: workspace of %zu bytes needed, %zu given", fn, bytes,
                    a->workspace ? a->workspace_bytes : (size_t)0);
    if (bytes && !aligned(a->workspace, 16)) return fail(GCL_ERR_INVALID_ARG, "%s: the workspace must be 16-byte aligned", fn);

    Params p{};
    p.q = rows(a->q); p.k = rows(a->k); p.v = rows(a->v);
    if (backward) {
        p.d_o = rows(a->d_o); p.dq = rows(a->dq); p.dk = rows(a->dk); p.dv = rows(a->dv);
        p.dht = a->dht; p.dh0 = a->dh0;
    } else {
        p.o = rows(a->o);
        p.ht = a->ht;
    }
    p.g = a->g; p.h0 = a->h0;
    p.cu = a->cu_seqlens; p.seq_order = a->seq_order; p.status = a->dev_status;
    p.t_max = a->t_max; p.n_max = a->n_max; p.H = a->H; p.K = a->K; p.V = a->V; p.scale = a->scale;
    p.n_rows = border_rows(a->t_max, seg);
    p.seg = (int32_t)(seg < a->t_max ? seg : a->t_max);
    const int both[2] = {kFwd, kDv}, out[3] = {kDq, kDv, kDk};
    cudaError_t e = cudaSuccess;
    if (bytes) {
        p.seg_fwd = static_cast<float *>(a->workspace);
        if (backward) p.seg_rev = p.seg_fwd + bytes / 2 / sizeof(float);
        e = launch(p, a->dtype, true, backward ? 2 : 1, both, s);
        if (e == cudaSuccess) e = launch_scan(p, backward, s);
    }
    if (e == cudaSuccess) e = launch(p, a->dtype, false, backward ? 3 : 1, backward ? out : both, s);
    return cuda_check(e, fn);
}

}  // namespace
}  // namespace dla
}  // namespace gcl

using namespace gcl;

extern "C" {

int64_t gcl_dla_segment_tokens(int64_t t_max, int32_t n_max, int32_t H, int32_t backward, int32_t dtype, int32_t K, int32_t V) {
    if (t_max < 1 || t_max >= (int64_t(1) << 31) || n_max < 1 || H < 1) return 0;
    return dla::segment_tokens(t_max, n_max, H, backward != 0, dtype, K, V);
}

size_t gcl_dla_fwd_workspace_bytes(const gcl_dla_args *a) { return a ? dla::segment_bytes(a, false, dla::plan(a, false)) : 0; }
size_t gcl_dla_bwd_workspace_bytes(const gcl_dla_args *a) { return a ? dla::segment_bytes(a, true, dla::plan(a, true)) : 0; }

gcl_status_t dla_chunk_fwd(const gcl_dla_args *a, gcl_stream_t stream) {
    return dla::run_chunk("dla_chunk_fwd", a, false, static_cast<cudaStream_t>(stream));
}

gcl_status_t dla_chunk_bwd(const gcl_dla_args *a, gcl_stream_t stream) {
    return dla::run_chunk("dla_chunk_bwd", a, true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
