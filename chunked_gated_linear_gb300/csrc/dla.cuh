// dla.cuh -- decayed linear attention (one fixed decay per head): what its kernels share.
//
// Forward and backward are one engine in four roles.  With gamma = exp(g_h), the recurrence
//   M <- gamma M + b_j c_j^T,   out_i = a_i M     (inclusive of j = i)
// over the tokens of a sequence, forwards or backwards in time, is
//   role  a    b    c    time       M            out          M before the first token
//   FWD   q    k    v    forwards   S   [K, V]   o / scale    h0
//   DQ    do   v    k    forwards   S^T [V, K]   dq / scale   h0^T
//   DV    k    q    do   backwards  G   [K, V]   dv           dht, met before a decay
//   DK    v    do   q    backwards  G^T [V, K]   dk           dht^T, likewise
// (G with scale q do^T as its increments.)  In chunk form, for the chunk's tokens i, j and len of
// them, with M the state that enters the chunk:
//   forwards   out_i = sum_{j <= i} gamma^(i-j) (a_i b_j) c_j + gamma^(i+1) a_i M
//              M'    = gamma^len M + sum_j gamma^(len-1-j) b_j c_j^T
//   backwards  out_i = sum_{j >= i} gamma^(j-i) (a_i b_j) c_j + gamma^(len-1-i) a_i M
//              M'    = gamma^len M + sum_j gamma^(j+1) b_j c_j^T
// where backwards M carries one decay more than G (it is gamma G), so that dht enters and dh0
// leaves as they are.
#pragma once

#include "gcl_internal.cuh"

namespace gcl {
namespace dla {

enum Role { kFwd = 0, kDq = 1, kDv = 2, kDk = 3 };

struct Rows {                      // a gcl_rows, strides in elements
    void *p;
    int64_t st, sh;
};

struct Params {
    Rows q, k, v, d_o, o, dq, dk, dv;
    const float *g, *h0, *dht;
    float *ht, *dh0;
    const int32_t *cu, *seq_order;
    int32_t *status;
    float *seg_fwd, *seg_rev;      // [n_rows, H, K, V], a row per border between segments: the own state of the
                                   // segment that it ends (in the role's time), after the scan the state there;
                                   // NULL for one segment per sequence
    int64_t t_max;
    int64_t n_rows;                // borders (capacity; 0: one segment per sequence)
    int32_t seg;                   // tokens per segment
    int32_t n_max, H, K, V;
    float scale;
    int32_t n_roles;               // roles of this launch: block b of (row, head) u has b = u n_roles + r
    uint32_t roles;                // role r, 2 bits each
};

// Host: the given roles whose states have shape 0 ([K, V]: kFwd, kDv; every role when K = V) or 1 ([V, K]).
inline bool take_roles(Params &p, int n_roles, const int *roles, int shape) {
    p.n_roles = 0;
    p.roles = 0;
    for (int i = 0; i < n_roles; ++i) {
        const bool trans = roles[i] == kDq || roles[i] == kDk;
        if (p.K != p.V ? trans == (shape == 1) : shape == 0) p.roles |= (uint32_t)roles[i] << (2 * p.n_roles++);
    }
    return p.n_roles > 0;
}

// Row t of head h.
template <typename T>
__host__ __device__ __forceinline__ T *row_ptr(const Rows &r, int64_t t, int h) {
    return static_cast<T *>(r.p) + t * r.st + h * r.sh;
}

// gamma^n (n >= 0): 1 for n = 0 whatever g is (also g = -inf).
__device__ __forceinline__ float decay_pow(float g, int64_t n) { return n == 0 ? 1.f : expf(g * (float)n); }

// The work of row j of the grid: sequence n, the segment's number i in it, its tokens [s0, s1), whether it is the
// sequence's last, and the row of its state among the segments' (-1: none).  Every thread of the block calls it
// (block barriers); the answer is the same for all.  False: nothing to do.
// The output kernels' first n_max rows are the sequence slots (in seq_order): each sequence's first segment in
// the role's time, which enters from h0 (dht) and needs nothing of the launches before.  The rows after
// them are the borders between two segments, sequence by sequence; the block adds up the sequences' borders,
// kBlock at a time, until row j falls into one.  Such a row's segment is the one that the border's state
// enters; of the own-state kernels (whose rows are the borders alone) the one that it leaves.
struct Item {
    int n, i;
    int64_t bos, eos, s0, s1, row;
    bool last;
};

__device__ __forceinline__ int borders(int64_t len, int32_t seg) { return len > seg ? (int)((len - 1) / seg) : 0; }

template <int kBlock, bool kOwn>
__device__ __forceinline__ bool find_item(const Params &p, int64_t j, bool rev, Item &it) {
    __shared__ int s_warp[32];
    __shared__ int s_hit[2], s_bad;
    const int tid = threadIdx.x;
    const bool cut = p.seg_fwd != nullptr || p.seg_rev != nullptr;
    if (!kOwn && j < p.n_max) {
        const int n = p.seq_order ? p.seq_order[j] : (int)j;
        if (n < 0 || n >= p.n_max) {
            if (tid == 0) status_set(p.status, GCL_DEV_BAD_RANGE);
            return false;
        }
        it.n = n;
        it.row = -1;
        it.bos = p.cu[n];
        it.eos = p.cu[n + 1];
        it.i = rev && cut ? borders(it.eos - it.bos, p.seg) : 0;
    } else {
        if (!kOwn) j -= p.n_max;
        if (tid == 0) { s_hit[0] = -1; s_bad = 0; }
        __syncthreads();
        int64_t base = 0;
        for (int n0 = 0; n0 < p.n_max; n0 += kBlock) {
            const int n = n0 + tid;
            int c = 0;
            bool bad = false;
            if (n < p.n_max) {
                const int64_t b = p.cu[n], e = p.cu[n + 1];
                bad = b < 0 || e < b || e > p.t_max;
                if (bad) s_bad = 1;
                else c = borders(e - b, p.seg);
            }
            int x = c;                                     // inclusive prefix over the block
            const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            if (lane == 31) s_warp[warp] = x;
            __syncthreads();
            int before = 0, total = 0;
            for (int w = 0; w < kBlock / 32; ++w) {
                if (w < warp) before += s_warp[w];
                total += s_warp[w];
            }
            const int64_t end = base + before + x;
            if (c > 0 && j < end && j >= end - c) {
                s_hit[0] = n;
                s_hit[1] = (int)(j - (end - c));
            }
            base += total;
            if (__syncthreads_or(bad || (c > 0 && j < end && j >= end - c))) break;
        }
        if (s_bad) {
            if (tid == 0) status_set(p.status, GCL_DEV_BAD_RANGE);
            return false;
        }
        if (s_hit[0] < 0) return false;
        it.n = s_hit[0];
        it.row = j;
        it.bos = p.cu[it.n];
        it.eos = p.cu[it.n + 1];
        it.i = s_hit[1] + (kOwn == rev ? 1 : 0);           // border k lies between segments k and k + 1
    }
    if (it.bos < 0 || it.eos < it.bos || it.eos > p.t_max) {
        if (tid == 0) status_set(p.status, GCL_DEV_BAD_RANGE);
        return false;
    }
    it.s0 = it.bos + (cut ? (int64_t)it.i * p.seg : 0);
    it.s1 = cut && it.s0 + p.seg < it.eos ? it.s0 + p.seg : it.eos;
    it.last = it.s1 == it.eos;
    return true;
}

// Whether the block does nothing, the status word having been set before the call; for the calls that go on past an index
// of their own out of range (bad(i) of i < n), whose blocks start before and after it is found and the word is set.  A word
// that holds GCL_DEV_BAD_RANGE stops the block only if the call has no such index: each block then takes
// the same way.  (Looked up in that case alone.)  Every thread of the block calls it (block barriers).
template <typename Bad>
__device__ __forceinline__ bool call_blocked(const int32_t *status, int64_t n, Bad bad) {
    __shared__ int s_word;
    if (threadIdx.x == 0) s_word = status ? *reinterpret_cast<const volatile int32_t *>(status) : 0;
    __syncthreads();
    if (s_word == 0) return false;
    if (s_word != GCL_DEV_BAD_RANGE) return true;
    bool own = false;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) own |= bad(i);
    return !__syncthreads_or(own);
}

// ---- host checks shared by the entry points that take gcl_rows ---------------
inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline Rows rows(const gcl_rows &r) { return Rows{r.ptr, r.token_stride, r.head_stride}; }
gcl_status_t check_rows(const char *fn, const char *name, const gcl_rows &r, int64_t tokens, int64_t heads, int32_t D,
                        int32_t esize, bool output);
gcl_status_t check_sizes(const char *fn, int32_t H, int32_t K, int32_t V, int32_t dtype);

// CTAs per SM that the CUDA-core engine is built for: two where shared memory and registers allow.
__host__ __device__ constexpr int simt_ctas(int na, int nv) { return na == 64 && nv == 64 ? 2 : 1; }

// ---- launchers ------------------------------------------------------------
// CUDA cores, fp32 arithmetic (fp32 and fp16 rows).  own_states: the segments' own states only (roles kFwd
// and kDv); otherwise the outputs of the given roles.
template <typename T>
cudaError_t launch_simt_t(const Params &p, bool own_states, int n_roles, const int *roles, cudaStream_t s);
cudaError_t launch(const Params &p, int dtype, bool own_states, int n_roles, const int *roles, cudaStream_t s);
// Tensor cores, bf16.
cudaError_t launch_tc(const Params &p, bool own_states, int n_roles, const int *roles, cudaStream_t s);
// The states at the segments' borders, in place of the segments' own.
cudaError_t launch_scan(const Params &p, bool backward, cudaStream_t s);

}  // namespace dla
}  // namespace gcl
