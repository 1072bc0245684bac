// linattn.cuh -- what the kernels of linear attention with a decay share: the
// cut of the sequences into chunks, and a chunk's decays.
//
// A chunk is up to C consecutive tokens of one sequence.  Without cu_seqlens
// every row holds ceil(T / C) chunks and they are found by arithmetic; packed
// sequences get a table, made on the device by table_kernel at the start of a
// call.  The tokens before the first and after the last packed sequence form
// filler chunks (seq -1), whose outputs are zeros.
#pragma once

#include <stdint.h>

#include "layer_ops.h"

namespace gdn {
namespace la {

// Where a call's tables and chunk states are.
struct View {
    const int4 *chunks;  // [n_chunks] {row, first token, tokens, sequence}; null without cu
    const int4 *seqs;    // [n_seq] {first chunk, chunks, first token, tokens}
    int n_chunks;        // of the call (with cu: at most)
    int per_row;         // chunks of a row (without cu)
};

struct Chunk {
    int row, t0, len, seq;
};

template <int C>
__device__ __forceinline__ Chunk chunk_at(const View &v, int T, int ci) {
    if (v.chunks) {
        const int4 e = v.chunks[ci];
        return {e.x, e.y, e.z, e.w};
    }
    const int row = ci / v.per_row, t0 = (ci - row * v.per_row) * C;
    return {row, t0, min(C, T - t0), row};
}

// {first chunk, chunks} of a sequence.
__device__ __forceinline__ int2 seq_at(const View &v, int s) {
    if (v.seqs) {
        const int4 e = v.seqs[s];
        return make_int2(e.x, e.y);
    }
    return make_int2(s * v.per_row, v.per_row);
}

// A sequence's tokens, cut to the row: also for offsets out of order or range.
struct Span {
    int start, len;
};
__device__ __forceinline__ Span span_of(const LinAttnArgs &a, int s) {
    if (!a.cu) return {0, a.T};
    const int start = min(max(a.cu[s], 0), a.T);
    return {start, max(min(a.cu[s + 1], a.T) - start, 0)};
}

inline int chunk_bound(const LinAttnArgs &a, int C) {
    if (a.cu) return a.T / C + a.n_seq + 2;
    return (int)((long long)a.B * ((a.T + C - 1) / C));
}

// {first chunk, chunks} of n chunks from `at` on in a table with room for
// `bound`.  In 64 bits: sequences of offsets out of order overlap, and up to
// 65534 of them may count every token.
__host__ __device__ inline int2 in_table(long long at, int n, int bound) {
    const long long room = at < bound ? bound - at : 0;
    return make_int2((int)(bound - room), (int)(n < room ? n : room));
}

// Bytes of the tables (a multiple of 256).
inline size_t table_bytes(const LinAttnArgs &a, int C) {
    if (!a.cu) return 0;
    return (((size_t)chunk_bound(a, C) + a.n_seq) * sizeof(int4) + 255) / 256 * 256;
}

// Fills the view of a call whose tables lie at `ws`, launching table_kernel
// where there is something to make.
int make_view(const LinAttnArgs &a, int C, void *ws, View *v, cudaStream_t stream);

// Log-decays below this are taken as it: exp(-100) is under the smallest
// normal fp32 number, and sums over a chunk stay finite (g = -inf clears the
// state).  A NaN stays one.
__device__ __forceinline__ float clamp_g(float g) { return g < -100.f ? -100.f : g; }

// A sum carried as hi + lo, to about 2^-45 (64-bit arithmetic is slow on this
// GPU: a chunk's sums took a warp 4,300 cycles in it, and take 700 so).
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair add(const Pair &a, const Pair &b) {
    const float s = a.hi + b.hi, bb = s - a.hi;
    const float e = ((a.hi - (s - bb)) + (b.hi - bb)) + (a.lo + b.lo);
    const float hi = s + e;
    return {hi, e - (hi - s)};
}

// The running sums of a chunk's log-decays, by one warp: cum[t] = g_0 + .. +
// g_t, and all of them.  Differences of two sums, (a.hi - b.hi) + (a.lo -
// b.lo), carry the error of the difference alone, not of its two large terms.
// Tokens past len count 0.
template <int C>
struct Gates {
    static constexpr int P = C / 32;  // lane's tokens: lane P .. lane P + P - 1
    Pair cum[P], all;
    __device__ __forceinline__ float to_end(int i) const { return (all.hi - cum[i].hi) + (all.lo - cum[i].lo); }
};

// The lane's gates, as loaded ..
template <int C>
__device__ __forceinline__ void load_gates(const float *g, long long step, int len, bool per_head,
                                           float (&gt)[C / 32]) {
#pragma unroll
    for (int i = 0; i < C / 32; ++i) {
        const int t = (threadIdx.x & 31) * (C / 32) + i;
        gt[i] = t < len ? clamp_g(per_head ? g[0] : g[t * step]) : 0.f;
    }
}

// .. and their sums over the warp.
template <int C>
__device__ __forceinline__ Gates<C> scan_gates(const float (&gt)[C / 32]) {
    constexpr int P = Gates<C>::P;
    const int lane = threadIdx.x & 31;
    Gates<C> r;
    r.cum[0] = {gt[0], 0.f};
#pragma unroll
    for (int i = 1; i < P; ++i) r.cum[i] = add(r.cum[i - 1], {gt[i], 0.f});
    Pair run = r.cum[P - 1];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const Pair y = {__shfl_up_sync(~0u, run.hi, m), __shfl_up_sync(~0u, run.lo, m)};
        const Pair z = add(run, y);
        if (lane >= m) run = z;
    }
    r.all = {__shfl_sync(~0u, run.hi, 31), __shfl_sync(~0u, run.lo, 31)};
    Pair before = {__shfl_up_sync(~0u, run.hi, 1), __shfl_up_sync(~0u, run.lo, 1)};
    if (lane == 0) before = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < P; ++i) r.cum[i] = add(before, r.cum[i]);
    return r;
}

template <int C>
__device__ __forceinline__ void gates(const float *g, long long step, int len, bool per_head, float *cum_hi,
                                      float *cum_lo, float *to_end) {
    float gt[C / 32];
    load_gates<C>(g, step, len, per_head, gt);
    const Gates<C> r = scan_gates<C>(gt);
#pragma unroll
    for (int i = 0; i < Gates<C>::P; ++i) {
        const int t = (threadIdx.x & 31) * Gates<C>::P + i;
        cum_hi[t] = r.cum[i].hi;
        cum_lo[t] = r.cum[i].lo;
        to_end[t] = r.to_end(i);
    }
}

// exp(cum[t] - cum[s]) from the pairs.
__device__ __forceinline__ float decay_between(float hi_t, float lo_t, float hi_s, float lo_s) {
    return expf((hi_t - hi_s) + (lo_t - lo_s));
}

// Where head h's log-decays of a chunk start.
__device__ __forceinline__ const float *gate_ptr(const LinAttnArgs &a, const Chunk &c, int h) {
    return (a.flags & GDN_G_PER_HEAD) ? a.g + h : a.g + c.row * a.sg.b + h * a.sg.h + c.t0 * a.sg.t;
}

// First element of head h of token t of a strided tensor.
template <typename T>
__device__ __forceinline__ T *at(T *p, const Strides &s, int row, int h, int t) {
    return p + row * s.b + h * s.h + t * s.t;
}

// Sums the value heads' shares [B,H,T,Dk] fp32 of the shared heads' gradients
// into dq and dk (strided, the tensors' type).
int launch_group_sum(const LinAttnArgs &a, const float *dqh, const float *dkh, cudaStream_t stream);
// dg[h] = sum over b, t of src [B,H,T].
int launch_head_sum(const float *src, float *dg, int B, int H, int T, cudaStream_t stream);

}  // namespace la

// The tensor-core path (linattn_tc.cu).
bool linattn_tc_supported(const LinAttnArgs &a);
size_t linattn_tc_fwd_workspace(const LinAttnArgs &a);
int launch_linattn_tc_fwd(const LinAttnArgs &a, cudaStream_t stream);
size_t linattn_tc_bwd_workspace(const LinAttnArgs &a);
int launch_linattn_tc_bwd(const LinAttnArgs &a, cudaStream_t stream);
int linattn_tc_read_clear_error();

}  // namespace gdn
