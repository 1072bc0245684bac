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

inline int chunk_bound(const LinAttnArgs &a, int C) {
    if (a.cu) return a.T / C + a.n_seq + 2;
    return (int)((long long)a.B * ((a.T + C - 1) / C));
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

// The running sums of a chunk's log-decays, by one warp: cum[t] = g_0 + .. +
// g_t as a pair hi + lo (so that cum[t] - cum[s] carries the error of the
// difference alone, not of its two large terms), and to_end[t] = g_{t+1} + ..
// The sums are made in 64 bits.  Tokens past len count 0.
template <int C>
struct Gates {
    static constexpr int P = C / 32;  // lane's tokens: lane P .. lane P + P - 1
    double cum[P], all;
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
    double sum = 0.;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        sum += gt[i];
        r.cum[i] = sum;
    }
    double run = sum;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const double y = __shfl_up_sync(~0u, run, m);
        if (lane >= m) run += y;
    }
    r.all = __shfl_sync(~0u, run, 31);
#pragma unroll
    for (int i = 0; i < P; ++i) r.cum[i] += run - sum;
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
        const float hi = (float)r.cum[i];
        cum_hi[t] = hi;
        cum_lo[t] = (float)(r.cum[i] - (double)hi);
        to_end[t] = (float)(r.all - r.cum[i]);
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

// Sums the value heads' shares of the shared heads' gradients: dst (strided,
// the tensors' type) [B,Hk,T,D] from src [B,H,T,D] fp32.
int launch_group_sum(const float *src, void *dst, const Strides &s, int B, int H, int Hk, int T, int D, int dtype,
                     cudaStream_t stream);
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
