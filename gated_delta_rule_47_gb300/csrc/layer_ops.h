// Internal declarations of the operators around a linear-attention layer:
// prompts (forward and backward), single-token steps, the residual norm and
// the pool of recurrent states.  Their entry points are in layer_api.cu.
#pragma once

#include <cstddef>
#include <cuda_runtime.h>

#include "gdn.h"

namespace gdn {

// Element strides of a [B,H,T,D] tensor whose last dimension is contiguous.
struct Strides {
    long long b, h, t;
};

// Arguments of one linear-attention prompt call, forward or backward.  Without
// cu every row b is one sequence of T tokens; with it (B = 1) sequence s holds
// tokens cu[s] .. cu[s+1]-1.
struct LinAttnArgs {
    const void *q, *k, *v;
    const float *g;  // [B,H,T], or [H] with GDN_G_PER_HEAD
    const float *s0;
    void *o;
    float *sf;
    const void *dout;
    const float *dsf;
    void *dq, *dk, *dv;
    float *dg, *ds0;
    const int *cu;
    Strides sq, sk, sv, so, sdo;  // of q, k, v, o / dout; gradients have their tensors' strides
    Strides sg;
    int n_seq;
    int B, H, Hk, T, Dk, Dv;
    float scale;
    unsigned flags;
    int dtype;
    void *ws;
    size_t ws_bytes;
};

size_t linattn_fwd_workspace(const LinAttnArgs &a);
int launch_linattn_fwd(const LinAttnArgs &a, cudaStream_t stream);
size_t linattn_bwd_workspace(const LinAttnArgs &a);
int launch_linattn_bwd(const LinAttnArgs &a, cudaStream_t stream);

struct StepArgs {
    const void *q, *k, *v, *beta;  // beta null: plain decay attention
    const float *g;
    const float *state;
    float *state_out;
    const int *slots;  // null: row b's state is page b
    void *o;
    int B, H, Hk, Dk, Dv, n_slots;
    float scale;
    unsigned flags;
    int dtype;
};
int launch_step(const StepArgs &a, cudaStream_t stream);

struct NormArgs {
    const void *x, *res;
    const float *w;
    void *y;
    float *scales;
    void *h;
    long long rows;
    int C, group;  // group 0: one scale a row
    float eps;
    int dtype, out_e4m3;
};
int launch_rms_norm(const NormArgs &a, cudaStream_t stream);

struct NormBwdArgs {
    const void *dy, *h, *dres;
    const float *w;
    void *dx;
    float *dw;
    long long rows;
    int C;
    float eps;
    int dtype;
    void *ws;
};
size_t rms_norm_bwd_workspace(long long rows, int C);
int launch_rms_norm_bwd(const NormBwdArgs &a, cudaStream_t stream);

// A pool of pages: [layers][n_slots][page_bytes].
struct PoolArgs {
    void *pool;
    int layers, n_slots;
    long long page_bytes;
};
int launch_pool_copy(const PoolArgs &p, const int *src, const int *dst, int n, cudaStream_t stream);
size_t pool_fork_workspace(int n_slots, int n);
int launch_pool_fork(const PoolArgs &p, unsigned char *live, const int *parents, int *children, int n, void *ws,
                     cudaStream_t stream);
int launch_pool_free(unsigned char *live, int n_slots, const int *slots, int n, cudaStream_t stream);
size_t pool_compact_workspace(int n_slots);
int launch_pool_compact(const PoolArgs &p, unsigned char *live, int *remap, int *n_live, void *ws,
                        cudaStream_t stream);

}  // namespace gdn
