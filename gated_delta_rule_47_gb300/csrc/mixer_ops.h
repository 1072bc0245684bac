// Internal declarations of the operators next to a recurrent layer's mixer: the
// short causal convolution, the selective state space scan, the gated norm by
// head and the norms around a block.  Their entry points are in mixer_api.cu.
#pragma once

#include <cstddef>
#include <cuda_runtime.h>

#include "gdn.h"

namespace gdn {

// Element strides of a [B,T,C] tensor whose channels are contiguous.
struct RowStrides {
    long long b, t;
};

// Arguments of one convolution, forward or backward.  Without cu every row b is
// one sequence of T tokens; with it (B = 1) sequence s holds tokens cu[s] ..
// cu[s+1]-1.
struct ConvArgs {
    const void *x;
    const float *w, *bias;
    const void *win;  // [n_seq,W-1,C] or null
    void *y, *win_out;
    const void *dy, *dwin_out;
    void *dx, *dwin;
    float *dw, *db;
    const int *cu;
    RowStrides sx, sy;  // of x (and dx: contiguous) and y / dy
    int n_seq, B, T, C, W;
    unsigned flags;
    int dtype;
    void *ws;
};
int launch_conv_fwd(const ConvArgs &a, cudaStream_t stream);
size_t conv_bwd_workspace(int B, int T, int C, int W);
int launch_conv_bwd(const ConvArgs &a, cudaStream_t stream);

struct ConvStepArgs {
    const void *x;
    const float *w, *bias;
    const void *win;
    void *win_out;
    const int *slots;  // null: row b's window is page b
    void *y;
    long long sx;  // row stride of x
    int B, C, W, n_slots;
    unsigned flags;
    int dtype;
};
int launch_conv_step(const ConvStepArgs &a, cudaStream_t stream);

// Arguments of one scan, forward or backward.
struct SsmArgs {
    const void *x, *dt, *Bt, *Ct, *z;
    const float *A, *D, *bias, *s0;
    void *y;
    float *sf;
    const void *dy;
    const float *dsf;
    void *dx, *ddt, *dB, *dC, *dz;  // contiguous
    float *dA, *dD, *dbias, *ds0;
    const int *cu;
    RowStrides sx, sdt, sB, sC, sz, sy;  // sy: of y or dy
    int n_seq, B, T, Di, N;
    unsigned flags;
    int dtype;
    void *ws;
};
size_t ssm_fwd_workspace(int B, int T, int Di, int N, int dtype);
int launch_ssm_fwd(const SsmArgs &a, cudaStream_t stream);
size_t ssm_bwd_workspace(int B, int T, int Di, int N, int dtype);
int launch_ssm_bwd(const SsmArgs &a, cudaStream_t stream);

struct SsmStepArgs {
    const void *x, *dt, *Bt, *Ct, *z;
    const float *A, *D, *bias, *state;
    float *state_out;
    const int *slots;  // null: row b's state is page b
    void *y;
    long long sx, sdt, sB, sC, sz;  // row strides
    int B, Di, N, n_slots;
    unsigned flags;
    int dtype;
};
int launch_ssm_step(const SsmStepArgs &a, cudaStream_t stream);

// Element strides of a [B,T,H,D] tensor whose last dimension is contiguous.
struct HeadStrides {
    long long b, t, h;
};
struct GatedNormArgs {
    const void *x, *gate;
    const float *w;
    void *y;
    const void *dy;
    void *dx, *dgate;  // dx: the strides of x; dgate: contiguous
    float *dw;
    HeadStrides sx, sg, sdy, sdx;  // y and dgate are contiguous
    int B, T, H, D;
    float eps;
    unsigned flags;
    int dtype;
    void *ws;
};
int launch_gated_norm(const GatedNormArgs &a, cudaStream_t stream);
size_t gated_norm_bwd_workspace(int B, int T, int H, int D, unsigned flags);
int launch_gated_norm_bwd(const GatedNormArgs &a, cudaStream_t stream);

struct BlockNormArgs {
    const void *x, *res;
    const float *w1, *s, *w2;  // weights of the norm after and before a block, scale [groups,C]
    void *y, *h;
    const void *dy, *dh;  // backward: h is an input
    void *dx, *dres;
    float *dw1, *ds, *dw2;
    long long rows;
    int C, groups;
    float eps;
    int dtype;
    void *ws;
};
int launch_block_norm(const BlockNormArgs &a, cudaStream_t stream);
size_t block_norm_bwd_workspace(long long rows, int C, int groups);
int launch_block_norm_bwd(const BlockNormArgs &a, cudaStream_t stream);

}  // namespace gdn
