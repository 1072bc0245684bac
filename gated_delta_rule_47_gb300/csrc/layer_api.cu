// layer_api.cu -- the extern "C" boundary of the operators around a
// linear-attention layer (layer_ops.h): host-side checks, status codes, the
// choice between the tensor-core and CUDA-core prompt kernels.  As in
// gdn_api.cu nothing is allocated, nothing waits and no exception crosses.
#include <cuda_runtime.h>

#include <algorithm>
#include <utility>

#include "api_util.h"
#include "gdn_internal.h"
#include "layer_ops.h"
#include "linattn.cuh"

namespace {

using gdn::LinAttnArgs;
using gdn::Range;
using gdn::Strides;
using gdn::aligned16;

bool bad_dims(int Dk, int Dv) { return (Dk != 64 && Dk != 128) || (Dv != 64 && Dv != 128); }

// Strides: 16-byte multiples that keep a vector load aligned.
bool bad_strides(const Strides &s, int dtype) {
    const long long m = dtype == GDN_BF16 ? 7 : 3;
    return ((s.b | s.h | s.t) & m) != 0;
}
bool negative(const Strides &s) { return s.b < 0 || s.h < 0 || s.t < 0; }

// Whether elements of a [B,H,T,D] tensor that is written may share memory: a
// dimension steps by less than those of smaller steps span.
bool overlaps(const Strides &s, int B, int H, int T, int D) {
    std::pair<long long, int> by[3] = {{s.b, B}, {s.h, H}, {s.t, T}};
    std::sort(by, by + 3);
    long long span = D;
    for (const auto &d : by) {
        if (d.second <= 1) continue;
        if (d.first < span) return true;
        span += d.first * (d.second - 1);
    }
    return false;
}

Strides dense(int H, int T, int D) { return {(long long)H * T * D, (long long)T * D, D}; }

// Sizes alone (also of a workspace query).
int check_sizes(const LinAttnArgs &a) {
    if (a.B < 0 || a.H < 0 || a.Hk < 0 || a.T < 0 || a.n_seq < 0) return GDN_ERR_INVALID_ARG;
    if (a.dtype != GDN_F32 && a.dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (a.flags & ~(GDN_PATH_SIMT | GDN_G_PER_HEAD)) return GDN_ERR_INVALID_ARG;
    if (a.H > 0 && (a.Hk == 0 || a.H % a.Hk != 0)) return GDN_ERR_INVALID_ARG;
    if (a.cu && a.B != 1) return GDN_ERR_INVALID_ARG;
    if (!a.cu && a.n_seq != a.B) return GDN_ERR_INVALID_ARG;
    if (bad_dims(a.Dk, a.Dv)) return GDN_ERR_UNSUPPORTED;
    if (a.H > 65535 || a.B > 65534 || a.n_seq > 65534 || a.T > (1 << 30)) return GDN_ERR_UNSUPPORTED;
    if (((long long)a.B * ((a.T + 63) / 64) + a.n_seq + 2) * (a.H ? a.H : 1) > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

void read_strides(LinAttnArgs *a, const long long *s) {
    a->sq = a->sk = dense(a->Hk, a->T, a->Dk);
    a->sv = a->so = a->sdo = dense(a->H, a->T, a->Dv);
    a->sg = dense(a->H, a->T, 1);
    if (!s) return;
    Strides *to[] = {&a->sq, &a->sk, &a->sv, &a->so, &a->sg};
    for (int i = 0; i < 5; ++i) *to[i] = {s[3 * i], s[3 * i + 1], s[3 * i + 2]};
    a->sdo = a->so;
}

int check_tensors(const LinAttnArgs &a) {
    const Strides *ss[] = {&a.sq, &a.sk, &a.sv, &a.so};
    for (const Strides *s : ss) {
        if (negative(*s)) return GDN_ERR_INVALID_ARG;
        if (bad_strides(*s, a.dtype)) return GDN_ERR_MISALIGNED;
    }
    if (negative(a.sg)) return GDN_ERR_INVALID_ARG;
    const void *ps[] = {a.q, a.k, a.v, a.o, a.dout, a.dq, a.dk, a.dv, a.s0, a.sf, a.dsf, a.ds0};
    for (const void *p : ps)
        if (p && !aligned16(p)) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}

// The state (or its gradient) where no token touches it.
int pass_state(const float *from, float *to, const LinAttnArgs &a, cudaStream_t stream) {
    const size_t bytes = sizeof(float) * (size_t)a.n_seq * a.H * a.Dk * a.Dv;
    if (!to || bytes == 0) return GDN_OK;
    const cudaError_t e = from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, stream)
                               : cudaMemsetAsync(to, 0, bytes, stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t fwd_workspace(const LinAttnArgs &a) {
    return gdn::linattn_tc_supported(a) ? gdn::linattn_tc_fwd_workspace(a) : gdn::linattn_fwd_workspace(a);
}
size_t bwd_workspace(const LinAttnArgs &a) {
    return gdn::linattn_tc_supported(a) ? gdn::linattn_tc_bwd_workspace(a) : gdn::linattn_bwd_workspace(a);
}

bool empty(const LinAttnArgs &a) { return (long long)a.B * a.H * a.T == 0; }

LinAttnArgs sized(int B, int H, int Hk, int T, int Dk, int Dv, int n_seq, bool packed, unsigned flags, int dtype) {
    static const int none = 0;
    LinAttnArgs a{};
    a.B = B, a.H = H, a.Hk = Hk, a.T = T, a.Dk = Dk, a.Dv = Dv;
    a.n_seq = n_seq, a.cu = packed ? &none : nullptr, a.flags = flags, a.dtype = dtype;  // cu: only whether it is null
    return a;
}

int check_step(const gdn::StepArgs &a, unsigned allowed) {
    if (a.B < 0 || a.H < 0 || a.Hk < 0 || a.n_slots < 0) return GDN_ERR_INVALID_ARG;
    if (a.dtype != GDN_F32 && a.dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (a.flags & ~allowed) return GDN_ERR_INVALID_ARG;
    if (a.H > 0 && (a.Hk == 0 || a.H % a.Hk != 0)) return GDN_ERR_INVALID_ARG;
    if (!a.slots && a.B > a.n_slots) return GDN_ERR_INVALID_ARG;
    if (bad_dims(a.Dk, a.Dv) || a.H > 65535) return GDN_ERR_UNSUPPORTED;
    if ((long long)a.B * a.H == 0) return GDN_OK;
    if (!a.q || !a.k || !a.v || !a.g || !a.state || !a.state_out || !a.o) return GDN_ERR_INVALID_ARG;
    const void *ps[] = {a.q, a.k, a.v, a.state, a.state_out, a.o};
    for (const void *p : ps)
        if (!aligned16(p)) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}

int check_pool(const gdn::PoolArgs &p) {
    if (p.layers < 0 || p.n_slots < 0 || p.page_bytes < 0) return GDN_ERR_INVALID_ARG;
    if (p.page_bytes % 16 != 0) return GDN_ERR_MISALIGNED;
    if (p.pool && !aligned16(p.pool)) return GDN_ERR_MISALIGNED;
    if (!p.pool && p.page_bytes * p.layers * p.n_slots != 0) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}
bool no_pages(const gdn::PoolArgs &p) { return p.page_bytes == 0 || p.layers == 0 || p.n_slots == 0; }

bool short_of(const void *ws, size_t bytes, size_t need) {
    return need > 0 && (ws == nullptr || bytes < need || !aligned16(ws));
}

}  // namespace

extern "C" {

size_t linattn_chunk_fwd_workspace_bytes(int B, int H, int Hk, int T, int Dk, int Dv, int n_seq, int packed,
                                         unsigned flags, int dtype) {
    const LinAttnArgs a = sized(B, H, Hk, T, Dk, Dv, n_seq, packed != 0, flags, dtype);
    if (check_sizes(a) != GDN_OK) return (size_t)-1;
    return empty(a) ? 0 : fwd_workspace(a);
}

int linattn_chunk_fwd(const void *q, const void *k, const void *v, const float *g, const float *initial_state,
                      void *o, float *final_state, const int *cu_seqlens, const long long *strides, int n_seq, int B,
                      int H, int Hk, int T, int Dk, int Dv, float scale, unsigned flags, int dtype, void *workspace,
                      size_t workspace_bytes, void *stream_v) {
    const Range nvtx_range("linattn_chunk_fwd");
    LinAttnArgs a = sized(B, H, Hk, T, Dk, Dv, n_seq, false, flags, dtype);
    a.q = q, a.k = k, a.v = v, a.g = g, a.s0 = initial_state, a.o = o, a.sf = final_state, a.cu = cu_seqlens;
    a.scale = scale, a.ws = workspace, a.ws_bytes = workspace_bytes;
    int st = check_sizes(a);
    if (st != GDN_OK) return st;
    read_strides(&a, strides);
    if (!empty(a) && (!q || !k || !v || !g || !o)) return GDN_ERR_INVALID_ARG;
    st = check_tensors(a);
    if (st != GDN_OK) return st;
    if (!empty(a) && overlaps(a.so, B, H, T, Dv)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    if (empty(a) || n_seq == 0) {
        if (!empty(a)) return GDN_ERR_INVALID_ARG;  // tokens, but no sequence that holds them
        return pass_state(a.s0, a.sf, a, stream);
    }
    if (short_of(workspace, workspace_bytes, fwd_workspace(a))) return GDN_ERR_WORKSPACE;
    return gdn::linattn_tc_supported(a) ? gdn::launch_linattn_tc_fwd(a, stream) : gdn::launch_linattn_fwd(a, stream);
}

size_t linattn_chunk_bwd_workspace_bytes(int B, int H, int Hk, int T, int Dk, int Dv, int n_seq, int packed,
                                         unsigned flags, int dtype) {
    const LinAttnArgs a = sized(B, H, Hk, T, Dk, Dv, n_seq, packed != 0, flags, dtype);
    if (check_sizes(a) != GDN_OK) return (size_t)-1;
    return empty(a) ? 0 : bwd_workspace(a);
}

int linattn_chunk_bwd(const void *q, const void *k, const void *v, const float *g, const float *initial_state,
                      const void *dout, const float *dfinal_state, void *dq, void *dk, void *dv, float *dg,
                      float *dinitial_state, const int *cu_seqlens, const long long *strides, int n_seq, int B, int H,
                      int Hk, int T, int Dk, int Dv, float scale, unsigned flags, int dtype, void *workspace,
                      size_t workspace_bytes, void *stream_v) {
    const Range nvtx_range("linattn_chunk_bwd");
    LinAttnArgs a = sized(B, H, Hk, T, Dk, Dv, n_seq, false, flags, dtype);
    a.q = q, a.k = k, a.v = v, a.g = g, a.s0 = initial_state, a.dout = dout, a.dsf = dfinal_state;
    a.dq = dq, a.dk = dk, a.dv = dv, a.dg = dg, a.ds0 = dinitial_state, a.cu = cu_seqlens;
    a.scale = scale, a.ws = workspace, a.ws_bytes = workspace_bytes;
    int st = check_sizes(a);
    if (st != GDN_OK) return st;
    read_strides(&a, strides);
    if (!empty(a) && (!q || !k || !v || !g || !dout || !dq || !dk || !dv || !dg)) return GDN_ERR_INVALID_ARG;
    st = check_tensors(a);
    if (st != GDN_OK) return st;
    // gradients have these strides
    if (!empty(a) && (overlaps(a.sq, B, Hk, T, Dk) || overlaps(a.sk, B, Hk, T, Dk) || overlaps(a.sv, B, H, T, Dv) ||
                      (!(flags & GDN_G_PER_HEAD) && overlaps(a.sg, B, H, T, 1))))
        return GDN_ERR_INVALID_ARG;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    if (empty(a) || n_seq == 0) {
        if (!empty(a)) return GDN_ERR_INVALID_ARG;
        if (dg && (flags & GDN_G_PER_HEAD) && H > 0 && cudaMemsetAsync(dg, 0, sizeof(float) * H, stream) != cudaSuccess)
            return GDN_ERR_CUDA;
        return pass_state(a.dsf, a.ds0, a, stream);
    }
    if (short_of(workspace, workspace_bytes, bwd_workspace(a))) return GDN_ERR_WORKSPACE;
    return gdn::linattn_tc_supported(a) ? gdn::launch_linattn_tc_bwd(a, stream) : gdn::launch_linattn_bwd(a, stream);
}

int linattn_step(const void *q, const void *k, const void *v, const float *g, const float *state, float *state_out,
                 const int *slots, void *o, int B, int H, int Hk, int Dk, int Dv, int n_slots, float scale,
                 unsigned flags, int dtype, void *stream) {
    const Range nvtx_range("linattn_step");
    const gdn::StepArgs a{q, k, v, nullptr, g, state, state_out, slots, o, B, H, Hk, Dk, Dv, n_slots, scale, flags, dtype};
    const int st = check_step(a, GDN_G_PER_HEAD);
    if (st != GDN_OK || (long long)B * H == 0) return st;
    return gdn::launch_step(a, static_cast<cudaStream_t>(stream));
}

int gdn_step(const void *q, const void *k, const void *v, const void *beta, const float *g, const float *state,
             float *state_out, const int *slots, void *o, int B, int H, int Hk, int Dk, int Dv, int n_slots,
             float scale, unsigned flags, int dtype, void *stream) {
    const Range nvtx_range("gdn_step");
    const gdn::StepArgs a{q, k, v, beta, g, state, state_out, slots, o, B, H, Hk, Dk, Dv, n_slots, scale, flags, dtype};
    const int st = check_step(a, GDN_G_PER_HEAD | GDN_QK_L2NORM);
    if (st != GDN_OK || (long long)B * H == 0) return st;
    if (!beta) return GDN_ERR_INVALID_ARG;
    return gdn::launch_step(a, static_cast<cudaStream_t>(stream));
}

int rms_norm_fwd(const void *x, const void *residual, const float *weight, void *y, float *scales, void *h,
                 long long rows, int C, int group, float eps, int out_e4m3, int dtype, void *stream) {
    const Range nvtx_range("rms_norm_fwd");
    if (rows < 0 || C < 1 || group < 0 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (rows > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    if (group > 0) {
        if (!out_e4m3 || C % group != 0) return GDN_ERR_INVALID_ARG;
        if ((group != 32 && group != 64 && group != 128) || C > 4096 * (dtype == GDN_BF16 ? 8 : 4)) return GDN_ERR_UNSUPPORTED;
    }
    if (rows == 0) return GDN_OK;
    if (!x || !y || (out_e4m3 && !scales)) return GDN_ERR_INVALID_ARG;
    const void *ps[] = {x, residual, weight, y, h};
    for (const void *p : ps)
        if (p && !aligned16(p)) return GDN_ERR_MISALIGNED;
    const gdn::NormArgs a{x, residual, weight, y, scales, h, rows, C, group, eps, dtype, out_e4m3};
    return gdn::launch_rms_norm(a, static_cast<cudaStream_t>(stream));
}

size_t rms_norm_bwd_workspace_bytes(long long rows, int C) {
    if (rows < 0 || C < 1) return (size_t)-1;
    return rows == 0 ? 0 : gdn::rms_norm_bwd_workspace(rows, C);
}

int rms_norm_bwd(const void *dy, const void *h, const float *weight, const void *dresidual, void *dx, float *dweight,
                 long long rows, int C, float eps, int dtype, void *workspace, size_t workspace_bytes,
                 void *stream_v) {
    const Range nvtx_range("rms_norm_bwd");
    if (rows < 0 || C < 1 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (!dweight) return GDN_ERR_INVALID_ARG;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    if (rows == 0) return cudaMemsetAsync(dweight, 0, sizeof(float) * C, stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    if (!dy || !h || !dx) return GDN_ERR_INVALID_ARG;
    const void *ps[] = {dy, h, weight, dresidual, dx, dweight};
    for (const void *p : ps)
        if (p && !aligned16(p)) return GDN_ERR_MISALIGNED;
    if (short_of(workspace, workspace_bytes, gdn::rms_norm_bwd_workspace(rows, C))) return GDN_ERR_WORKSPACE;
    const gdn::NormBwdArgs a{dy, h, dresidual, weight, dx, dweight, rows, C, eps, dtype, workspace};
    return gdn::launch_rms_norm_bwd(a, stream);
}

int state_pool_copy(void *pool, int layers, int n_slots, long long page_bytes, const int *src, const int *dst, int n,
                    void *stream) {
    const Range nvtx_range("state_pool_copy");
    const gdn::PoolArgs p{pool, layers, n_slots, page_bytes};
    const int st = check_pool(p);
    if (st != GDN_OK) return st;
    if (n < 0 || (n > 0 && (!src || !dst))) return GDN_ERR_INVALID_ARG;
    if (n == 0 || no_pages(p)) return GDN_OK;
    return gdn::launch_pool_copy(p, src, dst, n, static_cast<cudaStream_t>(stream));
}

size_t state_pool_fork_workspace_bytes(int n_slots, int n) {
    return n_slots < 0 || n < 0 ? (size_t)-1 : gdn::pool_fork_workspace(n_slots, n);
}

int state_pool_fork(void *pool, int layers, int n_slots, long long page_bytes, unsigned char *live,
                    const int *parents, int *children, int n, void *workspace, size_t workspace_bytes, void *stream) {
    const Range nvtx_range("state_pool_fork");
    const gdn::PoolArgs p{pool, layers, n_slots, page_bytes};
    const int st = check_pool(p);
    if (st != GDN_OK) return st;
    if (n < 0) return GDN_ERR_INVALID_ARG;
    if (n == 0) return GDN_OK;
    if (!parents || !children || (n_slots > 0 && !live)) return GDN_ERR_INVALID_ARG;
    if (short_of(workspace, workspace_bytes, gdn::pool_fork_workspace(n_slots, n))) return GDN_ERR_WORKSPACE;
    return gdn::launch_pool_fork(p, live, parents, children, n, workspace, static_cast<cudaStream_t>(stream));
}

int state_pool_free(unsigned char *live, int n_slots, const int *slots, int n, void *stream) {
    const Range nvtx_range("state_pool_free");
    if (n_slots < 0 || n < 0) return GDN_ERR_INVALID_ARG;
    if (n == 0 || n_slots == 0) return GDN_OK;
    if (!live || !slots) return GDN_ERR_INVALID_ARG;
    return gdn::launch_pool_free(live, n_slots, slots, n, static_cast<cudaStream_t>(stream));
}

size_t state_pool_compact_workspace_bytes(int n_slots) {
    return n_slots < 0 ? (size_t)-1 : gdn::pool_compact_workspace(n_slots);
}

int state_pool_compact(void *pool, int layers, int n_slots, long long page_bytes, unsigned char *live, int *remap,
                       int *n_live, void *workspace, size_t workspace_bytes, void *stream) {
    const Range nvtx_range("state_pool_compact");
    const gdn::PoolArgs p{pool, layers, n_slots, page_bytes};
    const int st = check_pool(p);
    if (st != GDN_OK) return st;
    if (!n_live || (n_slots > 0 && (!live || !remap))) return GDN_ERR_INVALID_ARG;
    if (short_of(workspace, workspace_bytes, gdn::pool_compact_workspace(n_slots))) return GDN_ERR_WORKSPACE;
    return gdn::launch_pool_compact(p, live, remap, n_live, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
