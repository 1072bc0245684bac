// mixer_api.cu -- the extern "C" boundary of the operators next to a mixer
// (mixer_ops.h): host-side checks and status codes.  As in gdn_api.cu nothing is
// allocated, nothing waits and no exception crosses.
#include <cuda_runtime.h>

#include <algorithm>
#include <utility>

#include "api_util.h"
#include "gdn_internal.h"
#include "mixer_ops.h"

namespace {

using gdn::Range;
using gdn::RowStrides;
using gdn::aligned16;

bool bad_type(int dtype) { return dtype != GDN_F32 && dtype != GDN_BF16; }
int wide(int dtype) { return dtype == GDN_BF16 ? 8 : 4; }  // elements of 16 bytes

bool misaligned(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p && !aligned16(p)) return true;
    return false;
}
bool short_of(const void *ws, size_t bytes, size_t need) { return need > 0 && (ws == nullptr || bytes < need || !aligned16(ws)); }

// Strides that are read: not negative, whole vectors.
int check_strides(const long long *s, int n, int dtype) {
    for (int i = 0; i < n; ++i) {
        if (s[i] < 0) return GDN_ERR_INVALID_ARG;
        if (s[i] % wide(dtype) != 0) return GDN_ERR_MISALIGNED;
    }
    return GDN_OK;
}

// Whether elements of a tensor that is written may share memory: a dimension steps
// by less than those of smaller steps span.
bool overlaps(std::initializer_list<std::pair<long long, int>> dims, int D) {
    std::pair<long long, int> by[3];
    int n = 0;
    for (const auto &d : dims) by[n++] = d;
    std::sort(by, by + n);
    long long span = D;
    for (int i = 0; i < n; ++i) {
        if (by[i].second <= 1) continue;
        if (by[i].first < span) return true;
        span += by[i].first * (by[i].second - 1);
    }
    return false;
}

// Rows and sequences of a convolution or scan.
int check_rows(const int *cu, int n_seq, int B, int T, int C) {
    if (B < 0 || T < 0 || C < 0 || n_seq < 0) return GDN_ERR_INVALID_ARG;
    if (cu ? B != 1 : n_seq != B) return GDN_ERR_INVALID_ARG;
    if (B > 65534 || n_seq > 65534 || T > (1 << 30) || C > (1 << 24)) return GDN_ERR_UNSUPPORTED;
    if ((long long)B * T > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// What a sequence carries, where there are no tokens.
int pass_on(const void *from, void *to, size_t bytes, cudaStream_t stream) {
    if (!to || bytes == 0) return GDN_OK;
    const cudaError_t e = from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, stream) : cudaMemsetAsync(to, 0, bytes, stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
int zeros(float *p, size_t n, cudaStream_t stream) { return pass_on(nullptr, p, n * sizeof(float), stream); }

int check_conv(int W, int C, unsigned flags, int dtype) {
    if (bad_type(dtype) || (flags & ~GDN_SILU)) return GDN_ERR_INVALID_ARG;
    if (W < 2 || W > 4 || C % wide(dtype) != 0) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}
int check_scan(int Di, int N, unsigned flags, int dtype) {
    if (bad_type(dtype) || (flags & ~GDN_DT_SOFTPLUS)) return GDN_ERR_INVALID_ARG;
    if ((N != 8 && N != 16 && N != 32) || Di % wide(dtype) != 0) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}
// CTAs and 32-bit places of a scan.
int check_scan_size(int B, int T, int Di, int N) {
    const long long items = (long long)B * ((T + 63) / 64) * ((Di + 31) / 32);
    return items > 0x7fffffffLL || (long long)Di * N > 0x7fffffffLL ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

int check_slots(const int *slots, int B, int n_slots) {
    if (B < 0 || n_slots < 0 || (!slots && B > n_slots)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

gdn::SsmArgs scan_args(const void *x, const void *dt, const float *A, const void *Bt, const void *Ct, const float *skip,
                       const void *z, const float *bias, const float *s0, const int *cu, const long long *st, int n_seq, int B,
                       int T, int Di, int N, unsigned flags, int dtype, void *ws) {
    gdn::SsmArgs a{};
    a.x = x, a.dt = dt, a.A = A, a.Bt = Bt, a.Ct = Ct, a.D = skip, a.z = z, a.bias = bias, a.s0 = s0, a.cu = cu;
    a.n_seq = n_seq, a.B = B, a.T = T, a.Di = Di, a.N = N, a.flags = flags, a.dtype = dtype, a.ws = ws;
    const RowStrides wide_row{(long long)T * Di, Di}, small{(long long)T * N, N};
    a.sx = a.sdt = a.sz = a.sy = wide_row, a.sB = a.sC = small;
    if (st) {
        RowStrides *to[] = {&a.sx, &a.sdt, &a.sB, &a.sC, &a.sz, &a.sy};
        for (int i = 0; i < 6; ++i) *to[i] = {st[2 * i], st[2 * i + 1]};
    }
    return a;
}

}  // namespace

extern "C" {

int causal_conv_fwd(const void *x, const float *weight, const float *bias, const void *initial_window, void *y,
                    void *final_window, const int *cu_seqlens, const long long *strides, int n_seq, int B, int T, int C, int W,
                    unsigned flags, int dtype, void *stream_v) {
    const Range nvtx_range("causal_conv_fwd");
    int st = check_rows(cu_seqlens, n_seq, B, T, C);
    if (st == GDN_OK) st = check_conv(W, C, flags, dtype);
    if (st == GDN_OK && strides) st = check_strides(strides, 4, dtype);
    if (st != GDN_OK) return st;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    if (misaligned({x, weight, bias, initial_window, y, final_window})) return GDN_ERR_MISALIGNED;
    if ((long long)B * T * C == 0)
        return pass_on(initial_window, final_window, (size_t)n_seq * (W - 1) * C * (dtype == GDN_BF16 ? 2 : 4), stream);
    if (!x || !weight || !y || n_seq == 0) return GDN_ERR_INVALID_ARG;
    gdn::ConvArgs a{};
    a.x = x, a.w = weight, a.bias = bias, a.win = initial_window, a.y = y, a.win_out = final_window, a.cu = cu_seqlens;
    a.sx = a.sy = {(long long)T * C, C};
    if (strides) a.sx = {strides[0], strides[1]}, a.sy = {strides[2], strides[3]};
    if (overlaps({{a.sy.b, B}, {a.sy.t, T}}, C)) return GDN_ERR_INVALID_ARG;
    a.n_seq = n_seq, a.B = B, a.T = T, a.C = C, a.W = W, a.flags = flags, a.dtype = dtype;
    return gdn::launch_conv_fwd(a, stream);
}

size_t causal_conv_bwd_workspace_bytes(int B, int T, int C, int W) {
    if (check_rows(nullptr, B, B, T, C) != GDN_OK || W < 2 || W > 4 || C % 4 != 0) return (size_t)-1;
    return (long long)B * T * C == 0 ? 0 : gdn::conv_bwd_workspace(B, T, C, W);
}

int causal_conv_bwd(const void *x, const float *weight, const float *bias, const void *dy, const void *initial_window,
                    const void *dfinal_window, void *dx, float *dweight, float *dbias, void *dinitial_window,
                    const int *cu_seqlens, const long long *strides, int n_seq, int B, int T, int C, int W, unsigned flags,
                    int dtype, void *workspace, size_t workspace_bytes, void *stream_v) {
    const Range nvtx_range("causal_conv_bwd");
    int st = check_rows(cu_seqlens, n_seq, B, T, C);
    if (st == GDN_OK) st = check_conv(W, C, flags, dtype);
    if (st == GDN_OK && strides) st = check_strides(strides, 4, dtype);
    if (st != GDN_OK) return st;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    if (misaligned({x, weight, bias, dy, initial_window, dfinal_window, dx, dweight, dbias, dinitial_window})) return GDN_ERR_MISALIGNED;
    if (C > 0 && !dweight) return GDN_ERR_INVALID_ARG;
    if ((long long)B * T * C == 0) {
        st = zeros(dweight, (size_t)C * W, stream);
        if (st == GDN_OK) st = zeros(dbias, C, stream);
        if (st != GDN_OK) return st;
        return pass_on(dfinal_window, dinitial_window, (size_t)n_seq * (W - 1) * C * (dtype == GDN_BF16 ? 2 : 4), stream);
    }
    if (!x || !weight || !dy || !dx || n_seq == 0) return GDN_ERR_INVALID_ARG;
    if (short_of(workspace, workspace_bytes, gdn::conv_bwd_workspace(B, T, C, W))) return GDN_ERR_WORKSPACE;
    gdn::ConvArgs a{};
    a.x = x, a.w = weight, a.bias = bias, a.dy = dy, a.win = initial_window, a.dwin_out = dfinal_window, a.dx = dx;
    a.dw = dweight, a.db = dbias, a.dwin = dinitial_window, a.cu = cu_seqlens, a.ws = workspace;
    a.sx = a.sy = {(long long)T * C, C};
    if (strides) a.sx = {strides[0], strides[1]}, a.sy = {strides[2], strides[3]};
    a.n_seq = n_seq, a.B = B, a.T = T, a.C = C, a.W = W, a.flags = flags, a.dtype = dtype;
    return gdn::launch_conv_bwd(a, stream);
}

int causal_conv_step(const void *x, const float *weight, const float *bias, const void *window, void *window_out,
                     const int *slots, void *y, long long x_stride, int B, int C, int W, int n_slots, unsigned flags, int dtype,
                     void *stream) {
    const Range nvtx_range("causal_conv_step");
    int st = check_slots(slots, B, n_slots);
    if (st == GDN_OK && C < 0) st = GDN_ERR_INVALID_ARG;
    if (st == GDN_OK) st = check_conv(W, C, flags, dtype);
    if (st == GDN_OK) st = check_strides(&x_stride, 1, dtype);
    if (st != GDN_OK) return st;
    if ((long long)B * (C / 4) > 0x7fffffffLL * 64) return GDN_ERR_UNSUPPORTED;
    if ((long long)B * C == 0) return GDN_OK;
    if (!x || !weight || !window || !window_out || !y) return GDN_ERR_INVALID_ARG;
    if (misaligned({x, weight, bias, window, window_out, y})) return GDN_ERR_MISALIGNED;
    const gdn::ConvStepArgs a{x, weight, bias, window, window_out, slots, y, x_stride, B, C, W, n_slots, flags, dtype};
    return gdn::launch_conv_step(a, static_cast<cudaStream_t>(stream));
}

size_t ssm_scan_fwd_workspace_bytes(int B, int T, int Di, int N, int dtype) {
    if (check_rows(nullptr, B, B, T, Di) != GDN_OK || check_scan(Di, N, 0, dtype) != GDN_OK || check_scan_size(B, T, Di, N) != GDN_OK)
        return (size_t)-1;
    return (long long)B * T * Di == 0 ? 0 : gdn::ssm_fwd_workspace(B, T, Di, N, dtype);
}

int ssm_scan_fwd(const void *x, const void *dt, const float *A, const void *Bt, const void *Ct, const float *skip, const void *z,
                 const float *dt_bias, const float *initial_state, void *y, float *final_state, const int *cu_seqlens,
                 const long long *strides, int n_seq, int B, int T, int Di, int N, unsigned flags, int dtype, void *workspace,
                 size_t workspace_bytes, void *stream_v) {
    const Range nvtx_range("ssm_scan_fwd");
    int st = check_rows(cu_seqlens, n_seq, B, T, Di);
    if (st == GDN_OK) st = check_scan(Di, N, flags, dtype);
    if (st == GDN_OK) st = check_scan_size(B, T, Di, N);
    if (st == GDN_OK && strides) st = check_strides(strides, 12, dtype);
    if (st != GDN_OK) return st;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    if (misaligned({x, dt, A, Bt, Ct, skip, z, dt_bias, initial_state, y, final_state})) return GDN_ERR_MISALIGNED;
    if ((long long)B * T * Di == 0) return pass_on(initial_state, final_state, sizeof(float) * (size_t)n_seq * Di * N, stream);
    if (!x || !dt || !A || !Bt || !Ct || !y || n_seq == 0) return GDN_ERR_INVALID_ARG;
    gdn::SsmArgs a = scan_args(x, dt, A, Bt, Ct, skip, z, dt_bias, initial_state, cu_seqlens, strides, n_seq, B, T, Di, N, flags,
                               dtype, workspace);
    a.y = y, a.sf = final_state;
    if (overlaps({{a.sy.b, B}, {a.sy.t, T}}, Di)) return GDN_ERR_INVALID_ARG;
    if (short_of(workspace, workspace_bytes, gdn::ssm_fwd_workspace(B, T, Di, N, dtype))) return GDN_ERR_WORKSPACE;
    return gdn::launch_ssm_fwd(a, stream);
}

size_t ssm_scan_bwd_workspace_bytes(int B, int T, int Di, int N, int dtype) {
    if (check_rows(nullptr, B, B, T, Di) != GDN_OK || check_scan(Di, N, 0, dtype) != GDN_OK || check_scan_size(B, T, Di, N) != GDN_OK)
        return (size_t)-1;
    return (long long)B * T * Di == 0 ? 0 : gdn::ssm_bwd_workspace(B, T, Di, N, dtype);
}

int ssm_scan_bwd(const void *x, const void *dt, const float *A, const void *Bt, const void *Ct, const float *skip, const void *z,
                 const float *dt_bias, const float *initial_state, const void *dy, const float *dfinal_state, void *dx, void *ddt,
                 float *dA, void *dB, void *dC, float *dskip, void *dz, float *ddt_bias, float *dinitial_state,
                 const int *cu_seqlens, const long long *strides, int n_seq, int B, int T, int Di, int N, unsigned flags, int dtype,
                 void *workspace, size_t workspace_bytes, void *stream_v) {
    const Range nvtx_range("ssm_scan_bwd");
    int st = check_rows(cu_seqlens, n_seq, B, T, Di);
    if (st == GDN_OK) st = check_scan(Di, N, flags, dtype);
    if (st == GDN_OK) st = check_scan_size(B, T, Di, N);
    if (st == GDN_OK && strides) st = check_strides(strides, 12, dtype);
    if (st != GDN_OK) return st;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    if (misaligned({x, dt, A, Bt, Ct, skip, z, dt_bias, initial_state, dy, dfinal_state, dx, ddt, dA, dB, dC, dskip, dz, ddt_bias,
                    dinitial_state}))
        return GDN_ERR_MISALIGNED;
    if (Di > 0 && !dA) return GDN_ERR_INVALID_ARG;
    if ((long long)B * T * Di == 0) {
        st = zeros(dA, (size_t)Di * N, stream);
        if (st == GDN_OK) st = zeros(dskip, Di, stream);
        if (st == GDN_OK) st = zeros(ddt_bias, Di, stream);
        const size_t small = (size_t)B * T * N * (dtype == GDN_BF16 ? 2 : 4);  // no channels, but tokens
        if (st == GDN_OK) st = pass_on(nullptr, dB, small, stream);
        if (st == GDN_OK) st = pass_on(nullptr, dC, small, stream);
        if (st != GDN_OK) return st;
        return pass_on(dfinal_state, dinitial_state, sizeof(float) * (size_t)n_seq * Di * N, stream);
    }
    if (!x || !dt || !A || !Bt || !Ct || !dy || !dx || !ddt || !dB || !dC || n_seq == 0 || (z && !dz)) return GDN_ERR_INVALID_ARG;
    if (short_of(workspace, workspace_bytes, gdn::ssm_bwd_workspace(B, T, Di, N, dtype))) return GDN_ERR_WORKSPACE;
    gdn::SsmArgs a = scan_args(x, dt, A, Bt, Ct, skip, z, dt_bias, initial_state, cu_seqlens, strides, n_seq, B, T, Di, N, flags,
                               dtype, workspace);
    a.dy = dy, a.dsf = dfinal_state, a.dx = dx, a.ddt = ddt, a.dA = dA, a.dB = dB, a.dC = dC, a.dD = dskip, a.dz = dz;
    a.dbias = ddt_bias, a.ds0 = dinitial_state;
    return gdn::launch_ssm_bwd(a, stream);
}

int ssm_step(const void *x, const void *dt, const float *A, const void *Bt, const void *Ct, const float *skip, const void *z,
             const float *dt_bias, const float *state, float *state_out, const int *slots, void *y, const long long *strides, int B,
             int Di, int N, int n_slots, unsigned flags, int dtype, void *stream) {
    const Range nvtx_range("ssm_step");
    int st = check_slots(slots, B, n_slots);
    if (st == GDN_OK && Di < 0) st = GDN_ERR_INVALID_ARG;
    if (st == GDN_OK) st = check_scan(Di, N, flags, dtype);
    if (st == GDN_OK && (long long)Di * N > 0x7fffffffLL) st = GDN_ERR_UNSUPPORTED;
    if (st == GDN_OK && strides) st = check_strides(strides, 5, dtype);
    if (st != GDN_OK || (long long)B * Di == 0) return st;
    if (!x || !dt || !A || !Bt || !Ct || !state || !state_out || !y) return GDN_ERR_INVALID_ARG;
    if (misaligned({x, dt, A, Bt, Ct, skip, z, dt_bias, state, state_out, y})) return GDN_ERR_MISALIGNED;
    gdn::SsmStepArgs a{x, dt, Bt, Ct, z, A, skip, dt_bias, state, state_out, slots, y, Di, Di, N, N, Di, B, Di, N, n_slots, flags, dtype};
    if (strides) a.sx = strides[0], a.sdt = strides[1], a.sB = strides[2], a.sC = strides[3], a.sz = strides[4];
    return gdn::launch_ssm_step(a, static_cast<cudaStream_t>(stream));
}

namespace {
int check_gated(int B, int T, int H, int D, float eps, unsigned flags, int dtype) {
    if (B < 0 || T < 0 || H < 0 || D < 0 || !(eps >= 0.f) || bad_type(dtype)) return GDN_ERR_INVALID_ARG;
    if (flags & ~(GDN_GATE_FIRST | GDN_GATE_SIGMOID | GDN_W_SHARED)) return GDN_ERR_INVALID_ARG;
    if (D % wide(dtype) != 0 || D > 8192) return GDN_ERR_UNSUPPORTED;
    if ((long long)H * D > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    // in two steps: the product of three ints may pass 64 bits
    if ((long long)B * T > 0x7fffffffLL || (long long)B * T * H > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}
}  // namespace

int gated_norm_fwd(const void *x, const void *gate, const float *weight, void *y, const long long *strides, int B, int T, int H,
                   int D, float eps, unsigned flags, int dtype, void *stream) {
    const Range nvtx_range("gated_norm_fwd");
    int st = check_gated(B, T, H, D, eps, flags, dtype);
    if (st == GDN_OK && strides) st = check_strides(strides, 6, dtype);
    if (st != GDN_OK || (long long)B * T * H * D == 0) return st;
    if (!x || !gate || !y) return GDN_ERR_INVALID_ARG;
    if (misaligned({x, gate, weight, y})) return GDN_ERR_MISALIGNED;
    gdn::GatedNormArgs a{};
    a.x = x, a.gate = gate, a.w = weight, a.y = y;
    a.sx = a.sg = {(long long)T * H * D, (long long)H * D, D};
    if (strides) a.sx = {strides[0], strides[1], strides[2]}, a.sg = {strides[3], strides[4], strides[5]};
    a.B = B, a.T = T, a.H = H, a.D = D, a.eps = eps, a.flags = flags, a.dtype = dtype;
    return gdn::launch_gated_norm(a, static_cast<cudaStream_t>(stream));
}

size_t gated_norm_bwd_workspace_bytes(int B, int T, int H, int D, unsigned flags) {
    if (check_gated(B, T, H, D, 0.f, flags, GDN_F32) != GDN_OK) return (size_t)-1;
    return (long long)B * T * H * D == 0 ? 0 : gdn::gated_norm_bwd_workspace(B, T, H, D, flags);
}

int gated_norm_bwd(const void *dy, const void *x, const void *gate, const float *weight, void *dx, void *dgate, float *dweight,
                   const long long *strides, int B, int T, int H, int D, float eps, unsigned flags, int dtype, void *workspace,
                   size_t workspace_bytes, void *stream_v) {
    const Range nvtx_range("gated_norm_bwd");
    int st = check_gated(B, T, H, D, eps, flags, dtype);
    if (st == GDN_OK && strides) st = check_strides(strides, 12, dtype);
    if (st != GDN_OK) return st;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    const size_t weights = (size_t)((flags & GDN_W_SHARED) ? 1 : H) * D;
    if (weights && !dweight) return GDN_ERR_INVALID_ARG;
    if ((long long)B * T * H * D == 0) return zeros(dweight, weights, stream);
    if (!dy || !x || !gate || !dx || !dgate) return GDN_ERR_INVALID_ARG;
    if (misaligned({dy, x, gate, weight, dx, dgate, dweight})) return GDN_ERR_MISALIGNED;
    if (short_of(workspace, workspace_bytes, gdn::gated_norm_bwd_workspace(B, T, H, D, flags))) return GDN_ERR_WORKSPACE;
    gdn::GatedNormArgs a{};
    a.dy = dy, a.x = x, a.gate = gate, a.w = weight, a.dx = dx, a.dgate = dgate, a.dw = dweight, a.ws = workspace;
    a.sx = a.sg = a.sdy = a.sdx = {(long long)T * H * D, (long long)H * D, D};
    if (strides) {
        gdn::HeadStrides *to[] = {&a.sx, &a.sg, &a.sdy, &a.sdx};
        for (int i = 0; i < 4; ++i) *to[i] = {strides[3 * i], strides[3 * i + 1], strides[3 * i + 2]};
    }
    if (overlaps({{a.sdx.b, B}, {a.sdx.t, T}, {a.sdx.h, H}}, D)) return GDN_ERR_INVALID_ARG;
    a.B = B, a.T = T, a.H = H, a.D = D, a.eps = eps, a.flags = flags, a.dtype = dtype;
    return gdn::launch_gated_norm_bwd(a, stream);
}

namespace {
int check_block(long long rows, int C, int groups, float eps, int dtype) {
    if (rows < 0 || C < 0 || groups < 0 || !(eps >= 0.f) || bad_type(dtype)) return GDN_ERR_INVALID_ARG;
    if (groups > 0 && rows % groups != 0) return GDN_ERR_INVALID_ARG;
    if (C % wide(dtype) != 0 || C > 8192 || rows > 0x7fffffffLL || groups > 65535) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}
}  // namespace

int block_norm_fwd(const void *x, const void *residual, const float *post_weight, const float *scale, const float *weight, void *y,
                   void *h, long long rows, int C, int groups, float eps, int dtype, void *stream) {
    const Range nvtx_range("block_norm_fwd");
    const int st = check_block(rows, C, groups, eps, dtype);
    if (st != GDN_OK) return st;
    if ((scale != nullptr) != (groups > 0)) return GDN_ERR_INVALID_ARG;
    if (rows * C == 0) return GDN_OK;
    if (!x || !residual || !y || !h) return GDN_ERR_INVALID_ARG;
    if (misaligned({x, residual, post_weight, scale, weight, y, h})) return GDN_ERR_MISALIGNED;
    gdn::BlockNormArgs a{};
    a.x = x, a.res = residual, a.w1 = post_weight, a.s = scale, a.w2 = weight, a.y = y, a.h = h;
    a.rows = rows, a.C = C, a.groups = groups, a.eps = eps, a.dtype = dtype;
    return gdn::launch_block_norm(a, static_cast<cudaStream_t>(stream));
}

size_t block_norm_bwd_workspace_bytes(long long rows, int C, int groups) {
    if (check_block(rows, C, groups, 0.f, GDN_F32) != GDN_OK) return (size_t)-1;
    return rows * C == 0 ? 0 : gdn::block_norm_bwd_workspace(rows, C, groups);
}

int block_norm_bwd(const void *dy, const void *dh, const void *x, const void *h, const float *post_weight, const float *scale,
                   const float *weight, void *dx, void *dresidual, float *dpost_weight, float *dscale, float *dweight,
                   long long rows, int C, int groups, float eps, int dtype, void *workspace, size_t workspace_bytes,
                   void *stream_v) {
    const Range nvtx_range("block_norm_bwd");
    int st = check_block(rows, C, groups, eps, dtype);
    if (st != GDN_OK) return st;
    if ((scale != nullptr) != (groups > 0) || (dscale && !scale)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    if (misaligned({dy, dh, x, h, post_weight, scale, weight, dx, dresidual})) return GDN_ERR_MISALIGNED;
    if (rows * C == 0) {
        st = zeros(dpost_weight, C, stream);
        if (st == GDN_OK) st = zeros(dscale, (size_t)groups * C, stream);
        return st == GDN_OK ? zeros(dweight, C, stream) : st;
    }
    if (!dy || !x || !h || !dx || !dresidual) return GDN_ERR_INVALID_ARG;
    if (short_of(workspace, workspace_bytes, gdn::block_norm_bwd_workspace(rows, C, groups))) return GDN_ERR_WORKSPACE;
    gdn::BlockNormArgs a{};
    a.dy = dy, a.dh = dh, a.x = x, a.h = const_cast<void *>(h), a.w1 = post_weight, a.s = scale, a.w2 = weight;
    a.dx = dx, a.dres = dresidual, a.dw1 = dpost_weight, a.ds = dscale, a.dw2 = dweight;
    a.rows = rows, a.C = C, a.groups = groups, a.eps = eps, a.dtype = dtype, a.ws = workspace;
    return gdn::launch_block_norm_bwd(a, stream);
}

}  // extern "C"
