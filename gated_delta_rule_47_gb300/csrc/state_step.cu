// state_step.cu -- one token of linear attention with a decay for each head,
// or of the gated delta rule, against a pool of fp32 states.
//
//   D = exp(g) S;   u = v (plain)  or  beta (v - D^T k) (delta rule)
//   S' = D + k u^T;  o = scale S'^T q = scale (D^T q + (q . k) u)
//
// Both products with D are sums over its rows for each column, so one read of
// S into registers, one exchange of partial sums and one write of S' is all
// that a token costs.  Columns are independent: a CTA owns W columns of one
// head, all Dk rows of them.  The bytes of S bound it (2 x 4 Dk Dv a head).
#include <cuda_bf16.h>

#include "gdn_internal.h"
#include "layer_ops.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float ldf(const float *p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void stf(float *p, float x) { *p = x; }
__device__ __forceinline__ void stf(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(~0u, x, m);
    return x;
}

// Measured, D 128, in place: 8192 heads 158 us for the delta rule and 156
// without it, 1.07 GB at 6.8 TB/s, as a plain copy; 16 heads 2.4 us.
// Grid: (Dv / W, H, B).  Thread (r, c): columns 4c..4c+3 of rows r, r + RP, ...
template <typename T, int DK, int DV, int W, bool DELTA>
__global__ void __launch_bounds__(kThreads) step_kernel(StepArgs a) {
    constexpr int LPR = W / 4;         // lanes per row
    constexpr int RP = kThreads / LPR; // rows per pass
    constexpr int R = DK / RP;         // rows per thread
    constexpr int NW = kThreads / 32;
    static_assert(R >= 1 && LPR <= 32, "tile");
    const int h = blockIdx.y, b = blockIdx.z, col0 = blockIdx.x * W;
    const int tid = threadIdx.x, c = tid % LPR, r0 = tid / LPR, warp = tid >> 5, lane = tid & 31;
    __shared__ float qs[DK], ks[DK];
    __shared__ float4 part[NW][DELTA ? 2 : 1][LPR];
    T *o = static_cast<T *>(a.o) + ((size_t)b * a.H + h) * DV + col0;
    const int slot = a.slots ? a.slots[b] : b;
    if (slot < 0 || slot >= a.n_slots) {  // an idle row
        if (tid < W) stf(o + tid, 0.f);
        return;
    }
    const size_t page = (((size_t)slot * a.H + h) * DK) * DV + col0;
    const float *S = a.state + page;
    float4 s[R];
#pragma unroll
    for (int i = 0; i < R; ++i) s[i] = __ldcs(reinterpret_cast<const float4 *>(S + (size_t)(r0 + i * RP) * DV) + c);
    const int hk = h / (a.H / a.Hk);
    const T *q = static_cast<const T *>(a.q) + ((size_t)b * a.Hk + hk) * DK;
    const T *k = static_cast<const T *>(a.k) + ((size_t)b * a.Hk + hk) * DK;
    if (tid < DK) {
        qs[tid] = ldf(q + tid);
        ks[tid] = ldf(k + tid);
    }
    const T *v = static_cast<const T *>(a.v) + ((size_t)b * a.H + h) * DV + col0 + 4 * c;
    float u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = ldf(v + j);
    const float decay = expf(a.g[(a.flags & GDN_G_PER_HEAD) ? h : b * a.H + h]);
    float beta = 1.f;
    if (DELTA) beta = ldf(static_cast<const T *>(a.beta) + (size_t)b * a.H + h);
    __syncthreads();
    float qk = 0.f, qq = 0.f, kk = 0.f;
#pragma unroll
    for (int i = lane; i < DK; i += 32) {
        qk = fmaf(qs[i], ks[i], qk);
        if (DELTA) {
            qq = fmaf(qs[i], qs[i], qq);
            kk = fmaf(ks[i], ks[i], kk);
        }
    }
    qk = warp_sum(qk);
    float qn = 1.f, kn = 1.f;
    if (DELTA && (a.flags & GDN_QK_L2NORM)) {
        qn = 1.f / fmaxf(sqrtf(warp_sum(qq)), 1e-12f);
        kn = 1.f / fmaxf(sqrtf(warp_sum(kk)), 1e-12f);
    }
    float4 zq = make_float4(0.f, 0.f, 0.f, 0.f), zk = zq;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        s[i].x *= decay, s[i].y *= decay, s[i].z *= decay, s[i].w *= decay;
        const float qi = qs[r0 + i * RP], ki = ks[r0 + i * RP];
        zq.x = fmaf(qi, s[i].x, zq.x), zq.y = fmaf(qi, s[i].y, zq.y);
        zq.z = fmaf(qi, s[i].z, zq.z), zq.w = fmaf(qi, s[i].w, zq.w);
        if (DELTA) {
            zk.x = fmaf(ki, s[i].x, zk.x), zk.y = fmaf(ki, s[i].y, zk.y);
            zk.z = fmaf(ki, s[i].z, zk.z), zk.w = fmaf(ki, s[i].w, zk.w);
        }
    }
#pragma unroll
    for (int m = LPR; m < 32; m <<= 1) {  // rows of one warp
        zq.x += __shfl_xor_sync(~0u, zq.x, m), zq.y += __shfl_xor_sync(~0u, zq.y, m);
        zq.z += __shfl_xor_sync(~0u, zq.z, m), zq.w += __shfl_xor_sync(~0u, zq.w, m);
        if (DELTA) {
            zk.x += __shfl_xor_sync(~0u, zk.x, m), zk.y += __shfl_xor_sync(~0u, zk.y, m);
            zk.z += __shfl_xor_sync(~0u, zk.z, m), zk.w += __shfl_xor_sync(~0u, zk.w, m);
        }
    }
    if (lane < LPR) {
        part[warp][0][lane] = zq;
        if (DELTA) part[warp][DELTA ? 1 : 0][lane] = zk;
    }
    __syncthreads();
    zq = make_float4(0.f, 0.f, 0.f, 0.f);
    zk = zq;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float4 p = part[w][0][c];
        zq.x += p.x, zq.y += p.y, zq.z += p.z, zq.w += p.w;
        if (DELTA) {
            const float4 n = part[w][DELTA ? 1 : 0][c];
            zk.x += n.x, zk.y += n.y, zk.z += n.z, zk.w += n.w;
        }
    }
    if (DELTA) {
        u[0] = beta * (u[0] - kn * zk.x), u[1] = beta * (u[1] - kn * zk.y);
        u[2] = beta * (u[2] - kn * zk.z), u[3] = beta * (u[3] - kn * zk.w);
    }
    float *Sn = a.state_out + page;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float ki = kn * ks[r0 + i * RP];
        s[i].x = fmaf(ki, u[0], s[i].x), s[i].y = fmaf(ki, u[1], s[i].y);
        s[i].z = fmaf(ki, u[2], s[i].z), s[i].w = fmaf(ki, u[3], s[i].w);
        __stcs(reinterpret_cast<float4 *>(Sn + (size_t)(r0 + i * RP) * DV) + c, s[i]);
    }
    if (r0 == 0) {
        const float m = a.scale * qn, w = qk * kn;
        stf(o + 4 * c + 0, m * fmaf(w, u[0], zq.x));
        stf(o + 4 * c + 1, m * fmaf(w, u[1], zq.y));
        stf(o + 4 * c + 2, m * fmaf(w, u[2], zq.z));
        stf(o + 4 * c + 3, m * fmaf(w, u[3], zq.w));
    }
}

template <typename T, int DK, int DV, bool DELTA>
void launch_w(const StepArgs &a, cudaStream_t stream) {
    // Slices of 32 columns while their CTAs are few (32 heads, D 128: 2.6 us
    // against 3.7), else a page's columns in one CTA, whose rows are whole
    // lines (128 heads 4.0 us against 5.0, 8192 heads 158 against 196).
    if ((long long)a.B * a.H * (DV / 32) > 2 * device_sm_count()) {
        step_kernel<T, DK, DV, DV, DELTA><<<dim3(1, a.H, a.B), kThreads, 0, stream>>>(a);
    } else {
        step_kernel<T, DK, DV, 32, DELTA><<<dim3(DV / 32, a.H, a.B), kThreads, 0, stream>>>(a);
    }
}

template <typename T, int DK, int DV>
void launch_d(const StepArgs &a, cudaStream_t stream) {
    if (a.beta) launch_w<T, DK, DV, true>(a, stream);
    else launch_w<T, DK, DV, false>(a, stream);
}

template <typename T>
void launch_t(const StepArgs &a, cudaStream_t stream) {
    if (a.Dk == 128 && a.Dv == 128) launch_d<T, 128, 128>(a, stream);
    else if (a.Dk == 128) launch_d<T, 128, 64>(a, stream);
    else if (a.Dv == 128) launch_d<T, 64, 128>(a, stream);
    else launch_d<T, 64, 64>(a, stream);
}

}  // namespace

int launch_step(const StepArgs &a, cudaStream_t stream) {
    // grid.z is limited to 65535 rows: larger batches go in pieces
    const size_t size = a.dtype == GDN_BF16 ? 2 : 4;
    for (int b0 = 0; b0 < a.B; b0 += 65535) {
        StepArgs p = a;
        p.B = a.B - b0 < 65535 ? a.B - b0 : 65535;
        auto at = [&](const void *x, size_t row) {
            return x ? static_cast<const char *>(x) + (size_t)b0 * row * size : nullptr;
        };
        p.q = at(a.q, (size_t)a.Hk * a.Dk);
        p.k = at(a.k, (size_t)a.Hk * a.Dk);
        p.v = at(a.v, (size_t)a.H * a.Dv);
        p.beta = at(a.beta, a.H);
        p.o = const_cast<char *>(at(a.o, (size_t)a.H * a.Dv));
        if (!(a.flags & GDN_G_PER_HEAD)) p.g = a.g + (size_t)b0 * a.H;
        if (a.slots) {
            p.slots = a.slots + b0;
        } else {  // page b is row b's
            p.state = a.state + (size_t)b0 * a.H * a.Dk * a.Dv;
            p.state_out = a.state_out + (size_t)b0 * a.H * a.Dk * a.Dv;
            p.n_slots = a.n_slots - b0;
        }
        if (a.dtype == GDN_BF16) launch_t<__nv_bfloat16>(p, stream);
        else launch_t<float>(p, stream);
        if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
        note_launch();
    }
    return GDN_OK;
}

}  // namespace gdn
