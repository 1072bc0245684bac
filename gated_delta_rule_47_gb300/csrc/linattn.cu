// linattn.cu -- linear attention with a decay for each head over whole
// prompts, forward and backward, on the CUDA cores in fp32.
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// Chunks of 64 tokens.  With c_t the sum of a chunk's log-decays up to token
// t, S the state that enters the chunk and G = c_63:
//
//   o_t  = scale (e^{c_t} S^T q_t + sum_{s<=t} e^{c_t - c_s} (q_t . k_s) v_s)
//   S'   = e^G S + sum_t e^{G - c_t} k_t v_t^T
//
// so a call is three launches: every chunk's own share of the state (a product
// over its tokens), the scan of these over a sequence's chunks, and every
// chunk's outputs.  The backward has the same shape twice, forwards for S and
// backwards for R, the gradient of the state that leaves a chunk,
//
//   R_before = e^G R + scale sum_t e^{c_t} q_t do_t^T,
//
// and then, with P_ts = scale e^{c_t-c_s} (q_t . k_s), N_ts = scale e^{c_t-c_s}
// (do_t . v_s) for s <= t,
//
//   dq_t = scale e^{c_t} S do_t + sum_s N_ts k_s
//   dk_s = e^{G-c_s} R v_s + sum_t N_ts q_t
//   dv_s = e^{G-c_s} R^T k_s + sum_t P_ts do_t
//   dg_u = sum_{t>=u} (x_t + sum_{s<t} A_ts - sum_{r>t} A_rt) + sum_{t<u} y_t + e^G <R, S>
//
// with A_ts = (q_t . k_s) N_ts, x_t = q_t . (S's part of dq_t) and y_t = k_t .
// (R's part of dk_t): what passes over the decay of token u, pair by pair.
#include <cuda_bf16.h>

#include "gdn_internal.h"
#include "linattn.cuh"
#include "simt_tile.cuh"

namespace gdn {
namespace la {
namespace {

constexpr int kC = 64;
constexpr int kTableThreads = 1024;

// One CTA: sequence s's first chunk from the running count, then every chunk's
// entry by a search for its sequence.  Bad offsets are cut to [0, T] and to
// the tables' room, so that no entry leads outside the tensors.
__global__ void __launch_bounds__(kTableThreads) table_kernel(const int *cu, int n_seq, int T, int C, int4 *chunks,
                                                              int4 *seqs, int bound) {
    __shared__ long long sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long first = 0;
    for (int s0 = 0; s0 < n_seq; s0 += kTableThreads) {
        const int s = s0 + threadIdx.x;
        int start = 0, len = 0;
        if (s < n_seq) {
            start = min(max(cu[s], 0), T);
            len = max(min(cu[s + 1], T) - start, 0);
        }
        const int n = (int)(((long long)len + C - 1) / C);
        long long y = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long t = __shfl_up_sync(~0u, y, m);
            if (lane >= m) y += t;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = y;
        __syncthreads();
        if (warp == 0) {
            long long z = sums[lane];
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const long long t = __shfl_up_sync(~0u, z, m);
                if (lane >= m) z += t;
            }
            sums[lane] = z;
        }
        __syncthreads();
        const int2 in = in_table(first + y - n + (warp ? sums[warp - 1] : 0), n, bound);
        first += sums[31];
        if (s < n_seq) seqs[s] = make_int4(in.x, in.y, start, len);
    }
    __syncthreads();
    const int count = in_table(first, 0, bound).x;
    const int head = min(max(cu[0], 0), T), tail = min(max(cu[n_seq], 0), T);
    const int fill0 = (head + C - 1) / C;
    for (int ci = threadIdx.x; ci < bound; ci += kTableThreads) {
        int4 e = make_int4(0, 0, 0, -1);
        if (ci >= count) {  // fillers, as far as there are any
            const int f = ci - count;
            const long long t = f < fill0 ? (long long)f * C : tail + (long long)(f - fill0) * C;
            const int end = f < fill0 ? head : T;
            if (t < end) e = make_int4(0, (int)t, min(C, end - (int)t), -1);
        } else {
            int lo = 0, hi = n_seq - 1;  // the last sequence whose first chunk is not after ci
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (seqs[mid].x <= ci) lo = mid;
                else hi = mid - 1;
            }
            const int4 q = seqs[lo];
            const int t = (ci - q.x) * C;
            e = make_int4(0, q.z + t, max(min(C, q.w - t), 0), lo);
        }
        chunks[ci] = e;
    }
}

// dq[b,hk,t,:] = sum of the value heads' shares dqh[b,h,t,:], in their order,
// and the same for dk: the second half of grid.x.  Bound by the bytes.
template <typename T>
__global__ void group_sum_kernel(LinAttnArgs a, const float4 *dqh, const float4 *dkh) {
    const int per = a.Dk / 4, rep = a.H / a.Hk, blocks = gridDim.x / 2;
    const bool key = blockIdx.x >= blocks;
    const long long n = (long long)a.T * per;
    const int hk = blockIdx.y, b = blockIdx.z;
    const float4 *src = key ? dkh : dqh;
    const Strides &s = key ? a.sk : a.sq;
    T *dst = static_cast<T *>(key ? a.dk : a.dq);
    for (long long i = (key ? blockIdx.x - blocks : blockIdx.x) * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)blocks * blockDim.x) {
        const int t = (int)(i / per), c = (int)(i - (long long)t * per);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < rep; ++r) {
            const float4 y = src[(((long long)b * a.H + hk * rep + r) * a.T + t) * per + c];
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        T *p = at(dst, s, b, hk, t) + 4 * c;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4 *>(p) = x;
        } else {
            __nv_bfloat162 y[2] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w)};
            *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(y);
        }
    }
}

__global__ void __launch_bounds__(1024) head_sum_kernel(const float *src, float *dg, int B, int H, int T) {
    __shared__ double s[32];
    const int h = blockIdx.x;
    double x = 0.;
    for (int b = 0; b < B; ++b) {
        const float *p = src + ((long long)b * H + h) * T;
        float part = 0.f;
        int n = 0;
        for (int t = threadIdx.x; t < T; t += 1024) {
            part += p[t];
            if (++n == 16) x += part, part = 0.f, n = 0;
        }
        x += part;
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(~0u, x, m);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x < 32) {
        x = s[threadIdx.x];
#pragma unroll
        for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(~0u, x, m);
        if (threadIdx.x == 0) dg[h] = (float)x;
    }
}

// ------------------------------------------------------------ chunk kernels
// Tiles have rows of D + 4 floats: 16-byte aligned, and a column of rows spreads
// over the banks.
template <int D>
constexpr int ld() { return D + 4; }

// acc[i][4 b + j] += sum_{k < K} A(m, k) B(k, n) with m = ty + (NT / 16) i and n =
// 4 tx + 64 b + j (tx = thread % 16, ty = thread / 16), A[m lda + k] and
// B[k ldb + n] in shared memory, all read 16 bytes at a time: for four k a
// warp's 2 x 8 outputs a thread take 18 shared-memory cycles and 64 multiply-adds.
template <int NT, int TI, int TB>
__device__ __forceinline__ void mm_kn(float (&acc)[TI][4 * TB], const float *A, int lda, const float *B, int ldb, int K) {
    constexpr int RS = NT / 16;
    const float *a0 = A + (threadIdx.x >> 4) * lda, *b0 = B + 4 * (threadIdx.x & 15);
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float4 a[TI];
#pragma unroll
        for (int i = 0; i < TI; ++i) a[i] = *reinterpret_cast<const float4 *>(a0 + RS * i * lda + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float4 b[TB];
#pragma unroll
            for (int c = 0; c < TB; ++c) b[c] = *reinterpret_cast<const float4 *>(b0 + (k + e) * ldb + 64 * c);
#pragma unroll
            for (int i = 0; i < TI; ++i) {
                const float x = e == 0 ? a[i].x : e == 1 ? a[i].y : e == 2 ? a[i].z : a[i].w;
#pragma unroll
                for (int c = 0; c < TB; ++c) {
                    acc[i][4 * c] = fmaf(x, b[c].x, acc[i][4 * c]);
                    acc[i][4 * c + 1] = fmaf(x, b[c].y, acc[i][4 * c + 1]);
                    acc[i][4 * c + 2] = fmaf(x, b[c].z, acc[i][4 * c + 2]);
                    acc[i][4 * c + 3] = fmaf(x, b[c].w, acc[i][4 * c + 3]);
                }
            }
        }
    }
}

__device__ __forceinline__ float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void st4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void st4(__nv_bfloat16 *p, float4 x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// Rows t < len of a strided [T][D] slice into a [64][D + 4] fp32 tile, zeros
// after them; f(t) scales row t.
template <typename T, int D, int NT, class F>
__device__ __forceinline__ void load_tile(float *dst, const T *src, long long step, int len, F f) {
#pragma unroll 4
    for (int i = threadIdx.x; i < kC * D / 4; i += NT) {
        const int t = i / (D / 4), d = i % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < len) {
            x = ld4(src + t * step + d);
            const float w = f(t);
            x.x *= w, x.y *= w, x.z *= w, x.w *= w;
        }
        *reinterpret_cast<float4 *>(dst + t * ld<D>() + d) = x;
    }
}
template <typename T, int D, int NT>
__device__ __forceinline__ void load_tile(float *dst, const T *src, long long step, int len) {
    load_tile<T, D, NT>(dst, src, step, len, [](int) { return 1.f; });
}

// Zeros in rows t < len of a strided [T][D] slice (tokens of no sequence).
template <typename T, int D, int NT>
__device__ __forceinline__ void zero_rows(T *dst, long long step, int len) {
    for (int i = threadIdx.x; i < len * D; i += NT) tile::st_f(dst + (i / D) * step + i % D, 0.f);
}

// A chunk's share of the state that leaves it, sum_t e^{G-c_t} k_t v_t^T (to
// U), and of the gradient before it, scale sum_t e^{c_t} q_t do_t^T (to R).
// Grid (chunks, H, 1 or, for the backward, 2); U, R [chunk][H][DK][DV],
// decay [chunk][H] = e^G.  A register-tiled product, bound by the CUDA cores:
// fp32, 2 x 4096 tokens of 16 heads, D 128: 136 us, 32 TFLOP/s.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(256) share_kernel(LinAttnArgs a, View v, float *U, float *R, float *decay) {
    const bool rev = blockIdx.z;
    extern __shared__ __align__(16) float sm[];
    float *X = sm, *Y = X + kC * ld<DK>(), *hi = Y + kC * ld<DV>(), *lo = hi + kC, *te = lo + kC;
    const int ci = blockIdx.x, h = blockIdx.y;
    const Chunk c = chunk_at<kC>(v, a.T, ci);
    if (c.len <= 0 || c.seq < 0) return;
    const int hk = h / (a.H / a.Hk);
    const T *xp = rev ? at(static_cast<const T *>(a.q), a.sq, c.row, hk, c.t0) : at(static_cast<const T *>(a.k), a.sk, c.row, hk, c.t0);
    const T *yp = rev ? at(static_cast<const T *>(a.dout), a.sdo, c.row, h, c.t0) : at(static_cast<const T *>(a.v), a.sv, c.row, h, c.t0);
    if (threadIdx.x < 32) gates<kC>(gate_ptr(a, c, h), a.sg.t, c.len, a.flags & GDN_G_PER_HEAD, hi, lo, te);
    load_tile<T, DV, 256>(Y, yp, rev ? a.sdo.t : a.sv.t, c.len);
    __syncthreads();
    load_tile<T, DK, 256>(X, xp, rev ? a.sq.t : a.sk.t, c.len, [&](int t) { return rev ? a.scale * expf(hi[t]) : expf(te[t]); });
    __syncthreads();
    // rows 4 ty + 64 i.., columns 4 tx + 64 j..: four and four at a time
    constexpr int MB = DK / 64, NB = DV / 64;
    float acc[4 * MB][4 * NB];
#pragma unroll
    for (int i = 0; i < 4 * MB; ++i)
#pragma unroll
        for (int j = 0; j < 4 * NB; ++j) acc[i][j] = 0.f;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 4
    for (int t = 0; t < kC; ++t) {
        float x[4 * MB], y[4 * NB];
#pragma unroll
        for (int i = 0; i < MB; ++i) *reinterpret_cast<float4 *>(x + 4 * i) = ld4(X + t * ld<DK>() + 4 * ty + 64 * i);
#pragma unroll
        for (int j = 0; j < NB; ++j) *reinterpret_cast<float4 *>(y + 4 * j) = ld4(Y + t * ld<DV>() + 4 * tx + 64 * j);
#pragma unroll
        for (int i = 0; i < 4 * MB; ++i)
#pragma unroll
            for (int j = 0; j < 4 * NB; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
    float *u = (rev ? R : U) + ((long long)ci * a.H + h) * DK * DV;
#pragma unroll
    for (int i = 0; i < 4 * MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            st4(u + (4 * ty + 64 * (i / 4) + i % 4) * DV + 4 * tx + 64 * j,
                make_float4(acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]));
    if (!rev && threadIdx.x == 0) decay[(long long)ci * a.H + h] = expf(hi[c.len - 1]);
}

// Turns the shares of a sequence's chunks into the states that enter them
// (forwards, from s0; the last one to sf), and into the gradients of the states
// that leave them (backwards, from dsf; the last one to ds0).
// Grid (blocks of a page, H, n_seq), twice as many blocks for both; a thread
// takes four elements.  Bound by the bytes of the chunks' states.
__global__ void __launch_bounds__(256) scan_kernel(LinAttnArgs a, View v, float *U, float *R, const float *decay, int page,
                                                   int blocks) {
    const bool rev = blockIdx.x >= blocks;
    const int e = ((rev ? blockIdx.x - blocks : blockIdx.x) * 256 + threadIdx.x) * 4, H = a.H, h = blockIdx.y, s = blockIdx.z;
    if (e >= page) return;
    if (rev) U = R;
    const float *start = rev ? a.dsf : a.s0;
    float *end = rev ? a.ds0 : a.sf;
    const int2 q = seq_at(v, s);
    const long long mine = ((long long)s * H + h) * page + e;
    float4 x = start ? *reinterpret_cast<const float4 *>(start + mine) : make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int A = 4;  // chunks read ahead
    float4 u[A];
    float d[A];
    auto slot = [&](int i) { return ((long long)(q.x + (rev ? q.y - 1 - i : i)) * H + h); };
#pragma unroll
    for (int j = 0; j < A; ++j)
        if (j < q.y) {
            u[j] = *reinterpret_cast<const float4 *>(U + slot(j) * page + e);
            d[j] = decay[slot(j)];
        }
    for (int i0 = 0; i0 < q.y; i0 += A) {
#pragma unroll
        for (int j = 0; j < A; ++j) {
            if (i0 + j >= q.y) break;
            const float4 w = u[j];
            const float f = d[j];
            if (i0 + j + A < q.y) {
                u[j] = *reinterpret_cast<const float4 *>(U + slot(i0 + j + A) * page + e);
                d[j] = decay[slot(i0 + j + A)];
            }
            *reinterpret_cast<float4 *>(U + slot(i0 + j) * page + e) = x;
            x.x = fmaf(f, x.x, w.x), x.y = fmaf(f, x.y, w.y), x.z = fmaf(f, x.z, w.z), x.w = fmaf(f, x.w, w.w);
        }
    }
    if (end) *reinterpret_cast<float4 *>(end + mine) = x;
}

constexpr int kT = tile::kThr;  // 512
constexpr int kP = kC + 4;      // rows of a [64][64] tile
constexpr int kSlab = 68;       // rows of 64 columns of a state

// Columns j0 .. j0 + 63 of a [DK][DV] state into [DK][68] (its rows) ..
template <int DK, int DV>
__device__ __forceinline__ void load_slab(float *dst, const float *S, int j0) {
#pragma unroll 4
    for (int i = threadIdx.x; i < DK * 16; i += kT) st4(dst + (i >> 4) * kSlab + (i & 15) * 4, ld4(S + (i >> 4) * DV + j0 + (i & 15) * 4));
}
// .. or transposed into [64][DK + 4].
template <int DK, int DV>
__device__ __forceinline__ void load_slab_t(float *dst, const float *S, int j0) {
#pragma unroll 4
    for (int i = threadIdx.x; i < DK * 64; i += kT) dst[(i & 63) * ld<DK>() + (i >> 6)] = S[(i >> 6) * DV + j0 + (i & 63)];
}

// A chunk's outputs.  Grid (chunks, H); S as scan_kernel left it.  Three products
// on the CUDA cores (fp32 operands, which the tensor cores would round): 397 us
// for the same, of 573 us in all.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kT) out_kernel(LinAttnArgs a, View v, const float *S) {
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *K = Q + kC * ld<DK>(), *V = K + kC * ld<DK>(), *P = V + kC * ld<DV>(), *slab = P + kC * kP;
    float *hi = slab + DK * kSlab, *lo = hi + kC, *te = lo + kC;
    const int ci = blockIdx.x, h = blockIdx.y;
    const Chunk c = chunk_at<kC>(v, a.T, ci);
    if (c.len <= 0) return;
    T *out = at(static_cast<T *>(a.o), a.so, c.row, h, c.t0);
    if (c.seq < 0) {
        zero_rows<T, DV, kT>(out, a.so.t, c.len);
        return;
    }
    const int hk = h / (a.H / a.Hk);
    if (threadIdx.x < 32)
        gates<kC>(gate_ptr(a, c, h), a.sg.t, c.len, a.flags & GDN_G_PER_HEAD, hi, lo, te);
    load_tile<T, DK, kT>(Q, at(static_cast<const T *>(a.q), a.sq, c.row, hk, c.t0), a.sq.t, c.len);
    load_tile<T, DK, kT>(K, at(static_cast<const T *>(a.k), a.sk, c.row, hk, c.t0), a.sk.t, c.len);
    load_tile<T, DV, kT>(V, at(static_cast<const T *>(a.v), a.sv, c.row, h, c.t0), a.sv.t, c.len);
    const float *Sc = S + ((long long)ci * a.H + h) * DK * DV;
    load_slab<DK, DV>(slab, Sc, 0);
    __syncthreads();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float p[2][4] = {};
    tile::mm_nt<kT, 2, 4>(p, Q, ld<DK>(), K, ld<DK>(), DK);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = ty + 32 * i, s = tx + 16 * j;
            P[t * kP + s] = s <= t ? p[i][j] * decay_between(hi[t], lo[t], hi[s], lo[s]) : 0.f;
        }
    for (int j0 = 0; j0 < DV; j0 += 64) {
        if (j0 > 0) {
            __syncthreads();
            load_slab<DK, DV>(slab, Sc, j0);
        }
        __syncthreads();
        float o[2][4] = {};
        mm_kn<kT, 2, 1>(o, Q, ld<DK>(), slab, kSlab, DK);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] *= expf(hi[ty + 32 * i]);
        mm_kn<kT, 2, 1>(o, P, kP, V + j0, ld<DV>(), kC);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (ty + 32 * i < c.len)
                st4(out + (ty + 32 * i) * a.so.t + j0 + 4 * tx,
                    make_float4(a.scale * o[i][0], a.scale * o[i][1], a.scale * o[i][2], a.scale * o[i][3]));
    }
}

// Sum over the 16 threads of a tile row; every one of them gets it.
__device__ __forceinline__ float row16(float x) {
#pragma unroll
    for (int m = 8; m; m >>= 1) x += __shfl_xor_sync(~0u, x, m);
    return x;
}

// A chunk's gradients.  Grid (chunks, H); S and R as the scans left them.
// dq and dk go to dqh, dkh [B,H,T,DK] fp32 where value heads share them.
// Nine products on the CUDA cores: 1.05 ms for the same.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kT, DK + DV == 128 ? 2 : 1) grad_kernel(LinAttnArgs a, View v, const float *S, const float *R, float *dqh,
                                                  float *dkh, float *dgt, Strides sdg) {
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *K = Q + kC * ld<DK>(), *V = K + kC * ld<DK>(), *O = V + kC * ld<DV>();
    // N by rows (N K), P by columns (P^T dO) and N by columns (N^T Q) in turn, from
    // the threads' registers; a slab of a state
    float *W = O + kC * ld<DV>(), *slab = W + kC * kP;
    constexpr int kSlabFloats = DK * kSlab > 64 * ld<DK>() ? DK * kSlab : 64 * ld<DK>();
    float *hi = slab + kSlabFloats, *lo = hi + kC, *te = lo + kC, *xq = te + kC, *xk = xq + kC, *xr = xk + kC, *xa = xr + kC, *red = xa + kC;
    const int ci = blockIdx.x, h = blockIdx.y;
    const Chunk c = chunk_at<kC>(v, a.T, ci);
    if (c.len <= 0) return;
    const int hk = h / (a.H / a.Hk);
    const bool shared = a.H != a.Hk;
    const long long out_row = (((long long)c.row * a.H + h) * a.T + c.t0) * DK;
    T *dq = at(static_cast<T *>(a.dq), a.sq, c.row, hk, c.t0), *dk = at(static_cast<T *>(a.dk), a.sk, c.row, hk, c.t0);
    T *dv = at(static_cast<T *>(a.dv), a.sv, c.row, h, c.t0);
    if (c.seq < 0) {
        if (shared) {
            zero_rows<float, DK, kT>(dqh + out_row, DK, c.len);
            zero_rows<float, DK, kT>(dkh + out_row, DK, c.len);
        } else {
            zero_rows<T, DK, kT>(dq, a.sq.t, c.len);
            zero_rows<T, DK, kT>(dk, a.sk.t, c.len);
        }
        zero_rows<T, DV, kT>(dv, a.sv.t, c.len);
        zero_rows<float, 1, kT>(at(dgt, sdg, c.row, h, c.t0), sdg.t, c.len);
        return;
    }
    if (threadIdx.x < 32)
        gates<kC>(gate_ptr(a, c, h), a.sg.t, c.len, a.flags & GDN_G_PER_HEAD, hi, lo, te);
    load_tile<T, DK, kT>(Q, at(static_cast<const T *>(a.q), a.sq, c.row, hk, c.t0), a.sq.t, c.len);
    load_tile<T, DK, kT>(K, at(static_cast<const T *>(a.k), a.sk, c.row, hk, c.t0), a.sk.t, c.len);
    load_tile<T, DV, kT>(V, at(static_cast<const T *>(a.v), a.sv, c.row, h, c.t0), a.sv.t, c.len);
    load_tile<T, DV, kT>(O, at(static_cast<const T *>(a.dout), a.sdo, c.row, h, c.t0), a.sdo.t, c.len);
    const float *Sc = S + ((long long)ci * a.H + h) * DK * DV, *Rc = R + ((long long)ci * a.H + h) * DK * DV;
    __syncthreads();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float p[2][4] = {}, n[2][4] = {};
    {
        tile::mm_nt<kT, 2, 4>(p, Q, ld<DK>(), K, ld<DK>(), DK);
        tile::mm_nt<kT, 2, 4>(n, O, ld<DV>(), V, ld<DV>(), DV);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = ty + 32 * i, s = tx + 16 * j;
                const float f = s <= t ? a.scale * decay_between(hi[t], lo[t], hi[s], lo[s]) : 0.f;
                const float nn = s <= t ? n[i][j] * f : 0.f;
                W[t * kP + s] = nn;
                slab[t * 65 + s] = s < t ? p[i][j] * nn : 0.f;  // A
                p[i][j] = s <= t ? p[i][j] * f : 0.f;
                n[i][j] = nn;
            }
    }
    __syncthreads();
    if (threadIdx.x < 2 * kC) {  // A's sums: rows, then columns
        const int t = threadIdx.x & (kC - 1);
        const bool rows = threadIdx.x < kC;
        float x = 0.f;
        for (int s = 0; s < kC; ++s) x += rows ? slab[t * 65 + s] : slab[s * 65 + t];
        (rows ? xa : xk)[t] = x;
    }
    auto columns = [&](const float (&x)[2][4]) {  // into W, which has been read
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) W[(tx + 16 * j) * kP + ty + 32 * i] = x[i][j];
    };
    constexpr int NB = DK / 64;
    // row sums of x against the rows of a tile
    auto along = [&](const float (&x)[2][4 * NB], const float *tile_, float *to) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float y = 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float4 q = ld4(tile_ + (ty + 32 * i) * ld<DK>() + 4 * tx + 64 * b);
                y = fmaf(q.x, x[i][4 * b], fmaf(q.y, x[i][4 * b + 1], fmaf(q.z, x[i][4 * b + 2], fmaf(q.w, x[i][4 * b + 3], y))));
            }
            y = row16(y);
            if (tx == 0) to[ty + 32 * i] = y;
        }
    };
    auto put = [&](const float (&x)[2][4 * NB], T *to, long long step, float *wide) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int t = ty + 32 * i, d = 4 * tx + 64 * b;
                const float4 y = make_float4(x[i][4 * b], x[i][4 * b + 1], x[i][4 * b + 2], x[i][4 * b + 3]);
                if (t < c.len) {
                    if (shared) st4(wide + out_row + (long long)t * DK + d, y);
                    else st4(to + t * step + d, y);
                }
            }
    };
    // dq: the part through S over its columns in slabs of 64, then the chunk's own
    {
        float acc[2][4 * NB] = {};
        for (int j0 = 0; j0 < DV; j0 += 64) {
            __syncthreads();
            load_slab_t<DK, DV>(slab, Sc, j0);
            __syncthreads();
            mm_kn<kT, 2, NB>(acc, O + j0, ld<DV>(), slab, ld<DK>(), 64);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4 * NB; ++j) acc[i][j] *= a.scale * expf(hi[ty + 32 * i]);
        along(acc, Q, xq);
        mm_kn<kT, 2, NB>(acc, W, kP, K, ld<DK>(), kC);
        put(acc, dq, a.sq.t, dqh);
    }
    // dk and dv, with R in the same slabs, both ways round; <R, S> on the way
    float dot = 0.f;
    {
        float acc[2][4 * NB] = {};
        for (int j0 = 0; j0 < DV; j0 += 64) {
            __syncthreads();
            load_slab_t<DK, DV>(slab, Rc, j0);
            if (j0 == 0) columns(p);
            __syncthreads();
            mm_kn<kT, 2, NB>(acc, V + j0, ld<DV>(), slab, ld<DK>(), 64);
            __syncthreads();
#pragma unroll 4
            for (int i = threadIdx.x; i < DK * 16; i += kT) {
                const float4 r = ld4(Rc + (i >> 4) * DV + j0 + (i & 15) * 4), s = ld4(Sc + (i >> 4) * DV + j0 + (i & 15) * 4);
                st4(slab + (i >> 4) * kSlab + (i & 15) * 4, r);
                dot = fmaf(r.x, s.x, fmaf(r.y, s.y, fmaf(r.z, s.z, fmaf(r.w, s.w, dot))));
            }
            __syncthreads();
            float w[2][4] = {};
            mm_kn<kT, 2, 1>(w, K, ld<DK>(), slab, kSlab, DK);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[i][j] *= expf(te[ty + 32 * i]);
            mm_kn<kT, 2, 1>(w, W, kP, O + j0, ld<DV>(), kC);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (ty + 32 * i < c.len)
                    st4(dv + (ty + 32 * i) * a.sv.t + j0 + 4 * tx, make_float4(w[i][0], w[i][1], w[i][2], w[i][3]));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4 * NB; ++j) acc[i][j] *= expf(te[ty + 32 * i]);
        along(acc, K, xr);
        __syncthreads();
        columns(n);
        __syncthreads();
        mm_kn<kT, 2, NB>(acc, W, kP, Q, ld<DK>(), kC);
        put(acc, dk, a.sk.t, dkh);
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(~0u, dot, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x < kC) {  // each token's own sums, in order
        const int u = threadIdx.x;
        if (u < c.len) {
            float x = 0.f, d = 0.f;
            for (int w = 0; w < kT / 32; ++w) d += red[w];
            for (int t = 0; t < kC; ++t) x += t < u ? xr[t] : xq[t] + (xa[t] - xk[t]);
            at(dgt, sdg, c.row, h, c.t0)[u * sdg.t] = fmaf(expf(hi[c.len - 1]), d, x);
        }
    }
}

size_t page_bytes(const LinAttnArgs &a) { return 4 * (size_t)a.H * a.Dk * a.Dv; }
size_t up(size_t x) { return (x + 255) / 256 * 256; }

template <class F>
int smem_limit(F f, int bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int launched() {
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    return GDN_OK;
}

#define LA_TRY(x)                       \
    do {                                \
        const int st_ = (x);            \
        if (st_ != GDN_OK) return st_;  \
    } while (0)

// The states that enter the chunks, to U; with R also their gradients.
template <typename T, int DK, int DV>
int run_states(const LinAttnArgs &a, const View &v, float *U, float *R, float *decay, cudaStream_t stream) {
    const int smem = 4 * (kC * (ld<DK>() + ld<DV>()) + 3 * kC), both = R ? 2 : 1, blocks = (DK * DV + 1023) / 1024;
    LA_TRY(smem_limit(share_kernel<T, DK, DV>, smem));
    share_kernel<T, DK, DV><<<dim3(v.n_chunks, a.H, both), 256, smem, stream>>>(a, v, U, R, decay);
    LA_TRY(launched());
    scan_kernel<<<dim3(both * blocks, a.H, a.n_seq), 256, 0, stream>>>(a, v, U, R, decay, DK * DV, blocks);
    return launched();
}

template <typename T, int DK, int DV>
int run_fwd(const LinAttnArgs &a, const View &v, float *U, float *decay, cudaStream_t stream) {
    LA_TRY((run_states<T, DK, DV>(a, v, U, nullptr, decay, stream)));
    const int smem = 4 * (kC * (2 * ld<DK>() + ld<DV>() + kP) + DK * kSlab + 3 * kC);
    LA_TRY(smem_limit(out_kernel<T, DK, DV>, smem));
    out_kernel<T, DK, DV><<<dim3(v.n_chunks, a.H), kT, smem, stream>>>(a, v, U);
    return launched();
}

struct BwdWs {
    float *U, *R, *decay, *dqh, *dkh, *dgt;
    size_t bytes;
};

BwdWs bwd_ws(const LinAttnArgs &a, void *ws) {
    const size_t tab = table_bytes(a, kC), n = chunk_bound(a, kC);
    const size_t heads = a.H != a.Hk ? up(4 * (size_t)a.B * a.H * a.T * a.Dk) : 0;
    const size_t gates = (a.flags & GDN_G_PER_HEAD) ? up(4 * (size_t)a.B * a.H * a.T) : 0;
    char *p = static_cast<char *>(ws) + tab;
    BwdWs w;
    w.U = reinterpret_cast<float *>(p), p += n * page_bytes(a);
    w.R = reinterpret_cast<float *>(p), p += n * page_bytes(a);
    w.decay = reinterpret_cast<float *>(p), p += up(4 * n * a.H);
    w.dqh = reinterpret_cast<float *>(p), p += heads;
    w.dkh = reinterpret_cast<float *>(p), p += heads;
    w.dgt = reinterpret_cast<float *>(p), p += gates;
    w.bytes = p - static_cast<char *>(ws);
    return w;
}

template <typename T, int DK, int DV>
int run_bwd(const LinAttnArgs &a, const View &v, const BwdWs &w, cudaStream_t stream) {
    LA_TRY((run_states<T, DK, DV>(a, v, w.U, w.R, w.decay, stream)));
    constexpr int slab = DK * kSlab > 64 * ld<DK>() ? DK * kSlab : 64 * ld<DK>();
    const int smem = 4 * (kC * (2 * ld<DK>() + 2 * ld<DV>() + kP) + slab + 7 * kC + 32);
    LA_TRY(smem_limit(grad_kernel<T, DK, DV>, smem));
    const bool per_head = a.flags & GDN_G_PER_HEAD;
    const Strides whole{(long long)a.H * a.T, a.T, 1};
    grad_kernel<T, DK, DV><<<dim3(v.n_chunks, a.H), kT, smem, stream>>>(a, v, w.U, w.R, w.dqh, w.dkh,
                                                                        per_head ? w.dgt : a.dg, per_head ? whole : a.sg);
    return launched();
}

template <typename T>
int fwd_t(const LinAttnArgs &a, const View &v, float *U, float *decay, cudaStream_t s) {
    if (a.Dk == 128) return a.Dv == 128 ? run_fwd<T, 128, 128>(a, v, U, decay, s) : run_fwd<T, 128, 64>(a, v, U, decay, s);
    return a.Dv == 128 ? run_fwd<T, 64, 128>(a, v, U, decay, s) : run_fwd<T, 64, 64>(a, v, U, decay, s);
}

template <typename T>
int bwd_t(const LinAttnArgs &a, const View &v, const BwdWs &w, cudaStream_t s) {
    if (a.Dk == 128) return a.Dv == 128 ? run_bwd<T, 128, 128>(a, v, w, s) : run_bwd<T, 128, 64>(a, v, w, s);
    return a.Dv == 128 ? run_bwd<T, 64, 128>(a, v, w, s) : run_bwd<T, 64, 64>(a, v, w, s);
}

}  // namespace

int make_view(const LinAttnArgs &a, int C, void *ws, View *v, cudaStream_t stream) {
    v->n_chunks = chunk_bound(a, C);
    v->per_row = (a.T + C - 1) / C;
    v->chunks = v->seqs = nullptr;
    if (!a.cu) return GDN_OK;
    int4 *chunks = static_cast<int4 *>(ws), *seqs = chunks + v->n_chunks;
    table_kernel<<<1, kTableThreads, 0, stream>>>(a.cu, a.n_seq, a.T, C, chunks, seqs, v->n_chunks);
    v->chunks = chunks, v->seqs = seqs;
    return launched();
}

int launch_group_sum(const LinAttnArgs &a, const float *dqh, const float *dkh, cudaStream_t stream) {
    const long long n = (long long)a.T * a.Dk / 4;
    const dim3 grid(2 * (unsigned)(n < 256 * 1024 ? (n + 255) / 256 : 1024), a.Hk, a.B);
    const float4 *q = reinterpret_cast<const float4 *>(dqh), *k = reinterpret_cast<const float4 *>(dkh);
    if (a.dtype == GDN_BF16) group_sum_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, q, k);
    else group_sum_kernel<float><<<grid, 256, 0, stream>>>(a, q, k);
    return launched();
}

int launch_head_sum(const float *src, float *dg, int B, int H, int T, cudaStream_t stream) {
    head_sum_kernel<<<H, 1024, 0, stream>>>(src, dg, B, H, T);
    return launched();
}

}  // namespace la

using namespace la;

size_t linattn_fwd_workspace(const LinAttnArgs &a) {
    return table_bytes(a, kC) + (size_t)chunk_bound(a, kC) * page_bytes(a) + up(4 * (size_t)chunk_bound(a, kC) * a.H);
}

int launch_linattn_fwd(const LinAttnArgs &a, cudaStream_t stream) {
    View v;
    LA_TRY(make_view(a, kC, a.ws, &v, stream));
    float *U = reinterpret_cast<float *>(static_cast<char *>(a.ws) + table_bytes(a, kC));
    float *decay = U + (size_t)v.n_chunks * page_bytes(a) / 4;
    return a.dtype == GDN_BF16 ? fwd_t<__nv_bfloat16>(a, v, U, decay, stream) : fwd_t<float>(a, v, U, decay, stream);
}

size_t linattn_bwd_workspace(const LinAttnArgs &a) { return bwd_ws(a, nullptr).bytes; }

int launch_linattn_bwd(const LinAttnArgs &a, cudaStream_t stream) {
    View v;
    LA_TRY(make_view(a, kC, a.ws, &v, stream));
    const bool shared = a.H != a.Hk, per_head = a.flags & GDN_G_PER_HEAD;
    const BwdWs w = bwd_ws(a, a.ws);
    LA_TRY(a.dtype == GDN_BF16 ? bwd_t<__nv_bfloat16>(a, v, w, stream) : bwd_t<float>(a, v, w, stream));
    if (shared) LA_TRY(launch_group_sum(a, w.dqh, w.dkh, stream));
    if (per_head) LA_TRY(launch_head_sum(w.dgt, a.dg, a.B, a.H, a.T, stream));
    return GDN_OK;
}

}  // namespace gdn
