// rms_norm.cu -- root-mean-square norm of a row after the residual's addition,
// with an output in the tensors' type or in e4m3 with scales; and its backward.
//
//   h = x + res;   y = w h / sqrt(mean(h^2) + eps)
//   e4m3: per group, scale = max(max|y| / 448, 1e-12) and y is stored as y / scale
//
// backward, for the row h that the forward stored (r = 1 / sqrt(...), C columns):
//   dh = r (w dy - h r^2 mean(h w dy)) + dres;   dw = sum over rows of dy h r
//
// One pass over the data: a CTA holds its row in registers between the sum of
// squares and the output.  The bytes of the rows bound both directions.
// Sums are in fp32; h enters the norm before it is rounded for the store.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "gdn_internal.h"
#include "layer_ops.h"

namespace gdn {
namespace {

constexpr float kTop = 448.f;  // the largest e4m3 value

// Vectors of N elements: 16 bytes (8 bf16 or 4 fp32), and what rows of other
// lengths divide into.
template <typename T>
constexpr int kWide = 16 / sizeof(T);
template <typename T, int N>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(uint4 p, float (&x)[8]) {
        const uint32_t u[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&t);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Vec<__nv_bfloat16, 2> {
    using Raw = uint32_t;
    static __device__ __forceinline__ void unpack(uint32_t p, float (&x)[2]) {
        x[0] = __uint_as_float(p << 16), x[1] = __uint_as_float(p & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t pack(const float (&x)[2]) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(x[0], x[1]);
        return *reinterpret_cast<const uint32_t *>(&t);
    }
};
template <>
struct Vec<__nv_bfloat16, 1> {
    using Raw = unsigned short;
    static __device__ __forceinline__ void unpack(unsigned short p, float (&x)[1]) { x[0] = __uint_as_float((uint32_t)p << 16); }
    static __device__ __forceinline__ unsigned short pack(const float (&x)[1]) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
    }
};
template <>
struct Vec<float, 1> {
    using Raw = uint32_t;
    static __device__ __forceinline__ void unpack(uint32_t p, float (&x)[1]) { x[0] = __uint_as_float(p); }
    static __device__ __forceinline__ uint32_t pack(const float (&x)[1]) { return __float_as_uint(x[0]); }
};
template <>
struct Vec<float, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(uint4 p, float (&x)[4]) {
        x[0] = __uint_as_float(p.x), x[1] = __uint_as_float(p.y);
        x[2] = __uint_as_float(p.z), x[3] = __uint_as_float(p.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

__device__ __forceinline__ float ldf(const float *p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void stf(float *p, float x) { *p = x; }
__device__ __forceinline__ void stf(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// max that keeps a NaN, so that a bad row shows in its scale
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A group's scale from its largest |y|, and what y is multiplied by.
__device__ __forceinline__ float scale_of(float top) { return max_nan(top * (1.f / kTop), 1e-12f); }
__device__ __forceinline__ float inverse(float x) { return __fdividef(1.f, x); }

// Sum / maximum over the CTA; every thread gets it.  `s` has room for 32, and
// nobody reads an earlier call's values from it any more.
template <int NT, bool MAX>
__device__ __forceinline__ float block_all(float x, float *s) {
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        const float y = __shfl_xor_sync(~0u, x, m);
        x = MAX ? max_nan(x, y) : x + y;
    }
    if (NT == 32) return x;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    x = s[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) x = MAX ? max_nan(x, s[w]) : x + s[w];
    return x;
}

// A vector's weights (1 where there are none).
template <int N>
__device__ __forceinline__ void load_weights(const float *w, int i, bool there, float (&x)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            float4 y = make_float4(1.f, 1.f, 1.f, 1.f);
            if (w && there) y = __ldg(reinterpret_cast<const float4 *>(w) + (i * N + e) / 4);
            x[e] = y.x, x[e + 1] = y.y, x[e + 2] = y.z, x[e + 3] = y.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = w && there ? __ldg(w + i * N + e) : 1.f;
    }
}

template <int N>
__device__ __forceinline__ void store_e4m3(void *p, const float (&y)[N], float inv) {
    if constexpr (N == 1) {
        *static_cast<unsigned char *>(p) = __nv_cvt_float_to_fp8(y[0] * inv, __NV_SATFINITE, __NV_E4M3);
        return;
    } else if constexpr (N == 2) {
        *static_cast<unsigned short *>(p) = __nv_cvt_float2_to_fp8x2(make_float2(y[0] * inv, y[1] * inv), __NV_SATFINITE, __NV_E4M3);
        return;
    } else {
        uint32_t u[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i] * inv, y[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2] * inv, y[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
            u[i] = lo | hi << 16;
        }
        if (N == 8) *static_cast<uint2 *>(p) = make_uint2(u[0], u[N / 4 - 1]);
        else *static_cast<uint32_t *>(p) = u[0];
    }
}

// Rows blockIdx.x, + gridDim.x, .. by a CTA of NT threads, V vectors a thread
// (vector j of thread t is number j NT + t, so a group's vectors are
// consecutive lanes of one warp).  The next row is on its way while this one is
// summed and written: a CTA that takes one row at a time has nothing to load
// for half of its life.  The weights stay in registers.  Instructions bound an
// 8-bit output before the bytes do: a thread takes two or four vectors, so that
// the sums over the CTA cost less of them, and y is not formed for it:
// y / scale = (h w) (r / scale).  Measured, bf16, 32760 x 2048 with a residual:
// to e4m3 in groups of 128 76 us (472 MB at 6.2 TB/s), to bf16 86 (6.2 TB/s);
// 8 rows 2.5 us.
// C is a multiple of the vector's width N: 16384 x 2046 bf16 with a residual 45 us
// in vectors of two, x 2047 56 in single elements (x 2048: 43).
template <typename T, int N, int NT, int V>
__global__ void __launch_bounds__(NT, V <= 2 ? 1024 / NT : 1) norm_kernel(NormArgs a) {
    using Raw = typename Vec<T, N>::Raw;
    __shared__ float red[2][32];
    const int nv = a.C / N;
    Raw px[V], pr[V];
    auto fetch = [&](long long row) {
        const Raw *x = reinterpret_cast<const Raw *>(static_cast<const T *>(a.x) + row * a.C);
        const Raw *res = reinterpret_cast<const Raw *>(static_cast<const T *>(a.res) + row * a.C);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = j * NT + threadIdx.x;
            px[j] = pr[j] = Raw{};
            if (row < a.rows && i < nv) {
                px[j] = __ldcs(x + i);
                if (a.res) pr[j] = __ldcs(res + i);
            }
        }
    };
    fetch(blockIdx.x);
    float w[V][N];
#pragma unroll
    for (int j = 0; j < V; ++j) load_weights(a.w, j * NT + threadIdx.x, j * NT + threadIdx.x < nv, w[j]);
    int buf = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
        float h[V][N];
        float sum = 0.f;
        Raw *ho = a.h ? reinterpret_cast<Raw *>(static_cast<T *>(a.h) + row * a.C) : nullptr;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = j * NT + threadIdx.x;
            Vec<T, N>::unpack(px[j], h[j]);
            if (a.res) {
                float r[N];
                Vec<T, N>::unpack(pr[j], r);
#pragma unroll
                for (int e = 0; e < N; ++e) h[j][e] += r[e];
            }
            if (ho && i < nv) __stcs(ho + i, Vec<T, N>::pack(h[j]));
#pragma unroll
            for (int e = 0; e < N; ++e) sum = fmaf(h[j][e], h[j][e], sum);
        }
        fetch(row + gridDim.x);
        sum = block_all<NT, false>(sum, red[buf]);
        const float r = rsqrtf(sum / a.C + a.eps);
        if (!a.out_e4m3) {
            Raw *y = reinterpret_cast<Raw *>(static_cast<T *>(a.y) + row * a.C);
#pragma unroll
            for (int j = 0; j < V; ++j) {
#pragma unroll
                for (int e = 0; e < N; ++e) h[j][e] *= r * w[j][e];
                if (j * NT + threadIdx.x < nv) __stcs(y + j * NT + threadIdx.x, Vec<T, N>::pack(h[j]));
            }
            continue;
        }
        unsigned char *y = static_cast<unsigned char *>(a.y) + row * a.C;
        float top[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            top[j] = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                h[j][e] *= w[j][e];
                top[j] = max_nan(top[j], fabsf(h[j][e]));
            }
        }
        if (a.group == 0) {
            float all = top[0];
#pragma unroll
            for (int j = 1; j < V; ++j) all = max_nan(all, top[j]);
            __syncthreads();  // the sum has been read by all
            const float scale = scale_of(r * block_all<NT, true>(all, red[buf]));
            if (threadIdx.x == 0) a.scales[row] = scale;
            const float inv = r * inverse(scale);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j * NT + threadIdx.x < nv) store_e4m3<N>(y + (size_t)(j * NT + threadIdx.x) * N, h[j], inv);
            continue;
        }
        const int lanes = a.group / N;  // a power of two, at most 32
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = j * NT + threadIdx.x;
            for (int m = lanes >> 1; m; m >>= 1) top[j] = max_nan(top[j], __shfl_xor_sync(~0u, top[j], m));
            const float scale = scale_of(r * top[j]);
            if (i < nv) {
                if ((i & (lanes - 1)) == 0) a.scales[row * (a.C / a.group) + i / lanes] = scale;
                store_e4m3<N>(y + (size_t)i * N, h[j], r * inverse(scale));
            }
        }
    }
}

// Any C, for rows that the registers do not hold: the row is read again after its
// sum of squares (and again for its maximum), element by element, from L2.
// Groups are not offered here.
template <typename T>
__global__ void __launch_bounds__(256) norm_any_kernel(NormArgs a) {
    __shared__ float red[2][32];
    const long long row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.C;
    const T *res = a.res ? static_cast<const T *>(a.res) + row * a.C : nullptr;
    T *ho = a.h ? static_cast<T *>(a.h) + row * a.C : nullptr;
    float sum = 0.f, top = 0.f;
    for (int i = threadIdx.x; i < a.C; i += 256) {
        const float h = ldf(x + i) + (res ? ldf(res + i) : 0.f);
        sum = fmaf(h, h, sum);
    }
    sum = block_all<256, false>(sum, red[0]);
    const float r = rsqrtf(sum / a.C + a.eps);
    float inv = 1.f;
    if (a.out_e4m3) {
        for (int i = threadIdx.x; i < a.C; i += 256) {
            const float h = ldf(x + i) + (res ? ldf(res + i) : 0.f);
            top = max_nan(top, fabsf(h * (r * (a.w ? a.w[i] : 1.f))));
        }
        top = block_all<256, true>(top, red[1]);
        const float scale = scale_of(top);
        if (threadIdx.x == 0) a.scales[row] = scale;
        inv = inverse(scale);
    }
    for (int i = threadIdx.x; i < a.C; i += 256) {
        const float h = ldf(x + i) + (res ? ldf(res + i) : 0.f);
        const float y = h * (r * (a.w ? a.w[i] : 1.f));
        // h after every read of x and res at this place, which it may overwrite
        if (ho) stf(ho + i, h);
        if (a.out_e4m3)
            static_cast<unsigned char *>(a.y)[row * a.C + i] = __nv_cvt_float_to_fp8(y * inv, __NV_SATFINITE, __NV_E4M3);
        else
            stf(static_cast<T *>(a.y) + row * a.C + i, y);
    }
}

// A grid of as many CTAs as the SMs hold at once (one more would run alone at
// the end), or of `rows` where that is less.
template <auto F, int NT>
unsigned resident(long long rows) {
    static const int per_sm = [] {
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, F, NT, 0) == cudaSuccess && n > 0 ? n : 1;
    }();
    const long long full = (long long)device_sm_count() * per_sm;
    return (unsigned)(rows < full ? rows : full);
}

template <typename T, int N, int NT, int V>
void launch_v(const NormArgs &a, cudaStream_t stream) {
    norm_kernel<T, N, NT, V><<<resident<norm_kernel<T, N, NT, V>, NT>(a.rows), NT, 0, stream>>>(a);
}

// Rows of narrow vectors: eight a thread.  Element by element in two passes they
// took 49 us where this takes 45 (16384 x 2047 bf16 without a residual), and the
// backward 108 where it takes 56.
template <typename T, int N>
void launch_narrow(const NormArgs &a, cudaStream_t stream) {
    const int nv = a.C / N;
    if (nv <= 64) launch_v<T, N, 32, 2>(a, stream);
    else if (nv <= 256) launch_v<T, N, 32, 8>(a, stream);
    else if (nv <= 512) launch_v<T, N, 64, 8>(a, stream);
    else if (nv <= 1024) launch_v<T, N, 128, 8>(a, stream);
    else if (nv <= 2048) launch_v<T, N, 256, 8>(a, stream);
    else if (nv <= 4096) launch_v<T, N, 512, 8>(a, stream);
    else norm_any_kernel<T><<<(unsigned)a.rows, 256, 0, stream>>>(a);
}

// Two vectors a thread, four from 4096 bf16 columns on: one leaves the sums over
// the CTA too large a share (32768 x 2048, a residual, to e4m3: 80 us against
// 75), eight too few warps (4096 columns: 97 against 75).
template <typename T>
void launch_t(const NormArgs &a, cudaStream_t stream) {
    constexpr int N = kWide<T>;
    const int nv = a.C / N;
    if (a.C % N != 0) {
        sizeof(T) == 2 && a.C % 2 == 0 ? launch_narrow<T, sizeof(T) == 2 ? 2 : 1>(a, stream) : launch_narrow<T, 1>(a, stream);
    } else if (nv > 4096) {
        norm_any_kernel<T><<<(unsigned)a.rows, 256, 0, stream>>>(a);
    } else if (nv <= 32) {
        launch_v<T, N, 32, 1>(a, stream);
    } else if (nv <= 64) {
        launch_v<T, N, 32, 2>(a, stream);
    } else if (nv <= 128) {
        launch_v<T, N, 64, 2>(a, stream);
    } else if (nv <= 256) {
        launch_v<T, N, 128, 2>(a, stream);
    } else if (nv <= 512) {
        launch_v<T, N, 128, 4>(a, stream);
    } else if (nv <= 1024) {
        launch_v<T, N, 256, 4>(a, stream);
    } else if (nv <= 2048) {
        launch_v<T, N, 512, 4>(a, stream);
    } else {
        launch_v<T, N, 512, 8>(a, stream);
    }
}

// ------------------------------------------------------------------ backward
constexpr int kBwdThreads = 256;

// Rows by groups of NT of the CTA's threads, a row each in turn, V vectors a
// thread as in norm_kernel: narrow rows would leave most of a CTA idle (512
// columns, 131072 rows: 259 us with 256 threads a row).  A thread's columns are
// the same in every row, so its share of dw stays in registers until the rows
// are done; then the groups' shares are added in order to part[blockIdx.x][C].
// Bound by the bytes: bf16, 16384 x 2048 with a residual's gradient 41 us, 268 MB
// at 6.6 TB/s (x 2046 45, x 2047 62).
template <typename T, int N, int NT, int V>
__global__ void __launch_bounds__(kBwdThreads, V == 1 ? 4 : V == 4 || V == 16 ? 1 : 2) norm_bwd_kernel(NormBwdArgs a, float *part) {
    using Raw = typename Vec<T, N>::Raw;
    constexpr int GROUPS = kBwdThreads / NT;
    __shared__ float red[2][2][kBwdThreads / 32];
    __shared__ __align__(16) float share[GROUPS > 1 ? kBwdThreads * N * V : 1];
    const int nv = a.C / N, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = threadIdx.x / NT, tid = threadIdx.x % NT, first = group * (NT / 32);
    const long long step = (long long)gridDim.x * GROUPS;
    float dw[V][N], w[V][N];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        load_weights(a.w, j * NT + tid, j * NT + tid < nv, w[j]);
#pragma unroll
        for (int e = 0; e < N; ++e) dw[j][e] = 0.f;
    }
    int buf = 0;
    Raw nh[V], nd[V], nr[V];
    auto fetch = [&](long long row) {  // the next row is on its way while this one is summed and written
        const Raw *h4 = reinterpret_cast<const Raw *>(static_cast<const T *>(a.h) + row * a.C);
        const Raw *dy4 = reinterpret_cast<const Raw *>(static_cast<const T *>(a.dy) + row * a.C);
        const Raw *dr4 = reinterpret_cast<const Raw *>(static_cast<const T *>(a.dres) + row * a.C);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = j * NT + tid;
            nh[j] = nd[j] = nr[j] = Raw{};
            if (row < a.rows && i < nv) {
                nh[j] = __ldcs(h4 + i);
                nd[j] = __ldcs(dy4 + i);
                if (a.dres) nr[j] = __ldcs(dr4 + i);
            }
        }
    };
    long long row = (long long)blockIdx.x * GROUPS + group;
    fetch(row);
    for (; row < a.rows; row += step, buf ^= 1) {
        Raw ph[V], pd[V], pr[V];
#pragma unroll
        for (int j = 0; j < V; ++j) ph[j] = nh[j], pd[j] = nd[j], pr[j] = nr[j];
        fetch(row + step);
        float ss = 0.f, sp = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float h[N], d[N];
            Vec<T, N>::unpack(ph[j], h);
            Vec<T, N>::unpack(pd[j], d);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                ss = fmaf(h[e], h[e], ss);
                sp = fmaf(h[e], d[e] * w[j][e], sp);
            }
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) {
            ss += __shfl_xor_sync(~0u, ss, m);
            sp += __shfl_xor_sync(~0u, sp, m);
        }
        if constexpr (NT > 32) {
            if (lane == 0) red[buf][0][warp] = ss, red[buf][1][warp] = sp;
            // one a row, of the group's threads: the buffers alternate
            if constexpr (GROUPS == 1) __syncthreads();
            else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(NT) : "memory");
            ss = sp = 0.f;
#pragma unroll
            for (int i = 0; i < NT / 32; ++i) ss += red[buf][0][first + i], sp += red[buf][1][first + i];
        }
        const float r = rsqrtf(ss / a.C + a.eps);
        const float m = r * r * (sp / a.C);
        Raw *dx = reinterpret_cast<Raw *>(static_cast<T *>(a.dx) + row * a.C);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = j * NT + tid;
            float h[N], d[N], g[N];
            Vec<T, N>::unpack(ph[j], h);
            Vec<T, N>::unpack(pd[j], d);
            Vec<T, N>::unpack(pr[j], g);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                g[e] = fmaf(r, fmaf(d[e], w[j][e], -h[e] * m), g[e]);
                dw[j][e] = fmaf(d[e], h[e] * r, dw[j][e]);
            }
            if (i < nv) __stcs(dx + i, Vec<T, N>::pack(g));
        }
    }
    float *to = part + (size_t)blockIdx.x * a.C;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = j * NT + tid;
        float *mine = GROUPS > 1 ? share + (group * V * NT + i) * N : to + (size_t)i * N;
        if (GROUPS > 1 || i < nv) {
            if constexpr (N % 4 == 0) {
#pragma unroll
                for (int e = 0; e < N; e += 4)
                    *reinterpret_cast<float4 *>(mine + e) = make_float4(dw[j][e], dw[j][e + 1], dw[j][e + 2], dw[j][e + 3]);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) mine[e] = dw[j][e];
            }
        }
    }
    if constexpr (GROUPS > 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < a.C; i += kBwdThreads) {
            float x = share[i];
#pragma unroll
            for (int g = 1; g < GROUPS; ++g) x += share[g * V * NT * N + i];
            to[i] = x;
        }
    }
}

// Any C, for rows that the registers do not hold: rows are read twice, and dw's
// share of a column is summed in `part` (8192 x 4095 bf16 took 223 us here).
template <typename T>
__global__ void __launch_bounds__(kBwdThreads) norm_bwd_any_kernel(NormBwdArgs a, float *part) {
    constexpr int NT = kBwdThreads;
    __shared__ float red[2][32];
    float *mine = part + (size_t)blockIdx.x * a.C;
    for (int i = threadIdx.x; i < a.C; i += NT) mine[i] = 0.f;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *h = static_cast<const T *>(a.h) + row * a.C, *dy = static_cast<const T *>(a.dy) + row * a.C;
        const T *dres = a.dres ? static_cast<const T *>(a.dres) + row * a.C : nullptr;
        float ss = 0.f, sp = 0.f;
        for (int i = threadIdx.x; i < a.C; i += NT) {
            const float x = ldf(h + i);
            ss = fmaf(x, x, ss);
            sp = fmaf(x, ldf(dy + i) * (a.w ? a.w[i] : 1.f), sp);
        }
        __syncthreads();  // the last row's sums have been read
        ss = block_all<NT, false>(ss, red[0]);
        sp = block_all<NT, false>(sp, red[1]);
        const float r = rsqrtf(ss / a.C + a.eps);
        const float m = r * r * (sp / a.C);
        for (int i = threadIdx.x; i < a.C; i += NT) {
            const float x = ldf(h + i), d = ldf(dy + i);
            mine[i] = fmaf(d, x * r, mine[i]);
            stf(static_cast<T *>(a.dx) + row * a.C + i,
                fmaf(r, fmaf(d, a.w ? a.w[i] : 1.f, -x * m), dres ? ldf(dres + i) : 0.f));
        }
    }
}

// dw[c] = the CTAs' shares: 32 columns a CTA, 32 strands of shares, then the
// strands in order.  3 us for 2048 columns of 304 shares: latency.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *part, float *dw, int n, int C) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, strand = threadIdx.x >> 5;
    float x = 0.f;
    if (c < C)
#pragma unroll 4
        for (int i = strand; i < n; i += 32) x += part[(size_t)i * C + c];
    s[strand][lane] = x;
    __syncthreads();
    if (strand == 0 && c < C) {
        x = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) x += s[j][lane];
        dw[c] = x;
    }
}

// The most shares of dw that a call makes (its workspace's size).
int bwd_ctas(long long rows) {
    const long long full = 4LL * device_sm_count();
    return (int)(rows < full ? rows : full);
}

// Launches with at most `most` CTAs (what the workspace holds) and says with how many.
template <auto F>
int launch_rows(const NormBwdArgs &a, int most, float *part, cudaStream_t stream) {
    const int fit = (int)resident<F, kBwdThreads>(a.rows), ctas = fit < most ? fit : most;
    F<<<ctas, kBwdThreads, 0, stream>>>(a, part);
    return ctas;
}

template <typename T, int N>
int launch_bwd_narrow(const NormBwdArgs &a, int most, float *part, cudaStream_t stream) {
    const int nv = a.C / N;
    if (nv <= 64) return launch_rows<norm_bwd_kernel<T, N, 32, 2>>(a, most, part, stream);
    if (nv <= 256) return launch_rows<norm_bwd_kernel<T, N, 32, 8>>(a, most, part, stream);
    if (nv <= 512) return launch_rows<norm_bwd_kernel<T, N, 64, 8>>(a, most, part, stream);
    if (nv <= 1024) return launch_rows<norm_bwd_kernel<T, N, 128, 8>>(a, most, part, stream);
    if (nv <= 2048) return launch_rows<norm_bwd_kernel<T, N, kBwdThreads, 8>>(a, most, part, stream);
    if (nv <= 4096) return launch_rows<norm_bwd_kernel<T, N, kBwdThreads, 16>>(a, most, part, stream);
    return launch_rows<norm_bwd_any_kernel<T>>(a, most, part, stream);
}

template <typename T>
int launch_bwd_t(const NormBwdArgs &a, int most, float *part, cudaStream_t stream) {
    constexpr int N = kWide<T>;
    const int nv = a.C / N;
    if (a.C % N != 0)
        return sizeof(T) == 2 && a.C % 2 == 0 ? launch_bwd_narrow<T, sizeof(T) == 2 ? 2 : 1>(a, most, part, stream)
                                              : launch_bwd_narrow<T, 1>(a, most, part, stream);
    if (nv > 4 * kBwdThreads) return launch_rows<norm_bwd_any_kernel<T>>(a, most, part, stream);
    // two vectors a thread, whose loads cover more of a row's sums than one's
    // (bf16, 131072 x 512: 82 us against 102)
    if (nv <= 32) return launch_rows<norm_bwd_kernel<T, N, 32, 1>>(a, most, part, stream);
    if (nv <= 64) return launch_rows<norm_bwd_kernel<T, N, 32, 2>>(a, most, part, stream);
    if (nv <= 128) return launch_rows<norm_bwd_kernel<T, N, 64, 2>>(a, most, part, stream);
    if (nv <= 256) return launch_rows<norm_bwd_kernel<T, N, 128, 2>>(a, most, part, stream);
    if (nv <= 2 * kBwdThreads) return launch_rows<norm_bwd_kernel<T, N, kBwdThreads, 2>>(a, most, part, stream);
    return launch_rows<norm_bwd_kernel<T, N, kBwdThreads, 4>>(a, most, part, stream);
}

}  // namespace

int launch_rms_norm(const NormArgs &a, cudaStream_t stream) {
    if (a.dtype == GDN_BF16) launch_t<__nv_bfloat16>(a, stream);
    else launch_t<float>(a, stream);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    return GDN_OK;
}

size_t rms_norm_bwd_workspace(long long rows, int C) { return 4 * (size_t)bwd_ctas(rows) * C; }

int launch_rms_norm_bwd(const NormBwdArgs &a, cudaStream_t stream) {
    float *part = static_cast<float *>(a.ws);
    const int most = bwd_ctas(a.rows);
    const int ctas = a.dtype == GDN_BF16 ? launch_bwd_t<__nv_bfloat16>(a, most, part, stream) : launch_bwd_t<float>(a, most, part, stream);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    norm_dw_kernel<<<(a.C + 31) / 32, 1024, 0, stream>>>(part, a.dw, ctas, a.C);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    return GDN_OK;
}

}  // namespace gdn
