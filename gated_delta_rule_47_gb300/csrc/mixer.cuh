// What the kernels next to a mixer share: where a token's sequence lies, the
// activations, and fixed-order sums of partial gradients.
#pragma once

#include <stdint.h>

#include "gdn_internal.h"
#include "mixer_ops.h"
#include "vec.cuh"

namespace gdn {
namespace mx {

// The tokens from some place on to `end` that belong to sequence `s`, which
// starts at `start`; s < 0: to no sequence.
struct Run {
    int s, start, end;
};

// Offsets outside 0..T count as cut to it; out of order they still give places
// within the row.
__device__ __forceinline__ int cut(int t, int T) { return min(max(t, 0), T); }

// The run that token t of a row is in: the last sequence that starts at or
// before it, which is not an empty one where t lies before its end.
__device__ __forceinline__ Run run_at(const int *cu, int n_seq, int T, int row, int t) {
    if (!cu) return {row, 0, T};
    int lo = 0, hi = n_seq + 1;  // offsets before lo are <= t, from hi on > t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    const int s = lo - 1;
    if (s < 0) return {-1, 0, cut(cu[0], T)};
    if (s >= n_seq) return {-1, cut(cu[n_seq], T), T};
    return {s, cut(cu[s], T), cut(cu[s + 1], T)};
}

// Whether sequence s has no tokens (its state or window is passed on).
__device__ __forceinline__ bool no_tokens(const int *cu, int T, int s) { return cut(cu[s + 1], T) <= cut(cu[s], T); }

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float inverse(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + exp(-x)); 0 where exp(-x) is infinite.
__device__ __forceinline__ float sigmoid(float x) { return inverse(1.f + exp2_fast(-kLog2e * x)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
// silu'(x) from sigmoid(x).
__device__ __forceinline__ float silu_slope(float x, float s) { return s * fmaf(x, 1.f - s, 1.f); }

// log(1 + e) / e for e in 0..1, by interpolation in Chebyshev's points: to 1.3e-7.
// lg2 would take twice an ex2's time and lose the value of small e against 1.
// Coefficient i, the highest power's first.
__device__ __forceinline__ float log1p_coefficient(int i) {
    const float c[10] = {-0.00317605701f, 0.0195425283f, -0.0563736148f, 0.105436236f, -0.152696669f,
                         0.196632743f, -0.249516159f, 0.333297104f, -0.499998927f, 1.f};
    return c[i];
}
__device__ __forceinline__ float log1p_over(float e) {
    float p = log1p_coefficient(0);
#pragma unroll
    for (int i = 1; i < 10; ++i) p = fmaf(p, e, log1p_coefficient(i));
    return p;
}
// log(1 + exp(v)) = max(v, 0) + log(1 + exp(-|v|)).
__device__ __forceinline__ float softplus(float v) {
    const float e = exp2_fast(-kLog2e * fabsf(v));
    return fmaf(e, log1p_over(e), fmaxf(v, 0.f));
}

// Two fp32 numbers for one instruction: half the issue slots of single ones at
// the same rate of operations.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 both(float x) { return pair(x, x); }
__device__ __forceinline__ void split(F2 p, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float sum(F2 p) {
    float a, b;
    split(p, a, b);
    return a + b;
}

// The activations of two at once: the exponentials and reciprocals are single.
__device__ __forceinline__ F2 softplus2(F2 v) {
    float a, b;
    split(v, a, b);
    const F2 e = pair(exp2_fast(-kLog2e * fabsf(a)), exp2_fast(-kLog2e * fabsf(b)));
    F2 p = both(log1p_coefficient(0));
#pragma unroll
    for (int i = 1; i < 10; ++i) p = fma2(p, e, both(log1p_coefficient(i)));
    return fma2(e, p, pair(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}
__device__ __forceinline__ F2 sigmoid2(F2 x) {
    float a, b;
    split(mul2(x, both(-kLog2e)), a, b);
    split(add2(pair(exp2_fast(a), exp2_fast(b)), both(1.f)), a, b);
    return pair(inverse(a), inverse(b));
}
__device__ __forceinline__ F2 silu2(F2 x) { return mul2(x, sigmoid2(x)); }
__device__ __forceinline__ F2 silu_slope2(F2 x, F2 s) { return mul2(s, fma2(x, fma2(s, both(-1.f), both(1.f)), both(1.f))); }
// N elements as pairs.
template <typename T, int N>
__device__ __forceinline__ void unpack2(const typename Vec<T, N>::Raw &p, F2 (&x)[N / 2]) {
    float v[N];
    Vec<T, N>::unpack(p, v);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) x[e] = pair(v[2 * e], v[2 * e + 1]);
}
template <typename T, int N>
__device__ __forceinline__ typename Vec<T, N>::Raw pack2(const F2 (&x)[N / 2]) {
    float v[N];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) split(x[e], v[2 * e], v[2 * e + 1]);
    return Vec<T, N>::pack(v);
}
// N fp32 weights from w on as pairs, 1 where there are none.
template <int N>
__device__ __forceinline__ void weights2(const float *w, bool there, F2 (&x)[N / 2]) {
#pragma unroll
    for (int e = 0; e < N / 2; e += 2) {
        float4 y = make_float4(1.f, 1.f, 1.f, 1.f);
        if (there) y = __ldg(reinterpret_cast<const float4 *>(w + 2 * e));
        x[e] = pair(y.x, y.y), x[e + 1] = pair(y.z, y.w);
    }
}

// The sum of column c of part's rows [n][C], in order: 32 columns a CTA, its
// strands of rows, then the strands; the first strand's threads get it.
template <int STRANDS>
__device__ __forceinline__ float column_sum(const float *part, int n, long long C, long long c) {
    __shared__ float s[STRANDS][33];
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    float x = 0.f;
    if (c < C)
#pragma unroll 8
        for (int i = strand; i < n; i += STRANDS) x += part[i * C + c];
    s[strand][lane] = x;
    __syncthreads();
    x = 0.f;
    if (strand == 0)
#pragma unroll
        for (int j = 0; j < STRANDS; ++j) x += s[j][lane];
    return x;
}

// A grid of as many CTAs as the SMs hold at once.
template <auto F, int NT>
int resident_ctas() {
    static const int n = [] {
        int k = 0;
        const bool ok = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k, F, NT, 0) == cudaSuccess && k > 0;
        return (ok ? k : 1) * device_sm_count();
    }();
    return n;
}

// A kernel that is launched with `follow` may begin as soon as every CTA of the one
// before it in the stream has called let_follow(); it calls follow_on() before it
// reads or writes what that one, or work before that one, writes or reads.  Measured:
// 2 us a call of two or three kernels (scan of 1999 x 512 fp32, backward, 61.6 to 59.4).
__device__ __forceinline__ void let_follow() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void follow_on() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
void follow(void (*kernel)(P...), unsigned ctas, int threads, int smem, cudaStream_t stream, const A &...args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(ctas), config.blockDim = dim3(threads), config.dynamicSmemBytes = smem, config.stream = stream;
    config.attrs = &early, config.numAttrs = 1;
    cudaLaunchKernelEx(&config, kernel, args...);  // a failure is the last error, as that of <<<>>>
}

inline int launched() {
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    return GDN_OK;
}

}  // namespace mx
}  // namespace gdn
