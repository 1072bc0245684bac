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

// 1 / (1 + exp(-x)).  Where exp(-x) is infinite the quotient is 0.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + exp2_fast(-kLog2e * x)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
// silu'(x) from sigmoid(x).
__device__ __forceinline__ float silu_slope(float x, float s) { return s * fmaf(x, 1.f - s, 1.f); }

// log(1 + e) / e for e in 0..1, by interpolation in Chebyshev's points: to 1.3e-7.
// lg2 would take twice an ex2's time and lose the value of small e against 1.
__device__ __forceinline__ float log1p_over(float e) {
    float p = -0.00317605701f;
    p = fmaf(p, e, 0.0195425283f);
    p = fmaf(p, e, -0.0563736148f);
    p = fmaf(p, e, 0.105436236f);
    p = fmaf(p, e, -0.152696669f);
    p = fmaf(p, e, 0.196632743f);
    p = fmaf(p, e, -0.249516159f);
    p = fmaf(p, e, 0.333297104f);
    p = fmaf(p, e, -0.499998927f);
    return fmaf(p, e, 1.f);
}
// log(1 + exp(v)) = max(v, 0) + log(1 + exp(-|v|)).
__device__ __forceinline__ float softplus(float v) {
    const float e = exp2_fast(-kLog2e * fabsf(v));
    return fmaf(e, log1p_over(e), fmaxf(v, 0.f));
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

inline int launched() {
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    return GDN_OK;
}

}  // namespace mx
}  // namespace gdn
