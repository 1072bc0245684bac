// ssm.cuh -- what the kernels of the selective state space scan share.
//
//   D_t = softplus(dt_t + bias) or dt_t + bias
//   h_t = exp(D_t A) h_{t-1} + D_t B_t x_t,   y_t = (C_t . h_t + skip x_t) silu(z_t)
//
// with a state of N numbers for each channel.  There is no product over channels
// or tokens in it that matrix instructions could take: every (token, channel,
// state) has a decay of its own, an exponential and four multiply-adds.
//
// Sequences are cut into chunks, of the row and not of a sequence: a chunk that a
// sequence starts in sets its state anew there.  What passes over chunks is the
// state that a chunk leaves when it starts from 0 and the sum of its steps, whose
// exponential with A is the chunk's whole decay.
#pragma once

#include "mixer.cuh"

namespace gdn {
namespace ssm {

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
// 2^x of both.
__device__ __forceinline__ F2 exp2_2(F2 x) {
    float a, b;
    split(x, a, b);
    return pair(mx::exp2_fast(a), mx::exp2_fast(b));
}

}  // namespace ssm
}  // namespace gdn
