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

using mx::F2;
using mx::both;
using mx::fma2;
using mx::mul2;
using mx::pair;
using mx::split;
using mx::sum;
// 2^x of both.
__device__ __forceinline__ F2 exp2_2(F2 x) {
    float a, b;
    split(x, a, b);
    return pair(mx::exp2_fast(a), mx::exp2_fast(b));
}

}  // namespace ssm
}  // namespace gdn
