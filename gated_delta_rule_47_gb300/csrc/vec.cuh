// Vectors of a row's elements, as they are loaded and as fp32: what the norms and
// the operators next to a mixer share.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace gdn {

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
struct Vec<__nv_bfloat16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(uint2 p, float (&x)[4]) {
        x[0] = __uint_as_float(p.x << 16), x[1] = __uint_as_float(p.x & 0xffff0000u);
        x[2] = __uint_as_float(p.y << 16), x[3] = __uint_as_float(p.y & 0xffff0000u);
    }
    static __device__ __forceinline__ uint2 pack(const float (&x)[4]) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
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
struct Vec<float, 2> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(uint2 p, float (&x)[2]) {
        x[0] = __uint_as_float(p.x), x[1] = __uint_as_float(p.y);
    }
    static __device__ __forceinline__ uint2 pack(const float (&x)[2]) {
        return make_uint2(__float_as_uint(x[0]), __float_as_uint(x[1]));
    }
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

}  // namespace gdn
