// Elements and rotations of rows of bf16 or fp32, shared by the kernels that turn
// rows (csa_rope.cu) and those that turn and quantise them (csa_quant.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace csa_dev {

template <int BYTES>
struct Chunk;
template <>
struct Chunk<16> {
    using type = uint4;
};
template <>
struct Chunk<8> {
    using type = uint2;
};
template <>
struct Chunk<4> {
    using type = uint32_t;
};
template <>
struct Chunk<2> {
    using type = uint16_t;
};
template <>
struct Chunk<1> {
    using type = uint8_t;
};

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) {
    return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// Sine and cosine of f 2^-64 turns.  The distance to the nearest quarter of a
// turn, an eighth at most, is exact in integers; it becomes a fp32 number x of
// half turns within 2^-23 relative, so that small angles keep their accuracy, and
// -f gives exactly the opposite angle.  The rest are the power series of sin(pi x)
// and cos(pi x) up to x^9 and x^10, the next terms below 3e-9 at |x| = 1/4, pi in
// two parts: each result within 2^-22 relative.  sincospif in their place, which
// reduces its argument once more: 30.6 us for 8192 tokens of 32 + 8 heads in bf16 and 2.9 us for
// one token each of 64 sequences, in a graph; with the series 29.5 and 2.4 us.
__device__ __forceinline__ void turn_by(unsigned long long f, float &sn, float &cs) {
    const unsigned lo = (unsigned)f, hi = (unsigned)(f >> 32) + 0x20000000u;
    const unsigned quarter = hi >> 30;
    // x = (h + l 2^-32) 2^-31, l being the signed low word
    const int h = (int)((hi & 0x3fffffffu) + (lo >> 31)) - 0x20000000, l = (int)lo;
    const float x = fmaf((float)h, 4.656612873077393e-10f, (float)l * 1.0842021724855044e-19f), y = x * x;
    float s = fmaf(y, 8.2145886e-02f, -5.9926453e-01f);  // pi^9/9!, -pi^7/7!
    s = fmaf(s, y, 2.5501640f);                          // pi^5/5!
    s = fmaf(s, y, -5.1677128f);                         // -pi^3/3!
    s = fmaf(s, y, -8.7422777e-08f);                     // pi less the next line's
    s = fmaf(x, 3.14159274f, x * s);
    float c = fmaf(y, -2.5806891e-02f, 2.3533063e-01f);  // -pi^10/10!, pi^8/8!
    c = fmaf(c, y, -1.3352628f);                         // -pi^6/6!
    c = fmaf(c, y, 4.0587121f);                          // pi^4/4!
    c = fmaf(c, y, -4.9348022f);                         // -pi^2/2!
    c = fmaf(c, y, 1.0f);
    const float a = quarter & 1 ? c : s, b = quarter & 1 ? s : c;
    sn = __uint_as_float(__float_as_uint(a) ^ (quarter & 2) << 30);
    cs = __uint_as_float(__float_as_uint(b) ^ ((quarter + 1) & 2) << 30);
}

}  // namespace csa_dev
