// Numbers of 8 bits: a row's scale from its largest magnitude, codes from values,
// and values from codes.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace csa_dev {

// Scale of a row whose largest magnitude has these bits, and the factor that its values
// are multiplied by to give codes.  True: the codes are 0 (an empty row, scale 0, or one
// with an infinity or NaN, scale NaN).
template <bool E4M3>
__device__ __forceinline__ bool row_scale(unsigned most, float &s, float &factor) {
    factor = 0.0f;
    if (most < (27u << 23)) {  // 2^-100
        s = 0.0f;
        return true;
    }
    if (most >= 0x7f800000u) {
        s = __uint_as_float(0x7fffffffu);
        return true;
    }
    if (E4M3) {
        // 448 = 1.75 * 2^8: the exponent of max, one more where its fraction is above 1.75, less 8
        const unsigned e = ((most + 0x1fffffu) >> 23) - 8;
        s = __uint_as_float(e << 23);
        factor = __uint_as_float((254u - e) << 23);  // 1 / s; e is 19 at least and 247 at most
    } else {
        s = __fdiv_rn(__uint_as_float(most), 127.0f);
        factor = __fdiv_rn(127.0f, __uint_as_float(most));
    }
    return false;
}

__device__ __forceinline__ uint32_t to_e4m3x4(const float (&x)[4], float factor) {
    uint16_t lo, hi;  // the second operand is the lower byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] * factor), "f"(x[0] * factor));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] * factor), "f"(x[2] * factor));
    return (uint32_t)hi << 16 | lo;
}

// x * factor is at most 127 (1 + 2^-23); the sum's last bits are the nearest integer's
__device__ __forceinline__ uint32_t to_int8x4(const float (&x)[4], float factor) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(fmaf(x[i], factor, 12582912.0f));
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// Two fp16 numbers from the codes in the low two bytes of `pair`, exactly.
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t pair) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)pair));
    return r;
}

// Four fp16 numbers from four codes, exactly: of int8 by the number 1024 + (code + 128),
// whose low byte is the code's with its sign bit flipped.
template <bool E4M3>
__device__ __forceinline__ void halves_of(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    if (E4M3) {
        lo = half2_of_e4m3(codes);
        hi = half2_of_e4m3(codes >> 16);
    } else {
        const uint32_t u = codes ^ 0x80808080u, magic = 0x64646464u;
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
        const uint32_t a = __byte_perm(u, magic, 0x4140), b = __byte_perm(u, magic, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off),
                      y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    }
}

// N values of a row of scale s from N codes.  AGAIN: they are rounded once more, to 16 bits, and the two roundings shall be as
// one.  Then a product is cut off, and its last bit set where the scale's fraction has one of its last eight: such a scale
// times a code's 8 bits is nowhere in the middle between two bf16 numbers (it would be a multiple of 2^15 units of the
// scale, a code of 2^7 at most), so that the bit stands for what was cut off or changes nothing; other products fit 24
// bits.  754 MB of int8 rows as bf16 in 117 us, 114 with the second rounding as it falls; a look at each product for the
// middle, and those put right that were moved: 139 us; the products two by two, in 50 registers: 121 us.
template <bool E4M3, bool AGAIN, int N, typename C>
__device__ __forceinline__ void values_of(const C &raw, float s, float (&x)[N]) {
    const unsigned rest = AGAIN && (__float_as_uint(s) & 0xffu) ? 1u : 0u;
    uint32_t words[(N + 3) / 4] = {};
    static_assert(sizeof(C) == N, "one byte each");
    memcpy(words, &raw, N);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        uint32_t h[2];
        halves_of<E4M3>(words[i / 4], h[0], h[1]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < N) {
                const __half2 p = *reinterpret_cast<const __half2 *>(&h[j / 2]);
                const float code = j & 1 ? __high2float(p) : __low2float(p);
                x[i + j] = AGAIN ? __uint_as_float(__float_as_uint(__fmul_rz(code, s)) | rest) : code * s;
            }
    }
}

}  // namespace csa_dev
