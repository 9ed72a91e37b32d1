// kv_quant.cuh -- rows of 16- or 32-bit numbers as e4m3 with a scale, and as
// e2m1 with a scale of their own for every 16 elements.
#pragma once

#include "kv.cuh"

namespace ss {

__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

template <typename T> __device__ __forceinline__ float2 open_pair(uint32_t u);
template <> __device__ __forceinline__ float2 open_pair<__nv_bfloat16>(uint32_t u) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
template <> __device__ __forceinline__ float2 open_pair<__half>(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// 16 elements over the scale, as e4m3, by a reciprocal and one correction: q =
// x r, then q - (q s - x) r, with r = 1 / s rounded.  That is the rounded
// quotient unless x / s lies within 2^-22 of a unit in the last place of the
// middle of two floats, which could matter only next to a tie of two e4m3
// values.  There, with X (11 bits), S (24) and T (5, of the tie) the integer
// significands, it takes |X 2^k - S (T 2^20 + 1)| < 8 with k >= 37, hence S =
// S1 2^20 + e with |e| < 8, 8 <= S1 <= 16 and T e + S1 = 0: only S = 2^24 - 1
// with T = 16, whose corrected quotient is (1 + 2^-24 + 2^-70) times the tie,
// on the same side of the middle as x / s.  (On the lower side, T e = S1 has no
// solution.)  So the e4m3 result is that of the division, and a zero keeps its
// sign: q s - x is then +0, and the correction -0, which changes no q, where
// r > 0.  Other scales, those for which a step could leave fp32's normal range,
// and non-finite elements are divided.
template <typename T> __device__ __forceinline__ uint4 quant16(const uint4 (&x)[2], float scale, float inverse) {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    float y[16], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 a = open_pair<T>(w[i]);
        const float q0 = a.x * inverse, q1 = a.y * inverse;
        y[2 * i] = fmaf(-fmaf(q0, scale, -a.x), inverse, q0);
        y[2 * i + 1] = fmaf(-fmaf(q1, scale, -a.y), inverse, q1);
        sum += fabsf(y[2 * i]) + fabsf(y[2 * i + 1]);
    }
    if (!(sum < INFINITY)) {  // an infinity or NaN among them, or no inverse
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 a = open_pair<T>(w[i]);
            y[2 * i] = __fdiv_rn(a.x, scale);
            y[2 * i + 1] = __fdiv_rn(a.y, scale);
        }
    }
    return make_uint4(quant4(y[0], y[1], y[2], y[3]), quant4(y[4], y[5], y[6], y[7]), quant4(y[8], y[9], y[10], y[11]),
                      quant4(y[12], y[13], y[14], y[15]));
}

// The reciprocal of a scale, NaN for those outside [2^-60, 2^60] and negative ones.
__device__ __forceinline__ float inverse_of(float s) {
    return s >= 0x1p-60f && s <= 0x1p60f ? __frcp_rn(s) : NAN;
}

// Eight fp32 numbers over the scale, in the same way: within 2^-23 of the quotient,
// and the same e4m3 value as quant16's where they have 11 bits.
__device__ __forceinline__ void quotients(const float (&x)[8], float scale, float inverse, float (&y)[8]) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = x[i] * inverse;
        y[i] = fmaf(-fmaf(q, scale, -x[i]), inverse, q);
        sum += fabsf(y[i]);
    }
    if (!(sum < INFINITY)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], scale);
    }
}

// Eight numbers as e2m1 codes, the first one lowest; ties to even, beyond 6 to 6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&z)[8]) {
    uint32_t w;
    asm("{.reg .b8 a, b, c, d; cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3; "
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7; mov.b32 %0, {a, b, c, d};}"
        : "=r"(w) : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
    return w;
}

// The larger of |x| and most; NaN stays.
__device__ __forceinline__ float abs_max(float most, float x) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(most), "f"(fabsf(x)));
    return y;
}

// The scale of a block of 16 elements whose largest is `most`: most / 6 as
// e4m3, at most 448; NaN where an element is.
struct BlockScale {
    uint32_t code;
    float value, inverse;  // 0 where the scale is 0 or NaN: elements become zeros
    __device__ __forceinline__ explicit BlockScale(float most) {
        code = (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(most, 6.0f), __NV_SATFINITE, __NV_E4M3);
        const bool some = code != 0 && code != 0x7f;
        value = some ? __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3))) : 0.0f;
        inverse = some ? __frcp_rn(value) : 0.0f;
    }
    // y over the scale, by the reciprocal and one correction.  The code of the
    // result is that of the rounded quotient: a tie t of two codes times the
    // scale is an fp32 number (3 and 4 bits), so that y is either that product,
    // where the correction gives t itself, or at least 2^-24 of it away, where
    // both stay on its side of t.  A zero keeps its sign.
    __device__ __forceinline__ float over(float y) const {
        y = fminf(fmaxf(y, -2688.0f), 2688.0f);  // 448 times 6: more gives the same code
        const float q = y * inverse;
        return fmaf(-fmaf(q, value, -y), inverse, q);
    }
};

}  // namespace ss
