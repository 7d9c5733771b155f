// int8.cuh -- rows in int8 with one binary32 scale each, as dispatch's int8
// payload has them: scale = max|v| / 127, q = rint(v / scale) (ties to even),
// 0 for a row of zeros. A row that holds an infinity or a NaN gets the scale NaN
// and codes 0, so that what is computed from it is NaN.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "experts.cuh"

namespace moe {

// The larger, or NaN if either is.
__device__ __forceinline__ float nan_max(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Int8Scale {
    float scale;
    float inv;  // rounded 1 / scale; 0 where every code is 0
    bool fast;  // inv is a normal number and so good to 2^-24, and scale is not near the smallest
};

__device__ __forceinline__ Int8Scale int8_scale(float most) {
    Int8Scale s;
    const bool fine = most <= 3.402823466e38f;  // not for NaN and infinity
    s.scale = fine ? __fdiv_rn(most, 127.f) : __uint_as_float(0x7fc00000u);
    const bool zero = !(s.scale > 0.f);
    s.inv = zero ? 0.f : __frcp_rn(s.scale);
    s.fast = s.inv >= 1.17549435e-38f && s.scale >= 0x1p-90f;
    return s;
}

// The low bytes of 8 numbers 1.5 * 2^23 + code.
__device__ __forceinline__ uint2 int8_bytes8(const float (&m)[8]) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(m[i]);
    return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}
constexpr float kWholeBits = 12582912.f;  // 1.5 * 2^23: added to a number below 2^22, it leaves the whole number in the low bits

// 8 values times inv to the nearest codes (|product| < 127.5).
__device__ __forceinline__ uint2 int8_near8(const float (&v)[8], float inv) {
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmaf(v[i], inv, kWholeBits);
    return int8_bytes8(m);
}

// rint(v / scale), divided.
static __device__ __noinline__ uint2 int8_divided8(float v0, float v1, float v2, float v3, float v4, float v5, float v6, float v7, float scale) {
    const float v[8] = {v0, v1, v2, v3, v4, v5, v6, v7};
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = fminf(fmaxf(rintf(__fdiv_rn(v[i], scale)), -127.f), 127.f);
        w[i >> 2] |= (static_cast<uint32_t>(static_cast<int32_t>(q)) & 0xffu) << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
}

// rint(v / scale) of 8 values, the quotient rounded as a division rounds it: v * inv is within two ulps
// of it, and adding what that leaves of v times inv rounds right where inv is the rounded reciprocal
// (P. Markstein, IBM Journal of Research and Development 34, 1990; every quotient of bf16 values is tested). What is left of v that matters, near a tie
// and so |v| >= scale / 4, is above 2^-26 scale: a scale from 2^-90 on keeps it a normal number. bf16 rows
// reach a tie often (127 v / max is a quotient of small whole numbers): 32768 x 7168 packed in 170 us when
// only products near one were divided, in 123 so. Codes are 0 under a scale of 0 or NaN.
__device__ __forceinline__ uint2 int8_codes8(const float (&v)[8], const Int8Scale& s) {
    if (s.inv == 0.f) return make_uint2(0u, 0u);
    if (!s.fast) return int8_divided8(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], s.scale);
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = v[i] * s.inv;
        m[i] = fmaf(fmaf(-q, s.scale, v[i]), s.inv, q) + kWholeBits;
    }
    return int8_bytes8(m);
}

// Four codes to four f16: code + 128 is the low byte of the f16 1024 + (code + 128).
__device__ __forceinline__ void halves4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    const uint32_t b = codes ^ 0x80808080u;
    const uint32_t u = __byte_perm(b, 0x64646464u, 0x4140), v = __byte_perm(b, 0x64646464u, 0x4342);
    const uint32_t off = 0x64806480u;  // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&off));
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&off));
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

}  // namespace moe
