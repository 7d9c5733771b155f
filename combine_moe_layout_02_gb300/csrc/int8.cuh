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
    bool fast;  // inv is a normal number and so good to 2^-24
};

__device__ __forceinline__ Int8Scale int8_scale(float most) {
    Int8Scale s;
    const bool fine = most <= 3.402823466e38f;  // not for NaN and infinity
    s.scale = fine ? __fdiv_rn(most, 127.f) : __uint_as_float(0x7fc00000u);
    const bool zero = !(s.scale > 0.f);
    s.inv = zero ? 0.f : __frcp_rn(s.scale);
    s.fast = s.inv <= 3.402823466e38f && s.inv >= 1.17549435e-38f && s.scale >= 1.17549435e-38f;
    return s;
}

// rint(v / scale) with the division's own rounding decided exactly: |v / scale| <=
// 127.13 (for scales down to the smallest denormal the rounding of most / 127 is
// within half a unit, and then the quotient is at most 127 * 1.5), v * inv is within 2^-15 of it,
// so only a product that near to a tie is divided.
__device__ __forceinline__ int32_t int8_code(float v, const Int8Scale& s) {
    const float t = v * s.inv;
    float q = rintf(t);
    if (!s.fast || fabsf(t - q) >= 0.5f - 0x1p-15f) q = s.inv == 0.f ? 0.f : rintf(__fdiv_rn(v, s.scale));
    return static_cast<int32_t>(fminf(fmaxf(q, -127.f), 127.f));
}

__device__ __forceinline__ uint2 int8_codes8(const float (&v)[8], const Int8Scale& s) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        w[h] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[h] |= (static_cast<uint32_t>(int8_code(v[4 * h + i], s)) & 0xffu) << (8 * i);
    }
    return make_uint2(w[0], w[1]);
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
