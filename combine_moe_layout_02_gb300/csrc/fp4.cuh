// fp4.cuh -- MXFP4 rows (OCP Microscaling Formats v1.0): the operand layout the
// packing, dispatch and product kernels share, and the rounding itself.
//
// A block of 32 consecutive elements of a row shares the power of two
// 2^(s - 127); an element is an e2m1 code (sign, 2 exponent bits, 1 fraction
// bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times it. For a block whose largest
// magnitude is m, s = max(0, floor(log2 m) + 127 - 2), so m lands in [4, 8)
// and magnitudes above 6 saturate to 6; codes are rounded to nearest, ties to
// the even code. A block holding an infinity or a NaN gets s = 255, which
// stands for NaN, and codes 0.
//
// Layout of an operand of `rows` x `width`: codes two to a byte (the even
// element in the low nibble), rows width / 2 bytes apart; scales in 512-byte
// chunks of 128 rows x 4 blocks, chunk (row / 128, block / 4), in which row
// m's 4 scales are the 32-bit word at byte (m % 32) * 16 + (m % 128) / 32 * 4.
// That is the order in which the tensor core takes scales from shared memory
// (32 lanes of 16 bytes), so the product copies chunks as they are.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "experts.cuh"

namespace moe {

constexpr int kFp4Tile = MOE_FP4_ROW_TILE;  // rows per scale chunk; experts' rows start at multiples
constexpr int kFp4Chunk = 128;              // elements per scale chunk
constexpr int kFp4ChunkBytes = 512;
constexpr int kPlanTileRows = MOE_PLAN_TILE_ROWS;

// A plan (include/moe.h): 4 header words, first rows, counts, row tiles.
__host__ __device__ __forceinline__ int64_t plan_tiles_at(int32_t E) { return 4 + 2 * round_up(E, 4); }

// Row tiles a plan of `ints` words can hold.
__host__ __device__ __forceinline__ int32_t plan_capacity(int32_t E, int64_t ints) {
    const int64_t n = (ints - plan_tiles_at(E)) / 4;
    return n < 0 ? 0 : (n > INT32_MAX ? INT32_MAX : static_cast<int32_t>(n));
}

// Row tiles that a plan of `ints` words can give of `rows` rows: experts' rows start at
// multiples of kFp4Tile, so no more tiles than that have any.
__host__ __forceinline__ int32_t plan_tiles_cap(int32_t E, int64_t ints, int64_t rows) {
    const int64_t n = plan_capacity(E, ints), most = rows / kFp4Tile + 1;
    return static_cast<int32_t>(n < most ? n : most);
}

// Byte of row m's scale word inside its chunk.
__host__ __device__ __forceinline__ int fp4_word_at(int m) { return (m & 31) * 16 + ((m >> 5) & 3) * 4; }

// Largest magnitude of the bf16 pairs in `w` and of both halves of `m`, as bit
// patterns: unsigned order is magnitude order, infinities and NaN above all.
__device__ __forceinline__ uint32_t fp4_absmax(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }

// Scale code of a block from the bit pattern of its largest magnitude.
__device__ __forceinline__ uint32_t fp4_scale_code(uint32_t bits) {
    const uint32_t e = bits >> 7;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 2^(127 - s): the factor that brings a block into e2m1's range (0 for s =
// 255). Exact: a power of two times a bf16 value, and what it underflows
// rounds to code 0 either way.
__device__ __forceinline__ float fp4_inverse(uint32_t s) { return s == 255u ? 0.f : __uint_as_float((254u - s) << 23); }

// 8 bf16 (four words) times `inv` to 8 codes. A NaN or an infinity (inv = 0)
// becomes code 0.
__device__ __forceinline__ uint32_t fp4_codes8(uint4 v, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __fmul_rn(__uint_as_float(w[i] << 16), inv);
        f[2 * i + 1] = __fmul_rn(__uint_as_float(w[i] & 0xffff0000u), inv);
    }
    uint32_t out;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(out)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return inv == 0.f ? 0u : out;
}

// 2^(s - 127) as a bf16 pair; NaN for 255.
__device__ __forceinline__ __nv_bfloat162 fp4_scale_pair(uint32_t s) {
    const uint32_t b = s == 0u ? 0x0040u : s == 255u ? 0x7fc0u : s << 7;
    const uint32_t w = b * 0x10001u;
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
}

// 8 codes to 8 bf16 e2m1 values times a power of two, exactly. The high and
// low bytes of a magnitude's bf16 pattern are looked up by byte permutation,
// four codes at once (0, 0x3f00, 0x3f80, 0x3fc0, 0x4000, 0x4040, 0x4080, 0x40c0).
__device__ __forceinline__ uint4 fp4_values8(uint32_t codes, __nv_bfloat162 scale) {
    uint32_t o[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t c = codes >> (16 * h);
        const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, c & 0x7777u);
        const uint32_t lo = __byte_perm(0xc0800000u, 0xc0804000u, c & 0x7777u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // the two codes' sign bits 3 and 7 go to bits 15 and 31
            const uint32_t sign = (((c >> (8 * i)) & 0x88u) * 0x01001000u) & 0x80008000u;
            const uint32_t w = __byte_perm(lo, hi, i ? 0x7362 : 0x5140) | sign;
            const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), scale);
            o[2 * h + i] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Source row of packed row m of a gated operand of `rows` rows: rows come in
// groups of 32, 16 gate rows and the 16 up rows that belong to them.
__host__ __device__ __forceinline__ int64_t fp4_gated_row(int64_t m, int64_t rows) {
    const int64_t b = m >> 5, i = m & 31;
    return b * 16 + (i & 15) + (i >= 16 ? rows / 2 : 0);
}

}  // namespace moe
