// product_int8_rows.cu -- the dense product of int8 operands for up to 16 rows
// (moe_expert_product_int8 without a plan; product_int8.cu has the others): the same
// sums as there, in whole numbers.
//
// Bound by the weights' bytes, and by how long the first of them take. A unit is 16
// weight rows, so that 4096 of them are 256 blocks and every SM loads (pairs of CTAs
// over 256 weight rows are 16 of 76 pairs: 27 us, 7168 -> 4096 gated, against 9 for up
// to 8 rows and 13 for 16). mma.sync m16n8k32 on 8-bit integers costs the same for one
// row as for eight, and its rate, low as it is on sm_103a, is several times what the
// bytes need. (Four products an instruction on the CUDA cores: 7.6 us for one row, 14
// for eight.)
//
// The order of K means nothing to a sum: a lane's 16 codes of a row, as they lie, are
// its elements of two instructions, for weights and rows alike. A warp takes 16 weight
// rows over a part of K, 512 codes of each at a time: 24 loads of 16 bytes in flight per
// lane; 1, 2, 4 or all 8 of a block's warps share the K of the same rows, and their
// sums are added.
#include <cuda_bf16.h>

#include "tensor.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kSteps = 8;            // of 64 codes of K at a time
constexpr int kChunk = 64 * kSteps;

// 16 bytes at p + k, or zeros past K.
__device__ __forceinline__ uint4 weights16(const int8_t* p, int32_t k, int32_t K) {
    return k < K ? ld_stream_u4(p + k) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ uint4 codes16(const int8_t* p, int32_t k, int32_t K) {
    return k < K ? __ldg(reinterpret_cast<const uint4*>(p + k)) : make_uint4(0, 0, 0, 0);
}

// 16 weight rows x 8 rows, 32 codes of each.
__device__ __forceinline__ void mma32(int32_t (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A block: 8 / parts times 16 weight rows (gated: 8 gate rows and their up rows).
// GROUPS: of 8 rows.
template <bool GATED, int GROUPS>
__global__ void __launch_bounds__(32 * kWarps, 2) product_int8_rows_kernel(const ProductInt8Args a, const int parts) {
    pdl_wait_then_release();
    __shared__ int32_t sums[kWarps][8 * GROUPS][16];  // [place * parts + part][row][weight row]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % parts, place = warp / parts, places = kWarps / parts;
    const int g = lane >> 2, q = lane & 3;  // of an operand: which row; which 16 of 64 codes
    const int n = static_cast<int>(a.rows);
    const uint32_t sixteens = static_cast<uint32_t>(a.N / 16), mine = blockIdx.x * places + place;
    // The 16 weight rows of a place start here; gated, 8 gate rows, then (16 behind them) their up rows.
    const auto first_of = [](uint32_t s) { return static_cast<int32_t>(GATED ? s / 2 * 32 + s % 2 * 8 : s * 16); };
    if (mine < sixteens) {  // the whole warp
        const int8_t* w = a.wq + static_cast<int64_t>(first_of(mine) + g) * a.K;
        const int8_t* w2 = w + static_cast<int64_t>(GATED ? 16 : 8) * a.K;
        int32_t c[GROUPS][4] = {};
        for (int32_t chunk = part * kChunk; chunk < a.K; chunk += parts * kChunk) {  // the whole warp alike
            const int32_t k0 = chunk + 16 * q;
            uint4 wv[kSteps], wv2[kSteps];
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                wv[j] = weights16(w, k0 + 64 * j, a.K);
                wv2[j] = weights16(w2, k0 + 64 * j, a.K);
            }
#pragma unroll
            for (int h = 0; h < GROUPS; ++h) {
                const int8_t* x = a.xq + min(8 * h + g, n - 1) * a.x_stride;  // the last row stands for those that are not there
                uint4 xv[kSteps];
#pragma unroll
                for (int j = 0; j < kSteps; ++j) xv[j] = codes16(x, k0 + 64 * j, a.K);
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
                    mma32(c[h], wv[j].x, wv2[j].x, wv[j].y, wv2[j].y, xv[j].x, xv[j].y);
                    mma32(c[h], wv[j].z, wv2[j].z, wv[j].w, wv2[j].w, xv[j].z, xv[j].w);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < GROUPS; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[warp][8 * h + 2 * q + (i & 1)][g + 8 * (i >> 1)] = c[h][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < places * GROUPS * 128; i += blockDim.x) {
        const int at = i / (GROUPS * 128), r = i / 16 % (8 * GROUPS), v0 = i & 15;
        const uint32_t m = blockIdx.x * places + at;
        if (r >= n || m >= sixteens || (GATED && v0 >= 8)) continue;
        const int32_t channel = first_of(m) + v0;
        const float xs = __ldg(reinterpret_cast<const float*>(a.xs + r * a.xs_stride));
        int32_t sum = 0, sum2 = 0;
        for (int p = 0; p < parts; ++p) {
            sum += sums[at * parts + p][r][v0];
            if (GATED) sum2 += sums[at * parts + p][r][v0 + 8];
        }
        float v = static_cast<float>(sum) * __ldg(a.ws + channel) * xs;
        if (GATED) v = gate_times_up(v, static_cast<float>(sum2) * __ldg(a.ws + channel + 16) * xs);
        uint16_t* y = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(a.y) + r * a.y_stride);
        y[GATED ? static_cast<int32_t>(m) * 8 + v0 : channel] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
}

}  // namespace

cudaError_t launch_product_int8_rows(const ProductInt8Args& a, cudaStream_t stream) {
    // As many warps to the same K as have a chunk of it each.
    const int64_t chunks = ceil_div(a.K, kChunk);
    const int parts = chunks >= 8 ? 8 : chunks >= 4 ? 4 : chunks >= 2 ? 2 : 1;
    const bool one = a.rows <= 8;
    const auto kernel = a.gated ? (one ? product_int8_rows_kernel<true, 1> : product_int8_rows_kernel<true, 2>)
                                : (one ? product_int8_rows_kernel<false, 1> : product_int8_rows_kernel<false, 2>);
    return launch_pdl(kernel, static_cast<unsigned>(ceil_div(a.N / 16, kWarps / parts)), 32u * kWarps, 0, stream, a, parts);
}

}  // namespace moe
