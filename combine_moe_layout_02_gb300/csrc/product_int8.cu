// product_int8.cu -- the experts' grouped product of int8 operands
// (moe_expert_product_int8): for every row r of expert e,
//   v[r][n] = ws_e[n] * xs[r] * sum over k of w_e[n][k] * x[r][k]
//   y[r] = bf16_rne(v[r]), or, gated, bf16_rne(silu(gate) * up) of the pairs.
//
// 64 weight rows x 64 rows per block, four products an instruction.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "int8.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 64, kPad = kStep + 4;

__device__ __forceinline__ float gate_times_up(float g, float u) {
    const float e = __expf(-fabsf(g));
    return __fdividef(g < 0.f ? g * e : g, 1.f + e) * u;
}

__global__ void __launch_bounds__(256) product_int8_kernel(const ProductInt8Args a) {
    pdl_wait_then_release();
    __shared__ __align__(16) int8_t ws[kTile][kPad], xs[kTile][kPad];
    __shared__ float v[kTile][kTile + 1];
    const int ntiles = static_cast<int>(ceil_div(a.N, kTile));
    const int64_t unit = blockIdx.x;
    const int n0 = static_cast<int>(unit % ntiles) * kTile;
    const int64_t part = unit / ntiles;  // a quarter of a row tile
    int4 t;
    if (a.plan) {
        if (part / 4 >= __ldg(a.plan)) return;
        t = __ldg(reinterpret_cast<const int4*>(a.plan + plan_tiles_at(a.E)) + part / 4);
    } else {
        const int64_t left = a.rows - part / 4 * kPlanTileRows;
        t = make_int4(0, static_cast<int32_t>(part / 4 * kPlanTileRows), static_cast<int32_t>(left < kPlanTileRows ? left : kPlanTileRows), 0);
    }
    if (t.x < 0 || t.x >= a.E || t.y < 0 || t.z < 0 || t.z > kPlanTileRows || t.y + static_cast<int64_t>(t.z) > a.rows) {
        raise_error(a.err, MOE_ERR_CAPACITY);
        return;
    }
    const int r0 = static_cast<int>(part % 4) * kTile, rows = min(kTile, t.z - r0);
    if (rows <= 0) return;
    const int8_t* w = a.wq + (static_cast<int64_t>(t.x) * a.N) * a.K;
    const int64_t row0 = t.y + r0;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int32_t acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kStep) {
        const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 16;
        uint4 wv = make_uint4(0, 0, 0, 0), xv = wv;
        if (n0 + r < a.N && k0 + c < a.K) wv = *reinterpret_cast<const uint4*>(w + static_cast<int64_t>(n0 + r) * a.K + k0 + c);
        if (r < rows && k0 + c < a.K) xv = *reinterpret_cast<const uint4*>(a.xq + (row0 + r) * a.x_stride + k0 + c);
        const uint32_t wa[4] = {wv.x, wv.y, wv.z, wv.w}, xa[4] = {xv.x, xv.y, xv.z, xv.w};
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<uint32_t*>(&ws[r][c + 4 * i]) = wa[i];
            *reinterpret_cast<uint32_t*>(&xs[r][c + 4 * i]) = xa[i];
        }
        __syncthreads();
        for (int k = 0; k < kStep; k += 4) {
            int32_t p[4], q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = *reinterpret_cast<const int32_t*>(&ws[tx + 16 * i][k]);
                q[i] = *reinterpret_cast<const int32_t*>(&xs[ty + 16 * i][k]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(p[i], q[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx + 16 * i, r = ty + 16 * j;
            if (n < a.N && r < rows)
                v[r][tx + 16 * i] = static_cast<float>(acc[i][j]) * __ldg(a.ws + static_cast<int64_t>(t.x) * a.N + n) *
                                    *reinterpret_cast<const float*>(a.xs + (row0 + r) * a.xs_stride);
        }
    __syncthreads();
    const int width = a.gated ? kTile / 2 : kTile;
    for (int i = threadIdx.x; i < rows * width; i += blockDim.x) {
        const int r = i / width, c = i % width;
        const int at = a.gated ? c / 16 * 32 + c % 16 : c;
        if (n0 + at >= a.N) continue;
        const float o = a.gated ? gate_times_up(v[r][at], v[r][at + 16]) : v[r][at];
        uint16_t* y = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(a.y) + (row0 + r) * a.y_stride);
        y[(a.gated ? n0 / 2 : n0) + c] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
    }
}

}  // namespace

cudaError_t launch_product_int8(const ProductInt8Args& a, cudaStream_t stream) {
    if (a.tile_cap == 0) return cudaSuccess;
    const int64_t blocks = static_cast<int64_t>(a.tile_cap) * 4 * ceil_div(a.N, kTile);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl(product_int8_kernel, static_cast<unsigned>(blocks), 256u, 0, stream, a);
}

}  // namespace moe
