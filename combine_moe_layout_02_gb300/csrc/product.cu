// product.cu -- the experts' grouped product of MXFP4 operands
// (moe_expert_product_fp4): for every row r of expert e,
//   v[r][n] = sum over k of w_e[n][k] * x[r][k]
//   y[r] = bf16_rne(v[r]), or, gated, bf16_rne(silu(gate) * up) of the pairs.
#include <cuda_bf16.h>

#include "fp4.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 32, kThreads = 256;

struct ProductArgs {
    int32_t E, N, K, gated, tile_cap;
    const uint8_t* wq;
    const uint8_t* wsf;
    const uint8_t* xq;
    const uint8_t* xsf;
    int64_t rows;
    const int32_t* plan;
    uint16_t* y;
    int64_t y_stride;
    int32_t* err;
};

// 64 rows x 64 weight rows per CTA, 4 x 4 values per thread, both operands
// decoded to binary32 in shared memory 32 elements (one block) at a time.
__global__ void __launch_bounds__(kThreads) product_kernel(const ProductArgs a) {
    pdl_wait_then_release();
    __shared__ float xs[kTile][kStep + 1], ws[kTile][kStep + 1];
    const int tid = threadIdx.x, tn = tid & 15, tm = tid >> 4;
    int32_t tiles = __ldg(a.plan);
    tiles = tiles < 0 ? 0 : (tiles > a.tile_cap ? a.tile_cap : tiles);
    const int64_t nt = ceil_div(a.N, kTile), chunks = ceil_div(a.K, kFp4Chunk), wtiles = ceil_div(a.N, kFp4Tile);
    const int4* list = reinterpret_cast<const int4*>(a.plan + plan_tiles_at(a.E));
    const int64_t units = static_cast<int64_t>(tiles) * 4 * nt;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int4 t = __ldg(list + u / (4 * nt));
        const int sub = static_cast<int>(u / nt % 4) * kTile;
        const int n0 = static_cast<int>(u % nt) * kTile;
        if (sub >= t.z) continue;
        if (t.x < 0 || t.x >= a.E || t.y < 0 || t.y % kFp4Tile != 0 || t.y + static_cast<int64_t>(t.z) > a.rows) {
            raise_error(a.err, MOE_ERR_CAPACITY);
            continue;
        }
        float acc[4][4] = {};
        for (int k0 = 0; k0 < a.K; k0 += kStep) {
            // 64 rows x 4 words of 8 codes of each operand
            const int m = tid >> 2, j = tid & 3;
            float f[8];
            {
                const int64_t row = t.y + sub + m;
                uint32_t c = 0, s = 0;
                if (sub + m < t.z) {
                    c = __ldg(reinterpret_cast<const uint32_t*>(a.xq + row * (a.K / 2) + k0 / 2) + j);
                    s = a.xsf[((row / kFp4Tile) * chunks + k0 / kFp4Chunk) * kFp4ChunkBytes +
                              fp4_word_at(static_cast<int>(row % kFp4Tile)) + (k0 >> 5 & 3)];
                }
                fp4_values8(c, f);
                for (int i = 0; i < 8; ++i) xs[m][j * 8 + i] = f[i] * fp4_scale(s);
            }
            {
                const int n = n0 + m;
                uint32_t c = 0, s = 0;
                if (n < a.N) {
                    c = __ldg(reinterpret_cast<const uint32_t*>(
                                  a.wq + (static_cast<int64_t>(t.x) * a.N + n) * (a.K / 2) + k0 / 2) + j);
                    s = a.wsf[((t.x * wtiles + n / kFp4Tile) * chunks + k0 / kFp4Chunk) * kFp4ChunkBytes +
                              fp4_word_at(n % kFp4Tile) + (k0 >> 5 & 3)];
                }
                fp4_values8(c, f);
                for (int i = 0; i < 8; ++i) ws[m][j * 8 + i] = f[i] * fp4_scale(s);
            }
            __syncthreads();
#pragma unroll 8
            for (int k = 0; k < kStep; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int h = 0; h < 4; ++h) acc[i][h] = fmaf(xs[tm + 16 * i][k], ws[tn + 16 * h][k], acc[i][h]);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = sub + tm + 16 * i;
            if (m >= t.z) continue;
            uint16_t* y = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(a.y) + (t.y + m) * a.y_stride);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int n = n0 + tn + 16 * h;
                if (n >= a.N) continue;
                if (!a.gated) {
                    y[n] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i][h]));
                } else if ((h & 1) == 0) {
                    const float g = acc[i][h], s = g / (1.f + __expf(-g));
                    y[n0 / 2 + 8 * h + tn] = __bfloat16_as_ushort(__float2bfloat16_rn(s * acc[i][h + 1]));
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_product(int32_t E, int32_t N, int32_t K, int32_t gated, const uint8_t* wq, const uint8_t* wsf,
                           const uint8_t* xq, const uint8_t* xsf, int64_t rows, const int32_t* plan, int64_t plan_ints,
                           uint16_t* y, int64_t y_stride, int32_t* err, cudaStream_t stream) {
    ProductArgs a{E, N, K, gated, plan_capacity(E, plan_ints), wq, wsf, xq, xsf, rows, plan, y, y_stride, err};
    if (a.tile_cap == 0) return cudaSuccess;
    int per_sm = 0;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(product_kernel), 0, kThreads, &per_sm);
    if (e != cudaSuccess) return e;
    return launch_pdl(product_kernel, static_cast<unsigned>(device_sm_count() * (per_sm < 1 ? 1 : per_sm)), kThreads, 0,
                      stream, a);
}

}  // namespace moe
