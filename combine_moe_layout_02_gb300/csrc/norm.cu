// norm.cu -- root-mean-square norm with the residual's addition (moe_rms_norm),
// its gradient (moe_rms_norm_grad), and int8 rows (moe_int8_pack, moe_int8_unpack).
// With h = x + residual of a row of H values:
//   rstd = 1 / sqrt(mean h^2 + eps),  y = h * rstd * weight
//   int8: scale = max |y| / 127,  q = rint(y / scale)
// and, with the gradients dy of y and dsum of the sum that is passed on,
//   dh = rstd * (weight dy - h rstd^2 mean(weight dy h)) + dsum
//   dweight = sum over rows of dy h rstd
//
// A row is a block's: a thread owns 8 consecutive values every 8 * blockDim and
// keeps them in registers, so every byte is read and written once. All
// arithmetic is binary32; y and the sum are rounded once, at their store.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "int8.cuh"

namespace moe {
namespace {

constexpr float kFarUnit = 0x1p-90f;  // brings every bf16 value's square, and sums of them, into binary32
constexpr float kFloatMax = 3.402823466e38f;
constexpr int kChunks = 4;  // 16-byte chunks of a thread's part of a row
constexpr int kPlanParts = 8;  // blocks that share a row tile of a plan

__device__ __forceinline__ void widen(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t pair_of(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
    return make_uint4(pair_of(f[0], f[1]), pair_of(f[2], f[3]), pair_of(f[4], f[5]), pair_of(f[6], f[7]));
}

// 16 bytes that are read once. Not through the read-only path: a result may replace an input.
__device__ __forceinline__ uint4 load16(const void* row, int chunk) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(static_cast<const uint8_t*>(row) + chunk * 16)
                 : "memory");
    return v;
}

// Sums over the block, the same in every thread; `at`: which of the block's scratch places.
template <int N, bool MAX>
__device__ __forceinline__ void block_join(float (&v)[N], float (*place)[32]) {
    const int warps = static_cast<int>(blockDim.x >> 5), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const float o = __shfl_xor_sync(0xffffffffu, v[i], d);
            v[i] = MAX ? nan_max(v[i], o) : v[i] + o;
        }
    if (warps == 1) return;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) place[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = place[i][0];
        for (int w = 1; w < warps; ++w) v[i] = MAX ? nan_max(v[i], place[i][w]) : v[i] + place[i][w];
    }
}

// rstd of a row whose squares add up past binary32: the sum is taken of h 2^-90. (An
// infinity or a NaN in the row gives 0 or NaN, as it does without this.) Whole blocks call it.
template <int C>
__device__ __noinline__ float far_rstd(const float (&h)[C][8], int32_t H, float (*place)[32]) {
    float sum[1] = {0.f};
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = h[j][i] * kFarUnit;
            sum[0] = fmaf(v, v, sum[0]);
        }
    block_join<1, false>(sum, place);
    return __frsqrt_rn(__fdiv_rn(sum[0], static_cast<float>(H))) * kFarUnit;
}

// NORM: root-mean-square norm; otherwise the rows are packed as they are.
template <int C, bool NORM>
__global__ void __launch_bounds__(NORM ? 512 : 1024) row_kernel(const NormArgs a) {
    pdl_wait_then_release();
    __shared__ float place[3][1][32];
    const int nch = a.H / 8;
    int64_t row = blockIdx.x, step = gridDim.x, end = a.rows;
    if (!NORM && a.plan) {
        const int32_t tile = static_cast<int32_t>(blockIdx.x / kPlanParts);
        if (tile >= __ldg(a.plan)) return;
        const int4 t = __ldg(reinterpret_cast<const int4*>(a.plan + plan_tiles_at(a.E)) + tile);
        if (t.y < 0 || t.z < 0 || t.z > kPlanTileRows || t.y + static_cast<int64_t>(t.z) > a.rows) return;
        row = t.y + blockIdx.x % kPlanParts;
        step = kPlanParts;
        end = t.y + t.z;
    }
    for (; row < end; row += step) {
        const int64_t from = a.gated ? row / a.group_rows * a.group_rows + fp4_gated_row(row % a.group_rows, a.group_rows) : row;
        const uint8_t* x = a.x + from * a.x_stride;
        float h[C][8];
        float sum[1] = {0.f};
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c >= nch) {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] = 0.f;
                continue;
            }
            widen(load16(x, c), h[j]);
            if (NORM && a.residual) {
                float r[8];
                widen(load16(a.residual + row * a.residual_stride, c), r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] += r[i];
            }
            if (NORM && a.sum) *reinterpret_cast<uint4*>(a.sum + row * a.sum_stride + c * 16) = narrow(h[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0] = fmaf(h[j][i], h[j][i], sum[0]);
        }
        if (NORM) {
            block_join<1, false>(sum, place[0]);
            float rstd = __frsqrt_rn(__fdiv_rn(sum[0], static_cast<float>(a.H)) + a.eps);
            if (!(sum[0] <= kFloatMax)) rstd = far_rstd<C>(h, a.H, place[2]);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int c = threadIdx.x + j * blockDim.x;
                if (c >= nch) continue;
                float w[8];
                widen(__ldg(reinterpret_cast<const uint4*>(a.weight) + c), w);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] = h[j][i] * rstd * w[i];
                if (a.y) *reinterpret_cast<uint4*>(a.y + row * a.y_stride + c * 16) = narrow(h[j]);
            }
        }
        if (!a.q) {
            __syncthreads();
            continue;
        }
        float most[1] = {0.f};
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) most[0] = nan_max(most[0], fabsf(h[j][i]));
        block_join<1, true>(most, place[1]);
        const Int8Scale s = int8_scale(most[0]);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < nch) *reinterpret_cast<uint2*>(a.q + row * a.q_stride + c * 8) = int8_codes8(h[j], s);
        }
        if (threadIdx.x == 0) *reinterpret_cast<float*>(a.q_scale + row * a.q_scale_stride) = s.scale;
        __syncthreads();
    }
}

template <int C>
__global__ void __launch_bounds__(512) norm_grad_kernel(const NormGradArgs a) {
    pdl_wait_then_release();
    __shared__ float place[4][32];
    const int nch = a.H / 8;
    float acc[C][8] = {};
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float h[C][8], b[C][8];  // the row, and dy
        float sums[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c >= nch) {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] = 0.f;
                continue;
            }
            float w[8];
            widen(load16(a.h + row * a.h_stride, c), h[j]);
            widen(load16(a.dy + row * a.dy_stride, c), b[j]);
            widen(__ldg(reinterpret_cast<const uint4*>(a.weight) + c), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sums[0] = fmaf(h[j][i], h[j][i], sums[0]);
                sums[1] = fmaf(b[j][i] * w[i], h[j][i], sums[1]);
            }
        }
        block_join<2, false>(sums, place);
        float rstd = __frsqrt_rn(__fdiv_rn(sums[0], static_cast<float>(a.H)) + a.eps);
        float back = sums[1] / static_cast<float>(a.H) * rstd * rstd;
        if (!(sums[0] <= kFloatMax)) {  // squares past binary32: all in h 2^-90, where eps is nothing
            sums[0] = sums[1] = 0.f;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int c = threadIdx.x + j * blockDim.x;
                if (c >= nch) continue;
                float w[8];
                widen(__ldg(reinterpret_cast<const uint4*>(a.weight) + c), w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = h[j][i] * kFarUnit;
                    sums[0] = fmaf(v, v, sums[0]);
                    sums[1] = fmaf(b[j][i] * w[i], v, sums[1]);
                }
            }
            block_join<2, false>(sums, place + 2);
            rstd = __frsqrt_rn(__fdiv_rn(sums[0], static_cast<float>(a.H)));
            back = sums[1] / static_cast<float>(a.H) * rstd * rstd * kFarUnit;
            rstd *= kFarUnit;
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c >= nch) continue;
            float w[8], d[8] = {};
            widen(__ldg(reinterpret_cast<const uint4*>(a.weight) + c), w);
            if (a.dsum) widen(load16(a.dsum + row * a.dsum_stride, c), d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[j][i] = fmaf(b[j][i], h[j][i] * rstd, acc[j][i]);
                d[i] += rstd * (b[j][i] * w[i] - h[j][i] * back);
            }
            *reinterpret_cast<uint4*>(a.dh + row * a.dh_stride + c * 16) = narrow(d);
        }
        __syncthreads();
    }
    if (a.parts == nullptr) return;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
        if (c >= nch) continue;
        float4* out = reinterpret_cast<float4*>(a.parts + static_cast<int64_t>(blockIdx.x) * a.H + c * 8);
        out[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        out[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
    }
}

// The blocks' sums of the weight's gradient, in ascending order.
__global__ void __launch_bounds__(256) norm_join_kernel(const float* parts, int n, int32_t H, float* dweight) {
    pdl_wait_then_release();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= H) return;
    float s = 0.f;
    for (int b = 0; b < n; ++b) s += parts[static_cast<int64_t>(b) * H + c];
    dweight[c] = s;
}

// codes * scale, rounded to bf16.
__global__ void __launch_bounds__(256) unpack_kernel(const NormArgs a) {
    pdl_wait_then_release();
    const int nch = a.H / 8;
    int64_t row = blockIdx.x, step = gridDim.x, end = a.rows;
    if (a.plan) {
        const int32_t tile = static_cast<int32_t>(blockIdx.x / kPlanParts);
        if (tile >= __ldg(a.plan)) return;
        const int4 t = __ldg(reinterpret_cast<const int4*>(a.plan + plan_tiles_at(a.E)) + tile);
        if (t.y < 0 || t.z < 0 || t.z > kPlanTileRows || t.y + static_cast<int64_t>(t.z) > a.rows) return;
        row = t.y + blockIdx.x % kPlanParts;
        step = kPlanParts;
        end = t.y + t.z;
    }
    for (; row < end; row += step) {
        const int64_t to = a.gated ? row / a.group_rows * a.group_rows + fp4_gated_row(row % a.group_rows, a.group_rows) : row;
        const float s = __ldg(reinterpret_cast<const float*>(a.q_scale + row * a.q_scale_stride));
        for (int c = threadIdx.x; c < nch; c += blockDim.x) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(a.q + row * a.q_stride) + c);
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = s * static_cast<float>(static_cast<int8_t>(((i < 4 ? v.x : v.y) >> (8 * (i & 3))) & 0xffu));
            *reinterpret_cast<uint4*>(a.y + to * a.y_stride + c * 16) = narrow(f);
        }
    }
}

// Threads of a row's block, and how many chunks each of them has.
unsigned row_threads(int32_t H) { return 32u * static_cast<unsigned>(ceil_div(ceil_div(H / 8, kChunks), 32)); }
int row_chunks(int32_t H) { return static_cast<int>(ceil_div(H / 8, row_threads(H))); }

unsigned row_grid(const NormArgs& a) {
    if (a.plan) return static_cast<unsigned>(a.tile_cap) * kPlanParts;
    return static_cast<unsigned>(a.rows < (1 << 30) ? a.rows : (1 << 30));
}

template <bool NORM>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t stream) {
    if (a.rows == 0 || (a.plan && a.tile_cap == 0)) return cudaSuccess;
    const int c = row_chunks(a.H);
    const auto kernel = c <= 1 ? row_kernel<1, NORM> : c == 2 ? row_kernel<2, NORM> : c == 3 ? row_kernel<3, NORM> : row_kernel<4, NORM>;
    return launch_pdl(kernel, row_grid(a), row_threads(a.H), 0, stream, a);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t stream) { return launch_rows<true>(a, stream); }
cudaError_t launch_int8_pack(const NormArgs& a, cudaStream_t stream) { return launch_rows<false>(a, stream); }

cudaError_t launch_int8_unpack(const NormArgs& a, cudaStream_t stream) {
    if (a.rows == 0 || (a.plan && a.tile_cap == 0)) return cudaSuccess;
    return launch_pdl(unpack_kernel, row_grid(a), 256u, 0, stream, a);
}

cudaError_t launch_rms_norm_grad(const NormGradArgs& a, float* dweight, cudaStream_t stream) {
    const unsigned blocks = static_cast<unsigned>(a.rows < kNormParts ? a.rows : kNormParts);
    if (blocks > 0) {
        const int c = row_chunks(a.H);
        const auto kernel = c <= 1 ? norm_grad_kernel<1> : c == 2 ? norm_grad_kernel<2> : c == 3 ? norm_grad_kernel<3> : norm_grad_kernel<4>;
        const cudaError_t e = launch_pdl(kernel, blocks, row_threads(a.H), 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    if (dweight == nullptr) return cudaSuccess;
    return launch_pdl(norm_join_kernel, static_cast<unsigned>(ceil_div(a.H, 256)), 256u, 0, stream,
                      static_cast<const float*>(a.parts), static_cast<int>(blocks), a.H, dweight);
}

}  // namespace moe
