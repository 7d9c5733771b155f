// gate.cu -- the router's gate and its gradient (moe_gate, moe_gate_grad). For a
// routed token g with logits z[e]:
//   p[e]   = exp(z[e] - max z) / sum over e of exp(z[e] - max z)
//   i_k    = the K largest logits in descending order, equal ones by ascending e
//   w_k    = scale * p[i_k] / D,  D = sum over k of p[i_k] (normalize) or 1
//   loss   = balance * E * sum over e of f[e] * P[e],  f[e] = count[e] / (K n),
//            P[e] = (sum over tokens of p[e]) / n,  n = routed tokens
// and, with the gradients dw of w and dl of loss,
//   a_k    = scale / D * (dw_k - [normalize] sum over j of dw_j p[i_j] / D)
//   c[e]   = dl * balance * E * f[e] / n              (counts are constants)
//   dz[e]  = p[e] * (c[e] + sum over k with i_k = e of a_k - T),
//   T      = sum over e of p[e] c[e] + sum over k of p[i_k] a_k
//
// A token is a warp's; its row is in shared memory. Selection compares whole
// numbers that order like the logits (NaN above all, -0 as 0), so ties are exact.
// Sums over tokens are binary32 per warp, joined in a fixed order.
#include <cuda_bf16.h>

#include "experts.cuh"

namespace moe {
namespace {

constexpr int kGateWarps = 4;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float logit(const float* z, int e) { return __ldg(z + e); }
__device__ __forceinline__ float logit(const __nv_bfloat16* z, int e) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(z) + e)) << 16);
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Whole numbers in the order of the logits; 0 is below all of them.
__device__ __forceinline__ uint32_t order_of(float z) {
    if (z != z) return 0xffffffffu;
    const uint32_t u = __float_as_uint(z + 0.f);  // -0 becomes 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kNoLogit = 0x007fffffu;  // order_of(-infinity): an expert that may not be chosen

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

template <typename T>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(const GateArgs a) {
    pdl_wait_then_release();
    extern __shared__ float smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* z = smem + static_cast<size_t>(warp) * 2 * a.E;  // the token's logits; the ones chosen are taken out
    float* sums = z + a.E;                                  // the warp's sums of p
    int32_t* count = reinterpret_cast<int32_t*>(smem + static_cast<size_t>(kGateWarps) * 2 * a.E);  // [E + 1]
    for (int e = lane; e < a.E; e += 32) sums[e] = 0.f;
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) count[e] = 0;
    __syncthreads();
    for (int64_t g = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp; g < a.S;
         g += static_cast<int64_t>(gridDim.x) * kGateWarps) {
        const T* row = reinterpret_cast<const T*>(static_cast<const uint8_t*>(a.logits) + g * a.row_stride);
        uint32_t most = 0;
        for (int e = lane; e < a.E; e += 32) {
            z[e] = logit(row, e);
            most = max(most, order_of(z[e]));
        }
        most = __reduce_max_sync(0xffffffffu, most);
        const bool routed = most > kNoLogit && (a.mask == nullptr || __ldg(a.mask + g) != 0);
        if (!routed) {
            if (lane < a.K) {
                a.topk_idx[g * a.K + lane] = -1;
                a.topk_weights[g * a.K + lane] = 0.f;
            }
            continue;
        }
        const uint32_t u = most & 0x80000000u ? most ^ 0x80000000u : ~most;
        const float top = __uint_as_float(u);  // NaN where most stands for one
        float sum = 0.f;
        for (int e = lane; e < a.E; e += 32) sum += __expf(z[e] - top);
        const float inv = __frcp_rn(warp_sum(sum));
        for (int e = lane; e < a.E; e += 32) sums[e] += __expf(z[e] - top) * inv;
        int32_t mine = -1;
        float p = 0.f;
        for (int k = 0; k < a.K; ++k) {
            uint32_t best = 0;
            int at = a.E;
            for (int e = lane; e < a.E; e += 32) {
                const uint32_t o = order_of(z[e]);
                if (o > best) {
                    best = o;
                    at = e;
                }
            }
            const uint32_t all = __reduce_max_sync(0xffffffffu, best);
            if (all <= kNoLogit) break;
            at = __reduce_min_sync(0xffffffffu, best == all ? at : a.E);
            if (lane == k) {
                mine = at;
                p = __expf(z[at] - top) * inv;
            }
            __syncwarp();
            if (lane == 0) {
                z[at] = kNegInf;
                atomicAdd(&count[at], 1);
            }
            __syncwarp();
        }
        const float d = a.normalize ? warp_sum(p) : 1.f;
        if (lane < a.K) {
            a.topk_idx[g * a.K + lane] = mine;
            a.topk_weights[g * a.K + lane] = mine < 0 ? 0.f : a.scale * __fdividef(p, d);
        }
        if (lane == 0) atomicAdd(&count[a.E], 1);
        __syncwarp();
    }
    __syncthreads();
    float* part = a.part_prob + static_cast<size_t>(blockIdx.x) * a.E;
    int32_t* part_count = a.part_count + static_cast<size_t>(blockIdx.x) * (a.E + 1);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        float s = 0.f;
        for (int w = 0; w < kGateWarps; ++w) s += smem[(static_cast<size_t>(w) * 2 + 1) * a.E + e];
        part[e] = s;
    }
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) part_count[e] = count[e];
}

// The blocks' sums to counts, mean probabilities and the loss.
__global__ void __launch_bounds__(1024) gate_join_kernel(const GateArgs a, int parts) {
    pdl_wait_then_release();
    __shared__ float partial[32];
    int32_t n = 0;
    for (int b = 0; b < parts; ++b) n += a.part_count[static_cast<size_t>(b) * (a.E + 1) + a.E];
    const float inv = n > 0 ? 1.f / static_cast<float>(n) : 0.f;
    float loss = 0.f;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int32_t c = 0;
        float s = 0.f;
        for (int b = 0; b < parts; ++b) {
            c += a.part_count[static_cast<size_t>(b) * (a.E + 1) + e];
            s += a.part_prob[static_cast<size_t>(b) * a.E + e];
        }
        s *= inv;
        a.expert_count[e] = c;
        if (a.expert_prob) a.expert_prob[e] = s;
        loss += static_cast<float>(c) * s;
    }
    if (threadIdx.x == 0) a.expert_count[a.E] = n;
    loss = warp_sum(loss);
    if ((threadIdx.x & 31) == 0) partial[threadIdx.x >> 5] = loss;
    __syncthreads();
    if (threadIdx.x == 0 && a.loss) {
        float s = 0.f;
        for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += partial[w];
        *a.loss = n > 0 ? a.balance * static_cast<float>(a.E) * (s / (static_cast<float>(n) * a.K)) : 0.f;
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kGateWarps) gate_grad_kernel(const GateArgs a) {
    pdl_wait_then_release();
    extern __shared__ float smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* c = smem;                                                // [E]
    float* add = smem + a.E + static_cast<size_t>(warp) * a.E;      // [E]: sum over k with i_k = e of a_k
    const int32_t n = __ldg(a.expert_count + a.E);
    const float unit = a.dloss && n > 0
                           ? __ldg(a.dloss) * a.balance * a.E / (static_cast<float>(n) * static_cast<float>(n) * a.K) : 0.f;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) c[e] = unit * static_cast<float>(__ldg(a.expert_count + e));
    for (int e = lane; e < a.E; e += 32) add[e] = 0.f;
    __syncthreads();
    for (int64_t g = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp; g < a.S;
         g += static_cast<int64_t>(gridDim.x) * kGateWarps) {
        const T* row = reinterpret_cast<const T*>(static_cast<const uint8_t*>(a.logits) + g * a.row_stride);
        T* out = reinterpret_cast<T*>(static_cast<uint8_t*>(a.dlogits) + g * a.dlogits_stride);
        uint32_t most = 0;
        for (int e = lane; e < a.E; e += 32) most = max(most, order_of(logit(row, e)));
        most = __reduce_max_sync(0xffffffffu, most);
        if (most <= kNoLogit || (a.mask != nullptr && __ldg(a.mask + g) == 0)) {
            for (int e = lane; e < a.E; e += 32) put(out + e, 0.f);
            continue;
        }
        const float top = __uint_as_float(most & 0x80000000u ? most ^ 0x80000000u : ~most);
        float sum = 0.f, t = 0.f;
        for (int e = lane; e < a.E; e += 32) {
            const float v = __expf(logit(row, e) - top);
            sum += v;
            t += v * c[e];
        }
        const float inv = __frcp_rn(warp_sum(sum));
        t = warp_sum(t) * inv;
        int32_t i = -1;
        float p = 0.f, dw = 0.f;
        if (lane < a.K) {
            i = __ldg(a.topk_idx + g * a.K + lane);
            if (i >= a.E) i = -1;
            if (i >= 0 && a.dweights) {
                dw = __ldg(a.dweights + g * a.K + lane);
                p = __expf(logit(row, i) - top) * inv;
            }
        }
        float d = 1.f, back = dw;
        if (a.normalize && a.dweights) {
            d = warp_sum(p);
            back = dw - warp_sum(dw * p) / d;
        }
        const float ak = i >= 0 && a.dweights ? a.scale * back / d : 0.f;
        t += warp_sum(p * ak);
        if (i >= 0) atomicAdd(&add[i], ak);
        __syncwarp();
        for (int e = lane; e < a.E; e += 32) put(out + e, __expf(logit(row, e) - top) * inv * (c[e] + add[e] - t));
        __syncwarp();
        if (i >= 0) add[i] = 0.f;
        __syncwarp();
    }
}

int gate_blocks(int64_t S) {
    const int64_t n = ceil_div(S, kGateWarps);
    return static_cast<int>(n < 1 ? 1 : n > kGateParts ? kGateParts : n);
}

}  // namespace

cudaError_t launch_gate(const GateArgs& a, cudaStream_t stream) {
    const size_t smem = (static_cast<size_t>(kGateWarps) * 2 * a.E + a.E + 1) * 4;
    const int blocks = gate_blocks(a.S);
    auto kernel = a.bf16 ? gate_kernel<__nv_bfloat16> : gate_kernel<float>;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), smem, 32 * kGateWarps, nullptr);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, static_cast<unsigned>(blocks), 32 * kGateWarps, smem, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(gate_join_kernel, 1u, 1024u, 0, stream, a, blocks);
}

cudaError_t launch_gate_grad(const GateArgs& a, cudaStream_t stream) {
    if (a.S == 0) return cudaSuccess;
    const size_t smem = static_cast<size_t>(kGateWarps + 1) * a.E * 4;
    auto kernel = a.bf16 ? gate_grad_kernel<__nv_bfloat16> : gate_grad_kernel<float>;
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), smem, 32 * kGateWarps, nullptr);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, static_cast<unsigned>(gate_blocks(a.S)), 32 * kGateWarps, smem, stream, a);
}

}  // namespace moe
