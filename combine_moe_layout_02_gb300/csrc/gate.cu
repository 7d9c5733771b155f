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
// (0 in the second sum where weights are normalized; p a_k is formed as scale (p[i_k] / D) (..), which is bounded).
//
// A token is a warp's, V of its logits a lane's, in registers; the next token's are
// loaded meanwhile. The logits are read once and the sums of p stay in registers over
// a warp's tokens. Bound by the selection's instructions (forward: 262144 tokens, 256
// experts, 8 picks 119-128 us, 2.2 TB/s, 0.74 instructions a cycle) and by memory (backward:
// 99-101 us, 5.5 TB/s). Up to 64 experts several tokens share a warp.
//
// Selection: whole numbers in the order of the logits, the low bits replaced by the
// expert's number counted down: one maximum over the warp then gives the next expert,
// equal logits by ascending expert. A lane sorts its V once and offers its largest. Where
// two of the K + 1 largest differ in the replaced bits only (a 16-bit logit has nothing
// in them), or there is a NaN, the token is selected again with whole numbers of all
// bits. (A maximum of all bits and then the lowest expert that has it, by two joins and a
// search of the lane's V for each of the K, took twice as long.)
//
// Sums over tokens are binary32 per warp, joined in a fixed order. More than 1024
// experts: a block to a token (the _wide kernels).
#include <cuda_bf16.h>

#include "experts.cuh"

namespace moe {
namespace {

constexpr int kGateWarps = 8;
constexpr int kOneBlock = 32;  // tokens that one block takes, sums joined on the spot
constexpr float kNegInf = -__builtin_huge_valf();
constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ float logit(const float* z, int e) { return __ldg(z + e); }
__device__ __forceinline__ float logit(const __nv_bfloat16* z, int e) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(z) + e)) << 16);
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Whole numbers in the order of the logits, -0 as 0, NaN above all; 0 is below all of them.
__device__ __forceinline__ uint32_t order_of(float z) {
    if (z != z) return 0xffffffffu;
    const uint32_t u = __float_as_uint(z + 0.f);  // -0 becomes 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t order) {
    return __uint_as_float(order & 0x80000000u ? order ^ 0x80000000u : ~order);
}
constexpr uint32_t kNoLogit = 0x007fffffu;  // order_of(-infinity): an expert that may not be chosen; numbers are above

// e^x for x <= 0 by the hardware's 2^x (to 2^-22; below 2^-126: 0); x log2 e is rounded once, which adds |x| 2^-24 at most,
// as much as the rounding of x = z - max does. With this and the reciprocal and quotient below, 262144 tokens of 256 experts have weights
// off by 6.0e-8 in the root mean square (binary32 torch: 5.7e-8); rounded reciprocals and quotients make it 5.8e-8 and the forward pass
// 128 -> 146 us, the product's lost bits added back 5.7e-8 and 153 us.
__device__ __forceinline__ float exp_of(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}

// 1 / x for 1 <= x < 2^126, to 2^-23.
__device__ __forceinline__ float inverse_of(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// Sums over lanes 0 to 15, in each of them (and over 16 to 31 in those).
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
    for (int d = 8; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// ---------------------------------------------------------------------------
// Up to 1024 experts

// 32-bit words of a lane in a warp's shared memory: V logits, V + 2 rows of lists.
constexpr int lists_of(int V) { return 2 * V + 2; }

// Expert of a lane's i-th logit, L lanes to a row: VEC neighbours to a load, ascending in i.
template <int VEC, int L = 32>
__device__ __forceinline__ int expert_of(int i, int lane) {
    return (i / VEC) * L * VEC + lane * VEC + i % VEC;
}

// A lane's raw logits of a row: VEC of them to a load of 16 bytes, or one by one.
template <typename T, int V, int VEC, int L = 32>
struct RowLoad {
    static constexpr int kWords = VEC > 1 ? V * static_cast<int>(sizeof(T)) / 4 : V;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const GateArgs& a, int64_t g, int lane) {
        const uint8_t* row = static_cast<const uint8_t*>(a.logits) + g * a.row_stride;
        if constexpr (VEC > 1) {
#pragma unroll
            for (int n = 0; n < V / VEC; ++n) {
                const int e = expert_of<VEC, L>(n * VEC, lane);
                constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // past the experts: -infinity
                uint4 v = make_uint4(kNone, kNone, kNone, kNone);
                if (e < a.E) v = __ldg(reinterpret_cast<const uint4*>(row + e * sizeof(T)));
                w[4 * n] = v.x;
                w[4 * n + 1] = v.y;
                w[4 * n + 2] = v.z;
                w[4 * n + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = expert_of<1, L>(i, lane);
                w[i] = __float_as_uint(e < a.E ? logit(reinterpret_cast<const T*>(row), e) : kNegInf);
            }
        }
    }
    __device__ __forceinline__ void values(float (&z)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (VEC > 1 && sizeof(T) == 2)
                z[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
            else
                z[i] = __uint_as_float(w[i]);
        }
    }
};

// The comparisons of odd-even merge sort (Batcher) for V numbers.
template <int V>
struct Network {
    int n = 0;
    short a[V * 8] = {}, b[V * 8] = {};

    constexpr Network() {
        for (int p = 1; p < V; p *= 2)
            for (int k = p; k >= 1; k /= 2)
                for (int j = k % p; j + k < V; j += 2 * k)
                    for (int i = 0; i < k && i + j + k < V; ++i)
                        if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                            a[n] = static_cast<short>(i + j);
                            b[n++] = static_cast<short>(i + j + k);
                        }
    }
};

template <int V>
__device__ __forceinline__ void sort_descending(uint32_t (&k)[V]) {
    constexpr Network<V> net;
#pragma unroll
    for (int i = 0; i < net.n; ++i) {
        const uint32_t x = k[net.a[i]], y = k[net.b[i]];
        k[net.a[i]] = max(x, y);
        k[net.b[i]] = min(x, y);
    }
}

// The K largest of the warp's logits: lane k's expert, or -1 in lanes past the last. SHORT: the
// logits are 16-bit numbers. lists [V + 2][32]: the warp's, in shared memory, a lane's
// column; row V is 0, row V + 1 takes what was picked.
template <int V, int VEC, bool SHORT>
__device__ __forceinline__ int32_t select(const float (&z)[V], int K, int lane, uint32_t* lists) {
    constexpr uint32_t kNumber = 32u * V - 1;  // the bits of an expert's number
    uint32_t* own = lists + lane;
    uint32_t head;
    {
        uint32_t k[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t u = __float_as_int(z[i] + 0.f);  // -0 becomes 0, any NaN the positive one of all ones
            k[i] = ((static_cast<uint32_t>(u >> 31) | 0x80000000u) ^ static_cast<uint32_t>(u)) & ~kNumber;
            k[i] |= kNumber - static_cast<uint32_t>(expert_of<VEC>(i, lane));
        }
        sort_descending(k);
        head = k[0];
#pragma unroll
        for (int i = 0; i < V; ++i) own[32 * i] = k[i];
    }
    uint32_t* picked = lists + 32 * (V + 1);
    const int picks = SHORT ? K : K + 1;  // one more, to see whether it is apart from the last
    constexpr int kAtOnce = SHORT ? 4 : 3;
    static_assert(MOE_MAX_TOPK + kAtOnce <= 32 && 32 * V >= 32, "picks: a lane each, no more than there are numbers");
    for (int j = 0; j < picks; j += kAtOnce) {
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n) {
            const uint32_t best = __reduce_max_sync(kAll, head);
            if (head == best) {  // one lane's: the numbers differ; and none is 0, where a lane that has no more stays
                picked[j + n] = best;
                own += 32;
            }
            head = *own;
        }
    }
    __syncwarp();
    const uint32_t mine = lane <= K ? picked[lane] : 0u;
    const uint32_t before = __shfl_up_sync(kAll, mine, 1);
    int32_t at = mine > kNoLogit && lane < K ? static_cast<int32_t>(kNumber - (mine & kNumber)) : -1;
    if (SHORT || !__any_sync(kAll, lane >= 1 && mine > kNoLogit && (mine | kNumber) == (before | kNumber))) return at;
    // All bits: the largest, then the lowest expert that has it.
    at = -1;
    uint32_t taken = 0;  // of the lane's V
    for (int j = 0; j < K; ++j) {
        uint32_t best = 0;
        int i0 = 0;
#pragma unroll
        for (int i = V - 1; i >= 0; --i) {  // of equal ones the lowest
            const uint32_t o = taken >> i & 1 ? 0u : order_of(z[i]);
            if (o >= best) {
                best = o;
                i0 = i;
            }
        }
        const uint32_t all = __reduce_max_sync(kAll, best);
        if (all <= kNoLogit) break;
        const int e = best == all ? expert_of<VEC>(i0, lane) : 1 << 20;
        const int first = __reduce_min_sync(kAll, e);
        if (lane == j) at = first;
        if (e == first) taken |= 1u << i0;
    }
    return at;
}

// A row's largest logit, NaN above all, as order_of() gives it.
template <int V>
__device__ __forceinline__ uint32_t row_top(const float (&z)[V]) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < V; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(z[i]));
    return __reduce_max_sync(kAll, order_of(m));
}

// The blocks' (parts') sums to counts, mean probabilities and the loss: expert e of this
// CTA's share from `first` on; the shares' part of the loss is returned to thread 0. 32
// experts at a time, a lane each, the warps' parts joined in ascending order.
__device__ __forceinline__ float join_parts(const GateArgs& a, int parts, int first, int end, int32_t* n_out) {
    __shared__ float sums[32][33];
    __shared__ int32_t counts[32][33];
    __shared__ int32_t routed[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    int32_t n = 0;
    for (int b = threadIdx.x; b < parts; b += blockDim.x) n += a.part_count[static_cast<size_t>(b) * (a.E + 1) + a.E];
    n = __reduce_add_sync(kAll, n);
    if (lane == 0) routed[warp] = n;
    __syncthreads();
    n = __reduce_add_sync(kAll, lane < warps ? routed[lane] : 0);
    *n_out = n;
    const float inv = n > 0 ? 1.f / static_cast<float>(n) : 0.f;
    float loss = 0.f;
    for (int e0 = first; e0 < end; e0 += 32) {
        const int e = e0 + lane;
        float s = 0.f;
        int32_t c = 0;
        constexpr int kAhead = 8;
        for (int b0 = warp; b0 < parts; b0 += kAhead * warps) {  // eight parts' loads at a time
            float ps[kAhead];
            int32_t pc[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int b = b0 + j * warps;
                const bool there = e < end && b < parts;
                ps[j] = there ? __ldg(a.part_prob + static_cast<size_t>(b) * a.E + e) : 0.f;
                pc[j] = there ? __ldg(a.part_count + static_cast<size_t>(b) * (a.E + 1) + e) : 0;
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                s += ps[j];
                c += pc[j];
            }
        }
        sums[warp][lane] = s;
        counts[warp][lane] = c;
        __syncthreads();
        if (warp == 0 && e < end) {
            s = 0.f;
            c = 0;
            for (int w = 0; w < warps; ++w) {
                s += sums[w][lane];
                c += counts[w][lane];
            }
            s *= inv;
            a.expert_count[e] = c;
            if (a.expert_prob) a.expert_prob[e] = s;
            loss += static_cast<float>(c) * s;
        }
        __syncthreads();
    }
    return warp == 0 ? warp_sum(loss) : 0.f;
}

__device__ __forceinline__ float loss_of(const GateArgs& a, float sum, int32_t n) {
    return n > 0 ? a.balance * static_cast<float>(a.E) * (sum / (static_cast<float>(n) * a.K)) : 0.f;
}

// A block's sums, sum_of(e), and counts to its part; a block alone joins them at once.
template <typename F>
__device__ __forceinline__ void leave_parts(const GateArgs& a, const int32_t* count, F sum_of) {
    if (gridDim.x > 1) {
        float* part = a.part_prob + static_cast<size_t>(blockIdx.x) * a.E;
        int32_t* part_count = a.part_count + static_cast<size_t>(blockIdx.x) * (a.E + 1);
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            part[e] = sum_of(e);
            part_count[e] = count[e];
        }
        if (threadIdx.x == 0) part_count[a.E] = count[a.E];
        return;
    }
    __shared__ float losses[32];
    const int32_t n = count[a.E];
    const float inv = n > 0 ? 1.f / static_cast<float>(n) : 0.f;
    float loss = 0.f;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        const float s = sum_of(e) * inv;
        a.expert_count[e] = count[e];
        if (a.expert_prob) a.expert_prob[e] = s;
        loss += static_cast<float>(count[e]) * s;
    }
    loss = warp_sum(loss);
    if (threadIdx.x % 32 == 0) losses[threadIdx.x / 32] = loss;
    __syncthreads();
    if (threadIdx.x > 0) return;
    loss = 0.f;
    for (unsigned w = 0; w < blockDim.x / 32; ++w) loss += losses[w];
    a.expert_count[a.E] = n;
    if (a.loss) *a.loss = loss_of(a, loss, n);
}

template <typename T, int V, int VEC>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(const GateArgs a) {
    pdl_wait_then_release();
    // Of each warp: a token's logits (in the end the sums of p), and its lists; then [E + 1] counts.
    extern __shared__ __align__(16) float smem[];
    constexpr int kMine = 32 * lists_of(V);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t* count = reinterpret_cast<int32_t*>(smem + kGateWarps * kMine);
    float* logits = smem + warp * kMine;
    uint32_t* lists = reinterpret_cast<uint32_t*>(logits + 32 * V);
    lists[32 * V + lane] = 0u;
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) count[e] = 0;
    __syncthreads();
    float acc[V] = {};
    int32_t routed_tokens = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGateWarps;
    int64_t g = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
    RowLoad<T, V, VEC> row;
    uint8_t masked = 0;
    const auto fetch = [&](int64_t t) {
        if (t >= a.S) return;
        row.load(a, t, lane);
        masked = a.mask != nullptr && __ldg(a.mask + t) == 0;
    };
    fetch(g);
    for (; g < a.S; g += step) {
        float z[V];
        row.values(z);
        const bool out = masked != 0;
        fetch(g + step);
        if constexpr (VEC > 1) {
#pragma unroll
            for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(logits + expert_of<VEC>(i, lane)) = make_float4(z[i], z[i + 1], z[i + 2], z[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) logits[expert_of<1>(i, lane)] = z[i];
        }
        __syncwarp();
        const int32_t at = out ? -1 : select<V, VEC, sizeof(T) == 2>(z, a.K, lane, lists);
        const float chosen = at >= 0 ? logits[at] : kNegInf;
        const float top = __shfl_sync(kAll, chosen, 0);  // the largest logit, NaN where there is one
        __syncwarp();  // the lists and the logits have been read
        if (top == kNegInf) {  // no expert was found
            if (lane < a.K) {
                a.topk_idx[g * a.K + lane] = -1;
                a.topk_weights[g * a.K + lane] = 0.f;
            }
            continue;
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            z[i] = exp_of(z[i] - top);
            sum += z[i];
        }
        const float p = at >= 0 ? exp_of(chosen - top) : 0.f;
        const float inv = inverse_of(warp_sum(sum));
        const float share = a.normalize ? __fdividef(a.scale, half_sum(p)) : a.scale * inv;  // of lanes below 16
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(z[i], inv, acc[i]);
        if (lane < a.K) {
            a.topk_idx[g * a.K + lane] = at;
            // a NaN or an infinity in the row: all its weights, of slots that found an expert, are NaN
            a.topk_weights[g * a.K + lane] = at < 0 ? 0.f : p * share + 0.f * inv;
            if (at >= 0) atomicAdd(&count[at], 1);
        }
        ++routed_tokens;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i) logits[expert_of<VEC>(i, lane)] = acc[i];
    if (lane == 0) atomicAdd(&count[a.E], routed_tokens);
    __syncthreads();
    leave_parts(a, count, [&](int e) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kGateWarps; ++w) s += smem[w * kMine + e];
        return s;
    });
}

// ---------------------------------------------------------------------------
// Up to 64 experts: L lanes to a token, 8 of its logits a lane's, 32 / L neighbouring tokens a
// warp's. Joins by shuffles among L lanes cost a warp more than one maximum, and serve 32 / L
// tokens. 262144 tokens, binary32, forward and backward: 8 experts, 2 picks 13 and 10 us (a warp
// to a token: 73 and 77), 16 experts 17 and 10 (73, 77), 32 experts, 4 picks 28 and 19 (80, 78),
// 64 experts, 6 picks 53 and 42 (87, 82); of 128 experts, 8 picks, two tokens to a warp would
// take 116 and 88 (95, 88). Bound by the selection's instructions; small logits by the launch.

constexpr int kTeamV = 8;
constexpr int kMostInTeams = 64;

template <int L>
constexpr int kTeams = 32 / L;
constexpr int kTeamPicks = MOE_MAX_TOPK + 5;  // of a token: K + 1, at a stride that spreads over the banks

// Word of expert e in a warp's columns [8][32], of the first team.
template <int VEC, int L>
__device__ __forceinline__ int column_of(int e) {
    return ((e / (VEC * L)) * VEC + e % VEC) * 32 + (e / VEC) % L;
}

template <int L>
__device__ __forceinline__ float team_sum(float v) {
#pragma unroll
    for (int d = L / 2; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
template <int L>
__device__ __forceinline__ uint32_t team_max(uint32_t v) {
#pragma unroll
    for (int d = L / 2; d; d >>= 1) v = max(v, __shfl_xor_sync(kAll, v, d));
    return v;
}
// NaN above all.
template <int L>
__device__ __forceinline__ float team_top(const float (&z)[kTeamV]) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < kTeamV; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(z[i]));
#pragma unroll
    for (int d = L / 2; d; d >>= 1) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(__shfl_xor_sync(kAll, m, d)));
    return m;
}

// As select(), for each team: picked[k] of the K largest, as team_pick() reads it. lists [9][32]:
// the warp's, the last row 0. live: the team has a token.
template <int L, int VEC, bool SHORT>
__device__ __forceinline__ void select_of_team(const float (&z)[kTeamV], int K, int lane, bool live, uint32_t* lists, uint32_t* picked) {
    constexpr int V = kTeamV;
    constexpr uint32_t kNumber = V * L - 1;
    const int l = lane % L;
    uint32_t* own = lists + lane;
    uint32_t head;
    {
        uint32_t k[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t u = __float_as_int(z[i] + 0.f);  // as in select()
            k[i] = ((static_cast<uint32_t>(u >> 31) | 0x80000000u) ^ static_cast<uint32_t>(u)) & ~kNumber;
            k[i] |= kNumber - static_cast<uint32_t>(expert_of<VEC, L>(i, l));
        }
        sort_descending(k);
        head = k[0];
#pragma unroll
        for (int i = 0; i < V; ++i) own[32 * i] = k[i];
    }
    const int picks = SHORT ? K : K + 1;
    for (int j = 0; j < picks; ++j) {
        const uint32_t best = team_max<L>(head);
        if (head == best) {
            picked[j] = best;
            if (best != 0u) own += 32;  // (a team may have fewer numbers than picks)
        }
        head = *own;
    }
    __syncwarp();
    if constexpr (!SHORT) {
        bool near = false;
        for (int s = l; s < K; s += L) near |= picked[s + 1] > kNoLogit && (picked[s] | kNumber) == (picked[s + 1] | kNumber);
        if (!__any_sync(kAll, live && near)) return;
        __syncwarp();
        uint32_t taken = 0;
        for (int j = 0; j < K; ++j) {
            uint32_t best = 0;
            int i0 = 0;
#pragma unroll
            for (int i = V - 1; i >= 0; --i) {
                const uint32_t o = taken >> i & 1 ? 0u : order_of(z[i]);
                if (o >= best) {
                    best = o;
                    i0 = i;
                }
            }
            const uint32_t all = team_max<L>(best);
            const uint32_t mine = best == all && all > kNoLogit ? kNumber - static_cast<uint32_t>(expert_of<VEC, L>(i0, l)) + 1u : 0u;
            const uint32_t first = team_max<L>(mine);  // the lowest expert's
            if (mine == first) {                       // one lane's, or all write a 0
                picked[j] = first ? ~kNumber | (first - 1u) : 0u;
                if (first) taken |= 1u << i0;
            }
        }
        __syncwarp();
    }
}

template <int L>
__device__ __forceinline__ int32_t team_pick(uint32_t picked) {
    constexpr uint32_t kNumber = kTeamV * L - 1;
    return picked > kNoLogit ? static_cast<int32_t>(kNumber - (picked & kNumber)) : -1;
}

// Words of a warp: a token's exponentials (in the end the sums of p), lists, picks.
template <int L>
constexpr int kTeamWords = 32 * kTeamV + 32 * (kTeamV + 1) + kTeams<L> * kTeamPicks;

template <typename T, int L, int VEC>
__global__ void __launch_bounds__(32 * kGateWarps) gate_team_kernel(const GateArgs a) {
    pdl_wait_then_release();
    constexpr int V = kTeamV, P = kTeams<L>, kMine = kTeamWords<L>;
    __shared__ float smem[kGateWarps * kMine];
    __shared__ int32_t count[kMostInTeams + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % L, team = lane / L;
    float* column = smem + warp * kMine;
    uint32_t* lists = reinterpret_cast<uint32_t*>(column + 32 * V);
    uint32_t* picked = lists + 32 * (V + 1) + team * kTeamPicks;
    lists[32 * V + lane] = 0u;
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) count[e] = 0;
    __syncthreads();
    float acc[V] = {};
    int32_t routed_tokens = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kGateWarps * P);
    int64_t first = (static_cast<int64_t>(blockIdx.x) * kGateWarps + warp) * P;  // the warp's first token
    RowLoad<T, V, VEC, L> row = {};
    uint8_t masked = 0;
    const auto fetch = [&](int64_t t) {
        if (t >= a.S) return;
        row.load(a, t, l);
        masked = a.mask != nullptr && __ldg(a.mask + t) == 0;
    };
    fetch(first + team);
    for (; first < a.S; first += step) {
        const int64_t g = first + team;
        float z[V];
        row.values(z);
        bool live = g < a.S && masked == 0;
        fetch(g + step);
        const float top = team_top<L>(z);
        live = live && top != kNegInf;
        select_of_team<L, VEC, sizeof(T) == 2>(z, a.K, lane, live, lists, picked);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            z[i] = exp_of(z[i] - top);
            sum += z[i];
            column[32 * i + lane] = z[i];
        }
        const float inv = inverse_of(team_sum<L>(sum));
        __syncwarp();
        const float* mine = column + team * L;
        float d = 0.f;
        if (a.normalize) {
            for (int s = l; s < a.K; s += L) {
                const int32_t at = team_pick<L>(picked[s]);
                d += at >= 0 ? mine[column_of<VEC, L>(at)] : 0.f;
            }
            d = team_sum<L>(d);
        }
        const float share = a.normalize ? __fdividef(a.scale, d) : a.scale * inv;
        if (g < a.S)
            for (int s = l; s < a.K; s += L) {
                const int32_t at = live ? team_pick<L>(picked[s]) : -1;
                a.topk_idx[g * a.K + s] = at;
                a.topk_weights[g * a.K + s] = at < 0 ? 0.f : mine[column_of<VEC, L>(at)] * share + 0.f * inv;
                if (at >= 0) atomicAdd(&count[at], 1);
            }
        if (live) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(z[i], inv, acc[i]);
            routed_tokens += l == 0;
        }
        __syncwarp();  // the columns and the picks have been read
    }
    routed_tokens = __reduce_add_sync(kAll, routed_tokens);
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int d = 16; d >= L; d >>= 1) acc[i] += __shfl_xor_sync(kAll, acc[i], d);
        column[32 * i + lane] = acc[i];
    }
    if (lane == 0) atomicAdd(&count[a.E], routed_tokens);
    __syncthreads();
    leave_parts(a, count, [&](int e) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kGateWarps; ++w) s += smem[w * kMine + column_of<VEC, L>(e)];
        return s;
    });
}

// One cluster: each CTA joins a share of the experts, the first one adds the shares' losses up.
constexpr int kJoinCtas = 8;
__global__ void __launch_bounds__(1024) gate_join_kernel(const GateArgs a, int parts) {
    pdl_wait_then_release();
    __shared__ float share;
    const int per = static_cast<int>(round_up(ceil_div(a.E, kJoinCtas), 32)), first = min(a.E, static_cast<int>(blockIdx.x) * per);
    int32_t n;
    const float loss = join_parts(a, parts, first, min(a.E, first + per), &n);
    if (threadIdx.x == 0) share = loss;
    cluster_sync_all();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        float s = 0.f;
        for (uint32_t r = 0; r < kJoinCtas; ++r) s += __int_as_float(ld_cluster_s32(cluster_map(&share, r)));
        a.expert_count[a.E] = n;
        if (a.loss) *a.loss = loss_of(a, s, n);
    }
    cluster_sync_all();
}

// The sum of the chosen exponentials below which they are formed again, from the largest chosen logit (a program has dropped
// the slots above it): from it down they lose bits, and 1 / sum leaves binary32.
constexpr float kFarSum = 0x1p-60f;

// The slots' part of the gradient, in lanes below K (K <= 16): expert (or -1), p, and p_k a_k summed
// over slots of the same expert in ascending order (in all of them); in all lanes t, the sum
// over k of p[i_k] a_k: scale / D times sum_k dw_k p_k - sum_j dw_j p_j = 0 of normalized
// weights, scale sum_k dw_k p_k of others. p_k a_k is scale (p_k / D) (dw_k - mean), whose factors are
// numbers however far the slots are below the row's largest logit. `chosen`: the slots' logits, `top` the row's largest;
// whose [E]: the warp's, in shared memory, or none (then the slots are compared).
struct Slots {
    int32_t i;
    float p, pa, t;
};
static_assert(MOE_MAX_TOPK <= 16, "slots in half a warp");
__device__ __forceinline__ Slots slots_of(const GateArgs& a, int lane, int32_t i, float dw, float chosen, float top, float inv,
                                          volatile uint8_t* whose) {
    float e = i >= 0 ? exp_of(chosen - top) : 0.f;
    Slots s{i, e * inv, 0.f, 0.f};
    if (a.dweights == nullptr) return s;
    float back = half_sum(dw * e);
    float own;
    if (a.normalize) {
        float d = half_sum(e);
        if (__any_sync(kAll, i >= 0 && !(d >= kFarSum))) {
            const uint32_t most = __reduce_max_sync(kAll, i >= 0 ? order_of(chosen) : 0u);
            e = i >= 0 && most > kNoLogit ? exp_of(chosen - logit_of(most)) : 0.f;
            back = half_sum(dw * e);
            d = half_sum(e);
        }
        const float each = __frcp_rn(d);  // (two divisions instead: 262144 x 256 115 us against 101)
        own = d > 0.f || d != d ? a.scale * (e * each * (dw - back * each)) : 0.f;  // (0: no slot, or none that counts)
    } else {
        own = a.scale * dw * s.p;
        s.t = __shfl_sync(kAll, a.scale * back * inv, 0);
    }
    s.pa = own;
    bool twice;
    if (whose != nullptr) {  // two slots of one expert read back one's lane
        if (i >= 0) whose[i] = static_cast<uint8_t>(lane);
        __syncwarp();
        twice = i >= 0 && whose[i] != lane;
    } else {
        twice = __popc(__match_any_sync(kAll, i)) > 1 && i >= 0;
    }
    if (__any_sync(kAll, twice)) {
        s.pa = 0.f;
        for (int k = 0; k < a.K; ++k) {
            const float o = __shfl_sync(kAll, own, k);
            if (__shfl_sync(kAll, i, k) == i) s.pa += o;
        }
    }
    __syncwarp();
    return s;
}

// dl * balance * E / (K n) / n.
__device__ __forceinline__ float loss_unit(const GateArgs& a) {
    const int32_t n = __ldg(a.expert_count + a.E);
    if (a.dloss == nullptr || n <= 0) return 0.f;
    return __ldg(a.dloss) * a.balance * a.E / (static_cast<float>(n) * static_cast<float>(n) * a.K);
}

// A lane's V of a row.
template <int V, int VEC, int L = 32, typename T>
__device__ __forceinline__ void put_row(T* to, int E, int lane, const float (&z)[V]) {
    if constexpr (VEC > 1) {
#pragma unroll
        for (int n = 0; n < V / VEC; ++n) {
            const int e = expert_of<VEC, L>(n * VEC, lane);
            if (e >= E) continue;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 2) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(z[n * VEC + 2 * j], z[n * VEC + 2 * j + 1]);
                    w[j] = *reinterpret_cast<const uint32_t*>(&b);
                } else {
                    w[j] = __float_as_uint(z[n * VEC + j]);
                }
            }
            *reinterpret_cast<uint4*>(to + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (expert_of<1, L>(i, lane) < E) put(to + expert_of<1, L>(i, lane), z[i]);
    }
}

template <typename T, int V, int VEC>
__global__ void __launch_bounds__(32 * kGateWarps) gate_grad_kernel(const GateArgs a) {
    pdl_wait_then_release();
    __shared__ float table[32 * V];  // c of each expert
    __shared__ uint8_t whose[kGateWarps][32 * V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float unit = loss_unit(a);
    for (int e = threadIdx.x; e < 32 * V; e += blockDim.x)
        table[e] = e < a.E ? unit * static_cast<float>(__ldg(a.expert_count + e)) : 0.f;
    __syncthreads();
    float c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = table[expert_of<VEC>(i, lane)];
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGateWarps;
    int64_t g = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
    RowLoad<T, V, VEC> row;
    uint8_t masked = 0;
    float chosen = 0.f, dw = 0.f;
    const auto ids = [&](int64_t t) {
        const int32_t i = t < a.S && lane < a.K ? __ldg(a.topk_idx + t * a.K + lane) : -1;
        return i < a.E ? i : -1;
    };
    // A token's logits, and its slots' by their ids, are loaded a token ahead, the ids two.
    const auto fetch = [&](int64_t t, int32_t i) {
        if (t >= a.S) return;
        row.load(a, t, lane);
        masked = a.mask != nullptr && __ldg(a.mask + t) == 0;
        chosen = i >= 0 ? logit(reinterpret_cast<const T*>(static_cast<const uint8_t*>(a.logits) + t * a.row_stride), i) : 0.f;
        dw = i >= 0 && a.dweights ? __ldg(a.dweights + t * a.K + lane) : 0.f;
    };
    int32_t idx = ids(g), idx_next = ids(g + step);
    fetch(g, idx);
    for (; g < a.S; g += step) {
        float z[V];
        row.values(z);
        const bool out = masked != 0;
        const int32_t i_now = idx;
        const float dw_now = dw, chosen_now = chosen;
        idx = idx_next;
        idx_next = ids(g + 2 * step);
        fetch(g + step, idx);
        T* to = reinterpret_cast<T*>(static_cast<uint8_t*>(a.dlogits) + g * a.dlogits_stride);
        const uint32_t most = row_top(z);
        const bool routed = !out && most > kNoLogit;
        float t = 0.f, inv = 0.f;
        Slots s{-1, 0.f, 0.f, 0.f};
        if (routed) {
            const float top = logit_of(most);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                z[i] = exp_of(z[i] - top);
                sum += z[i];
                t = fmaf(z[i], c[i], t);
            }
            inv = inverse_of(warp_sum(sum));
            t = warp_sum(t) * inv;
            s = slots_of(a, lane, i_now, dw_now, chosen_now, top, inv, whose[warp]);
            t += s.t;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = routed ? z[i] * inv * (c[i] - t) : 0.f;
        put_row<V, VEC>(to, a.E, lane, z);
        __syncwarp();  // the chosen experts' over what was stored for them
        if (s.i >= 0) put(to + s.i, fmaf(s.p, table[s.i] - t, s.pa));
        __syncwarp();
    }
}

// As gate_team_kernel. A token's slots are the team's, in turn; the lane that has a slot's expert
// adds p_k a_k to its column, in ascending order of k.
__device__ __forceinline__ void fetch_word(void* to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from)
                 : "memory");
}

template <typename T, int L, int VEC>
__global__ void __launch_bounds__(32 * kGateWarps) gate_team_grad_kernel(const GateArgs a) {
    pdl_wait_then_release();
    constexpr int V = kTeamV, P = kTeams<L>;
    const int slots = P * a.K;  // of a warp's tokens
    extern __shared__ __align__(16) float smem[];
    __shared__ float table[V * L];  // c of each expert
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % L, team = lane / L;
    float* column = smem + warp * (64 * V + 4 * slots);  // the exponentials
    float* add = column + 32 * V;                         // sum over k with i_k = e of p_k a_k
    int32_t* ids = reinterpret_cast<int32_t*>(add + 32 * V);
    float* dws = reinterpret_cast<float*>(ids + 2 * slots);
    const float unit = loss_unit(a);
    for (int e = threadIdx.x; e < V * L; e += blockDim.x)
        table[e] = e < a.E ? unit * static_cast<float>(__ldg(a.expert_count + e)) : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) add[32 * i + lane] = 0.f;
    __syncthreads();
    float c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = table[expert_of<VEC, L>(i, l)];
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kGateWarps * P);
    int64_t first = (static_cast<int64_t>(blockIdx.x) * kGateWarps + warp) * P;
    RowLoad<T, V, VEC, L> row = {};
    uint8_t masked = 0;
    // The next tokens' logits in registers, their slots in one of two places; a lane waits for what it has copied.
    const auto fetch = [&](int64_t f, int place) {
        if (a.dweights != nullptr && f < a.S) {
            const int n = static_cast<int>((a.S - f < P ? a.S - f : P)) * a.K;
            for (int s = lane; s < n; s += 32) {
                fetch_word(ids + place * slots + s, a.topk_idx + f * a.K + s);
                fetch_word(dws + place * slots + s, a.dweights + f * a.K + s);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (f + team < a.S) {
            row.load(a, f + team, l);
            masked = a.mask != nullptr && __ldg(a.mask + f + team) == 0;
        }
    };
    fetch(first, 0);
    for (int place = 0; first < a.S; first += step, place ^= 1) {
        const int64_t g = first + team;
        float z[V];
        row.values(z);
        bool live = g < a.S && masked == 0;
        fetch(first + step, place ^ 1);
        const float top = team_top<L>(z);
        live = live && top != kNegInf;
        float sum = 0.f, t = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            z[i] = live ? exp_of(z[i] - top) : 0.f;
            sum += z[i];
            t = fmaf(z[i], c[i], t);
            column[32 * i + lane] = z[i];
        }
        sum = team_sum<L>(sum);
        const float inv = live ? inverse_of(sum) : 0.f;
        t = team_sum<L>(t) * inv;
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        if (a.dweights != nullptr) {
            const int32_t* i_k = ids + place * slots + team * a.K;
            const float* dw_k = dws + place * slots + team * a.K;
            float back, d;
            const auto add_up = [&] {
                back = d = 0.f;
                if (live)
                    for (int s = l; s < a.K; s += L) {
                        const int32_t i = i_k[s];
                        if (i < 0 || i >= a.E) continue;
                        const float e = column[team * L + column_of<VEC, L>(i)];
                        back = fmaf(dw_k[s], e, back);
                        d += e;
                    }
                back = team_sum<L>(back);
                d = team_sum<L>(d);
            };
            add_up();
            const bool far = live && a.normalize && !(d >= kFarSum);
            if (__any_sync(kAll, far)) {  // the slots' columns from their largest logit
                const T* from = reinterpret_cast<const T*>(static_cast<const uint8_t*>(a.logits) + g * a.row_stride);
                uint32_t most = 0;
                if (far)
                    for (int s = l; s < a.K; s += L)
                        if (i_k[s] >= 0 && i_k[s] < a.E) most = max(most, order_of(logit(from, i_k[s])));
                most = team_max<L>(most);
                if (far && most > kNoLogit)
                    for (int s = l; s < a.K; s += L)
                        if (i_k[s] >= 0 && i_k[s] < a.E)
                            column[team * L + column_of<VEC, L>(i_k[s])] = exp_of(logit(from, i_k[s]) - logit_of(most));
                __syncwarp();
                add_up();
            }
            const float mean = a.normalize ? back / d : 0.f, each = a.normalize ? 1.f / d : inv;
            if (!a.normalize) t += a.scale * back * inv;
            if (live && (!a.normalize || d > 0.f || d != d))  // (0: no slot, or none that counts)
                for (int s = 0; s < a.K; ++s) {
                    const int32_t i = i_k[s];
                    if (i < 0 || i >= a.E || (i / VEC) % L != l) continue;
                    const int at = column_of<VEC, L>(i) - l + lane;
                    add[at] += a.scale * (column[at] * each * (dw_k[s] - mean));
                }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            z[i] = live ? fmaf(z[i] * inv, c[i] - t, add[32 * i + lane]) : 0.f;
            add[32 * i + lane] = 0.f;  // a lane's own
        }
        if (g < a.S) put_row<V, VEC, L>(reinterpret_cast<T*>(static_cast<uint8_t*>(a.dlogits) + g * a.dlogits_stride), a.E, l, z);
        __syncwarp();  // the columns and the slots have been read
    }
}

// ---------------------------------------------------------------------------
// More than 1024 experts: a block to a token, 512 of its logits a warp's, which finds the K
// largest of its own as above; the block's are among those. 16384 tokens, 4096 experts, 8 picks, binary32:
// forward 232 us, backward 95 (5.7 TB/s); as a warp to a token, rows in shared memory and searched for each
// pick, 1228 and 267. The forward pass is bound by its instructions.

constexpr int kWideV = 16;
constexpr int kWide = 32 * kWideV;  // experts of a warp
constexpr int kWideWarps = MOE_MAX_EXPERTS / kWide;
static_assert(MOE_MAX_EXPERTS % kWide == 0 && kWideWarps <= 8 && kWideWarps * MOE_MAX_TOPK <= 128, "a block's candidates, four a lane");

// The arguments as a warp's share of the experts has them.
template <typename T>
__device__ __forceinline__ GateArgs share_of(const GateArgs& a, int warp) {
    GateArgs mine = a;
    mine.logits = static_cast<const uint8_t*>(a.logits) + static_cast<size_t>(warp) * kWide * sizeof(T);
    mine.E = max(0, min(kWide, a.E - warp * kWide));
    return mine;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(32 * kWideWarps) gate_wide_kernel(const GateArgs a) {
    pdl_wait_then_release();
    // Of each warp as in gate_kernel; then [E + 1] counts.
    extern __shared__ __align__(16) float smem[];
    // By turns of two: a warp may be a token behind.
    __shared__ float sums[2][kWideWarps], found[2][kWideWarps * MOE_MAX_TOPK];
    __shared__ int32_t found_at[2][kWideWarps * MOE_MAX_TOPK];
    constexpr int V = kWideV, kMine = 32 * lists_of(V);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    int32_t* count = reinterpret_cast<int32_t*>(smem + warps * kMine);
    float* logits = smem + warp * kMine;
    uint32_t* lists = reinterpret_cast<uint32_t*>(logits + 32 * V);
    lists[32 * V + lane] = 0u;
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) count[e] = 0;
    __syncthreads();
    const GateArgs mine = share_of<T>(a, warp);
    float acc[V] = {};
    RowLoad<T, V, VEC> row = {};
    uint8_t masked = 0;
    const auto fetch = [&](int64_t t) {
        if (t >= a.S) return;
        row.load(mine, t, lane);
        masked = a.mask != nullptr && __ldg(a.mask + t) == 0;
    };
    int64_t g = blockIdx.x;
    fetch(g);
    for (int turn = 0; g < a.S; g += gridDim.x, turn ^= 1) {
        float z[V];
        row.values(z);
        const bool out = masked != 0;
        fetch(g + gridDim.x);
#pragma unroll
        for (int i = 0; i < V; ++i) logits[expert_of<VEC>(i, lane)] = z[i];
        __syncwarp();
        {
            const int32_t at = out ? -1 : select<V, VEC, sizeof(T) == 2>(z, a.K, lane, lists);
            if (lane < a.K) {
                found[turn][warp * a.K + lane] = at >= 0 ? logits[at] : kNegInf;
                found_at[turn][warp * a.K + lane] = warp * kWide + at;
            }
        }
        __syncthreads();
        const uint32_t most = __reduce_max_sync(kAll, lane < warps ? order_of(found[turn][lane * a.K]) : 0u);
        if (most <= kNoLogit) {  // no expert was found
            if (warp == 0 && lane < a.K) {
                a.topk_idx[g * a.K + lane] = -1;
                a.topk_weights[g * a.K + lane] = 0.f;
            }
            continue;
        }
        const float top = logit_of(most);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            z[i] = exp_of(z[i] - top);
            sum += z[i];
        }
        sum = warp_sum(sum);
        if (lane == 0) sums[turn][warp] = sum;
        __syncthreads();
        const float inv = inverse_of(warp_sum(lane < warps ? sums[turn][lane] : 0.f));
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(z[i], inv, acc[i]);
        if (warp != 0) continue;
        // The K largest of what the warps found, four a lane, of equal ones the lowest expert.
        uint32_t key[4];
        int32_t at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = lane + 32 * j;
            key[j] = c < warps * a.K ? order_of(found[turn][c]) : 0u;
            at[j] = c < warps * a.K ? found_at[turn][c] : 0;
        }
        int32_t pick = -1;
        float e = 0.f;
        for (int k = 0; k < a.K; ++k) {
            uint32_t best = key[0];
            int32_t best_at = at[0];
#pragma unroll
            for (int j = 1; j < 4; ++j)
                if (key[j] > best || (key[j] == best && at[j] < best_at)) {
                    best = key[j];
                    best_at = at[j];
                }
            const uint32_t all = __reduce_max_sync(kAll, best);
            if (all <= kNoLogit) break;
            const int32_t next = static_cast<int32_t>(__reduce_min_sync(kAll, best == all ? static_cast<uint32_t>(best_at) : 0x7fffffffu));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (key[j] == all && at[j] == next) key[j] = 0u;
            if (lane == k) {
                pick = next;
                e = exp_of(logit_of(all) - top);
            }
        }
        const float share = a.normalize ? __fdividef(a.scale, half_sum(e)) : a.scale * inv;  // of lanes below 16
        if (lane < a.K) {
            a.topk_idx[g * a.K + lane] = pick;
            a.topk_weights[g * a.K + lane] = pick < 0 ? 0.f : e * share + 0.f * inv;  // as in gate_kernel
            if (pick >= 0) atomicAdd(&count[pick], 1);
        }
        if (lane == 0) atomicAdd(&count[a.E], 1);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i) logits[expert_of<VEC>(i, lane)] = acc[i];
    __syncthreads();
    leave_parts(a, count, [&](int e) { return smem[e / kWide * kMine + e % kWide]; });
}

template <typename T, int VEC>
__global__ void __launch_bounds__(32 * kWideWarps) gate_wide_grad_kernel(const GateArgs a) {
    pdl_wait_then_release();
    __shared__ uint32_t tops[2][kWideWarps];  // by turns of two
    __shared__ float sums[2][2][kWideWarps];
    constexpr int V = kWideV;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const float unit = loss_unit(a);
    const GateArgs mine = share_of<T>(a, warp);
    float c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = expert_of<VEC>(i, lane);
        c[i] = e < mine.E ? unit * static_cast<float>(__ldg(a.expert_count + warp * kWide + e)) : 0.f;
    }
    RowLoad<T, V, VEC> row = {};
    uint8_t masked = 0;
    float chosen = 0.f, dw = 0.f;
    const auto ids = [&](int64_t t) {
        const int32_t i = t < a.S && lane < a.K ? __ldg(a.topk_idx + t * a.K + lane) : -1;
        return i < a.E ? i : -1;
    };
    const auto fetch = [&](int64_t t, int32_t i) {
        if (t >= a.S) return;
        row.load(mine, t, lane);
        masked = a.mask != nullptr && __ldg(a.mask + t) == 0;
        chosen = i >= 0 ? logit(reinterpret_cast<const T*>(static_cast<const uint8_t*>(a.logits) + t * a.row_stride), i) : 0.f;
        dw = i >= 0 && a.dweights ? __ldg(a.dweights + t * a.K + lane) : 0.f;
    };
    int64_t g = blockIdx.x;
    int32_t idx = ids(g), idx_next = ids(g + gridDim.x);
    fetch(g, idx);
    for (int turn = 0; g < a.S; g += gridDim.x, turn ^= 1) {
        float z[V];
        row.values(z);
        const bool out = masked != 0;
        const int32_t i_now = idx;
        const float dw_now = dw, chosen_now = chosen;
        idx = idx_next;
        idx_next = ids(g + 2 * static_cast<int64_t>(gridDim.x));
        fetch(g + gridDim.x, idx);
        T* to = reinterpret_cast<T*>(static_cast<uint8_t*>(a.dlogits) + g * a.dlogits_stride) + warp * kWide;
        uint32_t most = row_top(z);
        if (lane == 0) tops[turn][warp] = most;
        __syncthreads();
        most = __reduce_max_sync(kAll, lane < warps ? tops[turn][lane] : 0u);
        const bool routed = !out && most > kNoLogit;
        float t = 0.f, inv = 0.f;
        Slots s{-1, 0.f, 0.f, 0.f};
        if (routed) {
            const float top = logit_of(most);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                z[i] = exp_of(z[i] - top);
                sum += z[i];
                t = fmaf(z[i], c[i], t);
            }
            sum = warp_sum(sum);
            t = warp_sum(t);
            if (lane == 0) {
                sums[turn][0][warp] = sum;
                sums[turn][1][warp] = t;
            }
            __syncthreads();
            inv = inverse_of(warp_sum(lane < warps ? sums[turn][0][lane] : 0.f));
            t = warp_sum(lane < warps ? sums[turn][1][lane] : 0.f) * inv;
            s = slots_of(a, lane, i_now, dw_now, chosen_now, top, inv, nullptr);
            t += s.t;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = routed ? z[i] * inv * (c[i] - t) : 0.f;
        put_row<V, VEC>(to, mine.E, lane, z);
        __syncwarp();  // the warp's chosen experts' over what was stored for them
        const int at = s.i - warp * kWide;
        if (s.i >= 0 && at >= 0 && at < kWide) put(to + at, fmaf(s.p, unit * static_cast<float>(__ldg(a.expert_count + s.i)) - t, s.pa));
        __syncwarp();
    }
}

// ---------------------------------------------------------------------------

using Kernel = void (*)(const GateArgs);

// Loads of 16 bytes where rows are made of them.
bool by_16(const GateArgs& a, int64_t stride) {
    const int64_t elt = a.bf16 ? 2 : 4;
    return a.E * elt % 16 == 0 && stride % 16 == 0;
}

template <bool GRAD, typename T, int V, int VEC>
Kernel kernel_at() {
    if constexpr (GRAD)
        return gate_grad_kernel<T, V, VEC>;
    else
        return gate_kernel<T, V, VEC>;
}
constexpr int kMostInRegisters = 1024;  // of a warp
int logits_of_a_lane(int E) { return E <= 128 ? 4 : E <= 256 ? 8 : E <= 512 ? 16 : 32; }
int lanes_of_a_token(int E) { return E > kMostInTeams ? 32 : E <= 8 ? 1 : E <= 16 ? 2 : E <= 32 ? 4 : 8; }

template <bool GRAD, typename T, int L>
Kernel team_at(bool by) {
    constexpr int kVec = 16 / sizeof(T);
    if constexpr (GRAD)
        return by ? gate_team_grad_kernel<T, L, kVec> : gate_team_grad_kernel<T, L, 1>;
    else
        return by ? gate_team_kernel<T, L, kVec> : gate_team_kernel<T, L, 1>;
}

// by: rows are loaded 16 bytes at a time.
template <bool GRAD, typename T>
Kernel kernel_for(int E, bool by) {
    if (E > kMostInRegisters) {
        constexpr int kVec = 16 / sizeof(T);
        if constexpr (GRAD)
            return by ? gate_wide_grad_kernel<T, kVec> : gate_wide_grad_kernel<T, 1>;
        else
            return by ? gate_wide_kernel<T, kVec> : gate_wide_kernel<T, 1>;
    }
    switch (lanes_of_a_token(E)) {
        case 1: return team_at<GRAD, T, 1>(by);
        case 2: return team_at<GRAD, T, 2>(by);
        case 4: return team_at<GRAD, T, 4>(by);
        case 8: return team_at<GRAD, T, 8>(by);
        default: break;
    }
    // Of four logits to a lane 16-bit ones are no 16 bytes: they go one by one (262144 x 128, 8 picks: 99 us each way; 32-bit ones 98 and 87).
    constexpr int kVec = 16 / sizeof(T), kVec4 = kVec <= 4 ? kVec : 1;
    switch (logits_of_a_lane(E)) {
        case 4: return by ? kernel_at<GRAD, T, 4, kVec4>() : kernel_at<GRAD, T, 4, 1>();
        case 8: return by ? kernel_at<GRAD, T, 8, kVec>() : kernel_at<GRAD, T, 8, 1>();
        case 16: return by ? kernel_at<GRAD, T, 16, kVec>() : kernel_at<GRAD, T, 16, 1>();
        default: return by ? kernel_at<GRAD, T, 32, kVec>() : kernel_at<GRAD, T, 32, 1>();
    }
}

// A token's lanes, and a block's warps.
struct Geometry {
    int lanes, warps;
};
Geometry geometry(int E) {
    if (E > kMostInRegisters) return {kWide, static_cast<int>(ceil_div(E, kWide))};
    return {lanes_of_a_token(E), kGateWarps};
}

// Blocks: what is resident, or needed, at most kGateParts.
cudaError_t blocks_for(Kernel kernel, size_t smem, const Geometry& geo, int64_t S, unsigned* blocks) {
    const int warps = geo.warps, tokens = geo.lanes > 32 ? 1 : warps * 32 / geo.lanes;
    int per_sm = 0;
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), smem, 32 * warps, &per_sm);
    int64_t n = static_cast<int64_t>(device_sm_count()) * (per_sm > 0 ? per_sm : 1);
    if (n > kGateParts) n = kGateParts;
    const int64_t need = ceil_div(S, tokens);
    *blocks = static_cast<unsigned>(need < 1 ? 1 : need < n ? need : n);
    return e;
}

}  // namespace

cudaError_t launch_gate(const GateArgs& a, cudaStream_t stream) {
    const Geometry geo = geometry(a.E);
    const bool by = by_16(a, a.row_stride);
    const size_t smem = geo.lanes < 32 ? 0 : (static_cast<size_t>(geo.warps) * 32 * lists_of(geo.lanes > 32 ? kWideV : logits_of_a_lane(a.E)) + a.E + 1) * 4;
    const Kernel kernel = a.bf16 ? kernel_for<false, __nv_bfloat16>(a.E, by) : kernel_for<false, float>(a.E, by);
    unsigned blocks = 0;
    cudaError_t e = blocks_for(kernel, smem, geo, a.S, &blocks);
    if (e != cudaSuccess) return e;
    if (geo.lanes <= 32 && a.S <= kOneBlock) blocks = 1;
    e = launch_pdl(kernel, blocks, 32u * geo.warps, smem, stream, a);
    if (e != cudaSuccess || blocks == 1) return e;
    return launch_pdl_cluster(gate_join_kernel, kJoinCtas, 1024u, 0, kJoinCtas, stream, a, static_cast<int>(blocks));
}

cudaError_t launch_gate_grad(const GateArgs& a, cudaStream_t stream) {
    if (a.S == 0) return cudaSuccess;
    const Geometry geo = geometry(a.E);
    const bool by = by_16(a, a.row_stride) && by_16(a, a.dlogits_stride);
    const size_t smem = geo.lanes < 32 ? static_cast<size_t>(geo.warps) * (64 * kTeamV + 4 * (32 / geo.lanes) * a.K) * 4 : 0;
    const Kernel kernel = a.bf16 ? kernel_for<true, __nv_bfloat16>(a.E, by) : kernel_for<true, float>(a.E, by);
    unsigned blocks = 0;
    const cudaError_t e = blocks_for(kernel, smem, geo, a.S, &blocks);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, blocks, 32u * geo.warps, smem, stream, a);
}

}  // namespace moe
