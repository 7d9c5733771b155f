// combine_grad.cu -- the gradient of the weighted reduction
// (moe_combine_grad, moe_combine_expert_grad). With
//   out[g] = sum over returned rows r of c_r * y[r]
// and dout the gradient of out,
//   dy[r]    = bf16_rne(c_r * dout[g])
//   dw[g][k] = sum over h of dout[g][h] * y[r(k)][h]   (binary32)
// where r(k) is the row that slot k's expert answered in (rank layout: the row
// of its rank, shared by the token's slots on that rank; c_r is then the
// binary32 sum of their weights in ascending k, as in combine).
//
// Bound by memory: dout and y are read once, dy is written once, 2 operations
// per byte. One pass: a lane owns 16-byte column chunks, loads dout's chunk
// and the chunks of all the token's rows, adds the products to one partial sum
// per row and stores c_r * dout. A token is a warp's or four warps' (the rule is
// at the launch). Routing words are loaded one and two tokens ahead; the rank
// layout reads send_head only at its slots' ranks (a scan of all P ranks cost 3%
// at P = 128). Partial sums are joined in a fixed order (lanes by a butterfly,
// warps in ascending order), so the same inputs give the same bits.
// Measured: 131072 rows of 7168 (expert layout, 4.0 GB): 612 us, 6.5 TB/s, 0.96 of
// a copy's; 8192 tokens over 128 ranks: 281 us, 6.3 TB/s.
#include <cuda_bf16.h>

#include "experts.cuh"

namespace moe {
namespace {

constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / 32;
constexpr int kTeam = 4;           // warps per token, or 1
constexpr int kTeamHidden = 4096;

__device__ __forceinline__ float lo_of(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_of(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_of(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// One lane's routing words of a token, slot `lane`: its expert's rank (-1:
// none) and weight, and its row in the rank's partition. A row number needs the
// rank first (rank layout), so a token's ranks are loaded two tokens ahead and
// its row numbers one ahead.
struct GradSlot {
    int32_t idx;
    float w;
};

__device__ __forceinline__ GradSlot load_grad_slot(const CombineGradArgs& a, int64_t g, int lane) {
    GradSlot r{-1, 0.f};
    if (g < a.S && lane < a.K) {
        r.idx = __ldg(a.topk_idx + g * a.K + lane);
        if (a.topk_weights) r.w = __ldg(a.topk_weights + g * a.K + lane);
    }
    return r;
}

template <bool EXPERT>
__device__ __forceinline__ int32_t load_grad_place(const CombineGradArgs& a, int64_t g, int lane, int32_t idx) {
    if (idx < 0 || idx >= a.E) return -1;  // also the lanes past K and the tokens past S
    return EXPERT ? __ldg(a.slot_row + g * a.K + lane) : __ldg(a.send_head + g * a.P + idx / a.epr);
}

// Barrier of a token's warps.
template <int WARPS>
__device__ __forceinline__ void team_sync(int team) {
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * WARPS) : "memory");
}

// WARPS: warps per token.
template <int MAXR, bool EXPERT, int WARPS>
__global__ void __launch_bounds__(kGradThreads, MAXR >= 16 ? 1 : 2) combine_grad_kernel(const CombineGradArgs a) {
    pdl_wait_then_release();
    extern __shared__ __align__(16) int64_t prb[];  // [P+1]
    __shared__ float part[kGradWarps][MAXR];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i <= a.P; i += blockDim.x) prb[i] = a.part_row_base[i];
    __syncthreads();
    const int nchunks = a.H / 8;
    const int64_t tokens_at_once = static_cast<int64_t>(gridDim.x) * (kGradWarps / WARPS);
    const int team = warp / WARPS, member = warp % WARPS;  // the warps of a token
    const int first_chunk = member * 32 + lane;
    int64_t g = static_cast<int64_t>(blockIdx.x) * (kGradWarps / WARPS) + team;
    GradSlot cur = load_grad_slot(a, g, lane), next = load_grad_slot(a, g + tokens_at_once, lane);
    int32_t place = load_grad_place<EXPERT>(a, g, lane, cur.idx);
    for (; g < a.S; g += tokens_at_once) {
        const int32_t dk = (cur.idx >= 0 && cur.idx < a.E) ? cur.idx / a.epr : -1;
        const float w = cur.w;
        const int32_t sr = place;
        cur = next;
        place = load_grad_place<EXPERT>(a, g + tokens_at_once, lane, cur.idx);
        next = load_grad_slot(a, g + 2 * tokens_at_once, lane);
        // Rank layout: the first slot of each rank stands for its row, with the
        // sum of the weights of all of them.
        float c = w;
        bool valid = dk >= 0 && sr >= 0;
        if (!EXPERT) {
            c = 0.f;
            for (int k = 0; k < a.K; ++k) {
                const int32_t dkk = __shfl_sync(0xffffffffu, dk, k);
                const float wk = __shfl_sync(0xffffffffu, w, k);
                if (dkk == dk) {
                    c = __fadd_rn(c, wk);
                    if (k < lane) valid = false;
                }
            }
        }
        if (!a.topk_weights) c = 1.f;
        int64_t row = 0;
        if (valid) {
            const int64_t lo = prb[dk], hi = prb[dk + 1];
            row = lo + sr;
            valid = sr < hi - lo && row >= 0 && row < a.arena_rows;
            if (!valid) raise_error(a.err, MOE_ERR_CAPACITY);
        }
        // Lane r ends up with the r-th row, its weight and its rank (rank
        // layout) or slot (expert layout).
        int64_t my_row = 0;
        float my_c = 0.f;
        int32_t my_key = -1;
        uint32_t bal = __ballot_sync(0xffffffffu, valid);
        const int n = __popc(bal);  // at most min(K, P) <= MAXR
        for (int r = 0; r < n; ++r) {
            const int src = __ffs(bal) - 1;
            bal &= bal - 1;
            const int64_t p = __shfl_sync(0xffffffffu, row, src);
            const float cc = __shfl_sync(0xffffffffu, c, src);
            const int32_t d = __shfl_sync(0xffffffffu, dk, src);
            if (lane == r) {
                my_row = p;
                my_c = cc;
                my_key = EXPERT ? src : d;
            }
        }
        int64_t rows[MAXR];
        float coef[MAXR], dot[MAXR];
#pragma unroll
        for (int r = 0; r < MAXR; ++r) {
            rows[r] = __shfl_sync(0xffffffffu, my_row, r);
            coef[r] = __shfl_sync(0xffffffffu, my_c, r);
            dot[r] = 0.f;
        }
        const uint8_t* dout = reinterpret_cast<const uint8_t*>(a.dout + g * a.H);
        if (n > 0) {
            for (int j = first_chunk; j < nchunks; j += 32 * WARPS) {
                const size_t at = static_cast<size_t>(j) * 16;
                const uint4 dv = __ldg(reinterpret_cast<const uint4*>(dout + at));
                uint4 v[MAXR];
                if (a.dw) {
#pragma unroll
                    for (int r = 0; r < MAXR; ++r)
                        if (r < n) v[r] = ld_stream_u4(a.y + rows[r] * a.y_stride + at);
                }
                const uint32_t dw4[4] = {dv.x, dv.y, dv.z, dv.w};
                float d[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d[2 * i] = lo_of(dw4[i]);
                    d[2 * i + 1] = hi_of(dw4[i]);
                }
                if (a.dy) {
#pragma unroll
                    for (int r = 0; r < MAXR; ++r)
                        if (r < n) {
                            uint4 o;
                            o.x = pack_of(coef[r] * d[0], coef[r] * d[1]);
                            o.y = pack_of(coef[r] * d[2], coef[r] * d[3]);
                            o.z = pack_of(coef[r] * d[4], coef[r] * d[5]);
                            o.w = pack_of(coef[r] * d[6], coef[r] * d[7]);
                            *reinterpret_cast<uint4*>(a.dy + rows[r] * a.dy_stride + at) = o;
                        }
                }
                if (a.dw) {
#pragma unroll
                    for (int r = 0; r < MAXR; ++r)
                        if (r < n) {
                            const uint32_t y4[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
                            float s = 0.f;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                s = fmaf(d[2 * i], lo_of(y4[i]), s);
                                s = fmaf(d[2 * i + 1], hi_of(y4[i]), s);
                            }
                            dot[r] += s;
                        }
                }
            }
        }
        if (a.dw == nullptr) continue;
        // Lane r: row r's whole sum.
        float mine = 0.f;
#pragma unroll
        for (int r = 0; r < MAXR; ++r) {
            float s = dot[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == r) mine = s;
        }
        if (WARPS > 1) {
            if (lane < MAXR) part[warp][lane] = mine;
            team_sync<WARPS>(team);
            if (lane < MAXR) {
                mine = 0.f;
#pragma unroll
                for (int i = 0; i < WARPS; ++i) mine += part[team * WARPS + i][lane];
            }
            team_sync<WARPS>(team);  // part is free for the next token
            if (member != 0) continue;
        }
        // Slot k takes the sum of the row with its key, 0 if there is none.
        const int32_t want = EXPERT ? lane : dk;
        float res = 0.f;
        for (int r = 0; r < n; ++r) {
            const int32_t key = __shfl_sync(0xffffffffu, my_key, r);
            const float s = __shfl_sync(0xffffffffu, mine, r);
            if (dk >= 0 && key == want) res = s;
        }
        if (lane < a.K) a.dw[g * a.K + lane] = res;
    }
}

template <int MAXR, bool EXPERT, int WARPS>
cudaError_t launch_grad_t(const CombineGradArgs& a, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(a.P + 1) * 8;
    int per_sm = 0;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(combine_grad_kernel<MAXR, EXPERT, WARPS>), smem,
                                   kGradThreads, &per_sm);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) per_sm = 1;
    int64_t grid = static_cast<int64_t>(device_sm_count()) * per_sm;
    const int64_t needed = ceil_div(a.S, kGradWarps / WARPS);
    if (grid > needed) grid = needed;
    return launch_pdl(combine_grad_kernel<MAXR, EXPERT, WARPS>, static_cast<unsigned>(grid), kGradThreads, smem, stream, a);
}

template <int MAXR, bool EXPERT>
cudaError_t launch_grad_w(const CombineGradArgs& a, cudaStream_t stream) {
    // Four warps per token from kTeamHidden on, where each still has four rounds
    // of columns: fewer rows open at once per SM (131072 rows of 7168: 612 us,
    // one warp per token 640, eight 613; 262144 of 4096 688 against one's 709; 524288 of
    // 2048 697 against 714; 1048576 of 1024 774 against 712), and for few tokens, which
    // would leave SMs idle with a warp each (304 tokens of 1024 3.8 us against 6.2).
    const bool team = a.H >= kTeamHidden || a.S < static_cast<int64_t>(device_sm_count()) * kGradWarps;
    return team ? launch_grad_t<MAXR, EXPERT, kTeam>(a, stream) : launch_grad_t<MAXR, EXPERT, 1>(a, stream);
}

template <bool EXPERT>
cudaError_t launch_grad_mode(const CombineGradArgs& a, int maxr, cudaStream_t stream) {
    if (a.S == 0) return cudaSuccess;
    if (maxr <= 1) return launch_grad_w<1, EXPERT>(a, stream);
    if (maxr <= 2) return launch_grad_w<2, EXPERT>(a, stream);
    if (maxr <= 4) return launch_grad_w<4, EXPERT>(a, stream);
    if (maxr <= 8) return launch_grad_w<8, EXPERT>(a, stream);
    return launch_grad_w<16, EXPERT>(a, stream);
}

}  // namespace

cudaError_t launch_combine_grad(const moe_shape& s, const CombineGradArgs& a, cudaStream_t stream) {
    return launch_grad_mode<false>(a, s.K < s.P ? s.K : s.P, stream);
}

cudaError_t launch_combine_expert_grad(const moe_shape& s, const CombineGradArgs& a, cudaStream_t stream) {
    return launch_grad_mode<true>(a, s.K, stream);
}

}  // namespace moe
