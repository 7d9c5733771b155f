// norm.cu -- root-mean-square norm with the residual's addition (moe_rms_norm),
// its gradient (moe_rms_norm_grad), and int8 rows (moe_int8_pack, moe_int8_unpack).
// With h = x + residual of a row of H values:
//   rstd = 1 / sqrt(mean h^2 + eps),  y = h * rstd * weight
//   int8: scale = max |y| / 127,  q = rint(y / scale)
// and, with the gradients dy of y and dsum of the sum that is passed on,
//   dh = rstd * (weight dy - h rstd^2 mean(weight dy h)) + dsum
//   dweight = sum over rows of dy h rstd
//
// Bound by memory: every byte is read and written once. A row is a block's, a thread owns
// 8 consecutive values every 8 * blockDim of it, and the block's next rows are in
// flight to shared memory meanwhile (Ring), so that loads do not wait for a row's joins.
// All arithmetic is binary32; y and the sum are rounded once, at their store.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "int8.cuh"

namespace moe {
namespace {

constexpr float kFarUnit = 0x1p-90f;  // brings every bf16 value's square, and sums of them, into binary32
constexpr float kFloatMax = 3.402823466e38f;
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
// The largest of magnitudes, NaN above all: their bit patterns are in that order.
__device__ __forceinline__ float warp_most(float v) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v))); }

// SUMS sums, and (MOST) a magnitude's maximum behind them, over the block (one warp: over the
// warp), the same in every thread. Every warp joins the warps' values itself, by lanes.
template <int SUMS, bool MOST, bool WARP = false>
__device__ __forceinline__ void block_join(float (&v)[SUMS + MOST], float (*place)[32]) {
    const int warps = static_cast<int>(blockDim.x >> 5), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < SUMS + MOST; ++i) v[i] = i < SUMS ? warp_sum(v[i]) : warp_most(v[i]);
    if (WARP || warps == 1) return;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < SUMS + MOST; ++i) place[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SUMS + MOST; ++i) {
        v[i] = lane < warps ? place[i][lane] : 0.f;
        v[i] = i < SUMS ? warp_sum(v[i]) : warp_most(v[i]);
    }
}

// rstd of a row whose mean square and eps add up past binary32: the sum is taken of h 2^-90, and eps joins it by
// 2^-180, which no eps that counts leaves binary32 by. (An infinity or a NaN in the row gives 0 or NaN, as it does
// without this.) Whole blocks call it.
template <int C>
__device__ __forceinline__ float far_rstd(const float (&h)[C][8], int32_t H, float eps, float (*place)[32]) {
    float sum[1] = {0.f};
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = h[j][i] * kFarUnit;
            sum[0] = fmaf(v, v, sum[0]);
        }
    block_join<1, false>(sum, place);
    return __frsqrt_rn(__fdiv_rn(sum[0], static_cast<float>(H)) + eps * kFarUnit * kFarUnit) * kFarUnit;
}

// The tile of rows that a block of a plan's call shares with others: [row, end) by kPlanParts.
__device__ __forceinline__ bool plan_rows(const NormArgs& a, int64_t& row, int64_t& end) {
    const int32_t tile = static_cast<int32_t>(blockIdx.x / kPlanParts);
    if (tile >= __ldg(a.plan)) return false;
    const int4 t = __ldg(reinterpret_cast<const int4*>(a.plan + plan_tiles_at(a.E)) + tile);
    if (t.y < 0 || t.z < 0 || t.z > kPlanTileRows || t.y + static_cast<int64_t>(t.z) > a.rows) return false;
    row = t.y + blockIdx.x % kPlanParts;
    end = t.y + t.z;
    return true;
}

// A thread's own pieces of the block's next rows, in flight to shared memory while it works
// on one: no other thread reads them, so nothing but its own copies is waited for.
// IN arrays, DEPTH rows, C chunks a row; a thread's 16 bytes are next to its neighbours'.
template <int IN, int DEPTH, int C>
struct Ring {
    uint32_t base, place;
    int nch, tid, per;  // of a row: chunks; this thread, and threads

    __device__ __forceinline__ Ring(void* smem, int nch_, int tid_, int per_)
        : base(smem_addr(smem) + threadIdx.x * 16), place(0), nch(nch_), tid(tid_), per(per_) {}
    __device__ __forceinline__ uint32_t at(uint32_t p, int in, int j) const {
        return base + ((p * IN + in) * C + j) * blockDim.x * 16;
    }
    // The row's pieces, of each array that is there, to place (place + ahead) % DEPTH.
    __device__ __forceinline__ void fetch(const uint8_t* const (&rows)[IN], uint32_t ahead, bool in) {
        const uint32_t p = (place + ahead) % DEPTH;
        if (in)
#pragma unroll
            for (int k = 0; k < IN; ++k)
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    const int c = tid + j * per;
                    if (rows[k] && c < nch)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at(p, k, j)), "l"(rows[k] + c * 16) : "memory");
                }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory"); }
    __device__ __forceinline__ uint4 read(int in, int j) const {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at(place, in, j)) : "memory");
        return v;
    }
    __device__ __forceinline__ void next() { place = (place + 1) % DEPTH; }
};

// Rows of a block in shared memory: the one it works on and the next, or the next two (32768 x 7168, bf16 results:
// 285 us with 3, 310 with 2; int8, whose blocks are fewer to an SM with 3: 243 with 2, 267).
constexpr int kDepth = 2, kPlainDepth = 3;

// QUANT: int8 rows are wanted. Their scale is rstd max |h weight| / 127 and the codes are
// h weight 127 / max |h weight|, so that the row's sum and its maximum are joined at
// once. A code's quotient has two roundings (h weight, 127 / max) and is off by 127 * 2^-23 at most, so codes beside a tie
// may differ from those of rows that are normed first and divided by their scale. Where h weight leaves binary32's range on the way (and in rows of zeros) the
// values are formed first and their maximum joined by itself.
template <int C, bool QUANT>
__global__ void __launch_bounds__(512, QUANT ? 1 : 2) norm_kernel(const NormArgs a) {
    pdl_wait_then_release();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float places[2][4][32];  // rows by turns: a join's places are free two rows on
    const int nch = a.H / 8;
    constexpr int kDeep = QUANT ? kDepth : kPlainDepth;
    Ring<2, kDeep, C> ring(smem, nch, threadIdx.x, blockDim.x);
    const auto fetch = [&](int64_t row, uint32_t ahead) {
        const uint8_t* const rows[2] = {a.x + row * a.x_stride, a.residual ? a.residual + row * a.residual_stride : nullptr};
        ring.fetch(rows, ahead, row < a.rows);
    };
    const int64_t step = gridDim.x;
#pragma unroll
    for (int i = 0; i < kDeep - 1; ++i) fetch(blockIdx.x + i * step, i);
    float w[C][8];  // the thread's columns, for the codes (without them they are loaded where they are used: fewer registers)
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
        widen(c < nch ? __ldg(reinterpret_cast<const uint4*>(a.weight) + c) : make_uint4(0, 0, 0, 0), w[j]);
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += step, turn ^= 1, ring.next()) {
        float(*place)[32] = places[turn];
        fetch(row + (kDeep - 1) * step, kDeep - 1);
        ring.wait();
        float h[C][8];
        float joined[1 + QUANT] = {};  // sum of squares, max |h weight|
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c >= nch) {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] = 0.f;
                continue;
            }
            widen(ring.read(0, j), h[j]);
            if (a.residual) {
                float o[8];
                widen(ring.read(1, j), o);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] += o[i];
            }
            if (a.sum) *reinterpret_cast<uint4*>(a.sum + row * a.sum_stride + c * 16) = narrow(h[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                joined[0] = fmaf(h[j][i], h[j][i], joined[0]);
                if (QUANT) joined[QUANT] = nan_max(joined[QUANT], fabsf(h[j][i] * w[j][i]));
            }
        }
        block_join<1, QUANT>(joined, place);
        const float mean = __fdiv_rn(joined[0], static_cast<float>(a.H)) + a.eps;
        float rstd = __frsqrt_rn(mean);
        if (!(mean <= kFloatMax)) rstd = far_rstd<C>(h, a.H, a.eps, place + 2);
        if (a.y) {
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int c = threadIdx.x + j * blockDim.x;
                if (c >= nch) continue;
                float v[8], u[8];
                widen(__ldg(reinterpret_cast<const uint4*>(a.weight) + c), u);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = h[j][i] * rstd * u[i];
                *reinterpret_cast<uint4*>(a.y + row * a.y_stride + c * 16) = narrow(v);
            }
        }
        if (QUANT) {
            Int8Scale s;
            float most[1] = {joined[QUANT]};
            const bool near = joined[0] <= kFloatMax && most[0] >= 0x1p-60f && most[0] <= 0x1p100f;
            if (near) {
                s.scale = __fdiv_rn(most[0] * rstd, 127.f);
                s.inv = __fdiv_rn(127.f, most[0]);
            } else {
                most[0] = 0.f;
#pragma unroll
                for (int j = 0; j < C; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        h[j][i] *= rstd;
                        most[0] = nan_max(most[0], fabsf(h[j][i] * w[j][i]));
                    }
                block_join<0, true>(most, place + 3);
                s = int8_scale(most[0]);
            }
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int c = threadIdx.x + j * blockDim.x;
                if (c >= nch) continue;
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = h[j][i] * w[j][i];
                *reinterpret_cast<uint2*>(a.q + row * a.q_stride + c * 8) = near ? int8_near8(v, s.inv) : int8_codes8(v, s);
            }
            if (threadIdx.x == 0) *reinterpret_cast<float*>(a.q_scale + row * a.q_scale_stride) = s.scale;
        }
    }
}

// Rows of bf16 to int8, exactly as dispatch rounds them.
template <int C>
__global__ void __launch_bounds__(1024) pack_kernel(const NormArgs a) {
    pdl_wait_then_release();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float places[2][1][32];
    const int nch = a.H / 8;
    int64_t row = blockIdx.x, step = gridDim.x, end = a.rows;
    if (a.plan) {
        if (!plan_rows(a, row, end)) return;
        step = kPlanParts;
    }
    Ring<1, kDepth, C> ring(smem, nch, threadIdx.x, blockDim.x);
    const auto fetch = [&](int64_t r, uint32_t ahead) {
        const int64_t from = a.gated ? r / a.group_rows * a.group_rows + fp4_gated_row(r % a.group_rows, a.group_rows) : r;
        const uint8_t* const rows[1] = {a.x + from * a.x_stride};
        ring.fetch(rows, ahead, r < end);
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(row + i * step, i);
    for (int turn = 0; row < end; row += step, turn ^= 1, ring.next()) {
        fetch(row + (kDepth - 1) * step, kDepth - 1);
        ring.wait();
        uint4 xv[C];
        // Magnitudes are in the order of their bit patterns, infinities and NaN above all.
        uint32_t m2 = 0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            xv[j] = threadIdx.x + j * blockDim.x < nch ? ring.read(0, j) : make_uint4(0, 0, 0, 0);
            m2 = fp4_absmax(fp4_absmax(fp4_absmax(fp4_absmax(m2, xv[j].x), xv[j].y), xv[j].z), xv[j].w);
        }
        float most[1] = {__uint_as_float(max(m2 & 0xffffu, m2 >> 16) << 16)};
        block_join<0, true>(most, places[turn]);
        const Int8Scale s = int8_scale(most[0]);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c >= nch) continue;
            float v[8];
            widen(xv[j], v);
            *reinterpret_cast<uint2*>(a.q + row * a.q_stride + c * 8) = int8_codes8(v, s);
        }
        if (threadIdx.x == 0) *reinterpret_cast<float*>(a.q_scale + row * a.q_scale_stride) = s.scale;
    }
}

// A thread's columns of dweight stay in registers over the rows of its block; the rows
// themselves are read from the ring twice. TEAMS: rows of a block at a time, each a warp's
// (rows of up to 512 values), or 1.
template <int C, int TEAMS>
__global__ void __launch_bounds__(1024) norm_grad_kernel(const NormGradArgs a) {
    pdl_wait_then_release();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float places[2][4][32];
    const int nch = a.H / 8;
    const int team = TEAMS > 1 ? threadIdx.x >> 5 : 0, tid = TEAMS > 1 ? threadIdx.x & 31 : threadIdx.x;
    const int per = TEAMS > 1 ? 32 : blockDim.x;  // threads of a row
    Ring<3, kDepth, C> ring(smem, nch, tid, per);
    const auto fetch = [&](int64_t row, uint32_t ahead) {
        const uint8_t* const rows[3] = {a.h + row * a.h_stride, a.dy + row * a.dy_stride,
                                        a.dsum ? a.dsum + row * a.dsum_stride : nullptr};
        ring.fetch(rows, ahead, row < a.rows);
    };
    const int64_t first = static_cast<int64_t>(blockIdx.x) * TEAMS + team, step = static_cast<int64_t>(gridDim.x) * TEAMS;
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(first + i * step, i);
    float acc[C][8] = {};
    int turn = 0;
    for (int64_t row = first; row < a.rows; row += step, turn ^= 1, ring.next()) {
        float(*place)[32] = places[turn];
        fetch(row + (kDepth - 1) * step, kDepth - 1);
        ring.wait();
        // sum of (h unit)^2 and of weight dy h unit
        const auto add_up = [&](float unit, float (&sums)[2]) {
            sums[0] = sums[1] = 0.f;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int c = tid + j * per;
                if (c >= nch) continue;
                float h[8], b[8], w[8];
                widen(ring.read(0, j), h);
                widen(ring.read(1, j), b);
                widen(__ldg(reinterpret_cast<const uint4*>(a.weight) + c), w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = h[i] * unit;
                    sums[0] = fmaf(v, v, sums[0]);
                    sums[1] = fmaf(b[i] * w[i], v, sums[1]);
                }
            }
        };
        float sums[2];
        add_up(1.f, sums);
        block_join<2, false, (TEAMS > 1)>(sums, place);
        const float mean = __fdiv_rn(sums[0], static_cast<float>(a.H)) + a.eps;
        float rstd = __frsqrt_rn(mean);
        float back = sums[1] / static_cast<float>(a.H) * rstd * rstd;
        if (!(mean <= kFloatMax)) {  // past binary32: all in h 2^-90, as in far_rstd()
            add_up(kFarUnit, sums);
            block_join<2, false, (TEAMS > 1)>(sums, place + 2);
            rstd = __frsqrt_rn(__fdiv_rn(sums[0], static_cast<float>(a.H)) + a.eps * kFarUnit * kFarUnit);
            back = sums[1] / static_cast<float>(a.H) * rstd * rstd * kFarUnit;
            rstd *= kFarUnit;
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = tid + j * per;
            if (c >= nch) continue;
            float h[8], b[8], w[8], d[8] = {};
            widen(ring.read(0, j), h);
            widen(ring.read(1, j), b);
            widen(__ldg(reinterpret_cast<const uint4*>(a.weight) + c), w);
            if (a.dsum) widen(ring.read(2, j), d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[j][i] = fmaf(b[i], h[i] * rstd, acc[j][i]);
                d[i] = fmaf(rstd, fmaf(-h[i], back, b[i] * w[i]), d[i]);
            }
            *reinterpret_cast<uint4*>(a.dh + row * a.dh_stride + c * 16) = narrow(d);
        }
    }
    if (a.parts == nullptr) return;
    float* out = a.parts + static_cast<int64_t>(blockIdx.x) * a.H;
    if (TEAMS > 1) {  // the teams' sums, in ascending order
        float* sums = reinterpret_cast<float*>(smem);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int j = 0; j < C; ++j)
            if (tid + j * per < nch)
#pragma unroll
                for (int i = 0; i < 8; ++i) sums[team * a.H + (tid + j * per) * 8 + i] = acc[j][i];
        __syncthreads();
        for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
            float s = 0.f;
            for (int k = 0; k < TEAMS; ++k) s += sums[k * a.H + c];
            out[c] = s;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c = tid + j * per;
        if (c >= nch) continue;
        reinterpret_cast<float4*>(out + c * 8)[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        reinterpret_cast<float4*>(out + c * 8)[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
    }
}

// The blocks' sums of the weight's gradient: 32 columns a block, 32 threads a column,
// each every 32nd sum in ascending order, joined in ascending order.
__global__ void __launch_bounds__(1024) norm_join_kernel(const float* parts, int n, int32_t H, float* dweight) {
    pdl_wait_then_release();
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, first = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < H)
        for (int b = first; b < n; b += 32) s += parts[static_cast<int64_t>(b) * H + c];
    sums[first][lane] = s;
    __syncthreads();
    if (first != 0 || c >= H) return;
    s = 0.f;
    for (int b = 0; b < 32; ++b) s += sums[b][lane];
    dweight[c] = s;
}

// codes * scale, rounded to bf16. A row is a warp's, 8 codes at a time a lane's.
__global__ void __launch_bounds__(256) unpack_kernel(const NormArgs a) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pieces = a.H / 8;
    int64_t row = blockIdx.x, step = gridDim.x, end = a.rows;
    if (a.plan) {
        if (!plan_rows(a, row, end)) return;
        step = kPlanParts;
    }
    for (row += warp * step; row < end; row += 8 * step) {
        const int64_t to = a.gated ? row / a.group_rows * a.group_rows + fp4_gated_row(row % a.group_rows, a.group_rows) : row;
        const float s = __ldg(reinterpret_cast<const float*>(a.q_scale + row * a.q_scale_stride));
        const uint2* q = reinterpret_cast<const uint2*>(a.q + row * a.q_stride);
        uint4* y = reinterpret_cast<uint4*>(a.y + to * a.y_stride);
        constexpr int kAhead = 4;
        for (int c = lane; c < pieces; c += 32 * kAhead) {
            uint2 v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (c + 32 * u < pieces) v[u] = __ldg(q + c + 32 * u);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (c + 32 * u >= pieces) break;
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = s * static_cast<float>(static_cast<int8_t>((i < 4 ? v[u].x : v[u].y) >> (8 * (i & 3))));
                y[c + 32 * u] = narrow(f);
            }
        }
    }
}

// Threads of a row's block with up to `most` chunks for each of them, and how many they have. Rows of up to 1024 values are a block
// of one warp (norm to bf16: 65536 x 1024 50 us, 5.3 TB/s; 262144 x 128, where half the lanes have none, 57 us, 2.4 TB/s).
unsigned row_threads(int32_t H, int most) { return 32u * static_cast<unsigned>(ceil_div(ceil_div(H / 8, most), 32)); }
int row_chunks(int32_t H, int most) { return static_cast<int>(ceil_div(H / 8, row_threads(H, most))); }

// The blocks of a row kernel that are resident at once (in *blocks), with the ring's shared memory allowed.
cudaError_t resident_blocks(const void* kernel, size_t smem, unsigned threads, int64_t* blocks) {
    int per_sm = 0;
    const cudaError_t e = prepare_kernel(kernel, smem, static_cast<int>(threads), &per_sm);
    *blocks = static_cast<int64_t>(device_sm_count()) * (per_sm > 0 ? per_sm : 1);
    return e;
}

size_t ring_bytes(int in, int depth, int chunks, unsigned threads) { return static_cast<size_t>(in) * depth * chunks * threads * 16; }

}  // namespace

// Most chunks of 16 bytes that a thread has of a row. The norm's are the same whatever results are asked
// for, and so are their bits. The gradient has more to do with each: 32768 x 7168 330 us with 2, 345 with 4.
constexpr int kChunks = 4, kGradChunks = 2;

cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t stream) {
    if (a.rows == 0) return cudaSuccess;
    const int c = row_chunks(a.H, kChunks);
    const unsigned threads = row_threads(a.H, kChunks);
    const auto kernel = a.q ? (c <= 1   ? norm_kernel<1, true>
                               : c == 2 ? norm_kernel<2, true>
                               : c == 3 ? norm_kernel<3, true>
                                        : norm_kernel<4, true>)
                            : (c <= 1   ? norm_kernel<1, false>
                               : c == 2 ? norm_kernel<2, false>
                               : c == 3 ? norm_kernel<3, false>
                                        : norm_kernel<4, false>);
    const size_t smem = ring_bytes(2, a.q ? kDepth : kPlainDepth, c, threads);
    int64_t blocks = 0;
    const cudaError_t e = resident_blocks(reinterpret_cast<const void*>(kernel), smem, threads, &blocks);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, static_cast<unsigned>(a.rows < blocks ? a.rows : blocks), threads, smem, stream, a);
}

cudaError_t launch_int8_pack(const NormArgs& a, cudaStream_t stream) {
    if (a.rows == 0 || (a.plan && a.tile_cap == 0)) return cudaSuccess;
    const int c = row_chunks(a.H, kChunks);
    const unsigned threads = row_threads(a.H, kChunks);
    const auto kernel = c <= 1 ? pack_kernel<1> : c == 2 ? pack_kernel<2> : c == 3 ? pack_kernel<3> : pack_kernel<4>;
    const size_t smem = ring_bytes(1, kDepth, c, threads);
    int64_t blocks = 0;
    const cudaError_t e = resident_blocks(reinterpret_cast<const void*>(kernel), smem, threads, &blocks);
    if (e != cudaSuccess) return e;
    if (a.plan) blocks = static_cast<int64_t>(a.tile_cap) * kPlanParts;
    return launch_pdl(kernel, static_cast<unsigned>(!a.plan && a.rows < blocks ? a.rows : blocks), threads, smem, stream, a);
}

cudaError_t launch_int8_unpack(const NormArgs& a, cudaStream_t stream) {
    if (a.rows == 0 || (a.plan && a.tile_cap == 0)) return cudaSuccess;
    const int64_t eights = ceil_div(a.rows, 8), blocks = a.plan ? static_cast<int64_t>(a.tile_cap) * kPlanParts : eights;
    return launch_pdl(unpack_kernel, static_cast<unsigned>(blocks < (1 << 30) ? blocks : (1 << 30)), 256u, 0, stream, a);
}

cudaError_t launch_rms_norm_grad(const NormGradArgs& a, float* dweight, cudaStream_t stream) {
    int64_t blocks = 0;
    if (a.rows > 0) {
        constexpr int kTeams = 8;
        const int c = row_chunks(a.H, kGradChunks);
        const unsigned threads = row_threads(a.H, kGradChunks);
        const bool teams = threads == 32;
        const auto kernel = teams ? (c <= 1 ? norm_grad_kernel<1, kTeams> : norm_grad_kernel<2, kTeams>)
                                  : (c <= 1 ? norm_grad_kernel<1, 1> : norm_grad_kernel<2, 1>);
        const unsigned block = teams ? 32 * kTeams : threads;
        const size_t smem = ring_bytes(3, kDepth, c, block);
        cudaError_t e = resident_blocks(reinterpret_cast<const void*>(kernel), smem, block, &blocks);
        if (e != cudaSuccess) return e;
        const int64_t need = ceil_div(a.rows, teams ? kTeams : 1);
        if (blocks > kNormParts) blocks = kNormParts;
        if (blocks > need) blocks = need;
        e = launch_pdl(kernel, static_cast<unsigned>(blocks), block, smem, stream, a);
        if (e != cudaSuccess) return e;
    }
    if (dweight == nullptr) return cudaSuccess;
    return launch_pdl(norm_join_kernel, static_cast<unsigned>(ceil_div(a.H, 32)), 1024u, 0, stream,
                      static_cast<const float*>(a.parts), static_cast<int>(blocks), a.H, dweight);
}

}  // namespace moe
