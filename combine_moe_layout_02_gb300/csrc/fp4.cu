// fp4.cu -- MXFP4 rows: packing and unpacking (moe_fp4_pack, moe_fp4_unpack),
// the experts' row tiles (moe_expert_plan) and the expert-major dispatch that
// packs on the way (moe_dispatch_expert_fp4). Format and layout: fp4.cuh.
#include <cuda_bf16.h>

#include "fp4.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Packing and unpacking. The unit of work is one scale chunk: 128 rows x 128
// elements, one CTA of 256 threads. Eight threads share a row's 128 elements
// (16 each, half a block), and a thread takes rows r, r + 32, r + 64 and
// r + 96, whose scale words are the 16 bytes at r * 16 of the chunk.
//
// Bound by memory: 2 bytes in and 17/32 out per element, or the reverse. 128 bytes
// of loads per thread in flight; registers for three CTAs per SM (packing and
// unpacking 32768 x 7168 one after the other: 193 us; for two 200, for five 207,
// left to the compiler 209). Packing 32768 x 7168: 90 us, 6.6 TB/s; unpacking 105 us,
// 5.7 TB/s.

constexpr int kPackThreads = 256;

struct PackArgs {
    int64_t rows;        // rows per group (plain mode) or of the arena (plan mode)
    int32_t groups, width, gated;
    uint16_t* x;         // read by pack, written by unpack
    int64_t x_stride;    // bytes
    uint8_t* q;
    uint8_t* sf;
    const int32_t* plan;  // NULL: every row
    int32_t E, tile_cap;
};

// The rows of a unit: `n` of them from packed row `row0` of group `group`.
struct PackTile {
    int64_t group, row0;
    int32_t n;
};

__device__ __forceinline__ PackTile pack_tile(const PackArgs& a, int64_t t, int64_t tiles_per_group) {
    PackTile o;
    if (a.plan == nullptr) {
        o.group = t / tiles_per_group;
        o.row0 = (t - o.group * tiles_per_group) * kFp4Tile;
        const int64_t left = a.rows - o.row0;
        o.n = static_cast<int32_t>(left < kFp4Tile ? left : kFp4Tile);
        return o;
    }
    const int4 p = __ldg(reinterpret_cast<const int4*>(a.plan + plan_tiles_at(a.E)) + t / 2);
    const int half = static_cast<int>(t & 1) * kFp4Tile;
    o.group = 0;
    o.row0 = static_cast<int64_t>(p.y) + half;
    o.n = p.z - half;
    o.n = o.n < 0 ? 0 : (o.n > kFp4Tile ? kFp4Tile : o.n);
    // a plan that does not belong to this arena names no row of it
    if (p.y < 0 || p.y % kFp4Tile != 0 || o.row0 + o.n > a.rows) o.n = 0;
    return o;
}

__device__ __forceinline__ int64_t pack_units(const PackArgs& a, int64_t tiles_per_group, int64_t chunks) {
    if (a.plan == nullptr) return a.groups * tiles_per_group * chunks;
    int32_t n = __ldg(a.plan);
    n = n < 0 ? 0 : (n > a.tile_cap ? a.tile_cap : n);
    return 2 * static_cast<int64_t>(n) * chunks;
}

template <bool UNPACK>
__global__ void __launch_bounds__(kPackThreads, 3) pack_kernel(const PackArgs a) {
    pdl_wait_then_release();
    const int tid = threadIdx.x;
    const int r = tid >> 3, part = tid & 7;  // row of each quarter, part of its 128 elements
    const int64_t chunks = ceil_div(a.width, kFp4Chunk);
    const int64_t tiles_per_group = ceil_div(a.rows, kFp4Tile);
    const int64_t units = pack_units(a, tiles_per_group, chunks);
    const int half_width = a.width / 2;
    // Unit u is chunk c of tile t; the next one, gridDim.x further, without a division.
    const int64_t dt = gridDim.x / chunks, dc = gridDim.x - dt * chunks;
    int64_t t = blockIdx.x / chunks, c = blockIdx.x - t * chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x, t += dt, c += dc) {
        if (c >= chunks) {
            c -= chunks;
            ++t;
        }
        const PackTile tile = pack_tile(a, t, tiles_per_group);
        if (tile.n == 0) continue;  // the same for the whole block
        uint8_t* chunk = a.sf + ((tile.group * tiles_per_group + tile.row0 / kFp4Tile) * chunks + c) * kFp4ChunkBytes;
        // This thread's rows are 32 apart in the operand, and in x: 16 in gate / up order.
        const int64_t first = tile.row0 + r;
        const int left = tile.n - r;  // row p of the thread is in if 32 p < left
        const int col = static_cast<int>(c) * kFp4Chunk + part * (UNPACK ? 8 : 16);
        uint8_t* qp = a.q + (tile.group * a.rows + first) * half_width + col / 2;
        uint8_t* xp = reinterpret_cast<uint8_t*>(a.x) +
                      (tile.group * a.rows + (a.gated ? fp4_gated_row(first, a.rows) : first)) * a.x_stride + col * 2;
        const int64_t xstep = (a.gated ? 16 : 32) * a.x_stride;
        const int64_t qstep = 32 * static_cast<int64_t>(half_width);
        if (UNPACK) {
            // 8 elements at 8 * part and 8 more 64 on: the eight threads of a
            // row write 128 bytes side by side each time.
            const uint4 words = __ldg(reinterpret_cast<const uint4*>(chunk) + r);
            const uint32_t w[4] = {words.x, words.y, words.z, words.w};
            const bool in[2] = {col < a.width, col + 64 < a.width};
            uint32_t q[4][2];
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    q[p][h] = 32 * p < left && in[h] ? __ldg(reinterpret_cast<const uint32_t*>(qp + p * qstep + 32 * h)) : 0u;
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (32 * p >= left || !in[h]) continue;
                    // every value is a bf16 value: at most 2 significant bits, from 2^-128 on
                    const __nv_bfloat162 s = fp4_scale_pair((w[p] >> (8 * (2 * h + (part >> 2)))) & 255u);
                    *reinterpret_cast<uint4*>(xp + p * xstep + 128 * h) = fp4_values8(q[p][h], s);
                }
        } else {
            const bool in = col < a.width;  // a multiple of 32: a block is in or out as a whole
            uint4 v[4][2];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                v[p][0] = v[p][1] = make_uint4(0u, 0u, 0u, 0u);
                if (32 * p < left && in) {
                    const uint4* s = reinterpret_cast<const uint4*>(xp + p * xstep);
                    v[p][0] = __ldg(s);
                    v[p][1] = __ldg(s + 1);
                }
            }
            uint32_t mine = 0;  // this thread's block's scale codes, byte p for row r + 32 p
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                uint32_t m2 = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    m2 = fp4_absmax(m2, v[p][h].x);
                    m2 = fp4_absmax(m2, v[p][h].y);
                    m2 = fp4_absmax(m2, v[p][h].z);
                    m2 = fp4_absmax(m2, v[p][h].w);
                }
                m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
                const uint32_t most = max(m2 & 0xffffu, m2 >> 16);
                const uint32_t s = fp4_scale_code(most);
                mine |= s << (8 * p);
                if (32 * p < left && in) {
                    const float inv = fp4_inverse(s);
                    *reinterpret_cast<uint2*>(qp + p * qstep) =
                        make_uint2(fp4_codes8(v[p][0], inv), fp4_codes8(v[p][1], inv));
                }
            }
            // The row's word of quarter p holds the four blocks' codes: thread
            // pair p of the row's eight threads gathers byte p of each.
            const int p = part >> 1, lane0 = (tid & 31) & ~7;
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                word |= ((__shfl_sync(0xffffffffu, mine, lane0 + 2 * j) >> (8 * p)) & 255u) << (8 * j);
            if ((part & 1) == 0) *reinterpret_cast<uint32_t*>(chunk + r * 16 + p * 4) = word;
        }
    }
}

template <bool UNPACK>
cudaError_t launch_pack_t(const PackArgs& a, int64_t units_max, cudaStream_t stream) {
    if (units_max <= 0) return cudaSuccess;
    int per_sm = 0;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(pack_kernel<UNPACK>), 0, kPackThreads, &per_sm);
    if (e != cudaSuccess) return e;
    int64_t grid = static_cast<int64_t>(device_sm_count()) * (per_sm < 1 ? 1 : per_sm);
    if (grid > units_max) grid = units_max;
    return launch_pdl(pack_kernel<UNPACK>, static_cast<unsigned>(grid), kPackThreads, 0, stream, a);
}

// ---------------------------------------------------------------------------
// The experts' row tiles: one CTA, a thread per expert (several from 1024 on), no
// more threads than the experts need. A thread sums its expert's counts over the
// source ranks; then first rows and tile numbers are exclusive scans. Latency-bound:
// 8 ranks of 256 experts 2.2 us, 64 3.7, 128 5.2, 1024 of 1024 33. (1024 threads with
// the ranks split among those that the experts leave over, joined by shared atomics:
// 3.3, 5.7, 8.5 and 178.)

constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(int32_t P, int32_t E, int32_t align, int64_t max_slots, const int32_t* __restrict__ ntpe,
            int32_t* __restrict__ plan, int32_t tile_cap, int32_t* __restrict__ err) {
    pdl_wait_then_release();
    extern __shared__ __align__(16) int32_t sm_plan[];
    int32_t* counts = sm_plan;                     // [E]
    __shared__ int64_t row_part[32];
    __shared__ int32_t tile_part[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int threads = blockDim.x;
    // Thread t scans experts [t * per, (t + 1) * per).
    const int per = (E + threads - 1) / threads;
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e >= E) break;
        int32_t sum = 0;
#pragma unroll 8
        for (int s = 0; s < P; ++s) sum += __ldg(ntpe + static_cast<int64_t>(s) * E + e);
        counts[e] = sum;  // read by this thread only
    }
    int64_t rows = 0;
    int32_t tiles = 0;
    bool bad = false;
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e >= E) break;
        int32_t n = counts[e];
        if (n < 0 || n > max_slots) {  // not counts of this shape
            bad = true;
            counts[e] = n = 0;
        }
        rows += round_up(n, align);
        tiles += (n + kPlanTileRows - 1) / kPlanTileRows;
    }
    int64_t rincl = rows;
    int32_t tincl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ru = __shfl_up_sync(0xffffffffu, rincl, o);
        const int32_t tu = __shfl_up_sync(0xffffffffu, tincl, o);
        if (lane >= o) {
            rincl += ru;
            tincl += tu;
        }
    }
    if (lane == 31) {
        row_part[warp] = rincl;
        tile_part[warp] = tincl;
    }
    __syncthreads();
    if (warp == 0) {
        int64_t r = lane < threads / 32 ? row_part[lane] : 0;
        int32_t t = lane < threads / 32 ? tile_part[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t ru = __shfl_up_sync(0xffffffffu, r, o);
            const int32_t tu = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) {
                r += ru;
                t += tu;
            }
        }
        row_part[lane] = r;
        tile_part[lane] = t;
    }
    __syncthreads();
    // More rows than any routing of the shape needs: no plan. Else rows fit 32 bits (the
    // shape's own rule), and so do tile numbers.
    const bool none = row_part[31] > max_slots + static_cast<int64_t>(E) * (align - 1);
    bad |= none;
    int64_t row = none ? 0 : rincl - rows + (warp ? row_part[warp - 1] : 0);
    int32_t tile = none ? 0 : tincl - tiles + (warp ? tile_part[warp - 1] : 0);
    int4* list = reinterpret_cast<int4*>(plan + plan_tiles_at(E));
    const int e4 = static_cast<int>(round_up(E, 4));
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e >= E) break;
        const int32_t n = none ? 0 : counts[e];
        plan[4 + e] = static_cast<int32_t>(row);
        plan[4 + e4 + e] = n;
        for (int32_t at = 0; at < n; at += kPlanTileRows, ++tile) {
            if (tile >= tile_cap) {
                bad = true;
                break;
            }
            list[tile] = make_int4(e, static_cast<int32_t>(row + at), n - at < kPlanTileRows ? n - at : kPlanTileRows, 0);
        }
        row += round_up(n, align);
    }
    if (bad) raise_error(err, MOE_ERR_INCONSISTENT);
    if (tid == 0) {
        plan[0] = none ? 0 : tile_part[31] < tile_cap ? tile_part[31] : tile_cap;
        plan[1] = none ? 0 : static_cast<int32_t>(row_part[31]);
        plan[2] = E;
        plan[3] = 0;
    }
}

// ---------------------------------------------------------------------------
// Expert-major dispatch with an MXFP4 payload. The unit of work is a token, or
// a part of its columns when there are few tokens, and a warp takes one at a
// time: the columns are read once and rounded once, whatever the number of the
// token's slots; the packed columns are staged in shared memory and sent with
// one bulk store per slot, the scale words go straight to the slots' chunks.
//
// Bound by memory: S rows of 2H bytes in, a packed row per slot out. Measured (8
// slots per token, H = 7168): 4096 tokens 36 us, 5.1 TB/s; 32768 tokens 299 us, 4.9
// TB/s (331 before the scale words were kept in L2; without them at all 226: 4-byte
// words are what is left).

constexpr int kFp4DispatchWarps = 8;
// Units of work that every warp should have (8 slots, H = 7168, in a graph: 64 tokens
// 4.0 us, whole tokens 12.5; 2048 20.8 us, one unit per warp 21.4, four 30.7; 4096 35.7,
// 42.9 and 42.3; 1024 16.8, 11.6 and 16.8: one is better there alone).
constexpr int kFp4DispatchRounds = 2;

struct Fp4DispatchArgs {
    int32_t P, E, K, H, epr;
    int64_t S, T;
    const uint16_t* x;
    const int32_t* topk_idx;
    const float* topk_weights;
    const int32_t* slot_row;
    const int64_t* part_row_base;
    uint8_t* q;
    uint8_t* sf;
    int64_t arena_rows;
    int32_t* recv_src_idx;
    float* recv_weight;
    int32_t* err;
    int32_t qbytes, swords;  // packed row bytes, scale words per row
    int32_t keep_scales;
    int32_t parts, part_cols;  // parts of a token, columns of each (a multiple of 512; the last one's may be fewer)
};

// Staged codes and scale words of a part.
__host__ __device__ __forceinline__ size_t fp4_stage_bytes(int32_t cols) {
    return static_cast<size_t>(cols / 2 + cols / kFp4Chunk * 4);
}

__global__ void __launch_bounds__(kFp4DispatchWarps * 32) dispatch_fp4_kernel(const Fp4DispatchArgs a) {
    pdl_wait_then_release();
    extern __shared__ __align__(128) unsigned char smem_d4[];
    int64_t* prb = reinterpret_cast<int64_t*>(smem_d4);
    const size_t stage = fp4_stage_bytes(a.part_cols);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char* own = smem_d4 + round_up((a.P + 1) * 8, 128) + 2 * stage * warp;
    for (int i = threadIdx.x; i <= a.P; i += blockDim.x) prb[i] = a.part_row_base[i];
    __syncthreads();
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kFp4DispatchWarps;
    int buf = 0;
    // A sector of scales holds words of 8 rows, which come from tokens thousands
    // apart: asked to stay in L2, it is whole before it goes to memory. Only where
    // the call moves more than L2 holds: below that the request costs more than
    // it saves (512 tokens of 7168: 11.8 us with it, 9.9 without; 4096: 37 and 45).
    uint64_t keep;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
    const int64_t units = a.S * a.parts;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kFp4DispatchWarps + warp; u < units; u += warps) {
        const int64_t g = u / a.parts;
        const int part = static_cast<int>(u - g * a.parts);
        const int col0 = part * a.part_cols, cols = min(a.part_cols, a.H - col0);
        // Lane k < K: slot k's row, or -1.
        int64_t row = -1;
        if (lane < a.K) {
            const int32_t e = __ldg(a.topk_idx + g * a.K + lane);
            const int32_t sr = __ldg(a.slot_row + g * a.K + lane);
            if (e >= 0 && e < a.E && sr >= 0) {
                const int64_t lo = prb[e / a.epr], hi = prb[e / a.epr + 1];
                row = lo + sr;
                if (sr >= hi - lo || row < 0 || row >= a.arena_rows) {
                    raise_error(a.err, MOE_ERR_CAPACITY);
                    row = -1;
                }
            }
        }
        uint32_t live = __ballot_sync(0xffffffffu, row >= 0);
        if (live == 0) continue;
        unsigned char* q = own + buf * stage;
        uint32_t* words = reinterpret_cast<uint32_t*>(q + a.part_cols / 2);
        bulk_wait_read<1>();  // the stores of two tokens ago have read this buffer
        __syncwarp();
        const uint16_t* x = a.x + g * a.H + col0;
        const int swords = (cols + kFp4Chunk - 1) / kFp4Chunk;
#pragma unroll 2
        for (int c0 = 0; c0 < cols; c0 += 512) {
            const int col = c0 + lane * 16;
            uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
            if (col < cols) {
                v0 = __ldg(reinterpret_cast<const uint4*>(x + col));
                v1 = __ldg(reinterpret_cast<const uint4*>(x + col) + 1);
            }
            uint32_t m2 = fp4_absmax(fp4_absmax(fp4_absmax(fp4_absmax(0u, v0.x), v0.y), v0.z), v0.w);
            m2 = fp4_absmax(fp4_absmax(fp4_absmax(fp4_absmax(m2, v1.x), v1.y), v1.z), v1.w);
            m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
            const uint32_t s = fp4_scale_code(max(m2 & 0xffffu, m2 >> 16));
            if (col < cols) {
                const float inv = fp4_inverse(s);
                *reinterpret_cast<uint2*>(q + col / 2) = make_uint2(fp4_codes8(v0, inv), fp4_codes8(v1, inv));
            }
            // Eight lanes cover a chunk's four blocks: its word (0 past the width).
            uint32_t word = s << (8 * ((lane >> 1) & 3));
            word |= __shfl_xor_sync(0xffffffffu, word, 2);
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
            const int c = (c0 >> 7) + (lane >> 3);
            if ((lane & 7) == 0 && c < swords) words[c] = word;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (row >= 0) {
            bulk_store(a.q + row * a.qbytes + col0 / 2, q, static_cast<uint32_t>(cols / 2));
            if (part == 0 && a.recv_src_idx) a.recv_src_idx[row] = static_cast<int32_t>(g % a.T);
            if (part == 0 && a.recv_weight) a.recv_weight[row] = a.topk_weights ? __ldg(a.topk_weights + g * a.K + lane) : 1.f;
        }
        bulk_commit();
        while (live) {
            const int k = __ffs(live) - 1;
            live &= live - 1;
            const int64_t dst = __shfl_sync(0xffffffffu, row, k);
            uint8_t* base = a.sf + ((dst / kFp4Tile) * a.swords + col0 / kFp4Chunk) * kFp4ChunkBytes +
                            fp4_word_at(static_cast<int>(dst % kFp4Tile));
            if (a.keep_scales) {
                for (int c = lane; c < swords; c += 32)  // nothing here reads what this stores
                    asm volatile("st.global.L2::cache_hint.u32 [%0], %1, %2;" ::"l"(base + static_cast<int64_t>(c) * kFp4ChunkBytes),
                                 "r"(words[c]), "l"(keep));
            } else {
                for (int c = lane; c < swords; c += 32)
                    *reinterpret_cast<uint32_t*>(base + static_cast<int64_t>(c) * kFp4ChunkBytes) = words[c];
            }
        }
        __syncwarp();
        buf ^= 1;
    }
    bulk_wait<0>();
}

}  // namespace

cudaError_t launch_fp4_pack(bool unpack, int32_t groups, int64_t rows, int32_t width, int32_t gated, uint16_t* x,
                            int64_t x_stride, uint8_t* q, uint8_t* sf, const int32_t* plan, int32_t E,
                            int64_t plan_ints, cudaStream_t stream) {
    PackArgs a{};
    a.rows = rows;
    a.groups = groups;
    a.width = width;
    a.gated = gated;
    a.x = x;
    a.x_stride = x_stride;
    a.q = q;
    a.sf = sf;
    a.plan = plan;
    a.E = E;
    a.tile_cap = plan ? plan_capacity(E, plan_ints) : 0;
    const int64_t tiles = plan ? 2 * static_cast<int64_t>(a.tile_cap) : groups * ceil_div(rows, kFp4Tile);
    const int64_t units = tiles * ceil_div(width, kFp4Chunk);
    return unpack ? launch_pack_t<true>(a, units, stream) : launch_pack_t<false>(a, units, stream);
}

cudaError_t launch_expert_plan(const moe_shape& s, const int32_t* ntpe, int32_t* plan, int64_t plan_ints, int32_t* err,
                               cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(s.E) * 4;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(plan_kernel), smem, kPlanThreads, nullptr);
    if (e != cudaSuccess) return e;
    const int64_t threads = s.E < kPlanThreads ? round_up(s.E, 32) : kPlanThreads;
    return launch_pdl(plan_kernel, 1u, static_cast<unsigned>(threads), smem, stream, s.P, s.E, s.expert_alignment,
                      static_cast<int64_t>(s.S) * s.K, ntpe, plan, plan_capacity(s.E, plan_ints), err);
}

cudaError_t launch_dispatch_fp4(const moe_shape& s, const uint16_t* x, const int32_t* topk_idx, const float* topk_weights,
                                const int32_t* slot_row, const int64_t* part_row_base, uint8_t* q, uint8_t* sf,
                                int64_t arena_rows, int32_t* recv_src_idx, float* recv_weight, int32_t* err,
                                cudaStream_t stream) {
    if (s.S == 0) return cudaSuccess;
    Fp4DispatchArgs a{};
    a.P = s.P;
    a.E = s.E;
    a.K = s.K;
    a.H = s.H;
    a.epr = s.E / s.P;
    a.S = s.S;
    a.T = s.S / s.P;
    a.x = x;
    a.topk_idx = topk_idx;
    a.topk_weights = topk_weights;
    a.slot_row = slot_row;
    a.part_row_base = part_row_base;
    a.q = q;
    a.sf = sf;
    a.arena_rows = arena_rows;
    a.recv_src_idx = recv_src_idx;
    a.recv_weight = recv_weight;
    a.err = err;
    a.qbytes = s.H / 2;
    a.swords = static_cast<int32_t>(ceil_div(s.H, kFp4Chunk));
    const int64_t moved = static_cast<int64_t>(s.S) * (2 * s.H + static_cast<int64_t>(s.K) * a.qbytes);
    a.keep_scales = moved > device_l2_bytes();
    // Parts: halve the columns while every warp of the device would have fewer than
    // kFp4DispatchRounds of them.
    const int64_t blocks512 = ceil_div(s.H, 512);
    const int64_t warps = static_cast<int64_t>(device_sm_count()) * 4 * kFp4DispatchWarps;
    int64_t parts = 1;
    while (parts < blocks512 && s.S * parts < kFp4DispatchRounds * warps) parts *= 2;
    a.part_cols = static_cast<int32_t>(ceil_div(blocks512, parts) * 512);
    a.parts = static_cast<int32_t>(ceil_div(s.H, a.part_cols));
    const size_t smem = static_cast<size_t>(round_up((s.P + 1) * 8, 128)) + 2 * fp4_stage_bytes(a.part_cols) * kFp4DispatchWarps;
    int per_sm = 0;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(dispatch_fp4_kernel), smem, kFp4DispatchWarps * 32, &per_sm);
    if (e != cudaSuccess) return e;
    int64_t grid = static_cast<int64_t>(device_sm_count()) * (per_sm < 1 ? 1 : per_sm);
    const int64_t need = ceil_div(s.S * a.parts, kFp4DispatchWarps);
    if (grid > need) grid = need;
    return launch_pdl(dispatch_fp4_kernel, static_cast<unsigned>(grid), kFp4DispatchWarps * 32, smem, stream, a);
}

}  // namespace moe
