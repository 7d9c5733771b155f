// product.cu -- the experts' grouped product of MXFP4 operands
// (moe_expert_product_fp4): for every row r of expert e,
//   v[r][n] = sum over k of w_e[n][k] * x[r][k]
//   y[r] = bf16_rne(v[r]), or, gated, bf16_rne(silu(gate) * up) of the pairs.
//
// Tensor cores, tcgen05.mma kind::mxf4 with block scales: a pair of CTAs (one
// per SM) computes 256 weight rows x up to 256 of an expert's rows. The
// weights are the M side and the rows the N side, because N goes in steps of
// 32 down to 32: an expert with two rows costs a thin instruction, not a tile
// that is mostly padding, and the last tile of a long expert is cut to size.
// Each CTA holds its 128 weight rows, half of the rows (the pair shares them:
// every row is fetched into shared memory once per pair) and the scales.
//
// Warp 0 loads (TMA, 256 elements of K per stage, a ring of stages shared by
// the pair: both CTAs' bytes count on the leading CTA's barrier), warp 1 of the
// leading CTA copies the stage's scales to tensor memory and issues its four
// products of K = 64, warps 4-11 of both CTAs take the sums out of tensor
// memory (128 lanes = the CTA's weight rows, columns = the expert's rows),
// turn them with transposing matrix stores in shared memory and write 64 bytes
// (gated: 32) of a row per warp. Sums have two places in tensor memory, columns
// 0 and 224 on, so that a tile's sums are written while the next tile's are
// formed; two places of 256 columns and the scales' 24 would not fit the 512,
// so the places share 32 columns, which are read first and given back early.
//
// Bound by the weights' bytes while experts have few rows (64 tokens over 256
// experts of 7168 -> 4096: 506 us, 6.9 TB/s), by power and the SMs' intake when they
// have many: 256 x 256 x 64 takes the pair 128 cycles, a stage 512, and brings
// each SM 35 KB, 560 cycles at its 64 bytes per cycle (262144 rows: 2.53 ms, 6.1
// PFLOP/s at 1.55 GHz). A pair is the smallest tile that keeps the intake near the
// tensor pipe's pace; 256 columns are the widest instruction. Where rows of codes are
// no multiple of 128 bytes each load touches two lines of L2: 44800 rows 5984 -> 2048
// 226 us, 7168 -> 2048 214.
#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>

#include "fp4.cuh"

namespace moe {
namespace {

constexpr int kEpiWarps = 8;                 // two for each quarter of tensor memory's lanes
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kStages = 6;
constexpr int kMTile = 256;                  // weight rows of a CTA pair
constexpr int kStageK = 256;                 // elements of K per stage: one 128-byte swizzle row
constexpr uint32_t kWBytes = 128 * 128;      // a CTA's weight rows of a stage
constexpr uint32_t kXBox = 32 * 128;         // 32 rows of a stage
constexpr uint32_t kXBytes = 4 * kXBox;      // half of 256 rows
constexpr uint32_t kScaleBox = 2 * kFp4ChunkBytes;  // 128 rows' scales of a stage
constexpr uint32_t kOffX = kWBytes, kOffWS = kOffX + kXBytes, kOffXS = kOffWS + kScaleBox;
constexpr uint32_t kStageBytes = kOffXS + 2 * kScaleBox;  // a multiple of 1024
constexpr uint32_t kOutStride = 80;          // bytes per staged row: 64 and a shift of 4 banks per row
constexpr uint32_t kPackStride = 144;         // staged inner row of a CTA before packing: 128 bytes, shifted likewise
constexpr uint32_t kOutBytes = kEpiWarps * 16 * kOutStride;
static_assert(2 * 32 * kPackStride <= kOutBytes, "staging");
constexpr uint32_t kBarBytes = 256;
constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + kOutBytes + kBarBytes;
constexpr int kAcc1 = 224;                   // second place of the sums
constexpr long long kWaitCycles = 1ll << 32;
constexpr int kScaleCol = 480;               // scales of a stage: 8 columns of the weights', 16 of the rows'

struct ProductArgs {
    int32_t E, N, K, tile_cap;
    int64_t rows;
    const int32_t* plan;
    uint16_t* y;
    int64_t y_stride;
    uint8_t* hq;   // kPacked: the inner rows as MXFP4
    uint8_t* hsf;
    int32_t* err;
    int64_t wait_cycles;  // bound of a wait (kWaitCycles)
    int32_t quit_warp;    // test hook: a warp of each CTA that acts as if its first wait had run out, or -1
};

// What becomes of the sums: bf16; silu(gate) * up in bf16; that, packed to MXFP4.
enum ProductMode { kPlain = 0, kGated = 1, kPacked = 2 };

// Barriers of a CTA, and its abort flag.
struct Bars {
    uint64_t full[kStages];   // leading CTA: both CTAs' loads of a stage have landed
    uint64_t empty[kStages];  // each CTA: the products that read a stage are done
    uint64_t acc_full[2];     // each CTA: a tile's sums are complete
    uint64_t acc_empty[2];    // leading CTA: both CTAs have read a place
    uint64_t shared_free;     // leading CTA: both CTAs have read the tile's part of the shared columns
    uint64_t drain;           // leading CTA, after a failed wait: products in flight are done
    uint32_t tmem;
    uint32_t abort;
};
static_assert(sizeof(Bars) <= kBarBytes, "barriers");

// One tile of work.
struct Unit {
    int32_t e, row, n, m0;  // expert, first arena row, rows, first weight row of the pair
};

__device__ __forceinline__ uint32_t mma_n(int32_t rows) { return (rows + 31) & ~31; }

// Arrival on a barrier of the leading CTA. What it hands over is tensor memory that
// has been read (ordered by the tcgen05 fences), not data, so it releases at the
// CTA's scope: at the cluster's it waited for the thread's global stores, about
// a microsecond per tile (128 tokens, 1024 -> 14336: 456 us against 299).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// A wait has run out: the CTA's other roles are told, and the caller.
__device__ __forceinline__ void give_up(Bars* b, const ProductArgs& a) {
    *reinterpret_cast<volatile uint32_t*>(&b->abort) = 1u;
    raise_error(a.err, MOE_ERR_DEVICE_TIMEOUT);
}

// Bounded wait of a whole warp, by polls and by time (about two seconds: a poll
// may itself sleep); false if it ran out or another role of the CTA gave up.
__device__ __forceinline__ bool wait_for(Bars* b, uint64_t* bar, uint32_t parity, const ProductArgs& a) {
    if (__all_sync(0xffffffffu, mbar_try_wait_cluster(bar, parity))) return true;
    const long long began = clock64();
    for (uint32_t i = 0; i < kSpinLimit; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait_cluster(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(&b->abort) != 0u)) return false;
        if (__any_sync(0xffffffffu, clock64() - began > a.wait_cycles)) break;
    }
    give_up(b, a);
    return false;
}

// Whether all 128 threads that meet at barrier `id` say so.
__device__ __forceinline__ bool all_agree(int id, bool yes) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "bar.red.and.pred q, %1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(id), "r"(static_cast<uint32_t>(yes))
        : "memory");
    return all != 0;
}

// After a failed wait: what is in flight ends within microseconds, or (a peer
// gave up first) never.
__device__ __forceinline__ void drained(uint64_t* bar, uint32_t parity) {
    const long long began = clock64();
    while (!__any_sync(0xffffffffu, mbar_try_wait_cluster(bar, parity)) &&
           !__any_sync(0xffffffffu, clock64() - began > kWaitCycles / 64)) {
    }
}

// One lane of a converged warp. The loading and the issuing warp run their
// loops as whole warps on warp-uniform values and only the instructions
// themselves are one lane's: in a branch of one lane the compiler cannot keep
// descriptors in uniform registers, and each product then took about 100
// cycles to issue and each scale copy 80 (of 128 cycles of work; measured).
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

__device__ __forceinline__ int32_t uniform(int32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// TMA tile loads into this CTA's shared memory, counted on the barrier of the
// pair's leading CTA.
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                       uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Shared-memory matrix descriptors: rows of 128 bytes, swizzled, 8 rows to
// 1024 bytes; and scale chunks, 8 lanes of 16 bytes to 128 bytes.
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (8ull << 32) | (1ull << 46);
}

// Instruction descriptor: e2m1 x e2m1, ue8m0 scales, M = 256, N columns, both
// operands K-major; `half` selects which 2 of a word's 4 scales apply.
__device__ __forceinline__ uint32_t instr(uint32_t n, uint32_t half) {
    return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) | (16u << 24) | ((2u * half) << 29) | ((2u * half) << 4);
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                    uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(add)
        : "memory");
}

__device__ __forceinline__ void scales_to_tmem(uint32_t col, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(col), "l"(desc) : "memory");
}

// Arrives on `bar` of both CTAs once every product and copy issued so far is done.
__device__ __forceinline__ void commit_to(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 lanes x 16 columns of tensor memory: v[4 i + j], column 8 i + 2 (lane % 4) + j % 2,
// lane row lane / 4 + 8 (j / 2).
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(addr)
                 : "memory");
}

// Four 8 x 8 blocks of 16-bit values, transposed: lane 8 q + j gives the address
// of the 16 bytes that column j of block q goes to.
__device__ __forceinline__ void store_turned(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// silu(g) * u. e^-|g| <= 1, so nothing overflows and the denominator is in [1, 2].
__device__ __forceinline__ float gate_times_up(float g, float u) {
    const float e = __expf(-fabsf(g));
    return __fdividef(g < 0.f ? g * e : g, 1.f + e) * u;
}

// A pair's units, first, first + step, .. of the launch's. They run through groups of
// GROUP row tiles, the tiles of a group innermost (the rule is at four_tiles).
//
// A role steps from unit to unit without a division and holds the next one's plan
// words while it works on the current one. A unit of few stages is short of the time
// to find the next: 256 experts of a row or so, 512 -> 7008, 62 us against 67 with
// each unit found from its number; at width 256 50 against 51. A unit of a stage
// pays for the step instead (64 experts, 96 -> 4096 gated, 24 us against 23), and
// from width 1024 on the two are within 2%.
template <uint32_t GROUP>
struct Units {
    uint32_t tiles, per, group, in, step_group, step_in, left, m;
    int4 tile;

    __device__ __forceinline__ Units(const ProductArgs& a, uint32_t tiles_, uint32_t mtiles, uint32_t first, uint32_t step)
        : tiles(tiles_), per(mtiles * GROUP), m(0), tile(make_int4(0, 0, 0, 0)) {
        const uint32_t units = tiles * mtiles;
        left = first < units ? (units - first - 1) / step + 1 : 0;
        group = first / per;
        in = first - group * per;
        step_group = step / per;
        step_in = step - step_group * per;
        fetch(a);
    }
    __device__ __forceinline__ void fetch(const ProductArgs& a) {
        if (left == 0) return;
        uint32_t t = group;
        m = in;
        if (GROUP > 1) {
            const uint32_t size = min(GROUP, tiles - group * GROUP);  // the last group may be short
            m = size == GROUP ? in / GROUP : in / size;
            t = group * GROUP + in - m * size;
        }
        tile = __ldg(reinterpret_cast<const int4*>(a.plan + plan_tiles_at(a.E)) + t);
    }
    // The current unit, the same in every lane, or none (n = 0) where the plan's
    // tile is no tile of this arena; then on to the next.
    __device__ __forceinline__ Unit take(const ProductArgs& a) {
        Unit o{uniform(tile.x), uniform(tile.y), uniform(tile.z), static_cast<int32_t>(m) * kMTile};
        if (o.e < 0 || o.e >= a.E || o.row < 0 || o.row % kFp4Tile != 0 || o.n < 0 || o.n > kPlanTileRows ||
            o.row + static_cast<int64_t>(o.n) > a.rows) {
            raise_error(a.err, MOE_ERR_CAPACITY);
            o.n = 0;
        }
        --left;
        group += step_group;
        in += step_in;
        if (in >= per) {
            in -= per;
            ++group;
        }
        fetch(a);
        return o;
    }
};

// kPacked: silu(gate) * up of the CTA's 64 inner columns for the tile's rows,
// rounded to bf16 and then packed as moe_fp4_pack packs it. A block of 32 inner
// columns comes out of two warps, so four warps stage 32 rows in shared memory
// and each of their threads takes half a block. `group`: which of every two
// batches of 32 rows; its four warps meet at barrier 1 + group.
__device__ __forceinline__ void pack_tile_out(const ProductArgs& a, const Unit& t, uint32_t cta, uint32_t acc, int w,
                                              int lane, int group, bool place, unsigned char* stage, Bars* bars,
                                              uint64_t* acc_empty) {
    const int inner = a.N / 2, h0 = t.m0 / 2 + static_cast<int>(cta) * 64;  // the CTA's first inner column
    const int batches = static_cast<int>(mma_n(t.n) / 32);
    const int64_t chunks = ceil_div(inner, kFp4Chunk);
    const uint32_t to = smem_addr(stage) + ((lane & 7) + 8 * (lane >> 4)) * kPackStride + w * 32 + ((lane >> 3) & 1) * 16;
    const int id = w * 32 + lane;  // of the group's 128 threads
    for (int q = group; q < batches; q += 2) {
        const int c = place ? q : batches - 1 - q;
        uint32_t v[2][2][8];  // two halves of 16 columns, gate and up
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            tmem_load(acc + 32 * c + 16 * b, v[b][0]);
            tmem_load(acc + 32 * c + 16 * b + (16u << 16), v[b][1]);
        }
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (q == group) mbar_arrive_cluster(cluster_map(&bars->shared_free, 0));
            if (q + 2 >= batches) mbar_arrive_cluster(cluster_map(acc_empty, 0));
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)  // column block i / 2, inner columns 8 (i % 2) + lane / 4
                h[i] = bf16_pair(gate_times_up(__uint_as_float(v[b][0][2 * i]), __uint_as_float(v[b][1][2 * i])),
                                 gate_times_up(__uint_as_float(v[b][0][2 * i + 1]), __uint_as_float(v[b][1][2 * i + 1])));
            store_turned(to + 16 * b * kPackStride, h[0], h[1], h[2], h[3]);
        }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
        const int r = id >> 2, part = id & 3, block = h0 / 32 + (part >> 1);  // 16 of the row's 64 columns
        const bool in = block < inner / 32;
        const uint4* src = reinterpret_cast<const uint4*>(stage + r * kPackStride + part * 32);
        const uint4 x0 = src[0], x1 = src[1];
        uint32_t m2 = fp4_absmax(fp4_absmax(fp4_absmax(fp4_absmax(0u, x0.x), x0.y), x0.z), x0.w);
        m2 = fp4_absmax(fp4_absmax(fp4_absmax(fp4_absmax(m2, x1.x), x1.y), x1.z), x1.w);
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
        const uint32_t s = in ? fp4_scale_code(max(m2 & 0xffffu, m2 >> 16)) : 0u;  // scales past the width are 0
        if (32 * c + r < t.n) {
            const int64_t row = t.row + 32 * c + r;
            if (in) {
                const float inv = fp4_inverse(s);
                *reinterpret_cast<uint2*>(a.hq + row * (inner / 2) + h0 / 2 + part * 8) =
                    make_uint2(fp4_codes8(x0, inv), fp4_codes8(x1, inv));
            }
            if ((part & 1) == 0 && block < 4 * chunks)
                a.hsf[((row / kFp4Tile) * chunks + block / 4) * kFp4ChunkBytes + fp4_word_at(static_cast<int>(row % kFp4Tile)) +
                      (block & 3)] = static_cast<uint8_t>(s);
        }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");  // the staged rows have been read
    }
    if (group >= batches && lane == 0) {  // nothing of this tile is this group's
        mbar_arrive_cluster(cluster_map(&bars->shared_free, 0));
        mbar_arrive_cluster(cluster_map(acc_empty, 0));
    }
}

template <uint32_t GROUP, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const ProductArgs a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap wsmap,
               const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap xsmap) {
    extern __shared__ unsigned char smem_raw[];
    // The same offset in both CTAs of the pair (their shared windows are alike).
    unsigned char* smem = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    unsigned char* out_stage = smem + kStages * kStageBytes;
    Bars* bars = reinterpret_cast<Bars*>(out_stage + kOutBytes);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t cta = cluster_ctarank();  // of the pair; 0 leads

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->acc_full[i], 1);
            mbar_init(&bars->acc_empty[i], 2 * kEpiWarps);
        }
        mbar_init(&bars->shared_free, 2 * kEpiWarps);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        mbar_init_fence();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&bars->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (warp == 3 && elected())
        for (const CUtensorMap* map : {&wmap, &wsmap, &xmap, &xsmap})
            asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    pdl_wait_then_release();

    const int32_t planned = uniform(__ldg(a.plan));
    const uint32_t tiles = planned < 0 ? 0 : (planned > a.tile_cap ? a.tile_cap : planned);
    const uint32_t mtiles = (a.N + kMTile - 1) / kMTile;
    const uint32_t step = gridDim.x / 2, first = blockIdx.x / 2;
    const int nstages = static_cast<int>(ceil_div(a.K, kStageK));
    if (warp == a.quit_warp) give_up(bars, a);

    if (warp == 0) {
        const int32_t wtiles = static_cast<int32_t>(ceil_div(a.N, kFp4Tile));
        uint32_t s = 0, phase = 0;  // stage, and the parity its last use completed with
        int64_t issued = 0;
        bool ok = warp != a.quit_warp;
        Units<GROUP> list(a, tiles, mtiles, first, step);
        while (ok && list.left > 0) {
            const Unit t = list.take(a);
            if (t.n == 0) continue;
            const uint32_t n = mma_n(t.n);
            const int boxes = static_cast<int>((n / 2 + 31) / 32);
            const int halves = n > 128 ? 2 : 1;
            const uint32_t bytes = 2 * (kWBytes + boxes * kXBox + kScaleBox + halves * kScaleBox);
            const int32_t x0 = t.row + static_cast<int32_t>(cta * (n / 2));
            const int32_t m0 = t.m0 + static_cast<int32_t>(cta) * 128;
            const int32_t wtile = t.e * wtiles + m0 / kFp4Tile;
            for (int k = 0; k < nstages; ++k) {
                if (issued >= kStages && !wait_for(bars, &bars->empty[s], phase ^ 1, a)) {
                    ok = false;
                    break;
                }
                const uint32_t base = smem_addr(smem + s * kStageBytes);
                const uint32_t bar = cluster_map(&bars->full[s], 0);
                if (elected()) {
                    if (cta == 0) mbar_arrive_expect_tx(&bars->full[s], bytes);
                    tma_3d(base, &wmap, k * 128, m0, t.e, bar);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < boxes) tma_2d(base + kOffX + i * kXBox, &xmap, k * 128, x0 + 32 * i, bar);
                    tma_3d(base + kOffWS, &wsmap, 0, 2 * k, wtile, bar);
                    // Each CTA's tensor memory holds the scales of all the tile's rows.
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (h < halves) tma_3d(base + kOffXS + h * kScaleBox, &xsmap, 0, 2 * k, t.row / kFp4Tile + h, bar);
                }
                ++issued;
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && cta == 0) {  // bounded: what is in flight lands before the pair ends
            for (int i = 0; i < kStages && i < issued; ++i) {
                s = s == 0 ? kStages - 1 : s - 1;
                if (s == kStages - 1) phase ^= 1;
                drained(&bars->full[s], phase);
            }
        }
        __syncwarp();
    } else if (warp == 1 && cta == 0) {
        uint32_t s = 0, phase = 0, i = 0;  // i: tiles so far
        uint32_t last_n = 0;
        bool ok = warp != a.quit_warp;
        Units<GROUP> list(a, tiles, mtiles, first, step);
        while (ok && list.left > 0) {
            const Unit t = list.take(a);
            if (t.n == 0) continue;
            const uint32_t n = mma_n(t.n), place = i & 1;
            const uint32_t acc = tmem + (place ? kAcc1 : 0);
            // The place's last sums have been read; and, where this tile and
            // the one before it both reach the shared columns, that one's
            // part of them too.
            if (i >= 2) ok = wait_for(bars, &bars->acc_empty[place], ((i >> 1) - 1) & 1, a);
            if (ok && i >= 1 && (place ? last_n : n) > static_cast<uint32_t>(kAcc1))
                ok = wait_for(bars, &bars->shared_free, (i - 1) & 1, a);
            tc_fence_after();
            last_n = n;
            for (int k = 0; ok && k < nstages; ++k) {
                if (!wait_for(bars, &bars->full[s], phase, a)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t base = smem_addr(smem + s * kStageBytes);
                const int left = (a.K - k * kStageK + 63) / 64;
                if (elected()) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        scales_to_tmem(tmem + kScaleCol + 4 * c, desc_scales(base + kOffWS + c * kFp4ChunkBytes));
                        scales_to_tmem(tmem + kScaleCol + 8 + 8 * c, desc_scales(base + kOffXS + c * kFp4ChunkBytes));
                        if (n > 128)
                            scales_to_tmem(tmem + kScaleCol + 12 + 8 * c,
                                           desc_scales(base + kOffXS + kScaleBox + c * kFp4ChunkBytes));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < left)
                            mma(acc, desc_rows(base) + 2 * j, desc_rows(base + kOffX) + 2 * j, instr(n, j & 1),
                                tmem + kScaleCol + 4 * (j >> 1), tmem + kScaleCol + 8 + 8 * (j >> 1), k > 0 || j > 0);
                    commit_to(&bars->empty[s]);
                    if (k == nstages - 1) commit_to(&bars->acc_full[place]);
                }
                __syncwarp();
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
            ++i;
        }
        if (!ok) {  // bounded: products in flight end before tensor memory is given back
            if (elected())
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                 smem_addr(&bars->drain))
                             : "memory");
            drained(&bars->drain, 0);
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int w = warp & 3, half = (warp - 4) >> 2;  // lane quarter; which of every two chunks
        unsigned char* stage_ptr = out_stage + (warp - 4) * 16 * kOutStride;
        const uint32_t stage = smem_addr(stage_ptr);
        // stmatrix: block q of 8 lanes; ungated blocks are the warp's four
        // groups of 8 weight rows, gated two groups of each of two column blocks.
        const uint32_t to = stage + (lane & 7) * kOutStride + (lane >> 3) * 16;
        const uint32_t to_gated = stage + ((lane & 7) + 8 * (lane >> 4)) * kOutStride + ((lane >> 3) & 1) * 16;
        uint32_t i = 0;
        Units<GROUP> list(a, tiles, mtiles, first, step);
        while (list.left > 0) {
            const Unit t = list.take(a);
            if (t.n == 0) continue;
            const uint32_t place = i & 1;
            bool ok = warp != a.quit_warp && wait_for(bars, &bars->acc_full[place], (i >> 1) & 1, a);
            // Packing, four warps meet at barriers: they go on, or end, together. (One
            // whose wait ran out while another's came true would leave that one there.)
            if constexpr (MODE == kPacked) ok = all_agree(1 + half, ok);
            if (!ok) break;
            tc_fence_after();
            const int m = t.m0 + static_cast<int>(cta) * 128 + w * 32;  // the warp's weight rows
            const uint32_t acc = tmem + (place ? kAcc1 : 0) + (static_cast<uint32_t>(w * 32) << 16);
            if constexpr (MODE == kPacked) {
                pack_tile_out(a, t, cta, acc, w, lane, half, place != 0, out_stage + half * 32 * kPackStride, bars,
                              &bars->acc_empty[place]);
                ++i;
                continue;
            }
            const int chunks = static_cast<int>(mma_n(t.n) / 16);  // even: as many for either half
            // Place 0 has the shared columns at its end, place 1 at its start:
            // they are read first.
            for (int q = half; q < chunks; q += 2) {
                const int c = place ? q : chunks - 1 - q;
                uint32_t v[2][8];
                tmem_load(acc + 16 * c, v[0]);
                tmem_load(acc + 16 * c + (16u << 16), v[1]);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (q == half) mbar_arrive_cluster(cluster_map(&bars->shared_free, 0));
                    if (q + 2 >= chunks) mbar_arrive_cluster(cluster_map(&bars->acc_empty[place], 0));
                }
                const int c0 = 16 * c;  // first of the chunk's rows
                if (m >= a.N || c0 >= t.n) continue;
                uint8_t* y = reinterpret_cast<uint8_t*>(a.y) + (t.row + c0) * a.y_stride + (MODE == kGated ? m : 2 * m);
                if constexpr (MODE == kGated) {
                    uint32_t h[4];
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            h[2 * b + j] = bf16_pair(
                                gate_times_up(__uint_as_float(v[0][4 * b + 2 * j]), __uint_as_float(v[1][4 * b + 2 * j])),
                                gate_times_up(__uint_as_float(v[0][4 * b + 2 * j + 1]),
                                              __uint_as_float(v[1][4 * b + 2 * j + 1])));
                    store_turned(to_gated, h[0], h[1], h[2], h[3]);
                    __syncwarp();
                    const int r = lane >> 1;
                    if (c0 + r < t.n)
                        *reinterpret_cast<uint4*>(y + r * a.y_stride + (lane & 1) * 16) =
                            *reinterpret_cast<const uint4*>(stage_ptr + r * kOutStride + (lane & 1) * 16);
                } else {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t h[4];
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            h[g] = bf16_pair(__uint_as_float(v[g >> 1][4 * b + 2 * (g & 1)]),
                                             __uint_as_float(v[g >> 1][4 * b + 2 * (g & 1) + 1]));
                        store_turned(to + 8 * b * kOutStride, h[0], h[1], h[2], h[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const int r = 8 * p + (lane >> 2);
                        if (c0 + r < t.n)
                            *reinterpret_cast<uint4*>(y + r * a.y_stride + (lane & 3) * 16) =
                                *reinterpret_cast<const uint4*>(stage_ptr + r * kOutStride + (lane & 3) * 16);
                    }
                }
                __syncwarp();  // the staged rows have been read
            }
            ++i;
        }
    }

    // After a failed wait: loads that nobody waits for land before the cluster ends.
    if (*reinterpret_cast<volatile uint32_t*>(&bars->abort) != 0u)
        for (int i = 0; i < 200; ++i) __nanosleep(1000);
    // No CTA may leave while another's copies, products or arrivals can reach it.
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The CUDA driver's encoder, looked up once per process.
EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A map of codes (bytes, swizzled rows of 128) or scales (32-bit words, as they lie).
bool encode(CUtensorMap* map, bool codes, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    const cuuint32_t ones[3] = {1, 1, 1};
    return encoder()(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT32, rank,
                     const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     codes ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The next product of this host thread, when armed by moe_test_product_wait.
thread_local uint32_t t_test_wait_cycles = 0;
thread_local int32_t t_test_quit_warp = -1;

// Pairs that can be resident at once on the current device (cached).
template <uint32_t GROUP, int MODE>
int resident_pairs() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    const bool slot = dev >= 0 && dev < 64;
    if (slot && cache[dev].load(std::memory_order_relaxed) > 0) return cache[dev].load(std::memory_order_relaxed);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, product_kernel<GROUP, MODE>, &cfg) != cudaSuccess || n < 1) return -1;
    if (slot) cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <uint32_t GROUP, int MODE>
cudaError_t launch_pairs(const ProductArgs& a, const CUtensorMap& wmap, const CUtensorMap& wsmap, const CUtensorMap& xmap,
                         const CUtensorMap& xsmap, cudaStream_t stream) {
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(product_kernel<GROUP, MODE>), kSmem, kThreads, nullptr);
    if (e != cudaSuccess) return e;
    const int pairs = resident_pairs<GROUP, MODE>();
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    const int64_t most = a.tile_cap * ceil_div(a.N, kMTile);
    const unsigned grid = 2u * static_cast<unsigned>(most < pairs ? most : pairs);
    return launch_pdl_cluster(product_kernel<GROUP, MODE>, grid, kThreads, kSmem, 2u, stream, a, wmap, wsmap, xmap, xsmap);
}

// Whether four row tiles' units lie side by side, or one's. Four, whose pairs share
// an expert's weights, are faster in long calls: 262144 rows spread evenly over 256
// experts, 7168 -> 4096 2.46 ms against 2.63, 7168 -> 2048 1.31 against 1.37, 5984 ->
// 4096 2.76 against 2.97, 2048 -> 7168 1.49 against 1.51 (unevenly, 512 to 1536 rows
// each: 2.52 both, 2.86 against 2.93, 1.57 against 1.55). In shorter ones the order
// that spreads the short tiles better is the faster: 98304 rows over 128 experts 7168 ->
// 4096 1.06 ms against one's 1.02, 44800 rows over 32 experts 5984 -> 2048 232 us
// against 226, 65536 rows over 64 experts 7168 -> 4096 622 us against 630.
bool four_tiles(double rows, int32_t N, int32_t K) { return 2.0 * rows * N * K >= 7e12; }

}  // namespace

void arm_product_wait_test(uint32_t wait_cycles, int32_t quit_warp) {
    t_test_wait_cycles = wait_cycles;
    t_test_quit_warp = quit_warp;
}

cudaError_t launch_product(int32_t E, int32_t N, int32_t K, int32_t gated, const uint8_t* wq, const uint8_t* wsf,
                           const uint8_t* xq, const uint8_t* xsf, int64_t rows, const int32_t* plan, int64_t plan_ints,
                           uint16_t* y, int64_t y_stride, uint8_t* hq, uint8_t* hsf, int32_t* err, cudaStream_t stream) {
    ProductArgs a{E, N, K, plan_capacity(E, plan_ints), rows, plan, y, y_stride, hq, hsf, err, kWaitCycles, -1};
    if (t_test_wait_cycles != 0) {  // one call armed by moe_test_product_wait
        a.wait_cycles = t_test_wait_cycles;
        a.quit_warp = t_test_quit_warp;
        t_test_wait_cycles = 0;
        t_test_quit_warp = -1;
    }
    if (a.tile_cap == 0) return cudaSuccess;
    // Rows that the plan has room for: it has one tile per expert and one per 256 rows.
    const bool four = four_tiles(static_cast<double>(a.tile_cap - E) * kPlanTileRows, N, K);
    // Units are counted in 32 bits; what a plan of this arena can hold is far below.
    const int64_t most_tiles = rows / kFp4Tile + 1, room = (int64_t{1} << 31) / ceil_div(N, kMTile);
    if (a.tile_cap > most_tiles) a.tile_cap = static_cast<int32_t>(most_tiles);
    if (a.tile_cap > room) return cudaErrorInvalidValue;
    if (encoder() == nullptr) return cudaErrorNotSupported;
    const cuuint64_t kb = static_cast<cuuint64_t>(K) / 2, chunks = static_cast<cuuint64_t>(ceil_div(K, kFp4Chunk));
    const cuuint64_t wt = static_cast<cuuint64_t>(ceil_div(N, kFp4Tile));
    CUtensorMap wmap, wsmap, xmap, xsmap;
    {
        const cuuint64_t dims[3] = {kb, static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(E)};
        const cuuint64_t strides[2] = {kb, kb * static_cast<cuuint64_t>(N)};
        const cuuint32_t box[3] = {128, 128, 1};
        if (!encode(&wmap, true, wq, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t dims[2] = {kb, static_cast<cuuint64_t>(rows)};
        const cuuint64_t strides[1] = {kb};
        const cuuint32_t box[2] = {128, 32};
        if (!encode(&xmap, true, xq, 2, dims, strides, box)) return cudaErrorInvalidValue;
    }
    for (int side = 0; side < 2; ++side) {
        const cuuint64_t dims[3] = {kFp4ChunkBytes / 4, chunks,
                                    side ? static_cast<cuuint64_t>(rows / kFp4Tile) : wt * static_cast<cuuint64_t>(E)};
        const cuuint64_t strides[2] = {kFp4ChunkBytes, kFp4ChunkBytes * chunks};
        const cuuint32_t box[3] = {kFp4ChunkBytes / 4, 2, 1};
        if (!encode(side ? &xsmap : &wsmap, false, side ? xsf : wsf, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    const auto launch = hq ? (four ? launch_pairs<4, kPacked> : launch_pairs<1, kPacked>)
                           : gated ? (four ? launch_pairs<4, kGated> : launch_pairs<1, kGated>)
                                   : (four ? launch_pairs<4, kPlain> : launch_pairs<1, kPlain>);
    return launch(a, wmap, wsmap, xmap, xsmap, stream);
}

}  // namespace moe
