// product_int8.cu -- the experts' grouped product of int8 operands
// (moe_expert_product_int8): for every row r of expert e,
//   v[r][n] = ws_e[n] * xs[r] * sum over k of w_e[n][k] * x[r][k]
//   y[r] = bf16_rne(v[r]), or, gated, bf16_rne(silu(gate) * up) of the pairs.
//
// sm_103a's tensor cores multiply no 8-bit integers, but every int8 is an f16 and
// a product of two is exact in binary32, and so is a sum below 2^24 of them: the
// codes become f16 on their way to tcgen05.mma kind::f16. (An int8 as two e4m3
// parts would take four products at twice the rate.)
//
// A pair of CTAs (one per SM) computes 256 weight rows x up to 256 of an expert's
// rows; the weights are the M side, so that few rows cost a thin instruction. Each
// CTA has its 128 weight rows and half of the rows. Warp 0 loads codes (TMA, 128 of K
// to a stage, a ring of stages); four groups of four warps turn them into f16 -- the
// weights' straight into tensor memory, from where the instruction takes its A side,
// the rows' into shared memory, swizzled as its B side is --, two groups by turns at
// a stage, one at each half of its K; warp 1 of the leading CTA issues the products
// of K = 16; the warps from 4 on take the sums out, times the scales. A group has a place
// of its own for what it makes, so they work while others' places are multiplied.
//
// What bounds it. Many rows: the tensor pipe and power (262144 rows 7168 -> 4096 gated:
// 8.0-8.5 ms, 1.81-1.92 PFLOP/s; back to back for seconds 9.5-9.8).
// Weights through tensor memory save shared memory's rate: 64 of K are 16 KB of codes in,
// 16 out, 16 of f16 rows in and 16 out, 64 KB in the 512 cycles of their products, at 128
// bytes a cycle. Few rows: the weights' bytes (2 rows to each of 256 experts: 1.09 ms,
// 6.9 TB/s; 1.13 out of a cold L2). What it took there: four converting groups (two: 1.65 ms); one place to a
// group (two, which let groups run ahead of the products: 1.18); four warps for the sums
// (eight: 1.18); and arrivals and waits at the CTA's scope (all at the cluster's 3.6, and many
// rows 14.4; those of `ready` alone 2.0, and 10.7 against 8.1): why that holds for operands of the
// other CTA is said at mbar_arrive_cluster.
//
// Tensor memory: sums in two places, columns 0 and 128 on, which share 128 columns in
// tiles of more than 128 rows (read first and given back early), and the f16 weights,
// 32 columns to a place. Dense calls short of tiles cut them smaller, or let up to four
// pairs share a tile's K and join through each other's shared memory (the rule is at cut()).
#include <atomic>

#include "fp4.cuh"
#include "int8.cuh"
#include "tensor.cuh"

namespace moe {
namespace {

constexpr int kMTile = 256;                 // weight rows of a CTA pair
constexpr int kStageK = 128;                // codes of K per stage: one 128-byte swizzle row
constexpr uint32_t kWBytes = 128 * 128;     // a CTA's weight rows of a stage
constexpr uint32_t kXBox = 32 * 128;        // 32 rows of a stage
constexpr uint32_t kOutStride = 80;         // bytes per staged row: 64 and a shift of 4 banks per row
constexpr uint32_t kOutBytes = 16 * kOutStride;             // of a warp that takes sums out
constexpr uint32_t kScaleBytes = kPlanTileRows * 4;         // the rows' scales, for it
constexpr uint32_t kBarBytes = 512;
constexpr uint32_t kSentBytes = 128 * 64;  // a CTA's sums of 16 rows, binary32
constexpr int kAcc1 = 128;  // second place of the sums
constexpr int kSharedChunks = (256 - kAcc1) / 16;
constexpr int kMostStages = 10;
constexpr int kGroups = 4;     // of four converting warps: two by turns at a stage, one at each half of its K
constexpr int kACol = 512 - 32 * kGroups;  // the f16 weights: a place of 32 columns for each group

// Up to ROWS rows to a tile: fewer of them in shared memory make room for more stages. Their number is even: groups take
// stages by turns, so each place of the ring is always the same two groups', which see every use of it. (Of seven, a
// group saw every second use, of the same parity, and one that skips the short end of K, waiting for no product, could
// take the use in between for its own.)
template <int ROWS>
struct Cut {
    static constexpr int kStages = ROWS <= 64 ? 10 : ROWS <= 128 ? 6 : 4;
    static_assert(kStages % 2 == 0, "a place of the ring is the same groups' at every use");
    static constexpr int kEpiWarps = ROWS <= 128 ? 4 : 8;            // that take sums out: one or two for each quarter of the lanes
    static constexpr int kThreads = 128 + 32 * kEpiWarps + 128 * kGroups;
    static constexpr uint32_t kStageBytes = kWBytes + ROWS / 64 * kXBox;
    static constexpr uint32_t kHalfBytes = ROWS / 2 * 128;           // a CTA's rows of 64 f16
    static constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + kGroups * kHalfBytes + kEpiWarps * (kOutBytes + kScaleBytes) + kBarBytes;
    // parts of K: what the other pairs send of the chunks that a pair finishes, less than a tile's sums
    static_assert(ROWS / 16 * kSentBytes <= kStages * kStageBytes + kGroups * kHalfBytes, "room for sums");
    static_assert(kAcc1 + (ROWS < 256 ? ROWS : 256) <= kACol && kStages <= kMostStages && kSmem <= 227 * 1024, "room");
};

constexpr int kMostShare = 4;  // 8 CTAs, the largest portable cluster

struct Args {
    ProductInt8Args p;
    int32_t shift;        // tiles are 256 / 2^shift rows; a plan's are 256 and become 2^shift units, some of them empty
    int32_t split;        // pairs that share the K of a tile: 1, or 2 to kMostShare, one cluster (and one tile to it)
    int64_t wait_cycles;  // bound of a wait (kWaitCycles)
    int32_t quit_warp;    // test hook: a warp of each CTA that acts as if its first wait had run out, or -1
    int32_t* err;
};

// Barriers of a CTA, and its abort flag.
struct Bars {
    uint64_t full[kMostStages];   // each CTA: its loads of a stage have landed
    uint64_t empty[kMostStages];  // each CTA: both groups have read a stage
    uint64_t ready[kGroups];      // leading CTA: both CTAs' f16 operands of a group's place are there
    uint64_t used[kGroups];       // each CTA: the products that read it are done
    uint64_t acc_full[2];     // each CTA: a tile's sums are complete
    uint64_t acc_empty[2];    // leading CTA: both CTAs have read a place of the sums
    uint64_t may_send;        // each CTA, K in parts: the other pairs have room for its sums
    uint64_t joined;          // each CTA, K in parts: the other pairs' sums are there
    uint64_t shared_free;     // leading CTA: both CTAs have read the tile's part of the shared columns
    uint64_t drain;           // leading CTA, after a failed wait: products in flight are done
    uint32_t tmem;
    uint32_t abort;
};
static_assert(sizeof(Bars) <= kBarBytes, "barriers");

// One tile of work.
struct Unit {
    int32_t e, row, n, m0;  // expert, first row, rows, first weight row of the pair
};

__device__ __forceinline__ uint32_t mma_n(int32_t rows) { return (rows + 31) & ~31; }

// TMA tile loads into this CTA's shared memory, counted on its own barrier.
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// f16 x f16 to binary32, M = 256, N columns, A in tensor memory, B K-major.
__device__ __forceinline__ uint32_t instr(uint32_t n) { return (1u << 4) | ((n >> 3) << 17) | (16u << 24); }

__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

// Arrives on `bar` of both CTAs of the pair led by `lead` once every product issued so far is done.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint32_t lead) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3u << lead))
        : "memory");
}

// Arrival on a barrier of another CTA that hands over data written to it.
__device__ __forceinline__ void arrive_with_data(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void write_cluster(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint4 read_shared(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void write_shared(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 codes to 16 f16, two to a word.
__device__ __forceinline__ void halves16(uint4 v, uint32_t* h) {
    halves4(v.x, h[0], h[1]);
    halves4(v.y, h[2], h[3]);
    halves4(v.z, h[4], h[5]);
    halves4(v.w, h[6], h[7]);
}

// A lane's 32 words to 32 columns of tensor memory.
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&h)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7]), "r"(h[8]), "r"(h[9]),
        "r"(h[10]), "r"(h[11]), "r"(h[12]), "r"(h[13]), "r"(h[14]), "r"(h[15]), "r"(h[16]), "r"(h[17]), "r"(h[18]),
        "r"(h[19]), "r"(h[20]), "r"(h[21]), "r"(h[22]), "r"(h[23]), "r"(h[24]), "r"(h[25]), "r"(h[26]), "r"(h[27]),
        "r"(h[28]), "r"(h[29]), "r"(h[30]), "r"(h[31])
        : "memory");
}

// A pair's units, first, first + step, .. of the launch's; the weight rows are the
// inner index. A role steps from unit to unit without a division and holds the next
// one's plan words while it works on the current one. A plan's tile of more than
// ROWS rows is one unit of several tiles. (In ranges of even length for each pair, 2 rows each 7168 -> 4096 1098 -> 1280 us:
// pairs then read far apart.)
template <int ROWS>
struct Units {
    uint32_t per, part, in, step_part, step_in, left;
    int4 tile;
    int32_t skip;  // rows of the plan's tile that other units have
    Unit rest;     // what the current unit has left

    __device__ __forceinline__ Units(const Args& a, uint32_t tiles, uint32_t mtiles, uint32_t first, uint32_t step)
        : per(mtiles), tile(make_int4(0, 0, 0, 0)), skip(0), rest{0, 0, 0, 0} {
        const uint32_t units = (tiles << (a.p.plan ? a.shift : 0)) * mtiles;
        left = first < units ? (units - first - 1) / step + 1 : 0;
        part = first / per;
        in = first - part * per;
        step_part = step / per;
        step_in = step - step_part * per;
        fetch(a);
    }
    __device__ __forceinline__ void fetch(const Args& a) {
        if (left == 0) return;
        const int32_t size = kPlanTileRows >> a.shift;
        if (a.p.plan) {
            tile = __ldg(reinterpret_cast<const int4*>(a.p.plan + plan_tiles_at(a.p.E)) + (part >> a.shift));
            skip = static_cast<int32_t>(part & ((1u << a.shift) - 1)) * size;
        } else {
            const int64_t first = static_cast<int64_t>(part) * size, rows = a.p.rows - first;
            tile = make_int4(0, static_cast<int32_t>(first), static_cast<int32_t>(rows < size ? rows : size), 0);
        }
    }
    __device__ __forceinline__ bool more(const Args&) const { return left > 0 || rest.n > 0; }
    // The current tile, the same in every lane, or none (n = 0) where the plan's
    // tile is no tile of these rows; then on to the next.
    __device__ __forceinline__ Unit take(const Args& a) {
        Unit o = rest;
        if (rest.n == 0) {
            o = Unit{uniform(tile.x), uniform(tile.y), uniform(tile.z), static_cast<int32_t>(in) * kMTile};
            if (o.e < 0 || o.e >= a.p.E || o.row < 0 || o.n < 0 || o.n > kPlanTileRows ||
                o.row + static_cast<int64_t>(o.n) > a.p.rows) {
                raise_error(a.err, MOE_ERR_CAPACITY);
                o.n = 0;
            }
            const int32_t over = uniform(skip);
            o.row += over;
            o.n = max(0, min(o.n - over, kPlanTileRows >> a.shift));
            --left;
            part += step_part;
            in += step_in;
            if (in >= per) {
                in -= per;
                ++part;
            }
            fetch(a);
        }
        if (ROWS < kPlanTileRows) {
            const int32_t n = min(o.n, ROWS);
            rest = Unit{o.e, o.row + n, o.n - n, o.m0};
            o.n = n;
        }
        return o;
    }
};

// The same of tiles of up to 128 rows, which a plan's average asks for where some experts may have far more: both halves of a
// plan's tile are units, neighbours in the order, so that the pairs, which get units by turns, get as much to do. A warp holds
// 32 of the plan's tiles, a lane each. 8008 rows over 255 experts, one with 933, 2048 -> 7168 721 -> 705 us, 7168 -> 4096
// 1435 -> 1324, 31 rows each 636 -> 629. (Looking units up costs more than it gives where rows are few, 2 rows each 7168 -> 4096 in tiles of
// 64 1098 -> 1135, and where a tile is a unit anyway, 1024 rows each 8.28 -> 8.38 ms.)
struct HalfUnits {
    static constexpr int kSize = kPlanTileRows / 2;
    uint32_t per, part, in, step_part, step_in;
    uint32_t tiles;         // the plan's, or the rows'
    uint32_t base, before;  // first tile that is held, halves before it
    uint32_t upto, held;    // halves of the tiles that are held up to the lane's, and of all
    int4 tile;              // the lane's

    __device__ __forceinline__ HalfUnits(const Args& a, uint32_t all_tiles, uint32_t mtiles, uint32_t first, uint32_t step)
        : per(mtiles), tiles(all_tiles), base(0), before(0), upto(0), held(0), tile(make_int4(0, 0, 0, 0)) {
        part = first / per;
        in = first - part * per;
        step_part = step / per;
        step_in = step - step_part * per;
        if (a.p.plan) hold(a);
    }
    // (what is no count of rows is one, and skipped)
    __device__ __forceinline__ static uint32_t halves_of(int32_t n) { return n > kSize && n <= kPlanTileRows ? 2 : 1; }
    __device__ __forceinline__ void hold(const Args& a) {
        const uint32_t lane = threadIdx.x & 31, i = base + lane;
        if (i < tiles) tile = __ldg(reinterpret_cast<const int4*>(a.p.plan + plan_tiles_at(a.p.E)) + i);
        upto = i < tiles ? halves_of(tile.z) : 0;
#pragma unroll
        for (uint32_t d = 1; d < 32; d *= 2) {
            const uint32_t other = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += other;
        }
        held = __shfl_sync(0xffffffffu, upto, 31);
    }
    __device__ __forceinline__ bool more(const Args& a) {
        if (!a.p.plan) return part < tiles;
        while (part - before >= held) {
            if (base >= tiles) return false;
            base += 32;
            before += held;
            hold(a);
        }
        return true;
    }
    __device__ __forceinline__ Unit take(const Args& a) {
        const int32_t m0 = static_cast<int32_t>(in) * kMTile;
        Unit o;
        if (a.p.plan) {
            const int at = __ffs(__ballot_sync(0xffffffffu, part - before < upto)) - 1;
            o = Unit{uniform(__shfl_sync(0xffffffffu, tile.x, at)), uniform(__shfl_sync(0xffffffffu, tile.y, at)),
                     uniform(__shfl_sync(0xffffffffu, tile.z, at)), m0};
            const uint32_t end = uniform(__shfl_sync(0xffffffffu, upto, at));
            if (o.e < 0 || o.e >= a.p.E || o.row < 0 || o.n < 0 || o.n > kPlanTileRows ||
                o.row + static_cast<int64_t>(o.n) > a.p.rows) {
                raise_error(a.err, MOE_ERR_CAPACITY);
                o.n = 0;
            } else {
                const int32_t skip = kSize * static_cast<int32_t>(halves_of(o.n) - (end - (part - before)));
                o.row += skip;
                o.n = min(o.n - skip, kSize);
            }
        } else {
            const int64_t first = static_cast<int64_t>(part) * kSize, rows = a.p.rows - first;
            o = Unit{0, static_cast<int32_t>(first), static_cast<int32_t>(rows < kSize ? rows : kSize), m0};
        }
        part += step_part;
        in += step_in;
        if (in >= per) {
            in -= per;
            ++part;
        }
        return o;
    }
};

template <int ROWS>
struct ListOf {
    using Type = Units<ROWS>;
};
template <>
struct ListOf<128> {
    using Type = HalfUnits;
};

template <bool GATED, int ROWS>
__global__ void __launch_bounds__(Cut<ROWS>::kThreads, 1)
product_int8_kernel(const Args a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap) {
    constexpr int kStages = Cut<ROWS>::kStages, kEpiWarps = Cut<ROWS>::kEpiWarps, kParts = kEpiWarps / 4;
    constexpr uint32_t kStageBytes = Cut<ROWS>::kStageBytes, kHalfBytes = Cut<ROWS>::kHalfBytes;
    extern __shared__ unsigned char smem_raw[];
    // The same offset in both CTAs of the pair (their shared windows are alike).
    unsigned char* smem = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    unsigned char* halves = smem + kStages * kStageBytes;
    unsigned char* out_stage = halves + kGroups * kHalfBytes;
    float* scales = reinterpret_cast<float*>(out_stage + kEpiWarps * kOutBytes);
    Bars* bars = reinterpret_cast<Bars*>(out_stage + kEpiWarps * (kOutBytes + kScaleBytes));
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank(), cta = rank & 1, lead = rank & ~1u;  // of the pair, 0 leads; the leading CTA
    const int kpart = static_cast<int>(rank >> 1);                               // the pair's part of K

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 8);
        }
        for (int i = 0; i < kGroups; ++i) {
            mbar_init(&bars->ready[i], 8);
            mbar_init(&bars->used[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->acc_full[i], 1);
            mbar_init(&bars->acc_empty[i], 2 * kEpiWarps);
        }
        mbar_init(&bars->may_send, max(1, kEpiWarps * (a.split - 1)));
        mbar_init(&bars->joined, max(1, kEpiWarps * (a.split - 1)));
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
        for (const CUtensorMap* map : {&wmap, &xmap}) asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    pdl_wait_then_release();

    using List = typename ListOf<ROWS>::Type;
    uint32_t tiles = a.p.tile_cap;
    if (a.p.plan) {
        const int32_t planned = uniform(__ldg(a.p.plan));
        // More tiles than the rows have room for (tile_cap): the last ones lie outside and are not looked up.
        if (planned > a.p.tile_cap && blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, MOE_ERR_CAPACITY);
        tiles = max(0, min(planned, a.p.tile_cap));
    }
    const uint32_t mtiles = (a.p.N + kMTile - 1) / kMTile;
    const uint32_t step = gridDim.x / (2 * a.split), first = blockIdx.x / (2 * a.split);
    const int nstages = static_cast<int>(ceil_div(a.p.K, kStageK));
    const int k_first = nstages * kpart / a.split, k_end = nstages * (kpart + 1) / a.split;  // the pair's stages
    const bool short_end = a.p.K - (nstages - 1) * kStageK <= kStageK / 2;  // the last stage has one half
    if (warp == a.quit_warp) give_up(bars, a);

    if (warp == 0) {
        uint32_t s = 0, phase = 0;  // stage, and the parity its last use completed with
        int64_t issued = 0;
        bool ok = warp != a.quit_warp;
        List list(a, tiles, mtiles, first, step);
        while (ok && list.more(a)) {
            const Unit t = list.take(a);
            if (t.n == 0) continue;
            const uint32_t n = mma_n(t.n);
            const int boxes = static_cast<int>((n / 2 + 31) / 32);
            const uint32_t bytes = kWBytes + boxes * kXBox;
            const int32_t x0 = t.row + static_cast<int32_t>(cta * (n / 2));
            const int32_t m0 = t.m0 + static_cast<int32_t>(cta) * 128;
            for (int k = k_first; k < k_end; ++k) {
                if (issued >= kStages && !wait_here(bars, &bars->empty[s], phase ^ 1, a)) {
                    ok = false;
                    break;
                }
                const uint32_t base = smem_addr(smem + s * kStageBytes), bar = smem_addr(&bars->full[s]);
                if (elected()) {
                    mbar_arrive_expect_tx(&bars->full[s], bytes);
                    load_3d(base, &wmap, k * kStageK, m0, t.e, bar);
#pragma unroll
                    for (int i = 0; i < ROWS / 64; ++i)
                        if (i < boxes) load_2d(base + kWBytes + i * kXBox, &xmap, k * kStageK, x0 + 32 * i, bar);
                }
                ++issued;
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) {  // bounded: what is in flight lands before the pair ends
            for (int i = 0; i < kStages && i < issued; ++i) {
                s = s == 0 ? kStages - 1 : s - 1;
                if (s == kStages - 1) phase ^= 1;
                drained(&bars->full[s], phase);
            }
        }
        __syncwarp();
    } else if (warp == 1 && cta == 0) {
        uint32_t i = 0, last_n = 0;  // i: tiles so far
        uint32_t turn = 0, parity = 0;  // a bit a group: of its place's next use
        bool ok = warp != a.quit_warp;
        List list(a, tiles, mtiles, first, step);
        while (ok && list.more(a)) {
            const Unit t = list.take(a);
            if (t.n == 0) continue;
            const uint32_t n = mma_n(t.n), place = i & 1;
            const uint32_t acc = tmem + (place ? kAcc1 : 0);
            // The place's last sums have been read; and, where this tile and
            // the one before it both reach the shared columns, that one's
            // part of them too.
            if (i >= 2) ok = wait_here(bars, &bars->acc_empty[place], ((i >> 1) - 1) & 1, a);
            if (ok && i >= 1 && (place ? last_n : n) > static_cast<uint32_t>(kAcc1))
                ok = wait_here(bars, &bars->shared_free, (i - 1) & 1, a);
            tc_fence_after();
            last_n = n;
            for (int k = k_first; ok && k < k_end; ++k) {
                const bool end = k == k_end - 1, short_now = short_end && k == nstages - 1;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (half == 1 && short_now) break;
                    const uint32_t slot = 2 * turn + half;
                    if (!wait_here(bars, &bars->ready[slot], parity >> slot & 1, a)) {
                        ok = false;
                        break;
                    }
                    parity ^= 1u << slot;
                    tc_fence_after();
                    const uint64_t b = desc_rows(smem_addr(halves + slot * kHalfBytes));
                    if (elected()) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma(acc, tmem + kACol + 32 * slot + 8 * j, b + 2 * j, instr(n),
                                k > k_first || half > 0 || j > 0);
                        commit_pair(&bars->used[slot], lead);
                        if (end && (half == 1 || short_now)) commit_pair(&bars->acc_full[place], lead);
                    }
                    __syncwarp();
                }
                turn ^= 1;
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
    } else if (warp >= 4 + kEpiWarps) {
        // Four warps a group: of every two stages one, of its K one half.
        const int group = (warp - 4 - kEpiWarps) >> 2, half = group & 1, w = warp & 3;
        const int row = w * 32 + lane;           // lane of tensor memory and weight row
        const int xrow = 8 * w + (lane & 7), xpart = lane >> 3;  // of the rows: which one, and which 16 of 64 codes
        const uint32_t xfrom = ((4 * half + xpart) ^ (xrow & 7)) << 4, xto = ((2 * xpart) ^ (xrow & 7)) << 4;
        const uint32_t to = tmem + kACol + 32 * group + (static_cast<uint32_t>(w * 32) << 16);
        const uint32_t mine = smem_addr(halves) + group * kHalfBytes + xrow * 128;
        const uint32_t ready = cluster_map(bars->ready + group, lead);
        uint32_t s = 0, phase = 0, uses = 0, turn = 0;
        bool ok = warp != a.quit_warp;
        List list(a, tiles, mtiles, first, step);
        while (ok && list.more(a)) {
            const Unit t = list.take(a);
            if (t.n == 0) continue;
            const int rows = static_cast<int>(mma_n(t.n) / 2);
            for (int k = k_first; k < k_end; ++k) {
                const uint32_t at = s, parity = phase;
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1;
                }
                const uint32_t now = turn;
                turn ^= 1;
                if (now != static_cast<uint32_t>(group >> 1)) continue;
                if (!wait_here(bars, &bars->full[at], parity, a)) {
                    ok = false;
                    break;
                }
                const bool skip = half == 1 && short_end && k == nstages - 1;
                if (!skip) {
                    if (uses > 0 && !wait_here(bars, &bars->used[group], (uses - 1) & 1, a)) {
                        ok = false;
                        break;
                    }
                    ++uses;
                    // All codes first: a lane's weight row, and of every 32 rows 16 codes of one (the
                    // lanes of a warp are 8 rows x 4, so that neither side meets in a bank).
                    const uint32_t base = smem_addr(smem + at * kStageBytes);
                    uint4 wv[4], xv[ROWS / 64];
#pragma unroll
                    for (int c = 0; c < 4; ++c) wv[c] = read_shared(base + row * 128 + (((4 * half + c) ^ (row & 7)) << 4));
#pragma unroll
                    for (int j = 0; j < ROWS / 64; ++j)
                        if (32 * j + 8 * w < rows) xv[j] = read_shared(base + kWBytes + (xrow + 32 * j) * 128 + xfrom);
                    uint32_t h[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) halves16(wv[c], h + 8 * c);
                    tc_fence_after();
                    tmem_store(to, h);
#pragma unroll
                    for (int j = 0; j < ROWS / 64; ++j) {
                        if (32 * j + 8 * w >= rows) continue;
                        uint32_t x[8];
                        halves16(xv[j], x);
                        const uint32_t dst = mine + j * 32 * 128;
                        write_shared(dst + xto, x[0], x[1], x[2], x[3]);
                        write_shared(dst + (xto ^ 16), x[4], x[5], x[6], x[7]);
                    }
                    // Every lane's codes have been used and its f16 rows written, by the generic proxy: before the loader
                    // (the async proxy) writes the stage again, and before the tensor cores read the rows. A stage that
                    // went back once its codes were read, without the fence, was refilled under reads still in flight.
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->empty[at]);
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(ready);
                } else if (lane == 0) {
                    mbar_arrive(&bars->empty[at]);
                }
            }
        }
    } else if (warp >= 4) {
        const int w = warp & 3, part = (warp - 4) >> 2;  // lane quarter; which of every kParts chunks of 16 rows
        unsigned char* stage_ptr = out_stage + (warp - 4) * 16 * kOutStride;
        const uint32_t stage = smem_addr(stage_ptr);
        float* xs = scales + (warp - 4) * kPlanTileRows;
        // stmatrix: block q of 8 lanes; ungated blocks are the warp's four
        // groups of 8 weight rows, gated two groups of each of two column blocks.
        const uint32_t to = stage + (lane & 7) * kOutStride + (lane >> 3) * 16;
        const uint32_t to_gated = stage + ((lane & 7) + 8 * (lane >> 4)) * kOutStride + ((lane >> 3) & 1) * 16;
        uint32_t i = 0;
        List list(a, tiles, mtiles, first, step);
        while (list.more(a)) {
            const Unit t = list.take(a);
            if (t.n == 0) continue;
            const uint32_t place = i & 1;
            const int m = t.m0 + static_cast<int>(cta) * 128 + w * 32;  // the warp's weight rows
            // Scales, while the sums are formed: four weight rows' per lane, all rows' per warp.
            float ws[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = m + (lane >> 2) + 8 * j;
                ws[j] = n < a.p.N ? __ldg(a.p.ws + static_cast<int64_t>(t.e) * a.p.N + n) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < kPlanTileRows / 32; ++j) {
                const int r = lane + 32 * j;
                if (r < t.n) xs[r] = __ldg(reinterpret_cast<const float*>(a.p.xs + (t.row + static_cast<int64_t>(r)) * a.p.xs_stride));
            }
            __syncwarp();
            if (warp == a.quit_warp || !wait_here(bars, &bars->acc_full[place], (i >> 1) & 1, a)) break;
            tc_fence_after();
            const uint32_t acc = tmem + (place ? kAcc1 : 0) + (static_cast<uint32_t>(w * 32) << 16);
            const int chunks = static_cast<int>(mma_n(t.n) / 16);
            // K in parts: of every `split` chunks of 16 rows each pair finishes one and writes its sums of the
            // others to the shared memory of the pair that finishes those, where loads and products are done
            // by then, 16 a thread and chunk.
            const uint32_t sent = smem_addr(smem) + (w * 32 + lane) * 16;
            const int per = (chunks + a.split - 1) / a.split;  // chunks that a pair finishes
            if (a.split > 1) {
                if (lane == 0)
                    for (int p = 0; p < a.split; ++p)
                        if (p != kpart) arrive_with_data(cluster_map(&bars->may_send, 2 * p + cta));
                if (!wait_for(bars, &bars->may_send, 0, a)) break;
                for (int c = 0; c < chunks; ++c) {
                    const int o = c % a.split;
                    if (o == kpart || c / a.split % kParts != part) continue;
                    const uint32_t there = cluster_map(smem, 2 * o + cta) - smem_addr(smem) + sent +
                                           ((kpart < o ? kpart : kpart - 1) * per + c / a.split) * kSentBytes;
                    uint32_t v[2][8];
                    tmem_load(acc + 16 * c, v[0]);
                    tmem_load(acc + 16 * c + (16u << 16), v[1]);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        write_cluster(there + i * 2048, v[i >> 1][4 * (i & 1)], v[i >> 1][4 * (i & 1) + 1], v[i >> 1][4 * (i & 1) + 2],
                                      v[i >> 1][4 * (i & 1) + 3]);
                }
                __syncwarp();
                if (lane == 0)
                    for (int p = 0; p < a.split; ++p)
                        if (p != kpart) arrive_with_data(cluster_map(&bars->joined, 2 * p + cta));
                if (!wait_for(bars, &bars->joined, 0, a)) break;
            }
            // Place 0 has the shared columns at its end, place 1 at its start:
            // they are read first.
            for (int q = 0; q < chunks / kParts; ++q) {
                const int at = kParts * q + part;
                const int c = a.split > 1 ? at * a.split + kpart : place ? at : chunks - 1 - at;
                if (c >= chunks) break;  // of the pair's own there are fewer
                uint32_t v[2][8];
                tmem_load(acc + 16 * c, v[0]);
                tmem_load(acc + 16 * c + (16u << 16), v[1]);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (q == min(kSharedChunks, chunks) / kParts - 1) mbar_arrive_cluster(cluster_map(&bars->shared_free, lead));
                    if (q == chunks / kParts - 1) mbar_arrive_cluster(cluster_map(&bars->acc_empty[place], lead));
                }
                if (a.split > 1) {  // the parts' sums in ascending order
                    float s[2][8];
                    for (int p = 0; p < a.split; ++p)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t* own = &v[i >> 1][4 * (i & 1)];
                            uint4 o = make_uint4(own[0], own[1], own[2], own[3]);
                            if (p != kpart) o = read_shared(sent + ((p < kpart ? p : p - 1) * per + c / a.split) * kSentBytes + i * 2048);
                            float* to = &s[i >> 1][4 * (i & 1)];
                            const float f[4] = {__uint_as_float(o.x), __uint_as_float(o.y), __uint_as_float(o.z), __uint_as_float(o.w)};
#pragma unroll
                            for (int j = 0; j < 4; ++j) to[j] = p == 0 ? f[j] : to[j] + f[j];
                        }
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i >> 3][i & 7] = __float_as_uint(s[i >> 3][i & 7]);
                }
                const int c0 = 16 * c;  // first of the chunk's rows
                if (m >= a.p.N || c0 >= t.n) continue;
                float f[2][8];  // v times the scales
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float2 x = *reinterpret_cast<const float2*>(xs + c0 + 8 * b + 2 * (lane & 3));
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            f[h][4 * b + j] = __uint_as_float(v[h][4 * b + j]) * ws[2 * h + (j >> 1)] * (j & 1 ? x.y : x.x);
                }
                uint8_t* y = reinterpret_cast<uint8_t*>(a.p.y) + (t.row + c0) * a.p.y_stride + (GATED ? m : 2 * m);
                if constexpr (GATED) {
                    uint32_t h[4];
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            h[2 * b + j] = bf16_pair(gate_times_up(f[0][4 * b + 2 * j], f[1][4 * b + 2 * j]),
                                                     gate_times_up(f[0][4 * b + 2 * j + 1], f[1][4 * b + 2 * j + 1]));
                    store_turned(to_gated, h[0], h[1], h[2], h[3]);
                    __syncwarp();
                    const int r = lane >> 1;
                    if (c0 + r < t.n)
                        *reinterpret_cast<uint4*>(y + r * a.p.y_stride + (lane & 1) * 16) =
                            *reinterpret_cast<const uint4*>(stage_ptr + r * kOutStride + (lane & 1) * 16);
                } else {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t h[4];
#pragma unroll
                        for (int g = 0; g < 4; ++g) h[g] = bf16_pair(f[g >> 1][4 * b + 2 * (g & 1)], f[g >> 1][4 * b + 2 * (g & 1) + 1]);
                        store_turned(to + 8 * b * kOutStride, h[0], h[1], h[2], h[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const int r = 8 * p + (lane >> 2);
                        if (c0 + r < t.n)
                            *reinterpret_cast<uint4*>(y + r * a.p.y_stride + (lane & 3) * 16) =
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
    if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// A map of codes: swizzled rows of 128 bytes.
bool encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
    const cuuint32_t ones[3] = {1, 1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of `split` pairs that can be resident at once on the current device (cached); allows the kernel its shared memory.
template <bool GATED, int ROWS>
int resident_clusters(int split) {
    static std::atomic<int> cache[kMostShare][64];
    const int at = split - 1;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    const bool slot = dev >= 0 && dev < 64;
    if (slot && cache[at][dev].load(std::memory_order_relaxed) > 0) return cache[at][dev].load(std::memory_order_relaxed);
    if (prepare_kernel(reinterpret_cast<const void*>(product_int8_kernel<GATED, ROWS>), Cut<ROWS>::kSmem, Cut<ROWS>::kThreads, nullptr) != cudaSuccess)
        return -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * split);
    cfg.blockDim = dim3(Cut<ROWS>::kThreads);
    cfg.dynamicSmemBytes = Cut<ROWS>::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, product_int8_kernel<GATED, ROWS>, &cfg) != cudaSuccess || n < 1) return -1;
    if (slot) cache[at][dev].store(n, std::memory_order_relaxed);
    return n;
}

template <bool GATED>
int resident_clusters(int rows, int split) {
    return rows <= 64 ? resident_clusters<GATED, 64>(split) : rows <= 128 ? resident_clusters<GATED, 128>(split) : resident_clusters<GATED, 256>(split);
}

// How a call is cut: rows of a tile (256 >> shift; a plan's are 256), pairs to a tile's K, and the
// most rows that the kernel takes at a time.
struct Plan {
    int shift, split, rows;
};

// The cut whose rounds of units are over first, by what a unit of 256 / 128 / 64 / 32 rows takes: 0.27 / 0.19 / 0.175 /
// 0.17 us per 64 of K (the products, or the weights' conversion), 2.2 / 1.5 / 0.5 / 0 for its sums that nothing
// overlaps, and, where pairs share its K, 0.015 a row and 0.8 a pair to join them. They share it only where
// every cluster has one tile, and only there a plan's tiles are cut (of 1 / 2 / 3 / 4 pairs 76 / 36 / 23 / 15 clusters are resident). Microseconds from 1 to
// 4 pairs: 128 rows 7168 -> 512 in one tile 27.6, 20.4, 18.0, 16.1, in two 24.6, 17.1, 15.2, 13.2, in four
// 23.8, 15.9, 13.6, 13.0; 64 rows 2048 -> 2048 in two 9.9, 9.0, 9.7; 139 rows 736 -> 320 gated in three 7.2, 8.3, 9.2.
template <bool GATED>
bool cut(const ProductInt8Args& p, Plan* best) {
    constexpr double kOfK[] = {0.27, 0.19, 0.175, 0.17}, kSums[] = {2.2, 1.5, 0.5, 0.0};
    double least = 0;
    const int stages = static_cast<int>(ceil_div(p.K, kStageK));
    const int64_t each = p.plan ? p.plan_rows / p.E : kPlanTileRows;  // an expert's rows on average
    for (int shift = 0; shift <= 3; ++shift) {
        const int size = kPlanTileRows >> shift;
        const int64_t tiles = p.plan ? static_cast<int64_t>(p.tile_cap) << shift : ceil_div(p.rows, size), units = tiles * ceil_div(p.N, kMTile);
        int takes = shift;  // what a unit takes: as one of the rows that it has
        while (takes < 3 && each <= kPlanTileRows >> (takes + 1)) ++takes;
        for (int split = 1; split <= kMostShare; ++split) {
            const int clusters = resident_clusters<GATED>(size, split);
            if (clusters < 1) {
                if (split == 1) return false;
                continue;
            }
            if (split > 1 && (units > clusters || stages < 2 * split)) continue;
            if (p.plan && shift > 0 && units > clusters) continue;
            const double time = static_cast<double>(ceil_div(units, clusters)) * (ceil_div(2 * stages, split) * kOfK[takes] + kSums[takes]) +
                                (split > 1 ? 0.015 * (kPlanTileRows >> takes) + 0.8 * split : 0.0);
            if (shift + split == 1 || time < least) {
                *best = Plan{shift, split, size};
                least = time;
            }
        }
    }
    return true;
}

// The test hook's numbers are the same in every form: 0, 1 and 4 to 7 are the warps of these roles, 3 the last one that takes
// sums out, and 8 to 11 a warp of each converting group, each of another quarter of the lanes.
template <int ROWS>
int32_t quitting_warp(int32_t number) {
    return number >= 8 ? 4 + Cut<ROWS>::kEpiWarps + 5 * (number - 8) : number == 3 ? 3 + Cut<ROWS>::kEpiWarps : number;
}

template <bool GATED, int ROWS>
cudaError_t launch_pairs(Args a, cudaStream_t stream) {
    a.quit_warp = quitting_warp<ROWS>(a.quit_warp);
    const ProductInt8Args& p = a.p;
    const int clusters = resident_clusters<GATED, ROWS>(a.split);
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    const int64_t most = (static_cast<int64_t>(p.tile_cap) << (p.plan ? a.shift : 0)) * ceil_div(p.N, kMTile);
    if (most > INT32_MAX) return cudaErrorInvalidValue;  // units are counted in 32 bits
    if (encoder() == nullptr) return cudaErrorNotSupported;
    CUtensorMap wmap, xmap;
    {
        const cuuint64_t kb = static_cast<cuuint64_t>(p.K), n = static_cast<cuuint64_t>(p.N);
        const cuuint64_t dims[3] = {kb, n, static_cast<cuuint64_t>(p.E)}, strides[2] = {kb, kb * n};
        const cuuint32_t box[3] = {kStageK, 128, 1};
        if (!encode(&wmap, p.wq, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.K), static_cast<cuuint64_t>(p.rows)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.x_stride)};
        const cuuint32_t box[2] = {kStageK, 32};
        if (!encode(&xmap, p.xq, 2, dims, strides, box)) return cudaErrorInvalidValue;
    }
    const unsigned ctas = 2u * static_cast<unsigned>(a.split), grid = ctas * static_cast<unsigned>(most < clusters ? most : clusters);
    return launch_pdl_cluster(product_int8_kernel<GATED, ROWS>, grid, Cut<ROWS>::kThreads, Cut<ROWS>::kSmem, ctas, stream, a, wmap, xmap);
}

template <bool GATED>
cudaError_t launch_cut(Args a, cudaStream_t stream) {
    Plan plan{0, 1, 256};
    if (!cut<GATED>(a.p, &plan)) return cudaErrorInvalidConfiguration;
    if (a.p.plan) {
        // By the rows that the routing gives an expert on average: more stages where they are few, against experts of more
        // rows than the kernel takes at a time, whose weights are read again. 256 experts 7168 -> 4096 with 2 / 31 / 64 / 96 /
        // 140 rows each: 1091 / 1109 / 1134 / 2218 / 3326 us with 64 at a time, 1176 / 1192 / 1219 / 1281 / 2411 with 128,
        // 1259 / 1302 / 1339 / 1388 / 1550 with 256; 8008 rows, one expert with 933: 1607 with 64, 1326 with 128; 24576
        // rows, one with 2872: 1791 with 128, 1716 with 256.
        const int64_t each = a.p.plan_rows / a.p.E;
        if (plan.split == 1 && plan.shift == 0) plan.rows = each <= 24 ? 64 : each <= 96 ? 128 : 256;
    } else {
        a.p.tile_cap = static_cast<int32_t>(ceil_div(a.p.rows, kPlanTileRows >> plan.shift));
    }
    a.shift = plan.shift;
    a.split = plan.split;
    return plan.rows <= 64 ? launch_pairs<GATED, 64>(a, stream) : plan.rows <= 128 ? launch_pairs<GATED, 128>(a, stream) : launch_pairs<GATED, 256>(a, stream);
}

}  // namespace

cudaError_t launch_product_int8(const ProductInt8Args& p, cudaStream_t stream) {
    if (p.tile_cap == 0) return cudaSuccess;
    // Few rows, dense. Up to 8 cost product_int8_rows.cu one pass over the weights: always (1 to 8 rows, 8192 -> 16384: 28 us
    // against 33). Up to 16 cost it more than that, which pays where the pairs would be short of units (7168 -> 4096: 13 us
    // against 27; 8192 -> 16384 has 64 units for the 76 pairs).
    if (p.plan == nullptr && (p.rows <= 8 || (p.rows <= kInt8FewRows && ceil_div(p.N, kMTile) * 4 <= device_sm_count())))
        return launch_product_int8_rows(p, stream);
    Args a{p, 0, 1, kWaitCycles, -1, p.err};
    take_product_wait_test(&a.wait_cycles, &a.quit_warp);
    return p.gated ? launch_cut<true>(a, stream) : launch_cut<false>(a, stream);
}

}  // namespace moe
