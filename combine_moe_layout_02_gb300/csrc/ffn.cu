// ffn.cu -- moe_expert_ffn_fp4: the whole expert layer in one call. Routing
// (expert.cu), the packing dispatch (fp4.cu), gate and up product with SwiGLU and
// packing (product.cu), down product, weighted reduction (combine.cu): six
// launches (five for a batch of one routing chunk), each overlapping the start
// of the next.
//
// The call emulates no ranks: all experts' rows are one partition, which is
// why the rank tables of moe_layout and moe_notify are not needed.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.cuh"
#include "moe.h"

namespace moe {
namespace {

// The call's arrays in its workspace; with base == nullptr only the size.
struct FfnBuffers {
    int32_t *slot_row, *plan;
    int64_t* base;
    void* scratch;
    uint8_t *xq, *xsf, *hq, *hsf;
    uint16_t* y;
    int64_t rows, plan_ints, total;
};

FfnBuffers carve(const moe_shape& s, int32_t inner, unsigned char* base) {
    FfnBuffers b{};
    int64_t off = 0;
    auto take = [&](int64_t bytes) -> void* {
        void* p = base ? static_cast<void*>(base + off) : nullptr;
        off += round_up(bytes > 0 ? bytes : 1, 256);
        return p;
    };
    const int64_t slots = static_cast<int64_t>(s.S) * s.K;
    const int64_t hit = s.E < slots ? s.E : slots;  // experts that can have rows
    b.rows = round_up(slots + hit * (kFp4Tile - 1), kFp4Tile);
    b.plan_ints = plan_tiles_at(s.E) + 4 * (s.E + slots / kPlanTileRows);
    b.slot_row = static_cast<int32_t*>(take(slots * 4));
    b.base = static_cast<int64_t*>(take(16));
    b.plan = static_cast<int32_t*>(take(b.plan_ints * 4));
    b.scratch = take(expert_route_scratch_bytes(s));
    b.xq = static_cast<uint8_t*>(take(b.rows * (s.H / 2)));
    b.xsf = static_cast<uint8_t*>(take(moe_fp4_scale_bytes(b.rows, s.H)));
    b.hq = static_cast<uint8_t*>(take(b.rows * (inner / 2)));
    b.hsf = static_cast<uint8_t*>(take(moe_fp4_scale_bytes(b.rows, inner)));
    b.y = static_cast<uint16_t*>(take(b.rows * s.H * 2));
    b.total = off;
    return b;
}

moe_status check(const moe_shape* s, int32_t inner) {
    const moe_status st = moe_check_shape(s);
    if (st != MOE_OK) return st;
    if (inner < 1 || inner % 32 != 0 || s->H % 32 != 0) return MOE_ERR_INVALID_ARG;
    if (inner > MOE_FP4_MAX_WIDTH) return MOE_ERR_UNSUPPORTED;
    // rows are int32
    if (static_cast<int64_t>(s->S) * s->K + static_cast<int64_t>(s->E) * (kFp4Tile - 1) > INT32_MAX - kFp4Tile)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool bad(const void* p, uintptr_t align) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % align != 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int64_t moe_expert_ffn_fp4_workspace_bytes(const moe_shape* shape, int32_t inner) {
    if (check(shape, inner) != MOE_OK) return -1;
    return carve(*shape, inner, nullptr).total;
}

int64_t moe_expert_ffn_fp4_rows(const moe_shape* shape, int32_t inner) {
    if (check(shape, inner) != MOE_OK) return -1;
    return carve(*shape, inner, nullptr).rows;
}

moe_status moe_expert_ffn_fp4(const moe_shape* shape, int32_t inner, const uint16_t* x, const int32_t* topk_idx,
                              const float* topk_weights, const uint8_t* w1q, const uint8_t* w1sf, const uint8_t* w2q,
                              const uint8_t* w2sf, uint16_t* h, uint16_t* out, void* workspace,
                              int64_t workspace_bytes, int32_t* err, void* stream) {
    moe_status st = check(shape, inner);
    if (st != MOE_OK) return st;
    const moe_shape& s = *shape;
    if (bad(w1q, 16) || bad(w1sf, 16) || bad(w2q, 16) || bad(w2sf, 16) || bad(workspace, 256)) return MOE_ERR_INVALID_ARG;
    if ((h && bad(h, 16)) || (topk_weights && bad(topk_weights, 16)) || (err && bad(err, 4))) return MOE_ERR_INVALID_ARG;
    if (s.S > 0 && (bad(x, 16) || bad(topk_idx, 16) || bad(out, 16))) return MOE_ERR_INVALID_ARG;
    FfnBuffers b = carve(s, inner, static_cast<unsigned char*>(workspace));
    if (workspace_bytes < b.total) return MOE_ERR_INVALID_ARG;
    if (s.S == 0) return MOE_OK;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    moe_shape one = s;  // one partition
    one.P = 1;
    cudaError_t e = launch_expert_route(one, topk_idx, b.slot_row, b.base, b.plan, b.plan_ints, err, b.scratch, cs);
    if (e == cudaSuccess)
        e = launch_dispatch_fp4(one, x, topk_idx, topk_weights, b.slot_row, b.base, b.xq, b.xsf, b.rows, nullptr, nullptr,
                                err, cs);
    // The inner rows are packed as they come out of the first product; a caller
    // that wants them in bf16 too has them written and packed by another launch.
    if (e == cudaSuccess)
        e = launch_product(s.E, 2 * inner, s.H, 1, w1q, w1sf, b.xq, b.xsf, b.rows, b.plan, b.plan_ints, h,
                           2 * static_cast<int64_t>(inner), h ? nullptr : b.hq, h ? nullptr : b.hsf, err, cs);
    if (h && e == cudaSuccess)
        e = launch_fp4_pack(false, 1, b.rows, inner, 0, h, 2 * static_cast<int64_t>(inner), b.hq, b.hsf, b.plan, s.E,
                            b.plan_ints, cs);
    if (e == cudaSuccess)
        e = launch_product(s.E, s.H, inner, 0, w2q, w2sf, b.hq, b.hsf, b.rows, b.plan, b.plan_ints, b.y,
                           2 * static_cast<int64_t>(s.H), nullptr, nullptr, err, cs);
    if (e == cudaSuccess) {
        CombineArgs c{};
        c.P = 1;
        c.E = s.E;
        c.K = s.K;
        c.H = s.H;
        c.epr = s.E;
        c.S = s.S;
        c.y = reinterpret_cast<const uint8_t*>(b.y);
        c.y_stride = 2 * static_cast<int64_t>(s.H);
        c.part_row_base = b.base;
        c.arena_rows = b.rows;
        c.topk_idx = topk_idx;
        c.topk_weights = topk_weights;
        c.out = out;
        c.err = err;
        c.slot_row = b.slot_row;
        e = launch_combine_expert(one, c, cs);
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
