// experts.cuh -- launchers of the experts' operators (combine_grad.cu, fp4.cu,
// product.cu, expert.cu), called by the C-ABI layer and by ffn.cu. Arguments are
// validated before these run.
#pragma once

#include "moe_device.cuh"

namespace moe {

struct CombineGradArgs {
    int32_t P, E, K, H, epr;
    int64_t S;
    const uint16_t* dout;
    const uint8_t* y;
    int64_t y_stride;
    const int64_t* part_row_base;
    int64_t arena_rows;
    const int32_t* send_head;  // rank layout
    const int32_t* slot_row;   // expert layout
    const int32_t* topk_idx;
    const float* topk_weights;
    uint8_t* dy;
    int64_t dy_stride;
    float* dw;
    int32_t* err;
};
cudaError_t launch_combine_grad(const moe_shape& s, const CombineGradArgs& a, cudaStream_t stream);
cudaError_t launch_combine_expert_grad(const moe_shape& s, const CombineGradArgs& a, cudaStream_t stream);

// MXFP4 (fp4.cu, product.cu).
cudaError_t launch_fp4_pack(bool unpack, int32_t groups, int64_t rows, int32_t width, int32_t gated, uint16_t* x,
                            int64_t x_stride, uint8_t* q, uint8_t* sf, const int32_t* plan, int32_t E,
                            int64_t plan_ints, cudaStream_t stream);
cudaError_t launch_expert_plan(const moe_shape& s, const int32_t* ntpe, int32_t* plan, int64_t plan_ints, int32_t* err,
                               cudaStream_t stream);
cudaError_t launch_dispatch_fp4(const moe_shape& s, const uint16_t* x, const int32_t* topk_idx, const float* topk_weights,
                                const int32_t* slot_row, const int64_t* part_row_base, uint8_t* q, uint8_t* sf,
                                int64_t arena_rows, int32_t* recv_src_idx, float* recv_weight, int32_t* err,
                                cudaStream_t stream);
cudaError_t launch_product(int32_t E, int32_t N, int32_t K, int32_t gated, const uint8_t* wq, const uint8_t* wsf,
                           const uint8_t* xq, const uint8_t* xsf, int64_t rows, const int32_t* plan, int64_t plan_ints,
                           uint16_t* y, int64_t y_stride, uint8_t* hq, uint8_t* hsf, int32_t* err,
                           cudaStream_t stream);  // hq, hsf: packed gated rows instead of y
// Test hook behind moe_test_product_wait (this host thread's next product).
constexpr int kProductWarps = 12;  // warps of a product's CTA
void arm_product_wait_test(uint32_t wait_cycles, int32_t quit_warp);

// Rows and plan of the expert layer from topk_idx alone (one partition, experts
// at multiples of MOE_FP4_ROW_TILE rows).
int64_t expert_route_scratch_bytes(const moe_shape& s);
cudaError_t launch_expert_route(const moe_shape& s, const int32_t* topk_idx, int32_t* slot_row, int64_t* base,
                                int32_t* plan, int64_t plan_ints, int32_t* err, void* scratch, cudaStream_t stream);

// L2 cache of the current device, in bytes (cached).
int device_l2_bytes();

}  // namespace moe
