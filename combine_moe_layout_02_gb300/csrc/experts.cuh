// experts.cuh -- launchers of the operators around the experts (combine_grad.cu,
// fp4.cu, product.cu, expert.cu, gate.cu, norm.cu, product_int8.cu), called by the
// C-ABI layer and by ffn.cu. Arguments are validated before these run.
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
void take_product_wait_test(int64_t* wait_cycles, int32_t* quit_warp);  // leaves both where nothing is armed

// Rows and plan of the expert layer from topk_idx alone (one partition, experts
// at multiples of MOE_FP4_ROW_TILE rows).
int64_t expert_route_scratch_bytes(const moe_shape& s);
cudaError_t launch_expert_route(const moe_shape& s, const int32_t* topk_idx, int32_t* slot_row, int64_t* base,
                                int32_t* plan, int64_t plan_ints, int32_t* err, void* scratch, cudaStream_t stream);

// The router's gate and its gradient (gate.cu).
constexpr int kGateParts = 1216;  // most blocks that leave sums in the scratch
struct GateArgs {
    int32_t E, K, bf16, normalize;
    int64_t S;
    float scale, balance;
    const void* logits;
    int64_t row_stride;
    const uint8_t* mask;
    int32_t* topk_idx;  // read by the gradient
    float* topk_weights;
    int32_t* expert_count;  // [E + 1]; read by the gradient
    float* expert_prob;
    float* loss;
    float* part_prob;     // [kGateParts][E]
    int32_t* part_count;  // [kGateParts][E + 1]
    const float* dweights;
    const float* dloss;
    void* dlogits;
    int64_t dlogits_stride;
};
cudaError_t launch_gate(const GateArgs& a, cudaStream_t stream);
cudaError_t launch_gate_grad(const GateArgs& a, cudaStream_t stream);

// Root-mean-square norm, int8 rows (norm.cu). Strides are in bytes.
constexpr int kNormParts = 1216;  // most blocks that leave sums in the gradient's scratch
struct NormArgs {
    int64_t rows;
    int32_t H;
    float eps;
    const uint8_t* x;  // packing: the rows; unpacking: not used
    int64_t x_stride;
    const uint8_t* residual;
    int64_t residual_stride;
    const uint8_t* weight;
    uint8_t* sum;
    int64_t sum_stride;
    uint8_t* y;  // unpacking: the values
    int64_t y_stride;
    uint8_t* q;
    int64_t q_stride;
    uint8_t* q_scale;
    int64_t q_scale_stride;
    int32_t gated;       // packing: operands of group_rows rows whose gate and up rows go by turns
    int64_t group_rows;
    const int32_t* plan;  // packing: only the rows that it gives to experts
    int32_t E, tile_cap;
};
struct NormGradArgs {
    int64_t rows;
    int32_t H;
    float eps;
    const uint8_t* dy;
    int64_t dy_stride;
    const uint8_t* h;
    int64_t h_stride;
    const uint8_t* weight;
    const uint8_t* dsum;
    int64_t dsum_stride;
    uint8_t* dh;
    int64_t dh_stride;
    float* parts;  // [kNormParts][H], or NULL: no gradient of the weight
};
cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t stream);
cudaError_t launch_rms_norm_grad(const NormGradArgs& a, float* dweight, cudaStream_t stream);
cudaError_t launch_int8_pack(const NormArgs& a, cudaStream_t stream);
cudaError_t launch_int8_unpack(const NormArgs& a, cudaStream_t stream);

// Product of int8 operands (product_int8.cu). Strides are in bytes.
struct ProductInt8Args {
    int32_t E, N, K, gated, tile_cap;
    int64_t rows;
    const int8_t* wq;
    const float* ws;
    const int8_t* xq;
    int64_t x_stride;
    const uint8_t* xs;
    int64_t xs_stride;
    const int32_t* plan;  // NULL: all rows are the one expert's
    int64_t plan_rows;    // rows of the routings that the plan is made for, to a multiple of a tile's below
    uint16_t* y;
    int64_t y_stride;
    int32_t* err;
};
cudaError_t launch_product_int8(const ProductInt8Args& a, cudaStream_t stream);
// Dense calls of few rows (product_int8_rows.cu): of 1..kInt8FewRows.
constexpr int kInt8FewRows = 16;
cudaError_t launch_product_int8_rows(const ProductInt8Args& a, cudaStream_t stream);

// L2 cache of the current device, in bytes (cached).
int device_l2_bytes();

}  // namespace moe
