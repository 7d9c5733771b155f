/*
 * moe.h -- C ABI of libmoe.so, the GB300 (sm_103a) MoE dispatch/combine path.
 *
 * The path moves the hidden rows of S tokens to the expert-parallel ranks that
 * own their Top-K experts and reduces the experts' answers back:
 *
 *   moe_layout   topk_idx            -> per-rank / per-expert counts, token->rank table
 *   moe_notify   counts + table      -> prefix matrices, receive offsets, send_head
 *   moe_dispatch x + send_head       -> receive slots in P rank partitions (+ side arrays)
 *   moe_combine  expert rows (y)     -> out[S,H] = weighted sum over ranks
 *
 * The P expert-parallel ranks are P disjoint partitions of one receive arena
 * in this GPU's memory; "sending" a row to rank d means storing it in d's
 * partition. Source rank s owns global tokens [s*T, (s+1)*T), T = S / P.
 *
 * Problem statement followed ("Ascend DeepEP MoE Dispatch Optimization",
 * section "一条 token 如何走完 MoE"): inputs x[S,H], topk_idx[S,K],
 * topk_weights[S,K]; dst_rank = expert_id / experts_per_rank and
 * dst_local_expert = expert_id % experts_per_rank; one copy of the row per
 * distinct destination rank; combine returns the rows and reduces them by the
 * Top-K weights.
 *
 * Conventions for every entry point:
 *   - All array pointers are DEVICE pointers, owned and allocated by the
 *     caller. The library never allocates device or pinned memory.
 *   - Every call only enqueues work on `stream` (a cudaStream_t; NULL is the
 *     legacy default stream) and returns; results are ready when the stream
 *     reaches them. Nothing synchronises with the host.
 *   - The one exception to the two rules above is moe_run_host, the serving
 *     loop: it takes HOST buffers for the batches, uses its own streams and
 *     returns when the results are in host memory (see its declaration).
 *   - Arguments are validated on the host before anything is enqueued; a bad
 *     argument returns MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED and enqueues
 *     nothing. MOE_ERR_CUDA means a launch failed.
 *   - Data-dependent problems (an expert id >= E, a receive row outside its
 *     partition or the arena, an inconsistent send_head) cannot be seen on the
 *     host. The kernels skip the offending element -- they never read or
 *     write out of bounds -- and store a moe_status code into the caller's
 *     device word `err` (may be NULL). moe_layout and moe_dispatch_fused
 *     always write `err` (0 or a code); the other calls only ever write a
 *     non-zero code into it.
 *   - Row-major layouts; int32 counts; the bf16 payload is passed as uint16
 *     bit patterns.
 *   - Alignment: every array pointer must be 16-byte aligned (the error word
 *     4-byte, scratch 256-byte); allocations from cudaMalloc or the PyTorch
 *     caching allocator are 256-byte aligned. y_row_stride is a multiple of 16.
 *   - Results are deterministic: the same inputs give the same bits on every
 *     run (no floating-point atomics, fixed reduction orders).
 */
#ifndef MOE_H_
#define MOE_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,        /* bad pointer, size, alignment or shape      */
    MOE_ERR_TOPK_OUT_OF_RANGE = 2,  /* device: an expert id was >= E              */
    MOE_ERR_CAPACITY = 3,           /* device: a receive row fell outside its partition or the arena */
    MOE_ERR_CUDA = 4,               /* a CUDA launch or attribute call failed     */
    MOE_ERR_UNSUPPORTED = 5,        /* shape beyond the limits below              */
    MOE_ERR_DEVICE_TIMEOUT = 6,     /* device: a bounded wait on a copy gave up   */
    MOE_ERR_INCONSISTENT = 7        /* device: send_head names more ranks than the token's experts allow */
} moe_status;

/* Limits (the pages' CAM limits are P <= 384, E <= 512, K <= 16, H <= 7168). */
#define MOE_MAX_RANKS 1024
#define MOE_MAX_EXPERTS 4096
#define MOE_MAX_TOPK 16
#define MOE_MAX_HIDDEN 16384
/* Also S*K + E*(expert_alignment-1) <= INT32_MAX, so that every per-rank row
 * count and offset fits int32; larger shapes return MOE_ERR_UNSUPPORTED. */

/* Shape of one call. The tiling record of "HCCL Window 模式 (Non-SHMEM)
 * 代码深度剖析", section 8.1 (epWorldSize, moeExpertNum, quantMode, bs, k, h)
 * reduced to what the path needs. */
typedef struct moe_shape {
    int32_t P;                 /* expert-parallel ranks, 1..MOE_MAX_RANKS                  */
    int32_t E;                 /* experts, E % P == 0, P <= E <= MOE_MAX_EXPERTS            */
    int32_t S;                 /* global tokens, S % P == 0 (T = S / P per source rank), >= 0 */
    int32_t K;                 /* Top-K slots per token, 1..MOE_MAX_TOPK                    */
    int32_t H;                 /* hidden size, multiple of 8 (of 16 when quant = 1)          */
    int32_t num_channels;      /* C >= 1: shapes the channel prefix matrices only           */
    int32_t expert_alignment;  /* >= 1: per-expert receive counts are rounded up to it      */
    int32_t quant;             /* 0: bf16 payload; 1: int8 payload + fp32 scale             */
} moe_shape;

/* Human-readable name of a status code (static string). */
const char* moe_status_string(int32_t status);

/* Host-side check of a shape against the rules above. */
moe_status moe_check_shape(const moe_shape* shape);

/* Bytes per receive slot ("HCCL Window 模式 (Non-SHMEM) 代码深度剖析",
 * section 2.3 token format and section 8.2 size check):
 *   Ceil(Ceil(H * elt, 32) + 44, 512), elt = 2 (bf16) or 1 (int8).
 * Slot layout: payload [0, H*elt); fp32 scale at byte Ceil(H*elt, 32)
 * (int8 only; its 32-byte block is written, zero after the scale); int32
 * triple (source rank, source-local token, lowest k whose expert is on this
 * rank) at byte Ceil(H*elt, 32) + 32 (its 32-byte block is written, zero
 * after the triple); the rest is padding and is not written.
 * 14848 bytes for H = 7168 bf16. Returns -1 for H < 1. */
int64_t moe_slot_stride(int32_t H, int32_t quant);

/* Scratch bytes moe_layout, moe_notify, moe_notify_expert and
 * moe_dispatch_fused need for this shape (the calls may share one buffer; its
 * contents do not carry over between calls). */
int64_t moe_scratch_bytes(const moe_shape* shape);

/* Receive rows that always suffice when partitions are packed back to back
 * (part_row_base from moe_notify): S * min(K, P). */
int64_t moe_max_recv_rows(const moe_shape* shape);

/*
 * moe_layout -- the routing tables ("Ascend DeepEP MoE Dispatch
 * Optimization", sections "从 Python 接口进入真实调用链" and "Dispatch handle
 * 六项分别保存什么": num_tokens_per_rank, num_tokens_per_expert and the [S,P]
 * boolean is_token_in_rank).
 *
 *   topk_idx               int32 [S,K]  expert ids; any negative value is a
 *                                       masked slot; ids >= E are skipped and
 *                                       reported as MOE_ERR_TOPK_OUT_OF_RANGE
 *   num_tokens_per_rank    int32 [P,P]  [s][d] = tokens of source rank s with
 *                                       at least one expert on rank d
 *   num_tokens_per_expert  int32 [P,E]  [s][e] = slots of s's tokens equal to e
 *   is_token_in_rank       uint8 [S,P]  1 if token g has an expert on rank d
 *   is_token_in_rank_bits  uint32 [S,ceil(P/32)] or NULL: the same table packed,
 *                                       bit d%32 of word d/32
 *   err                    int32 device word or NULL; always written (0 or 2)
 *   scratch                >= moe_scratch_bytes(shape) bytes, 256-byte aligned
 */
moe_status moe_layout(const moe_shape* shape, const int32_t* topk_idx,
                      int32_t* num_tokens_per_rank, int32_t* num_tokens_per_expert,
                      uint8_t* is_token_in_rank, uint32_t* is_token_in_rank_bits,
                      int32_t* err, void* scratch, int64_t scratch_bytes, void* stream);

/*
 * moe_notify -- counts and prefixes ("Ascend DeepEP MoE Dispatch
 * Optimization", section "Notify 先交换数量和前缀"; per-expert alignment from
 * "internode.cu", section 1 notify_dispatch; receive position from section
 * "Device 侧如何把 channel 变成远端 Put").
 *
 *   inputs: num_tokens_per_rank [P,P], num_tokens_per_expert [P,E],
 *           is_token_in_rank [S,P] (as written by moe_layout)
 *   rank_prefix_matrix         int32 [P,P]   [s][d] = sum over s' <= s of num_tokens_per_rank[s'][d]
 *   channel_prefix_matrix      int32 [P,P,C] [s][d][c] = tokens of s in channels 0..c bound for d
 *                                            (channel c = c-th block of the balanced split of T
 *                                            tokens over C, first T % C blocks one larger:
 *                                            "HCCL Window 模式 (Non-SHMEM) 代码深度剖析", section 8.3)
 *   recv_channel_prefix_matrix int32 [P,P,C] [d][s][c] = first row of (s, c)'s tokens in d's partition
 *   num_recv_tokens            int32 [P]     rows received by each rank
 *   num_recv_tokens_per_expert int32 [P,E/P] slots per local expert, rounded up to expert_alignment
 *   recv_expert_offset         int32 [P,E/P] exclusive scan of the line above, per rank
 *   send_head                  int32 [S,P]   row of token g inside d's partition, or -1 if not sent:
 *                                            rank_prefix[s-1][d] + channel_prefix[s][d][c-1] +
 *                                            running count inside the channel
 *   part_row_base              int64 [P+1]   exclusive scan of num_recv_tokens: partitions packed
 *                                            back to back; part_row_base[P] = total rows
 *   scratch                    >= moe_scratch_bytes(shape) bytes, 256-byte aligned
 */
moe_status moe_notify(const moe_shape* shape, const int32_t* num_tokens_per_rank,
                      const int32_t* num_tokens_per_expert, const uint8_t* is_token_in_rank,
                      int32_t* rank_prefix_matrix, int32_t* channel_prefix_matrix,
                      int32_t* recv_channel_prefix_matrix, int32_t* num_recv_tokens,
                      int32_t* num_recv_tokens_per_expert, int32_t* recv_expert_offset,
                      int32_t* send_head, int64_t* part_row_base,
                      void* scratch, int64_t scratch_bytes, void* stream);

/*
 * moe_dispatch -- the permutation ("HCCL Window 模式 (Non-SHMEM) 代码深度剖析",
 * section 3.6 InputToShare with the dynamic quantisation steps and FillTriple;
 * one copy per distinct rank as in "Ascend DeepEP MoE Dispatch Optimization").
 *
 * For every token g and rank d with send_head[g][d] >= 0, slot row
 * part_row_base[d] + send_head[g][d] of the arena receives:
 *   quant = 0: the bf16 row x[g], bit for bit;
 *   quant = 1: q[h] = clamp(rint(f32(x[g][h]) / scale), -127, 127) as int8 and
 *              scale = amax / 127 (binary32, round to nearest even; amax = max|x[g]|;
 *              amax == 0 gives scale 0 and q 0). Defined for finite x: a row with
 *              an infinity or NaN gets unspecified codes and scale (no error);
 *   the triple (g / T, g % T, lowest k with topk_idx[g][k] / (E/P) == d).
 * Side arrays (each may be NULL), indexed by arena row:
 *   recv_src_idx      int32 [arena_rows]    g % T
 *   recv_topk_idx     int32 [arena_rows,K]  topk_idx % (E/P) where the expert is on d, else -1
 *   recv_topk_weights float [arena_rows,K]  topk_weights where the expert is on d, else 0
 *
 *   x                bf16 bits [S,H], 16-byte aligned
 *   topk_idx         int32 [S,K]; topk_weights float [S,K] (may be NULL when
 *                    recv_topk_weights is NULL)
 *   part_row_base    int64 [P+1] device: first arena row of each partition;
 *                    moe_notify's packed bases, or any caller-chosen bases
 *                    (e.g. d * capacity for fixed-capacity partitions)
 *   recv_arena       arena_rows * moe_slot_stride(H, quant) bytes, 16-byte aligned
 *   err              int32 device word or NULL: rows outside [part_row_base[d],
 *                    part_row_base[d+1]) or beyond arena_rows are skipped and
 *                    raise MOE_ERR_CAPACITY
 */
moe_status moe_dispatch(const moe_shape* shape, const uint16_t* x, const int32_t* topk_idx,
                        const float* topk_weights, const int32_t* send_head,
                        const int64_t* part_row_base, void* recv_arena, int64_t arena_rows,
                        int32_t* recv_src_idx, int32_t* recv_topk_idx, float* recv_topk_weights,
                        int32_t* err, void* stream);

/*
 * moe_combine -- the inverse permutation and weighted reduction ("HCCL Window
 * 模式 (Non-SHMEM) 代码深度剖析", section 7.8 ReadBufferAndWeightedSum: FP32
 * accumulator, Cast -> Muls -> Add per returned row, one CAST_RINT to BF16).
 *
 *   out[g][h] = bf16_rne( sum over d ascending with send_head[g][d] >= 0 of
 *                         c[g][d] * f32(y[part_row_base[d] + send_head[g][d]][h]) )
 *   c[g][d]   = sum, in ascending k, of topk_weights[g][k] over the slots whose
 *               expert is on d; 1 for every rank when topk_weights is NULL.
 * The accumulator starts at +0.0f; each product and each sum is rounded to
 * binary32 on its own (no fused multiply-add). A token with no valid rank
 * gives +0.
 *
 *   y             bf16 rows, y_row_stride bytes apart (a multiple of 16, >= 2H);
 *                 pass the dispatch arena with moe_slot_stride(H, 0) for
 *                 identity experts
 *   part_row_base int64 [P+1] device, as for moe_dispatch; arena_rows bounds the rows read
 *   send_head     int32 [S,P]; topk_idx int32 [S,K]; topk_weights float [S,K] or NULL
 *   out           bf16 bits [S,H], 16-byte aligned
 *   err           int32 device word or NULL (MOE_ERR_CAPACITY, MOE_ERR_INCONSISTENT)
 */
moe_status moe_combine(const moe_shape* shape, const void* y, int64_t y_row_stride,
                       const int64_t* part_row_base, int64_t arena_rows,
                       const int32_t* send_head, const int32_t* topk_idx,
                       const float* topk_weights, uint16_t* out, int32_t* err, void* stream);

/*
 * moe_dispatch_fused -- moe_layout + moe_notify + moe_dispatch in one launch,
 * for the small-message regime where the fixed cost of the routing tables
 * dominates the payload ("Ascend DeepEP MoE Dispatch Optimization", section
 * "128P 为什么会放大问题"; the single-kernel counting + prefix + copy shape of
 * "DeepEP Warp Specialization 深度分析", dispatch_impl). Every output has the
 * meaning, layout and value of the three separate calls with packed partitions
 * (part_row_base is written here and used for the rows).
 *
 * One cooperative persistent kernel (two CTAs per SM when their row buffers
 * fit in half an SM's shared memory, else one) with two bounded grid barriers;
 * the barrier counter lives in scratch and is zeroed by a one-thread kernel
 * launched on the stream just before. `err` is always written: cleared by the kernel, then
 * raised to MOE_ERR_TOPK_OUT_OF_RANGE, MOE_ERR_CAPACITY or
 * MOE_ERR_DEVICE_TIMEOUT if needed.
 * Supported: P <= 64, E <= 1024, H <= 8192, K <= 16, P * num_channels <= 4096,
 * quant = 0; other shapes return MOE_ERR_UNSUPPORTED (use the separate calls).
 * scratch >= moe_scratch_bytes.
 */
moe_status moe_dispatch_fused(const moe_shape* shape, const uint16_t* x, const int32_t* topk_idx,
                              const float* topk_weights, int32_t* num_tokens_per_rank,
                              int32_t* num_tokens_per_expert, uint8_t* is_token_in_rank,
                              uint32_t* is_token_in_rank_bits, int32_t* rank_prefix_matrix,
                              int32_t* channel_prefix_matrix, int32_t* recv_channel_prefix_matrix,
                              int32_t* num_recv_tokens, int32_t* num_recv_tokens_per_expert,
                              int32_t* recv_expert_offset, int32_t* send_head, int64_t* part_row_base,
                              void* recv_arena, int64_t arena_rows, int32_t* recv_src_idx,
                              int32_t* recv_topk_idx, float* recv_topk_weights, int32_t* err, void* scratch,
                              int64_t scratch_bytes, void* stream);

/*
 * Expert-major receive layout ("HCCL Window 模式 (Non-SHMEM) 代码深度剖析",
 * section 3.6 InputToShare and section 7.8 ReadBufferAndWeightedSum). Instead of
 * one row per (token, destination rank), every valid (token, k) slot gets its
 * own row, and rank d's partition holds its experts' rows expert by expert:
 * local expert l starts at recv_expert_offset[d][l] (counts rounded up to
 * expert_alignment; rows in the alignment gaps are not written), and inside an
 * expert the slots are in (token, k) order. Each expert's rows are contiguous,
 * ready for a grouped expert GEMM.
 *
 * moe_max_expert_rows: arena rows that always suffice: S*K + E*(expert_alignment-1).
 *
 * moe_notify_expert -- after moe_layout and moe_notify:
 *   topk_idx                   int32 [S,K]
 *   num_recv_tokens_per_expert int32 [P,E/P] and recv_expert_offset int32 [P,E/P] from moe_notify
 *   slot_row                   int32 [S,K]   row of slot (g,k) inside rank (topk_idx/(E/P))'s
 *                                            partition: recv_expert_offset[e] + the number of
 *                                            earlier slots (token-major order) of expert e;
 *                                            -1 for a masked or out-of-range slot
 *   expert_part_base           int64 [P+1]   exclusive scan of the ranks' aligned row totals
 *   scratch                    >= moe_scratch_bytes(shape) bytes, 256-byte aligned
 *
 * moe_dispatch_expert -- for every valid slot, row expert_part_base[d] + slot_row[g][k]
 *   receives the payload (bf16, or int8 + scale, as moe_dispatch), the triple
 *   (g / T, g % T, k), recv_src_idx[row] = g % T and recv_weight[row] =
 *   topk_weights[g][k] (1 if topk_weights is NULL). Side arrays may be NULL.
 *   Rows outside their partition or the arena are skipped (MOE_ERR_CAPACITY in err).
 *
 * moe_combine_expert --
 *   out[g] = bf16_rne( sum over k ascending with a valid slot of
 *                      w[g][k] * f32(y[expert_part_base[d] + slot_row[g][k]]) )
 *   binary32 accumulator from +0, each product and sum rounded on its own, w = 1
 *   when topk_weights is NULL. y rows are y_row_stride bytes apart.
 */
int64_t moe_max_expert_rows(const moe_shape* shape);
moe_status moe_notify_expert(const moe_shape* shape, const int32_t* topk_idx,
                             const int32_t* num_recv_tokens_per_expert, const int32_t* recv_expert_offset,
                             int32_t* slot_row, int64_t* expert_part_base, void* scratch,
                             int64_t scratch_bytes, void* stream);
moe_status moe_dispatch_expert(const moe_shape* shape, const uint16_t* x, const int32_t* topk_idx,
                               const float* topk_weights, const int32_t* slot_row,
                               const int64_t* expert_part_base, void* recv_arena, int64_t arena_rows,
                               int32_t* recv_src_idx, float* recv_weight, int32_t* err, void* stream);
moe_status moe_combine_expert(const moe_shape* shape, const void* y, int64_t y_row_stride,
                              const int64_t* expert_part_base, int64_t arena_rows, const int32_t* slot_row,
                              const int32_t* topk_idx, const float* topk_weights, uint16_t* out,
                              int32_t* err, void* stream);

/*
 * moe_combine_grad / moe_combine_expert_grad -- the backward pass of
 * moe_combine / moe_combine_expert. With dout the gradient of out,
 *
 *   dy[row]  = bf16_rne( c * f32(dout[g]) ) for every row that one of token g's
 *              slots has (rank layout: the rows of its slots' ranks, where
 *              send_head has one); c is that row's weight as in the forward call
 *              (rank layout: the sum, in ascending k, of the token's weights on
 *              the rank; 1 when topk_weights is NULL), one binary32 product;
 *   dw[g][k] = sum over h of f32(dout[g][h]) * f32(y[row of slot k][h]) in
 *              binary32; slots whose experts share a rank share its row (rank
 *              layout). 0 for a masked slot or a row that is skipped.
 *
 *   dout  bf16 bits [S,H]; y, y_row_stride, part_row_base (expert_part_base),
 *         arena_rows, send_head (slot_row), topk_idx, topk_weights: as in the
 *         forward call (y may be NULL when dw is)
 *   dy    bf16 rows, dy_row_stride bytes apart (a multiple of 16, >= 2H), in the
 *         arena's rows; NULL for no dy. Rows that no token owns (alignment gaps,
 *         rows past a partition's tokens) are not written. May not overlap y or dout.
 *   dw    float [S,K], every element written; NULL for no dw
 *   err   int32 device word or NULL (MOE_ERR_CAPACITY)
 *
 * The backward pass of dispatch (each row a copy of x[g]) is the forward
 * combine without weights: moe_combine / moe_combine_expert with topk_weights =
 * NULL sums the rows' gradients into dx[g].
 */
moe_status moe_combine_grad(const moe_shape* shape, const uint16_t* dout, const void* y, int64_t y_row_stride,
                            const int64_t* part_row_base, int64_t arena_rows, const int32_t* send_head,
                            const int32_t* topk_idx, const float* topk_weights, void* dy, int64_t dy_row_stride,
                            float* dw, int32_t* err, void* stream);
moe_status moe_combine_expert_grad(const moe_shape* shape, const uint16_t* dout, const void* y, int64_t y_row_stride,
                                   const int64_t* expert_part_base, int64_t arena_rows, const int32_t* slot_row,
                                   const int32_t* topk_idx, const float* topk_weights, void* dy,
                                   int64_t dy_row_stride, float* dw, int32_t* err, void* stream);

/*
 * MXFP4 rows (OCP Microscaling Formats v1.0: e2m1 elements under one ue8m0
 * power of two per 32 of them), for the experts' products.
 *
 * A row of `width` elements (a multiple of 32) is width / 2 bytes of codes, the
 * even element in the low nibble, rows packed back to back, and width / 32
 * scale bytes. A block whose largest magnitude is m has scale code
 * s = max(0, floor(log2 m) + 125) and its elements are rounded to the nearest
 * e2m1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6) times 2^(s - 127), ties to the even
 * code; magnitudes above 6 become 6. A block that holds an infinity or a NaN gets
 * s = 255 (NaN) and codes 0. Packing is exact to the bit.
 *
 * The scales of `rows` rows are ceil(rows / 128) * ceil(width / 128) chunks of
 * 512 bytes (moe_fp4_scale_bytes): chunk [row / 128][block / 4], in which the
 * 4 scales of row m are the bytes from (m % 32) * 16 + (m % 128) / 32 * 4 on. Scales
 * past the width are 0.
 *
 * Weights of E experts with N rows each are E such operands back to back
 * (groups = E, rows = N). Gated weights hold gate and up rows by turns: 16 gate
 * rows, then the 16 up rows that belong to them; gated = 1 makes moe_fp4_pack
 * take them from the usual order (all N / 2 gate rows, then all up rows).
 */
#define MOE_FP4_ROW_TILE 128
int64_t moe_fp4_scale_bytes(int64_t rows, int32_t width);

/*
 * moe_fp4_pack / moe_fp4_unpack -- bf16 rows to MXFP4, and back to the bf16
 * values they stand for (exact for every scale code that packing gives; under the
 * codes 253 and 254 the largest values are past bf16's range and become infinite).
 *
 *   groups, rows   groups >= 0 operands of rows >= 0 rows each; x and q hold
 *                  groups * rows rows, sf groups * moe_fp4_scale_bytes(rows, width) bytes
 *   width          a multiple of 32, at most MOE_FP4_MAX_WIDTH
 *   gated          0, or 1: x in gate / up order, the operand by turns (rows % 32 == 0)
 *   x              bf16 bits, rows x_row_stride bytes apart (a multiple of 16, >= 2 * width)
 *   q              uint8 [groups * rows, width / 2], 16-byte aligned
 *   sf             uint8, 16-byte aligned
 *   plan           NULL, or a plan of moe_expert_plan for E experts (plan_ints words):
 *                  only the rows that it gives to experts are read and written
 *                  (groups = 1, gated = 0, rows = the arena's, a multiple of 128).
 *                  Scales of the other rows of a 128-row tile become 0.
 */
#define MOE_FP4_MAX_WIDTH 32768
moe_status moe_fp4_pack(int32_t groups, int64_t rows, int32_t width, int32_t gated, const uint16_t* x,
                        int64_t x_row_stride, uint8_t* q, uint8_t* sf, int32_t E, const int32_t* plan,
                        int64_t plan_ints, void* stream);
moe_status moe_fp4_unpack(int32_t groups, int64_t rows, int32_t width, int32_t gated, const uint8_t* q,
                          const uint8_t* sf, uint16_t* x, int64_t x_row_stride, int32_t E, const int32_t* plan,
                          int64_t plan_ints, void* stream);

/*
 * moe_expert_plan -- where the experts' rows lie in the expert-major arena, and
 * the row tiles that the products run over. expert_alignment must be a multiple
 * of MOE_FP4_ROW_TILE, so that an expert's rows start at a scale chunk.
 *
 *   num_tokens_per_expert int32 [P,E] (from moe_layout)
 *   plan   int32 [plan_ints], plan_ints >= moe_expert_plan_ints(shape), 16-byte aligned:
 *          [0] row tiles, [1] arena rows in use (gaps included), [2] E, [3] 0;
 *          then, E4 = E rounded up to a multiple of 4: first arena row of each expert
 *          [E4], rows of each expert [E4], and the tiles [.., 4]: expert, first arena
 *          row, rows (1..MOE_PLAN_TILE_ROWS), 0
 *   err    int32 device word or NULL: MOE_ERR_INCONSISTENT if the counts are not
 *          those of a routing of this shape: an expert's sum over the ranks negative
 *          or more than S * K (it then has no rows), or more rows in all than
 *          moe_max_expert_rows (no expert then has any), or more tiles than fit
 */
#define MOE_PLAN_TILE_ROWS 256
int64_t moe_expert_plan_ints(const moe_shape* shape);
moe_status moe_expert_plan(const moe_shape* shape, const int32_t* num_tokens_per_expert, int32_t* plan,
                           int64_t plan_ints, int32_t* err, void* stream);

/*
 * moe_dispatch_expert_fp4 -- moe_dispatch_expert with an MXFP4 payload in the
 * products' operand layout: every valid slot's arena row expert_part_base[d] +
 * slot_row[g][k] of q / sf receives x[g] packed as by moe_fp4_pack (each token is
 * read and rounded once). H must be a multiple of 32; shape->quant is ignored.
 * The scales of other rows are not written.
 *
 *   q           uint8 [arena_rows, H / 2]; sf uint8 [moe_fp4_scale_bytes(arena_rows, H)]
 *   recv_src_idx int32 [arena_rows], recv_weight float [arena_rows] (each may be
 *               NULL), err: as for moe_dispatch_expert
 */
moe_status moe_dispatch_expert_fp4(const moe_shape* shape, const uint16_t* x, const int32_t* topk_idx,
                                   const float* topk_weights, const int32_t* slot_row,
                                   const int64_t* expert_part_base, uint8_t* q, uint8_t* sf, int64_t arena_rows,
                                   int32_t* recv_src_idx, float* recv_weight, int32_t* err, void* stream);

/*
 * moe_expert_product_fp4 -- the experts' linear layer on MXFP4 operands. For
 * every row r that the plan gives to expert e:
 *
 *   v[n] = sum over k of w_e[n][k] * x[r][k]           (products exact, binary32 sum)
 *   gated = 0: y[r][n] = bf16_rne(v[n]),               n < N
 *   gated = 1: y[r][i] = bf16_rne(silu(gate_i) * up_i), i < N / 2, gate_i and up_i the
 *              i-th gate and up row's v (weights held by turns), silu(a) = a / (1 + e^-a)
 *
 *   E, N, K     experts, weight rows per expert and row width: N and K multiples of
 *               32, N <= MOE_FP4_MAX_WIDTH * 2, K <= MOE_FP4_MAX_WIDTH
 *   wq, wsf     the weights' E operands of N x K
 *   xq, xsf     the rows' operand of arena_rows x K (arena_rows a multiple of 128; with
 *               0 rows nothing is enqueued, and err is not written)
 *   plan        moe_expert_plan's, plan_ints words
 *   y           bf16 rows of the same arena, y_row_stride bytes apart (a multiple of
 *               16, at least 2 bytes per value); rows that are no expert's are not written
 *   err         int32 device word or NULL: MOE_ERR_CAPACITY for a tile outside the arena
 *               or of no expert (skipped), MOE_ERR_DEVICE_TIMEOUT
 * All of q, sf, x, y 16-byte aligned. A row holding a NaN block gives NaN; no row
 * affects another.
 */
moe_status moe_expert_product_fp4(int32_t E, int32_t N, int32_t K, int32_t gated, const uint8_t* wq,
                                  const uint8_t* wsf, const uint8_t* xq, const uint8_t* xsf, int64_t arena_rows,
                                  const int32_t* plan, int64_t plan_ints, uint16_t* y, int64_t y_row_stride,
                                  int32_t* err, void* stream);

/*
 * moe_expert_ffn_fp4 -- the whole expert layer of one GPU:
 *
 *   out[g] = bf16_rne( sum over k ascending with a valid slot of
 *                      w[g][k] * f32(y_e) ),   y_e = W2_e h,  h = silu(gate) * up,  (gate, up) = W1_e x[g]
 *
 * with x and h rounded to MXFP4 (moe_fp4_pack) before each product, h and y to
 * bf16 after it, and combine's arithmetic. The same bits as moe_dispatch_expert_fp4,
 * moe_expert_product_fp4 (gated), moe_fp4_pack, moe_expert_product_fp4 and
 * moe_combine_expert give one after another, in one call and without the rank
 * tables. P, num_channels, expert_alignment and quant of the shape are only checked.
 *
 *   inner       a multiple of 32 (and H), at most MOE_FP4_MAX_WIDTH
 *   x           bf16 bits [S,H]; topk_idx int32 [S,K] (negative: masked; >= E: skipped and
 *               MOE_ERR_TOPK_OUT_OF_RANGE); topk_weights float [S,K] or NULL (1)
 *   w1q, w1sf   gated weights, E operands of 2 * inner x H; w2q, w2sf: E of H x inner
 *   h           NULL, or bf16 [moe_expert_ffn_fp4_rows(shape, inner), inner]: receives the
 *               inner rows, experts in order, each from a multiple of 128 on, in (token, k) order
 *   out         bf16 bits [S,H]
 *   workspace   >= moe_expert_ffn_fp4_workspace_bytes(shape, inner) bytes, 256-byte aligned;
 *               its contents do not carry over between calls
 *   err         int32 device word or NULL; only non-zero codes are written
 */
int64_t moe_expert_ffn_fp4_workspace_bytes(const moe_shape* shape, int32_t inner);
int64_t moe_expert_ffn_fp4_rows(const moe_shape* shape, int32_t inner);
moe_status moe_expert_ffn_fp4(const moe_shape* shape, int32_t inner, const uint16_t* x, const int32_t* topk_idx,
                              const float* topk_weights, const uint8_t* w1q, const uint8_t* w1sf, const uint8_t* w2q,
                              const uint8_t* w2sf, uint16_t* h, uint16_t* out, void* workspace,
                              int64_t workspace_bytes, int32_t* err, void* stream);

/*
 * moe_gate -- the router: Top-K experts, their weights, the experts' counts and
 * the balance loss, from the gate's logits. For token g, z = logits[g],
 * p = softmax(z):
 *
 *   topk_idx[g][k]     = the expert of the k-th largest logit; equal logits by
 *                        ascending expert (-0 equals 0)
 *   topk_weights[g][k] = scale * p[i_k] / D,  D = the sum of the token's chosen p
 *                        (normalize = 1) or 1 (normalize = 0)
 *   expert_count[e]    = slots that chose e;  expert_count[E] = n, tokens routed
 *   expert_prob[e]     = (sum over routed tokens of p[e]) / n, 0 for n = 0
 *   loss               = balance * E * sum over e of
 *                        (expert_count[e] / (K n)) * expert_prob[e], 0 for n = 0
 *
 * A token is not routed where mask[g] is 0 or all its logits are -infinity: its
 * ids are -1, its weights 0 and it is in no sum. An expert whose logit is
 * -infinity is not chosen: slots that find no expert hold -1 and 0. NaN counts as
 * the largest logit; a row with a NaN or +infinity has valid ids and weights NaN
 * (and makes expert_prob and the loss NaN). Ids and counts are exact; the exponentials
 * are the hardware's (binary32, off by up to 2^-21 + |z - max| 2^-23, relative).
 *
 *   shape        E, S and K are used; the rest is only checked
 *   type         of the logits (and of their gradient): MOE_F32 or MOE_BF16
 *   row_stride   bytes from row to row, a multiple of the element's size
 *   mask         uint8 [S] or NULL (all tokens)
 *   topk_idx     int32 [S,K]; topk_weights float [S,K]; expert_count int32 [E + 1]
 *   expert_prob  float [E] or NULL; loss float [1] or NULL
 *   scratch      >= moe_gate_scratch_bytes(shape) bytes, 256-byte aligned; its
 *                contents do not carry over between calls
 *
 * moe_gate_grad -- the gradient of the logits, from the gradients of the weights
 * (as combine's gradient gives them) and of the loss. Ids and counts are
 * constants of it:
 *
 *   a_k     = scale / D * (dw_k - (normalize ? sum over j of dw_j p[i_j] / D : 0))
 *   c[e]    = dloss * balance * E * expert_count[e] / (K n) / n
 *   dz[e]   = p[e] * (c[e] + sum over k with i_k = e of a_k - T),
 *   T       = sum over e of p[e] c[e] + sum over k of p[i_k] a_k
 *
 * and 0 for a token that is not routed. Slots with an id outside [0, E) take no
 * part (the forward call's -1, or slots that a program has dropped since: D is
 * then the sum over the others); an id that is there twice counts twice.
 *
 *   logits, mask, normalize, scale, balance   as in the forward call
 *   topk_idx, expert_count                    its results
 *   dweights     float [S,K] or NULL (0); dloss float [1] or NULL (0)
 *   dlogits      rows of `type`, dlogits_stride bytes apart; may not overlap logits (the
 *                same address is refused)
 */
#define MOE_F32 0
#define MOE_BF16 1
int64_t moe_gate_scratch_bytes(const moe_shape* shape);
moe_status moe_gate(const moe_shape* shape, int32_t type, const void* logits, int64_t row_stride, const uint8_t* mask,
                    int32_t normalize, float scale, float balance, int32_t* topk_idx, float* topk_weights,
                    int32_t* expert_count, float* expert_prob, float* loss, void* scratch, int64_t scratch_bytes,
                    void* stream);
moe_status moe_gate_grad(const moe_shape* shape, int32_t type, const void* logits, int64_t row_stride,
                         const uint8_t* mask, int32_t normalize, float scale, float balance, const int32_t* topk_idx,
                         const int32_t* expert_count, const float* dweights, const float* dloss, void* dlogits,
                         int64_t dlogits_stride, void* stream);

/*
 * moe_rms_norm -- root-mean-square norm of x + residual, rows of H bf16 values:
 *
 *   h = x + residual (binary32),  rstd = 1 / sqrt(mean h^2 + eps)
 *   sum = bf16_rne(h),  y = bf16_rne(v),  v = h * rstd * weight
 *   q_scale = max|v| / 127,  q = v / q_scale to the nearest whole number; a quotient
 *             within 2^-15 of a tie may go either way (v is not rounded on the way, so these
 *             are not moe_int8_pack's codes of y, which alone are dispatch's bit for bit).
 *             A row of zeros: 0; a row whose v holds an infinity or a NaN: q_scale NaN, codes 0
 *
 * Every result may be NULL, but not all of them.
 *
 *   rows, H      rows >= 0; H a multiple of 8 (of 16 with q), at most MOE_MAX_HIDDEN
 *   x, residual  bf16 bits; residual may be NULL (0)
 *   weight       bf16 bits [H]
 *   eps          finite, at least 2^-126
 *   q, q_scale   int8 rows and one float per row, both or none
 *   strides      bytes from row to row: multiples of 16, at least a row's bytes;
 *                q_scale_stride a multiple of 4 >= 4 (int8 slots of dispatch hold the
 *                scale behind the row: any pair of strides will do)
 * sum may be x or residual itself, y may be x, residual or neither (not also sum), with
 * the same stride; no other overlap.
 *
 * moe_rms_norm_grad -- its gradient at h (the sum as it was kept), without int8:
 *
 *   dh      = bf16_rne(rstd * (weight dy - h rstd^2 mean(weight dy h)) + dsum)
 *   dweight = sum over rows of dy h rstd            (binary32, fixed order)
 *
 * dh is the gradient of x and of the residual alike. dsum: the gradient of the
 * sum that was passed on, or NULL. dweight: float [H] or NULL; with it scratch
 * holds moe_rms_norm_grad_scratch_bytes(rows, H) bytes (256-byte aligned). dh may be
 * dy or dsum itself, with the same stride; no other overlap.
 */
moe_status moe_rms_norm(int64_t rows, int32_t H, float eps, const uint16_t* x, int64_t x_stride,
                        const uint16_t* residual, int64_t residual_stride, const uint16_t* weight, uint16_t* sum,
                        int64_t sum_stride, uint16_t* y, int64_t y_stride, int8_t* q, int64_t q_stride, float* q_scale,
                        int64_t q_scale_stride, void* stream);
int64_t moe_rms_norm_grad_scratch_bytes(int64_t rows, int32_t H);
moe_status moe_rms_norm_grad(int64_t rows, int32_t H, float eps, const uint16_t* dy, int64_t dy_stride,
                             const uint16_t* h, int64_t h_stride, const uint16_t* weight, const uint16_t* dsum,
                             int64_t dsum_stride, uint16_t* dh, int64_t dh_stride, float* dweight, void* scratch,
                             int64_t scratch_bytes, void* stream);

/*
 * moe_int8_pack / moe_int8_unpack -- bf16 rows to int8 with a scale per row, bit
 * for bit as dispatch's int8 payload (quant = 1) has them, and back to
 * bf16_rne(q * scale). A row that holds an infinity or a NaN gets the scale NaN and
 * codes 0. Weights are packed by output channel: a channel is a row.
 *
 *   groups, rows   groups >= 0 operands of rows >= 0 rows each, back to back
 *   width          a multiple of 16, at most MOE_INT8_MAX_WIDTH
 *   gated          0, or 1: x holds all gate rows, then all up rows of an operand
 *                  (rows % 32 == 0), the operand 16 gate rows and their 16 up rows by turns
 *   x              bf16 bits, rows x_row_stride bytes apart (a multiple of 16, >= 2 * width);
 *                  it and q may not overlap
 *   q              int8, rows q_row_stride bytes apart (a multiple of 16, >= width)
 *   scale          float, scale_stride bytes apart (a multiple of 4, >= 4)
 *   plan           NULL, or a plan of moe_expert_plan for E experts (plan_ints words):
 *                  only the rows that it gives to experts are read and written
 *                  (groups = 1, gated = 0)
 */
#define MOE_INT8_MAX_WIDTH 32768
moe_status moe_int8_pack(int32_t groups, int64_t rows, int32_t width, int32_t gated, const uint16_t* x,
                         int64_t x_row_stride, int8_t* q, int64_t q_row_stride, float* scale, int64_t scale_stride,
                         int32_t E, const int32_t* plan, int64_t plan_ints, void* stream);
moe_status moe_int8_unpack(int32_t groups, int64_t rows, int32_t width, int32_t gated, const int8_t* q,
                           int64_t q_row_stride, const float* scale, int64_t scale_stride, uint16_t* x,
                           int64_t x_row_stride, int32_t E, const int32_t* plan, int64_t plan_ints, void* stream);

/*
 * moe_expert_product_int8 -- the linear layer on int8 rows and weights, a scale per
 * row and per output channel. For every row r of expert e:
 *
 *   v[n] = (sum over k of wq_e[n][k] * xq[r][k]) * ws_e[n] * xs[r]
 *          (products exact, binary32 sum: exact below 2^24)
 *   gated = 0: y[r][n] = bf16_rne(v[n]),               n < N
 *   gated = 1: y[r][i] = bf16_rne(silu(gate_i) * up_i), i < N / 2, gate_i and up_i the
 *              i-th gate and up row's v (weights held by turns, as moe_int8_pack
 *              makes them), silu(a) = a / (1 + e^-a)
 *
 *   E, N, K        experts, weight rows per expert (a multiple of 32, at most
 *                  2 * MOE_INT8_MAX_WIDTH) and row width (a multiple of 16, at most
 *                  MOE_INT8_MAX_WIDTH)
 *   wq, ws         int8 [E,N,K], float [E,N]
 *   xq             int8 rows, x_row_stride bytes apart (a multiple of 16, >= K)
 *   xs             float, xs_stride bytes apart (a multiple of 4, >= 4). Of dispatch's
 *                  int8 slots xq is the arena, xs the arena + Ceil(H, 32), and both
 *                  strides moe_slot_stride(H, 1)
 *   rows           rows of xq and y (with 0 nothing is enqueued, and err is not written)
 *   plan           moe_expert_plan's for E experts, plan_ints words; or NULL with E = 1:
 *                  all rows are the one expert's (a dense layer)
 *   y              bf16 rows, y_row_stride bytes apart (a multiple of 16, at least 2
 *                  bytes per value); rows that are no expert's are not written
 *   err            int32 device word or NULL: MOE_ERR_CAPACITY for a tile outside the rows
 *                  or of no expert (skipped), MOE_ERR_DEVICE_TIMEOUT
 * A row whose scale is NaN gives NaN; no row affects another.
 */
moe_status moe_expert_product_int8(int32_t E, int32_t N, int32_t K, int32_t gated, const int8_t* wq, const float* ws,
                                   const int8_t* xq, int64_t x_row_stride, const float* xs, int64_t xs_stride,
                                   int64_t rows, const int32_t* plan, int64_t plan_ints, uint16_t* y,
                                   int64_t y_row_stride, int32_t* err, void* stream);

/*
 * moe_pad_partitions -- fixed-length receive partitions ("Ascend DeepEP MoE
 * Dispatch Optimization", section "输出长度有动态和固定两种模式": with a fixed
 * output length, num_worst_tokens, the host reads no count back and the rows
 * past the received count are padding -- x, scales and weights 0, topk_idx -1).
 *
 * With fixed-capacity partitions (part_row_base[d] = d * capacity, passed to
 * moe_dispatch) this fills, for every rank d, the rows from
 * part_row_base[d] + num_recv_tokens[d] up to part_row_base[d+1] (and below
 * arena_rows): payload 0, the scale block 0 (int8 slots), the triple
 * (-1, -1, -1), recv_src_idx -1, recv_topk_idx -1, recv_topk_weights 0 (each
 * side array may be NULL). A partition that overflowed (count > capacity) has
 * no padding; moe_dispatch reports the overflow rather than truncating.
 *
 *   num_recv_tokens int32 [P] (from moe_notify); part_row_base int64 [P+1];
 *   recv_arena / side arrays as for moe_dispatch. Only padding rows are written.
 */
moe_status moe_pad_partitions(const moe_shape* shape, const int32_t* num_recv_tokens,
                              const int64_t* part_row_base, void* recv_arena, int64_t arena_rows,
                              int32_t* recv_src_idx, int32_t* recv_topk_idx, float* recv_topk_weights,
                              void* stream);

/*
 * moe_layout_static_scratch -- moe_layout without a caller-provided scratch
 * buffer. The pages have no counterpart: this entry point exists for callers
 * that cannot allocate device memory, such as code hosted by an engine that
 * owns all device memory and forbids allocation after start-up, or serving
 * loops where cudaMalloc would stall the device. Inputs, outputs and results
 * are those of moe_layout; the one scratch array moe_layout needs (an
 * out-of-range flag per source rank, folded into err) is a buffer of
 * MOE_LAYOUT_STATIC_SCRATCH_BYTES compiled into the library, which every GPU
 * that loads the library holds until the process exits.
 *   - The buffer holds the flags of the largest shape moe_check_shape
 *     accepts (MOE_MAX_RANKS source ranks). A shape needing more is refused
 *     with MOE_ERR_UNSUPPORTED before anything is enqueued (moe_check_shape
 *     already refuses every such shape the same way).
 *   - The first call on each device looks up the buffer's device address
 *     (with that device current) and keeps it for the life of the process;
 *     make that first call before any stream capture. The kept address
 *     assumes the device's primary context is never reset or destroyed
 *     (cudaDeviceReset): after a reset, do not call this entry point again
 *     in the same process.
 *   - All calls share the buffer, which keeps the last call's contents;
 *     every flag is written before it is read, so nothing needs to start at
 *     zero. Calls that overlap on the GPU (different streams or threads)
 *     race on it: serialise them. Calls enqueued one after another on one
 *     stream are serialised by the stream.
 *   - Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 */
#define MOE_LAYOUT_STATIC_SCRATCH_BYTES (MOE_MAX_RANKS * 4u)
moe_status moe_layout_static_scratch(const moe_shape* shape, const int32_t* topk_idx,
                                     int32_t* num_tokens_per_rank, int32_t* num_tokens_per_expert,
                                     uint8_t* is_token_in_rank, uint32_t* is_token_in_rank_bits,
                                     int32_t* err, void* stream);

/*
 * moe_run_host -- the whole path (moe_layout -> moe_notify -> moe_dispatch ->
 * moe_combine, or moe_dispatch_fused -> moe_combine) over n_batches batches
 * held in HOST memory, end to end: each batch's x, topk_idx and topk_weights
 * are copied to the device, routed, exchanged and reduced, and its combined
 * rows are copied back to out_host[i]. The pages have no single call for
 * this; it is the serving loop around the path ("Ascend DeepEP MoE Dispatch
 * Optimization", section "一条 token 如何走完 MoE": route, exchange, reduce,
 * per batch).
 *
 * Three internal streams overlap consecutive batches: while batch i computes,
 * batch i + 1's inputs are copied in and batch i - 1's output is copied out.
 * Inputs and outputs are double-buffered in the workspace; all other buffers
 * are used in batch order. The call is blocking: it first waits for all work
 * already submitted to the device, and returns when every copy has landed in
 * host memory. It is not capturable in a CUDA graph.
 *
 *   x_host[i]            bf16 bits [S,H] of batch i (pinned host memory for
 *                        copies that overlap; any host memory is accepted)
 *   topk_idx_host[i]     int32 [S,K]
 *   topk_weights_host    NULL (unit weights, as in moe_combine) or an array of
 *                        n_batches pointers to float [S,K]
 *   out_host[i]          bf16 bits [S,H], written with batch i's combine
 *                        result; entries may alias (batches are written back
 *                        in order)
 *   y, y_row_stride      expert outputs read by combine, device memory of at
 *                        least max(moe_max_recv_rows, moe_max_expert_rows)
 *                        rows; NULL means identity experts (combine reads the
 *                        bf16 dispatch arena, quant must be 0)
 *   flags                0 (rank-major layout), MOE_RUN_FUSED (use
 *                        moe_dispatch_fused when it supports the shape,
 *                        otherwise the separate calls) or MOE_RUN_EXPERT (the
 *                        expert-major layout: moe_notify_expert,
 *                        moe_dispatch_expert, moe_combine_expert); not both
 *   workspace            >= moe_run_host_workspace_bytes(shape, n_batches)
 *                        device bytes, 256-byte aligned, owned by the caller
 *   err_host             NULL or int32 [n_batches] host array: each batch's
 *                        device error word (0, or a moe_status code)
 * Returns MOE_OK, a host-side error (nothing run), MOE_ERR_CUDA, or the first
 * nonzero device error word in batch order.
 */
#define MOE_RUN_FUSED 1
#define MOE_RUN_EXPERT 2
int64_t moe_run_host_workspace_bytes(const moe_shape* shape, int32_t n_batches);
moe_status moe_run_host(const moe_shape* shape, int32_t n_batches, const uint16_t* const* x_host,
                        const int32_t* const* topk_idx_host, const float* const* topk_weights_host,
                        uint16_t* const* out_host, const void* y, int64_t y_row_stride, int32_t flags,
                        void* workspace, int64_t workspace_bytes, int32_t* err_host);

/*
 * moe_exchange_plan -- HOST function, for the path spread over P GPUs (one
 * expert-parallel rank each). After every rank has run moe_layout on its own
 * T tokens, the ranks all-gather their rows of num_tokens_per_rank and
 * num_tokens_per_expert ("internode.cu", section 1 notify_dispatch: counts
 * exchanged, then global prefix sums; "Ascend DeepEP MoE Dispatch
 * Optimization", section "Notify 先交换数量和前缀"). From the gathered tables
 * this computes what rank `self` needs before any row moves; every value is
 * the one moe_notify computes from the full tables.
 *
 *   ntpr_all [P,P], ntpe_all [P,E]   int32, host: row s = rank s's layout row
 *   rank_prefix_matrix [P,P]         int32, host (or NULL): inclusive column prefix
 *   num_recv_tokens [P]              int32, host (or NULL): rows each rank receives
 *   send_row_base [P]                int64, host (or NULL): first row of self's
 *                                    tokens inside rank d's receive partition
 *   self_recv_tokens_per_expert [E/P] int32, host (or NULL): self's experts'
 *                                    receive counts, rounded up to expert_alignment
 *   self_recv_expert_offset [E/P]    int32, host (or NULL): their exclusive scan
 *   part_row_base [P+1]              int64, host (or NULL): the packed bases of all
 *                                    partitions (the one-GPU emulation's layout)
 * Touches no device. Returns MOE_ERR_INVALID_ARG for a bad rank or a negative
 * count, MOE_ERR_UNSUPPORTED if a count overflows int32.
 */
moe_status moe_exchange_plan(const moe_shape* shape, int32_t self, const int32_t* ntpr_all,
                             const int32_t* ntpe_all, int32_t* rank_prefix_matrix, int32_t* num_recv_tokens,
                             int64_t* send_row_base, int32_t* self_recv_tokens_per_expert,
                             int32_t* self_recv_expert_offset, int64_t* part_row_base);

/*
 * moe_test_fused_barrier -- test hook for the bounded waits of
 * moe_dispatch_fused; the pages have no counterpart. It arms the NEXT
 * moe_dispatch_fused call made by this host thread (and that call only):
 * each of its grid barriers gives up after `spin_limit` polls (instead of
 * several million), and if skip_cta >= 0 the CTA with that index leaves out
 * its arrival at the first barrier. Every CTA's wait then runs out: the call
 * records MOE_ERR_DEVICE_TIMEOUT in err, each CTA waits (bounded) for its own
 * row loads to land and returns, and the context stays usable. It exists so
 * that tests can make a device-side wait time out without a fault. Returns
 * MOE_ERR_INVALID_ARG for spin_limit = 0.
 */
moe_status moe_test_fused_barrier(uint32_t spin_limit, int32_t skip_cta);

/*
 * moe_test_product_wait -- test hook for the bounded waits of the experts'
 * products. It arms the NEXT product of this host thread (moe_expert_product_fp4,
 * moe_expert_product_int8 but for dense calls of few rows, which wait on nothing, or
 * the first product of moe_expert_ffn_fp4; that one only): its waits give up
 * after `wait_cycles` clock cycles (instead of 2^32), and if quit_warp >= 0 that
 * warp of each CTA (0 loads, 1 issues, 4..11 take the sums out; of int8 codes
 * 4..7 and 3, the last of its kind, take the sums out and 8..11 are one of each
 * group that converts) acts as if its first wait had run out. The call records MOE_ERR_DEVICE_TIMEOUT in err, every
 * role ends, what is in flight lands (bounded), and the context stays usable;
 * results are undefined. Returns MOE_ERR_INVALID_ARG for wait_cycles = 0 or a
 * quit_warp outside -1..11.
 */
moe_status moe_test_product_wait(uint32_t wait_cycles, int32_t quit_warp);

/*
 * moe_profile_attach -- profile builds only (compiled with -DMOE_PROFILE into
 * libmoe_profile.so; the default libmoe.so has no such symbol and its kernels
 * record nothing). The pages' "Ascend DeepEP MoE Dispatch Optimization",
 * section "Device 侧计时": per-core phase times written to exclusive slots
 * behind a compile-time switch that costs nothing when off.
 *
 * Points every instrumented kernel at `slots`, a device array of
 * MOE_PROF_KERNELS * MOE_PROF_CTAS * MOE_PROF_PHASES uint64 (bytes >= that
 * times 8, 16-byte aligned), or detaches them (slots = NULL). Thereafter CTA b
 * of kernel k writes row (k * MOE_PROF_CTAS + b) * MOE_PROF_PHASES:
 *   slot 0: %globaltimer (ns) when the CTA starts its work (after waiting for
 *           the previous kernel on the stream);
 *   slot p >= 1: the CTA's clock64 cycles from then to the end of phase p,
 *           or, for the int8 consumer's per-token steps, that step's cycles
 *           summed over the CTA's first consumer warp's tokens (added to:
 *           clear the array before a run).
 *   slot MOE_PROF_PHASES - 1: 1 + the SM the CTA ran on (%smid).
 * Kernel ids: 0 layout, 1 notify (either kernel), 2 dispatch bf16, 3 dispatch
 * int8, 4 combine, 5 fused, 6 notify_expert's rows kernel, 7 its count
 * kernel. CTAs at or beyond MOE_PROF_CTAS record nothing. Synchronous (a copy to each kernel unit's device pointer); call it
 * with no work of this library in flight. Outputs are unchanged.
 */
#define MOE_PROF_KERNELS 8
#define MOE_PROF_CTAS 4096
#define MOE_PROF_PHASES 16
#ifdef MOE_PROFILE
moe_status moe_profile_attach(void* slots, int64_t bytes);
#endif

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* MOE_H_ */
