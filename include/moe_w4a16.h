/*
 * libmoe_w4a16 — mixture-of-experts FFN layer with 4-bit (E2M1) expert weights and bf16 activations
 * (W4A16), hand-written HIP for AMD Instinct MI355X (gfx950).
 *
 * Pages this interface follows (cited by title and section):
 *   [Atlas] "告别Python堆栈：Atlas用纯Rust重写LLM推理，在GB10上跑赢vLLM",
 *           section "编译时内核选择和W4A16 Grouped GEMM": one launch per projection covering all
 *           experts (gate_up, then down); packed FP4 weights dequantized inside the matmul with no
 *           bf16 weight write-back; a grid sized by the number of row tiles per expert (max_m_tiles).
 *           Section "KV Cache量化、MTP推测解码和调试工具链": missing zero-initialisation and a broken
 *           max_m_tiles heuristic as MoE failure modes (so outputs here never rely on the caller
 *           zeroing them, and tile counts are computed exactly on the device).
 *   [ATOM]  "AMD ATOM推理引擎：如何用分页KV缓存和分段编译实现大模型推理性能翻倍",
 *           section "8.1 MoE 路径：路由、专家并行与 MORI 通信": routing, top-k selection, expert
 *           compute and the final combine.  Section "8.2 量化并非单一格式，而是一套执行契约": dtype,
 *           scale shape and layout form the kernel's contract.  Section "6.1 Linear：按量化类型分派
 *           GEMM": per-1x32 scaling of 4-bit weights.
 *   [RustDL] "Rust 实现深度学习推理引擎：从计算图到异构硬件加速", section "四、算子融合：性能翻倍的关键":
 *           the activation (SiLU) fused into the producing matmul.
 *
 * Conventions for every call
 *   - Pointers are DEVICE pointers unless stated; bf16 values are passed as their uint16_t bits.
 *   - Every device pointer must be 16-byte aligned (128-bit loads) unless stated otherwise.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).  Calls only enqueue
 *     work on it and return; there is no host<->device synchronisation.
 *   - The caller allocates and owns every buffer, workspaces included.  The library allocates
 *     nothing, frees nothing and keeps no pointer after a call returns.
 *   - Inputs are read-only.  Outputs are fully overwritten; no zero-initialisation is expected.
 *   - Arguments are validated on the host before anything is launched; a failing call returns a
 *     negative status, launches nothing and records a message for moe_last_error().
 *   - Results are deterministic: identical inputs give identical output bits (no floating-point
 *     atomics).
 *   - Calls that share a workspace or output buffer must not overlap in time.
 *
 * Weight format (the layer's contract)
 *   - Element: E2M1 (1 sign, 2 exponent bits with bias 1, 1 mantissa bit; values 0, ±0.5, ±1, ±1.5,
 *     ±2, ±3, ±4, ±6).  Two codes per byte: byte j of a row holds element 2j in bits 0..3 and element
 *     2j+1 in bits 4..7.
 *   - Scale: one bf16 per 32 consecutive K elements of a row.  Weight value = E2M1(code) * scale.
 *   - gate_up weights: codes w13_q [E, 2I, H/2], scales w13_s [E, 2I, H/32]; rows [0, I) are the
 *     gate projection, rows [I, 2I) the up projection.
 *   - down weights: codes w2_q [E, H, I/2], scales w2_s [E, H, I/32].
 *
 * Packed layout (optional, from moe_w4_prepack; same values, same total size): for each block of
 *   16 consecutive rows and 128 consecutive K elements (blocks ordered expert, row block, K block),
 *   1024 bytes of codes in the order the kernel's 64 lanes consume them, then separately 128 bytes
 *   of scales [16 rows][4 groups].  It exists so that each wave-level load is one contiguous block
 *   (the ATOM page, 8.2, lists weight pre-rearrangement as part of a quantized format's contract).
 *   Requires N % 16 == 0 and K % 128 == 0; a gate_up tensor read with SILU_MUL also needs
 *   N % 32 == 0, so that its up rows (from N/2) start a block.  A grouped GEMM gives the same bits
 *   with either layout; the layer does too, except where the packed layout's 128-row tiles take the
 *   exact fp16 path below (canonical weights never do), which agrees within the layer tolerance.
 *
 * Numerics: E2M1 codes are exact in bf16; each 32-element group is reduced by bf16 MFMA into an
 * fp32 partial that is multiplied by the group's scale in fp32; accumulation is fp32.  h (the
 * SiLU-mul output) is stored as bf16 (round to nearest even), the down-projection output as fp16
 * with an in-band power-of-two exponent per row and 8 columns (MOE_OUT_F16E), and the combine sums the k
 * slots in fp32 in slot order before one rounding of y to bf16.  Layers whose experts average more
 * than 256 rows with packed weights (128-row tiles) run the exact fp16 path instead: x in fp16 with a
 * power-of-two exponent per row (moe_x_to_f16), weights formed exactly in fp16 as code * scale and
 * reduced by fp16 MFMA with fp32 accumulation, and h in fp16 with exponents per row and 32 columns
 * (moe_grouped_gemm_w4f16).
 */
#ifndef MOE_W4A16_H
#define MOE_W4A16_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t moe_status_t;

#define MOE_OK 0
#define MOE_ERR_INVALID_ARG (-1)       /* NULL pointer, negative size, k > E, bad enum */
#define MOE_ERR_UNSUPPORTED_SHAPE (-2) /* size outside the supported range (see each call) */
#define MOE_ERR_MISALIGNED (-3)        /* a pointer is not 16-byte aligned */
#define MOE_ERR_WORKSPACE (-4)         /* workspace or tile buffer smaller than required */
#define MOE_ERR_HIP (-5)               /* a HIP launch failed */

#define MOE_EPI_NONE 0     /* C[r, n] = sum_k A[row(r), k] * W_e[n, k]                          */
#define MOE_EPI_SILU_MUL 1 /* C[r, j] = silu(G[r, j]) * G[r, N/2 + j], G the NONE result, j < N/2 */

#define MOE_OUT_BF16 0
#define MOE_OUT_F32 1
/* fp16 with an in-band power-of-two exponent per row and 8-column segment: a segment is 8 plain
 * fp16 values (round to nearest even) when its largest finite magnitude m is 0 or in [2^-6, 2^15) and
 * it holds no non-finite value; otherwise it is scaled by 2^-exp, exp = floor(log2 m) - 14 clamped to
 * [-110, 113] (exact), its first element is replaced by a marker, the fp16 quiet NaN
 * 0x7E00 | (exp + 256), and that element's scaled value is written to C_side[row, col / 8] (fp32).
 * Every value of a marked segment is then (fp16 or side value) * 2^exp.  No unmarked segment holds a
 * NaN.  The layer writes the down projection this way: half the bytes of fp32, 3 more significant
 * bits than bf16, and fp32's range. */
#define MOE_OUT_F16E 3
/* SiLU*mul output of moe_grouped_gemm_w4f16: h as fp16 [R_out, N/2] (round to nearest even) with a
 * signed exponent per row and block of 32 columns: row r's values in block j are fp16(h / 2^exp), exp =
 * 0 unless the row's largest finite |h| m in that block is 2^15 or more, or below 2^-6 but not 0 (then
 * exp = floor(log2 m) - 14 clamped to [-110, 113], which scales m into [2^14, 2^15) exactly).  C_aux
 * uint8 [max_tiles, ceil(N/2/32)] flags, per tile and block, whether any row of the tile has a nonzero
 * exponent there; C_aux2 int8 [R_out, ceil(N/2/32)] holds the exponents, written only for flagged
 * blocks. */
#define MOE_OUT_H16 4

#define MOE_LAYOUT_CANONICAL 0 /* the weight format above */
#define MOE_LAYOUT_PACKED 1    /* the same codes and scales re-laid out by moe_w4_prepack */

#define MOE_MAX_EXPERTS 1024

/* Version of this interface (incremented on any incompatible change). */
int32_t moe_abi_version(void);

/* Static text of a status code. */
const char* moe_status_string(moe_status_t status);

/* Text of the most recent failure on the calling host thread ("" if none).  Valid until the
 * thread's next call into the library. */
const char* moe_last_error(void);

/*
 * Top-k routing [ATOM, 8.1]: for each token t, softmax over the E router logits, keep the k
 * largest probabilities and renormalise them to sum to 1.
 *   logits    fp32 [T, E] row-major, finite values.
 *   topk_ids  int32 [T, k] out: expert ids; slot 0 holds the largest logit.  Equal logits are
 *             ordered by lower expert id; the ids of one token are distinct.
 *   topk_w    fp32 [T, k] out: renormalised weights, w_s = exp(l_s - l_0) / sum_j exp(l_j - l_0).
 * Shapes: T >= 0 (T == 0 launches nothing), 1 <= k <= E <= MOE_MAX_EXPERTS.
 * Alignment: 4 bytes suffices for all three pointers.
 */
moe_status_t moe_route_topk(const float* logits, int32_t T, int32_t E, int32_t k, int32_t* topk_ids,
                            float* topk_w, void* stream);

/*
 * Upper bound on the number of row tiles moe_align can emit: floor(T*k / block_m) + min(E, T*k).
 * Host-only, pure.  Returns -1 for invalid arguments.
 */
int32_t moe_max_tiles(int32_t T, int32_t k, int32_t E, int32_t block_m);

/* Device scratch bytes moe_align needs for these sizes (0 when it runs in one workgroup). */
size_t moe_align_workspace_bytes(int32_t T, int32_t k, int32_t E);

/*
 * Token -> expert permutation (moe_align) [Atlas, 编译时内核选择和W4A16 Grouped GEMM: per-expert
 * row tiles; KV Cache量化…调试工具链: the max_m_tiles failure mode].  A stable counting sort of the
 * R = T*k flat slots f = t*k + s by expert id topk_ids[f]:
 *   expert_counts  int32 [E]    out: rows routed to each expert.
 *   expert_offsets int32 [E+1]  out: exclusive prefix sum of the counts; offsets[E] = R.
 *   sorted_ids     int32 [R]    out: the flat slot at permuted row r; within an expert the slots
 *                               appear in ascending f, experts in ascending id.
 *   inv_perm       int32 [R]    out: permuted row of flat slot f (inverse of sorted_ids).
 *   tiles          int32 [max_tiles, 3] out: (expert, first permuted row, rows <= block_m) for each
 *                               block of up to block_m consecutive rows of one expert, experts
 *                               ascending then rows ascending.  Entries past *num_tiles are unused.
 *   num_tiles      int32 [1]    out: number of tiles written (stays on the device).
 *   workspace      device scratch of at least moe_align_workspace_bytes(T, k, E) bytes (may be
 *                  NULL when that is 0).
 * Shapes: T >= 0, 1 <= k <= E <= MOE_MAX_EXPERTS, 1 <= block_m <= 4096,
 *         max_tiles >= moe_max_tiles(T, k, E, block_m), T*k < 2^26.
 * topk_ids must hold ids in [0, E) with no repeats within a token (as moe_route_topk produces).
 */
moe_status_t moe_align(const int32_t* topk_ids, int32_t T, int32_t k, int32_t E, int32_t block_m,
                       int32_t* expert_counts, int32_t* expert_offsets, int32_t* sorted_ids,
                       int32_t* inv_perm, int32_t* tiles, int32_t max_tiles, int32_t* num_tiles,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Re-lay out one weight tensor from the canonical layout into the packed layout (see above).
 *   w_q [E, N, K/2], w_s [E, N, K/32] (canonical, device) -> packed_q (E*N*K/2 bytes) and packed_s
 *   (E*N*K/32 bf16), device buffers owned by the caller, not overlapping the inputs.
 * Shapes: 1 <= E <= MOE_MAX_EXPERTS, N >= 16, N % 16 == 0, K >= 128, K % 128 == 0.
 * Alignment: w_q, packed_q 16 bytes; w_s, packed_s 2 bytes (packed_s 8 bytes for use by the GEMMs).
 * Done once per weight tensor (e.g. at load time); every later call can read the packed copy.
 */
moe_status_t moe_w4_prepack(const uint8_t* w_q, const uint16_t* w_s, int32_t E, int32_t N, int32_t K,
                            uint8_t* packed_q, uint16_t* packed_s, void* stream);

/*
 * Grouped W4A16 GEMM, one launch over all experts [Atlas, 编译时内核选择和W4A16 Grouped GEMM].
 * For every tile (e, row0, rows) of `tiles` and every permuted row r in [row0, row0+rows):
 *   a(r) = a_row_of ? a_row_of[r] / a_row_div : r                (activation row)
 *   G[r, n] = sum_{kk<K} A[a(r), kk] * E2M1(Wq[e, n, kk]) * Ws[e, n, kk/32]      (n < N)
 *   MOE_EPI_NONE:     C[r, n] = G[r, n]                                  C is [R_out, N]
 *   MOE_EPI_SILU_MUL: C[r, j] = silu(G[r, j]) * G[r, N/2 + j]            C is [R_out, N/2]
 * with silu(g) = g / (1 + exp(-g)) [RustDL, 四、算子融合].  Rows of C that no tile covers are not
 * written.
 *   A          bf16 [*, K] row-major activations (gate_up: the tokens x, with a_row_of = sorted_ids
 *              and a_row_div = k; down: h in permuted order with a_row_of = NULL).
 *   Wq, Ws     [E, N, K/2] codes and [E, N, K/32] bf16 scales (the weight format above), in
 *              weight_layout MOE_LAYOUT_CANONICAL or MOE_LAYOUT_PACKED (then N % 16 == 0 -- with
 *              SILU_MUL N % 32 == 0 --, K % 128 == 0 and Ws 8-byte aligned).
 *   tiles, num_tiles  as written by moe_align with the same block_m; max_tiles is the capacity
 *              passed to moe_align (it sizes the launch; tiles past *num_tiles cost nothing).
 *   block_m    one of 16, 32, 64, 128.  With block_m 16 and max_tiles <= 32 the four waves of a
 *              workgroup split K (fp32 partial sums added in wave order), so bits can differ from a
 *              call with a larger capacity; both stay within the same error bound, and identical
 *              arguments always give identical bits.
 *   out_dtype  MOE_OUT_BF16 (round to nearest even), MOE_OUT_F32, or (NONE only) MOE_OUT_F16E:
 *              C fp16 [R_out, N] with side values C_side fp32 [R_out, ceil(N/8)] (see
 *              MOE_OUT_F16E; C_side is written only for marked segments, and is ignored for the
 *              other kinds and may then be NULL).  SILU_MUL requires BF16.
 * Shapes: 1 <= E <= MOE_MAX_EXPERTS, N >= 1 (N even for SILU_MUL), K % 32 == 0, K >= 32,
 *         N*K/2 < 4 GiB (one expert's codes).
 * Alignment: A, Wq, C 16 bytes; Ws 2 bytes.
 */
moe_status_t moe_grouped_gemm_w4a16(const uint16_t* A, const int32_t* a_row_of, int32_t a_row_div,
                                    const uint8_t* Wq, const uint16_t* Ws, int32_t weight_layout,
                                    int32_t E, int32_t N,
                                    int32_t K, const int32_t* tiles, int32_t max_tiles,
                                    const int32_t* num_tiles, int32_t block_m, int32_t epilogue,
                                    void* C, int32_t out_dtype, float* C_side, void* stream);

/*
 * Activations for the exact fp16 path of the grouped GEMM (moe_grouped_gemm_w4f16):
 *   x16[t, c] = fp16(x[t, c] * 2^-x_exp[t]) (round to nearest even), x_exp[t] = floor(log2 m) - 14
 *   where m is row t's largest finite |x| (x_exp = 0 for an all-zero row; clamped to [-110, 113]).
 * The row's largest magnitude lands in [2^14, 2^15): every value at most 2^31 below it is exact in
 * fp16; non-finite values stay non-finite.
 *   x bf16 [T, H]; x16 fp16 [T, H]; x_exp int32 [T].  Shapes: T >= 0, H % 8 == 0.
 */
moe_status_t moe_x_to_f16(const uint16_t* x, int32_t T, int32_t H, uint16_t* x16, int32_t* x_exp, void* stream);

/*
 * Grouped W4A16 GEMM, exact fp16 form [Atlas, 编译时内核选择和W4A16 Grouped GEMM: dequantization inside
 * the matmul]: the same result as moe_grouped_gemm_w4a16 with activations given in fp16 with power-
 * of-two exponents.  Each weight E2M1(code) * scale is formed in fp16, exact when the bf16 scale has
 * an exponent in [-16, 12], so every product is exact and the fp32 MFMA accumulation carries the group
 * scales with it.  A K step holding any other scale (zero, subnormal, non-finite, out of that range),
 * or h blocks with exponents, takes a general form: the scale is split into an fp16-exact part and a
 * power of two, and the fp32 accumulators are scaled by that power of two (exactly) around each group.
 *   A          fp16 [*, K]: with a_row_of (gathered rows, e.g. x16 of moe_x_to_f16) activation row a
 *              is A[a] * 2^a_row_exp[a] (a_row_exp NULL: exponents 0); with a_row_of NULL (h of the
 *              previous SILU_MUL call, with its two exponent arrays as a_blk_flag and a_row_blk_exp)
 *              row r's values in K columns [32j, 32j+32) are A * 2^a_row_blk_exp[r * ceil(K/32) + j]
 *              when a_blk_flag[i * ceil(K/32) + j] is nonzero for r's tile i, else A (a_blk_flag
 *              NULL: no exponents).
 *   block_m    64, or 128 with MOE_LAYOUT_PACKED weights (the tile list of moe_align with it).
 *   epilogue   MOE_EPI_SILU_MUL with out_dtype MOE_OUT_H16 (C fp16 [R_out, N/2], C_aux and C_aux2 the
 *              exponent flags and exponents, see MOE_OUT_H16), or MOE_EPI_NONE with MOE_OUT_F32 (C
 *              fp32) or MOE_OUT_F16E (C fp16, C_aux fp32 side values [R_out, ceil(N/8)]); C_aux2 is
 *              used by SILU_MUL only.
 * Other arguments, shapes and alignment as for moe_grouped_gemm_w4a16.
 */
moe_status_t moe_grouped_gemm_w4f16(const uint16_t* A, const int32_t* a_row_exp, const uint8_t* a_blk_flag,
                                    const uint8_t* a_row_blk_exp, const int32_t* a_row_of, int32_t a_row_div,
                                    const uint8_t* Wq, const uint16_t* Ws, int32_t weight_layout, int32_t E, int32_t N,
                                    int32_t K, const int32_t* tiles, int32_t max_tiles, const int32_t* num_tiles,
                                    int32_t block_m, int32_t epilogue, void* C, int32_t out_dtype, void* C_aux,
                                    uint8_t* C_aux2, void* stream);

/*
 * Routing-weighted scatter-reduce (combine) [ATOM, 8.1]:
 *   y[t, c] = bf16( sum_{s=0}^{k-1} topk_w[t, s] * O[inv_perm[t*k + s], c]  (+ shared[t, c]) )
 * summed in fp32 in ascending slot order, then the shared term (if any) added, rounded once to bf16.
 *   O          expert outputs in permuted row order, [T*k, H]: o_dtype MOE_OUT_F32 (fp32, O_side
 *              ignored) or MOE_OUT_F16E (fp16 with in-band exponents and side values O_side fp32
 *              [T*k, H/8], the down projection's output kind in the layer; each value decodes
 *              exactly to fp32);
 *   inv_perm int32 [T*k]; topk_w fp32 [T, k]; shared fp32 [T, H] or NULL (the shared-expert output
 *   of moe_dense_ffn_w4a16, added with weight 1 [Atlas, KV Cache量化、MTP推测解码和调试工具链]);
 *   y bf16 [T, H] out.
 * Shapes: T >= 0, k >= 1, H % 8 == 0.
 */
moe_status_t moe_combine(const void* O, int32_t o_dtype, const float* O_side, const int32_t* inv_perm,
                         const float* topk_w, const float* shared, int32_t T, int32_t k, int32_t H, uint16_t* y,
                         void* stream);

/*
 * Router gate logits [Atlas, KV Cache量化、MTP推测解码和调试工具链: the gate input and the gate logits
 * of each MoE layer; ATOM, 8.1: the logits the top-k routing reads]:
 *   logits[t, e] = sum_h x[t, h] * w_router[e, h], bf16 products accumulated in fp32 (MFMA order,
 *   so not bit-identical to another summation order).
 *   x bf16 [T, H]; w_router bf16 [E, H]; logits fp32 [T, E] out (4-byte aligned).
 * Shapes: 0 <= T < 2^26 (T == 0 launches nothing), 1 <= E <= MOE_MAX_EXPERTS, H % 32 == 0, H >= 32.
 */
moe_status_t moe_router_logits(const uint16_t* x, const uint16_t* w_router, int32_t T, int32_t H, int32_t E,
                               float* logits, void* stream);

/* Workspace bytes moe_dense_ffn_w4a16 needs (host-only, pure; 0 on invalid sizes). */
size_t moe_dense_ffn_workspace_bytes(int32_t T, int32_t H, int32_t I);

/*
 * Dense W4A16 SwiGLU FFN: one expert applied to every token (the shared expert of an MoE block
 * [Atlas, KV Cache量化、MTP推测解码和调试工具链]), on the same grouped-GEMM kernels with every row in
 * one group:
 *   out[t] = W2 ( silu(W1 x[t]) * (W3 x[t]) ), h rounded to bf16 between the projections.
 *   x bf16 [T, H]; w13_q [2I, H/2], w13_s [2I, H/32], w2_q [H, I/2], w2_s [H, I/32] in the weight
 *   format above (one expert, E = 1), all in weight_layout; out fp32 [T, H].
 *   workspace: device scratch of at least moe_dense_ffn_workspace_bytes(T, H, I) bytes (holds h).
 * Shapes: T >= 0 (T == 0 launches nothing), H and I positive multiples of 32 (of 128 when packed),
 *         T < 2^26.
 */
moe_status_t moe_dense_ffn_w4a16(const uint16_t* x, int32_t T, int32_t H, int32_t I, const uint8_t* w13_q,
                                 const uint16_t* w13_s, const uint8_t* w2_q, const uint16_t* w2_s,
                                 int32_t weight_layout, float* out, void* workspace, size_t workspace_bytes,
                                 void* stream);

/* Row-tile height (block_m) moe_ffn_forward uses for these sizes and weight layout (host-only,
 * pure; -1 on invalid sizes or layout).  Lets a caller run the same launch configuration through
 * the separate entry points.  moe_ffn_workspace_bytes covers every layout's choice. */
int32_t moe_ffn_block_m(int32_t T, int32_t E, int32_t k, int32_t weight_layout);

/* Workspace bytes moe_ffn_forward needs for these sizes (host-only, pure; 0 on invalid sizes). */
size_t moe_ffn_workspace_bytes(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k);

/*
 * The whole MoE FFN layer [ATOM, 8.1; Atlas, 编译时内核选择和W4A16 Grouped GEMM]:
 *   route (moe_route_topk) -> permute (moe_align) -> gate_up grouped GEMM with SiLU*mul fused
 *   -> down grouped GEMM -> combine, all enqueued on `stream`:
 *   y[t] = sum_s w[t,s] * W2_e(s) ( silu(W1_e(s) x[t]) * (W3_e(s) x[t]) ),  e(s) = topk_ids[t, s].
 *   x bf16 [T, H]; router_logits fp32 [T, E]; weights in the format above, all four tensors in
 *   weight_layout (MOE_LAYOUT_PACKED needs H % 128 == 0 and I % 128 == 0); y bf16 [T, H] out.
 *   topk_ids_out int32 [T, k], topk_w_out fp32 [T, k]: optional copies of the routing (NULL = skip).
 *   workspace: device scratch of at least moe_ffn_workspace_bytes(T, H, I, E, k) bytes.
 * Shapes: T >= 0 (T == 0 launches nothing), 1 <= k <= E <= MOE_MAX_EXPERTS, H % 32 == 0,
 *         I % 32 == 0, H >= 32, I >= 32, T*k < 2^26, H*I < 4 GiB (one expert's gate_up codes).
 * Diagnostics: with MOE_DUMP=1 in the environment (read on every call), the call then synchronises
 *   `stream` and prints one line to stderr: shape, tile height and count, rows per expert (least,
 *   most, experts without rows), most tiles of one expert, the ten largest logits of token 0 and
 *   the L2 norms of x and y [Atlas, KV Cache量化、MTP推测解码和调试工具链: per-layer expert-id dump].
 *   Results are unchanged; nothing is printed for a stream under graph capture; a failing copy
 *   returns MOE_ERR_HIP.  moe_ffn_block_forward does the same; moe_ffn_forward_noalloc never dumps.
 */
moe_status_t moe_ffn_forward(const uint16_t* x, const float* router_logits, int32_t T, int32_t H,
                             int32_t I, int32_t E, int32_t k, const uint8_t* w13_q,
                             const uint16_t* w13_s, const uint8_t* w2_q, const uint16_t* w2_s,
                             int32_t weight_layout, uint16_t* y, int32_t* topk_ids_out, float* topk_w_out, void* workspace,
                             size_t workspace_bytes, void* stream);

/* Bytes of the static device scratch array that moe_ffn_forward_noalloc works in (64 MiB). */
#define MOE_NOALLOC_SCRATCH_BYTES (64u << 20)
size_t moe_ffn_noalloc_scratch_bytes(void);

/*
 * moe_ffn_forward for callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation.  Same arguments, layouts, results and
 * errors as moe_ffn_forward minus the workspace: the intermediate buffers (routing, permutation,
 * tile list, h, O) live in one static device array of MOE_NOALLOC_SCRATCH_BYTES inside the library.
 * The call allocates nothing (no hipMalloc, no allocating library routine) and launches exactly the
 * kernels moe_ffn_forward launches, so its outputs are bit-identical to moe_ffn_forward's.
 *   - Limit: sizes whose moe_ffn_workspace_bytes exceeds MOE_NOALLOC_SCRATCH_BYTES are rejected with
 *     MOE_ERR_WORKSPACE before anything touches the device (the 800-token, 256-expert, H = 2048,
 *     I = 512 layer needs about 39 MB; every decode batch of a few hundred tokens fits).
 *   - Each GPU holds its own copy of the array from the first call on that device (the calling
 *     thread's current device, which `stream` must belong to) until the process ends.
 *   - All calls on one GPU share that GPU's array: calls that overlap in time on one GPU (two streams,
 *     two host threads) race and must be serialised by the caller.
 */
moe_status_t moe_ffn_forward_noalloc(const uint16_t* x, const float* router_logits, int32_t T, int32_t H, int32_t I,
                                     int32_t E, int32_t k, const uint8_t* w13_q, const uint16_t* w13_s,
                                     const uint8_t* w2_q, const uint16_t* w2_s, int32_t weight_layout, uint16_t* y,
                                     int32_t* topk_ids_out, float* topk_w_out, void* stream);

/* Workspace bytes moe_ffn_block_forward needs (host-only, pure; 0 on invalid sizes).  Is = 0 means
 * no shared expert. */
size_t moe_ffn_block_workspace_bytes(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k, int32_t Is);

/*
 * The whole MoE block from the hidden states [Atlas, KV Cache量化、MTP推测解码和调试工具链: gate input,
 * gate logits, routed output and shared-expert output of a layer]:
 *   logits = moe_router_logits(x, w_router); (when Is > 0) s = moe_dense_ffn_w4a16(x, shared weights);
 *   y = moe_ffn_forward(x, logits, ...) with s added in the combine (weight 1).
 *   w_router bf16 [E, H]; the routed weights as for moe_ffn_forward; Is = shared-expert intermediate
 *   size (0 = none, the four shared pointers are then ignored), shared weights w13s_q [2Is, H/2],
 *   w13s_s [2Is, H/32], w2s_q [H, Is/2], w2s_s [H, Is/32] in weight_layout.
 *   logits_out fp32 [T, E], topk_ids_out int32 [T, k], topk_w_out fp32 [T, k]: optional copies
 *   (NULL = skip).  workspace: at least moe_ffn_block_workspace_bytes(T, H, I, E, k, Is) bytes.
 * Shapes: those of moe_ffn_forward; Is >= 0, and Is > 0 follows the rules for I.
 */
moe_status_t moe_ffn_block_forward(const uint16_t* x, const uint16_t* w_router, int32_t T, int32_t H, int32_t I,
                                   int32_t E, int32_t k, const uint8_t* w13_q, const uint16_t* w13_s,
                                   const uint8_t* w2_q, const uint16_t* w2_s, int32_t Is, const uint8_t* w13s_q,
                                   const uint16_t* w13s_s, const uint8_t* w2s_q, const uint16_t* w2s_s,
                                   int32_t weight_layout, uint16_t* y, float* logits_out, int32_t* topk_ids_out,
                                   float* topk_w_out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * ---- MXFP4 (W4A4) variant ------------------------------------------------------------------------
 * [ATOM, 6.1: per-1x32 MXFP4 served by an a4w4 GEMM; ATOM, 8.2: dynamic activation quantization is
 * part of a format's contract.]  Weights and activations are E2M1 codes (as above) with one E8M0
 * scale byte per 32 consecutive K elements: value = E2M1(code) * 2^(byte - 127) (byte 255 = NaN is
 * not accepted in weights).  Activations are quantized on the fly, per row and block of 32, by the
 * OCP MX conversion: X = 2^(floor(log2(max |v|)) - 2) clamped to [2^-127, 2^127] (an all-zero block
 * takes byte 0), code = nearest E2M1 value of v / X, ties to the even code, saturating at +-6.
 * Products run on the gfx950 scaled FP4 matrix instruction with fp32 accumulation.
 */

/* x bf16 [rows, K] -> codes q [rows, K/2] and scale bytes s [rows, K/32] (MX conversion above).
 * Shapes: 0 <= rows < 2^26, K a positive multiple of 32.  x and q 16-byte aligned. */
moe_status_t moe_mx_quantize(const uint16_t* x, int32_t rows, int32_t K, uint8_t* q, uint8_t* s, void* stream);

/* Activation layouts of the MXFP4 GEMM. */
#define MOE_ACT_ROWS 0   /* row-major [*, K/2] codes and [*, K/32] scales, rows gathered through a_row_of */
#define MOE_ACT_TILED 1  /* tile-blocked: the tile list's rows, tile by tile, in the packed block order */

/*
 * Packed MXFP4 weight layout (same bytes, MFMA lane order): the [E, N, K] matrix cut into blocks of
 * 16 rows x 128 K elements ordered (expert, row block, K block), K fastest; per block 1024 bytes of
 * codes (bytes [16l, 16l+16) = row l % 16, K elements [32 (l / 16), +32)) and, separately, 64 scale
 * bytes (byte l = the same row and 32-block).  w_q [E, N, K/2], w_e [E, N, K/32] canonical in,
 * packed_q / packed_e of the same sizes out.  Needs N % 16 == 0, K % 128 == 0 [ATOM, 8.2: weight
 * pre-rearrangement is part of a quantized format's contract].
 */
moe_status_t moe_mx_prepack(const uint8_t* w_q, const uint8_t* w_e, int32_t E, int32_t N, int32_t K, uint8_t* packed_q,
                            uint8_t* packed_e, void* stream);

/*
 * x quantized (as moe_mx_quantize) and gathered into the tile-blocked activation layout of a tile
 * list: tile t's rows r = tiles[t].row0 + i (i < tiles[t].rows), source row a_row_of[r] / a_row_div
 * (or r), padded to block_m rows; blocks of 16 rows x 128 K ordered (tile, 16-row group, K block) with
 * K fastest, each 1024 code bytes in the packed lane order plus 64 scale bytes.  Padding rows and
 * tiles past *num_tiles are left unwritten.  q: max_tiles * block_m * K/2 bytes, s: max_tiles *
 * block_m * K/32 bytes.  Needs K % 128 == 0, block_m 16, 32 or 64.
 */
moe_status_t moe_mx_quantize_tiles(const uint16_t* x, int32_t T, int32_t K, const int32_t* a_row_of,
                                  int32_t a_row_div, const int32_t* tiles, int32_t max_tiles, const int32_t* num_tiles,
                                  int32_t block_m, uint8_t* q, uint8_t* s, void* stream);

/*
 * Grouped MXFP4 GEMM over the tile list of moe_align [Atlas, 编译时内核选择和W4A16 Grouped GEMM: one
 * launch over all experts]: for each permuted row r of expert e, activation row
 * a = (a_row_of ? a_row_of[r] / a_row_div : r):
 *   G[r, n] = sum_k A[a, k] * W_e[n, k],  A = (Aq [*, K/2], As [*, K/32]), W = (Wq [E, N, K/2], We [E, N, K/32]).
 *   epilogue NONE:     C [rows, N] fp32 or bf16 (out_dtype); Cs unused.
 *   epilogue SILU_MUL: h[r, j] = silu(G[r, j]) * G[r, N/2 + j] in fp32, then quantized per 32 columns:
 *                      C = codes [rows, N/4], Cs = scale bytes [rows, N/64] (out_dtype ignored).
 * weight_layout: MOE_LAYOUT_CANONICAL or MOE_LAYOUT_PACKED (moe_mx_prepack; needs N % 16 == 0 and
 * K % 128 == 0).  act_layout: MOE_ACT_ROWS, or MOE_ACT_TILED (packed weights only; A from
 * moe_mx_quantize_tiles or a previous SILU_MUL output, a_row_of unused; a SILU_MUL output is then
 * written tile-blocked too, for K = N/2 of the next projection, which needs N/2 % 128 == 0).
 * Results are bit-identical across layouts.  block_m 16, 32, 64 or 128 (the tile height moe_align
 * used); 128 runs a 128 x 256 LDS-staged kernel (bit-identical to the others) that needs
 * K % 128 == 0, MOE_ACT_ROWS and 4-byte aligned As and We.  K % 32 == 0; SILU_MUL needs N % 64 == 0.
 */
moe_status_t moe_grouped_gemm_mxfp4(const uint8_t* Aq, const uint8_t* As, const int32_t* a_row_of, int32_t a_row_div,
                                    const uint8_t* Wq, const uint8_t* We, int32_t weight_layout, int32_t act_layout,
                                    int32_t E, int32_t N, int32_t K,
                                    const int32_t* tiles, int32_t max_tiles, const int32_t* num_tiles, int32_t block_m,
                                    int32_t epilogue, void* C, uint8_t* Cs, int32_t out_dtype, void* stream);

/* Row-tile height and workspace bytes of moe_ffn_forward_mxfp4 (host-only, pure; -1 / 0 on invalid sizes). */
int32_t moe_ffn_mxfp4_block_m(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k);
size_t moe_ffn_mxfp4_workspace_bytes(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k);

/*
 * The whole MXFP4 (W4A4) layer [ATOM, 6.1 and 8.1-8.2]: route -> permute -> x quantized -> gate_up
 * (SiLU*mul, h quantized in the epilogue) -> down (fp32) -> combine, all enqueued on `stream`:
 *   y[t] = sum_s w[t,s] * W2_e(s) Q( silu(W1_e(s) Q(x[t])) * (W3_e(s) Q(x[t])) ),  Q = MX quantization.
 *   x bf16 [T, H]; router_logits fp32 [T, E]; w13_q [E, 2I, H/2], w13_e [E, 2I, H/32],
 *   w2_q [E, H, I/2], w2_e [E, H, I/32], all four in weight_layout (MOE_LAYOUT_PACKED from
 *   moe_mx_prepack needs H % 128 == 0 and I % 128 == 0; the quantized activations are then kept in
 *   the same blocked order internally; results are bit-identical to the canonical layout);
 *   y bf16 [T, H].  Optional routing copies as for moe_ffn_forward.  With experts of more than 128
 *   rows on average (and H, I multiples of 128) the 128-row kernel runs, on row-major activations,
 *   and the scale arrays need 4-byte alignment.
 *   workspace: at least moe_ffn_mxfp4_workspace_bytes(T, H, I, E, k) bytes (either layout).
 * Shapes: as moe_ffn_forward (H, I positive multiples of 32).
 */
moe_status_t moe_ffn_forward_mxfp4(const uint16_t* x, const float* router_logits, int32_t T, int32_t H, int32_t I,
                                   int32_t E, int32_t k, const uint8_t* w13_q, const uint8_t* w13_e,
                                   const uint8_t* w2_q, const uint8_t* w2_e, int32_t weight_layout, uint16_t* y,
                                   int32_t* topk_ids_out, float* topk_w_out, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * ---- W4A8 variant (MXFP8 activations on the MXFP4 weights) -----------------------------------------
 * [ATOM, 6.1: the MX formats served by the scaled-instruction GEMMs; ATOM, 8.2: dynamic activation
 * quantization is part of a format's contract.]  Weights exactly as the MXFP4 variant (either layout,
 * the same moe_mx_prepack).  Activations are MXFP8: OCP FP8 E4M3 codes (one byte per element; 1 sign,
 * 4 exponent bits with bias 7, 3 mantissa bits, largest finite 448) with one E8M0 scale byte per 32
 * consecutive K elements: value = E4M3(code) * 2^(byte - 127).  Quantization per row and block of 32:
 * X = 2^(floor(log2(max |v|)) - 8) clamped to [2^-127, 2^127] (an all-zero block takes byte 0), code =
 * nearest E4M3 value of v / X, ties to the even code, saturating at +-448.  Products run on the gfx950
 * scaled matrix instruction with E4M3 x E2M1 operands and fp32 accumulation.
 */

/* x bf16 [rows, K] -> codes q [rows, K] and scale bytes s [rows, K/32] (MXFP8 conversion above).
 * Shapes: 0 <= rows < 2^26, K a positive multiple of 32.  x and q 16-byte aligned. */
moe_status_t moe_mx8_quantize(const uint16_t* x, int32_t rows, int32_t K, uint8_t* q, uint8_t* s, void* stream);

/*
 * x quantized to MXFP8 (as moe_mx8_quantize) and gathered into the tile-blocked layout of a tile list
 * (rows as for moe_mx_quantize_tiles): blocks of 16 rows x 128 K ordered (tile, 16-row group, K block),
 * K fastest, each 2048 code bytes in the instruction's 8-bit lane order with the halves apart: bytes
 * [16l, 16l+16) = row l % 16, K [16 (l / 16), +16) of the block; bytes [1024 + 16l, +16) = the same row,
 * K [64 + 16 (l / 16), +16); and, separately, 64 scale bytes (byte l = row l % 16, 32-block l / 16).
 * Padding rows and tiles past *num_tiles are left unwritten.  q: max_tiles * block_m * K bytes, s:
 * max_tiles * block_m * K/32 bytes.  Needs K % 128 == 0, block_m 16, 32 or 64.
 */
moe_status_t moe_mx8_quantize_tiles(const uint16_t* x, int32_t T, int32_t K, const int32_t* a_row_of,
                                   int32_t a_row_div, const int32_t* tiles, int32_t max_tiles, const int32_t* num_tiles,
                                   int32_t block_m, uint8_t* q, uint8_t* s, void* stream);

/*
 * Grouped W4A8 GEMM over the tile list of moe_align (as moe_grouped_gemm_mxfp4): for each permuted
 * row r of expert e, activation row a = (a_row_of ? a_row_of[r] / a_row_div : r):
 *   G[r, n] = sum_k A[a, k] * W_e[n, k],  A = (Aq [*, K] E4M3 codes, As [*, K/32]), W = (Wq [E, N, K/2], We [E, N, K/32]).
 *   epilogue NONE:     C [rows, N] fp32 or bf16 (out_dtype); Cs unused.
 *   epilogue SILU_MUL: h[r, j] = silu(G[r, j]) * G[r, N/2 + j] in fp32, then quantized to MXFP8 per 32
 *                      columns: C = codes [rows, N/2], Cs = scale bytes [rows, N/64] (out_dtype ignored).
 * weight_layout: MOE_LAYOUT_CANONICAL or MOE_LAYOUT_PACKED (moe_mx_prepack; needs N % 16 == 0 and
 * K % 128 == 0).  act_layout: MOE_ACT_ROWS, or MOE_ACT_TILED (packed weights and block_m <= 64; A from
 * moe_mx8_quantize_tiles or a previous SILU_MUL output, a_row_of unused; a SILU_MUL output is then
 * written tile-blocked too, which needs N/2 % 128 == 0).  Results are bit-identical across layouts.
 * block_m 16, 32, 64 or 128 (the tile height moe_align used); 128 runs a 128 x 256 LDS-staged kernel
 * (bit-identical to the others) that needs K % 128 == 0, MOE_ACT_ROWS and 4-byte aligned As and We.
 * K % 32 == 0; SILU_MUL needs N % 64 == 0.  Aq, Wq and C 16-byte aligned.
 */
moe_status_t moe_grouped_gemm_w4a8(const uint8_t* Aq, const uint8_t* As, const int32_t* a_row_of, int32_t a_row_div,
                                   const uint8_t* Wq, const uint8_t* We, int32_t weight_layout, int32_t act_layout,
                                   int32_t E, int32_t N, int32_t K, const int32_t* tiles, int32_t max_tiles,
                                   const int32_t* num_tiles, int32_t block_m, int32_t epilogue, void* C, uint8_t* Cs,
                                   int32_t out_dtype, void* stream);

/* Row-tile height and workspace bytes of moe_ffn_forward_w4a8 (host-only, pure; -1 / 0 on invalid sizes):
 * the MXFP4 layer's choice (128 for experts averaging more than 128 rows with H, I multiples of 128). */
int32_t moe_ffn_w4a8_block_m(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k);
size_t moe_ffn_w4a8_workspace_bytes(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k);

/*
 * The whole W4A8 layer [ATOM, 6.1 and 8.1-8.2]: route -> permute -> x quantized to MXFP8 -> gate_up
 * (SiLU*mul, h quantized to MXFP8 in the epilogue) -> down (fp32) -> combine, all enqueued on `stream`:
 *   y[t] = sum_s w[t,s] * W2_e(s) Q8( silu(W1_e(s) Q8(x[t])) * (W3_e(s) Q8(x[t])) ),  Q8 = MXFP8 quantization.
 *   Arguments as moe_ffn_forward_mxfp4 (the same MXFP4 weights in either layout; packed needs
 *   H % 128 == 0 and I % 128 == 0, results bit-identical to the canonical layout); y bf16 [T, H].
 *   With packed weights the quantized activations are kept tile-blocked internally.  With experts of
 *   more than 128 rows on average (and H, I multiples of 128) the 128-row kernel runs, on row-major
 *   activations, and the scale arrays need 4-byte alignment.
 *   workspace: at least moe_ffn_w4a8_workspace_bytes(T, H, I, E, k) bytes.
 * Shapes: as moe_ffn_forward (H, I positive multiples of 32).
 */
moe_status_t moe_ffn_forward_w4a8(const uint16_t* x, const float* router_logits, int32_t T, int32_t H, int32_t I,
                                  int32_t E, int32_t k, const uint8_t* w13_q, const uint8_t* w13_e,
                                  const uint8_t* w2_q, const uint8_t* w2_e, int32_t weight_layout, uint16_t* y,
                                  int32_t* topk_ids_out, float* topk_w_out, void* workspace, size_t workspace_bytes,
                                  void* stream);

/*
 * ---- FP8 (W8A8, per-1x128) variant ----------------------------------------------------------------
 * [ATOM, 6.1: per-1x128 FP8 served by an a8w8 block-scale GEMM; ATOM, 8.1: the FP8 path of the fused
 * MoE; ATOM, 8.2: dynamic activation quantization is part of a format's contract.]  Weights and
 * activations are OCP FP8 E4M3 codes (1 sign, 4 exponent bits with bias 7, 3 mantissa bits; exponent
 * field 0 subnormal; largest finite 448; the NaN codes 0x7F / 0xFF are not accepted in weights), one
 * byte per element, rows K-contiguous, with one fp32 scale per row and block of 128 consecutive K
 * elements: value = E4M3(code) * scale.  Activations are quantized on the fly, per row and block:
 * s = max |v| / 448 (fp32 division), code = the E4M3 value nearest to the fp32 quotient v / s, ties to
 * the even code; an all-zero block gets s = 0 and codes 0.  Products run on the gfx950 FP8 matrix
 * instruction, one 128-element K block per instruction, whose fp32 partial is multiplied by the two
 * block scales in fp32; accumulation is fp32.
 */
#define MOE_IN_BF16 0
#define MOE_IN_F32 1
#define MOE_OUT_F8 2  /* SILU_MUL output of moe_grouped_gemm_f8 quantized per 1x128 (codes + fp32 scales) */

/* x [rows, K] (bf16 bits, or fp32 with in_dtype MOE_IN_F32) -> codes q [rows, K] and fp32 scales
 * s [rows, K/128] (the conversion above).  Shapes: 0 <= rows < 2^26, K a positive multiple of 128.
 * Alignment: x and q 16 bytes, s 4 bytes. */
moe_status_t moe_f8_quantize(const void* x, int32_t in_dtype, int32_t rows, int32_t K, uint8_t* q, float* s,
                             void* stream);

/*
 * Grouped FP8 GEMM over the tile list of moe_align [Atlas, 编译时内核选择和W4A16 Grouped GEMM: one
 * launch over all experts]: for each permuted row r of expert e, activation row
 * a = (a_row_of ? a_row_of[r] / a_row_div : r):
 *   G[r, n] = sum_k A[a, k] * W_e[n, k],  A = (Aq [*, K], As [*, K/128]), W = (Wq [E, N, K], Ws [E, N, K/128]).
 *   epilogue NONE:     C [rows, N], fp32 or bf16 (out_dtype).
 *   epilogue SILU_MUL: h[r, j] = silu(G[r, j]) * G[r, N/2 + j] in fp32, stored as
 *                      out_dtype MOE_OUT_F32: C [rows, N/2] fp32 (moe_f8_quantize then quantizes it), or
 *                      out_dtype MOE_OUT_F8: quantized in the epilogue exactly as moe_f8_quantize would,
 *                      C = codes [rows, N/2], Cs = fp32 scales [rows, N/256]; needs block_m 128 and
 *                      N/2 % 128 == 0.  Cs is unused (may be NULL) for the other output types.
 * Rows of C that no tile covers are not written.  block_m 16, 32, 64 or 128 (the tile height
 * moe_align used).  With block_m 16 or 32 the waves of a workgroup split K (four ways when block_m
 * is 16 and max_tiles <= 32, else two) and add their fp32 partials in wave order, so bits can
 * differ between tile heights and capacities; identical arguments always give identical bits.
 * 128 runs a 128 x 256 LDS-staged kernel, bit-identical to the 64-row one.
 * Shapes: 1 <= E <= MOE_MAX_EXPERTS, N >= 1 (N even for SILU_MUL), K a positive multiple of 128,
 *         K <= 32768.  Alignment: Aq, Wq, C 16 bytes; As, Ws 4 bytes.
 */
moe_status_t moe_grouped_gemm_f8(const uint8_t* Aq, const float* As, const int32_t* a_row_of, int32_t a_row_div,
                                 const uint8_t* Wq, const float* Ws, int32_t E, int32_t N, int32_t K,
                                 const int32_t* tiles, int32_t max_tiles, const int32_t* num_tiles, int32_t block_m,
                                 int32_t epilogue, void* C, float* Cs, int32_t out_dtype, void* stream);

/* Row-tile height and workspace bytes of moe_ffn_forward_f8 (host-only, pure; -1 / 0 on invalid sizes). */
int32_t moe_ffn_f8_block_m(int32_t T, int32_t E, int32_t k);
size_t moe_ffn_f8_workspace_bytes(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k);

/*
 * The whole FP8 (W8A8, per-1x128) layer [ATOM, 6.1 and 8.1-8.2]: route -> permute -> x quantized ->
 * gate_up (SiLU*mul, h in fp32) -> h quantized (in the gate_up epilogue with 128-row tiles) -> down
 * (fp32) -> combine, all enqueued on `stream`:
 *   y[t] = sum_s w[t,s] * W2_e(s) Q( silu(W1_e(s) Q(x[t])) * (W3_e(s) Q(x[t])) ),  Q = FP8 quantization.
 *   x bf16 [T, H]; router_logits fp32 [T, E]; w13_q [E, 2I, H], w13_s [E, 2I, H/128] fp32,
 *   w2_q [E, H, I], w2_s [E, H, I/128] fp32; y bf16 [T, H].  Optional routing copies as for
 *   moe_ffn_forward.  workspace: at least moe_ffn_f8_workspace_bytes(T, H, I, E, k) bytes.
 * Shapes: as moe_ffn_forward, with H and I positive multiples of 128, H and I <= 32768.
 */
moe_status_t moe_ffn_forward_f8(const uint16_t* x, const float* router_logits, int32_t T, int32_t H, int32_t I,
                                int32_t E, int32_t k, const uint8_t* w13_q, const float* w13_s, const uint8_t* w2_q,
                                const float* w2_s, uint16_t* y, int32_t* topk_ids_out, float* topk_w_out,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * ---- Ragged products: INT8 (W8A8, per token and channel) and 16-bit expert weights ----------------
 * [ATOM, 6.1: linears dispatched by quantization type; ATOM, 8.1: expert compute.]  These products take
 * their groups as expert_offsets int32 [E + 1] on the device (as moe_align writes them; nothing of it is
 * read by the host): expert e owns the rows [offsets[e], offsets[e + 1]) of R rows in all.  Offsets are
 * ascending and within [0, R]; the kernels clamp them to that range.  Rows that no expert owns (past
 * offsets[E]) are not written.  Experts without rows cost nothing.
 * a_row_of, a_row_div: activation row of row r = a_row_of ? a_row_of[r] / a_row_div : r (with a_row_of the
 * sorted_ids of moe_align and a_row_div = k, the token of the row).  Unlike the offsets these indexes are not
 * checked: for every row that an expert owns, the activation row has to lie within the activations.
 * One expert's weights stay below 4 GiB.
 */
#define MOE_IN_F16 2
#define MOE_OUT_F16 5
#define MOE_RAGGED_MAX_DIM (1 << 20) /* largest N and K */
#define MOE_I8_MAX_K (1 << 17)       /* sums of K products of int8 codes in [-127, 127] stay exact in int32 (and with
                                        -128 too, unless all K products of a sum are -128 * -128 at the largest K) */

/*
 * Rows quantized to int8: s[r] = fp32(max |x[r, :]| / 127), q[r, c] = the integer nearest to x[r, c] / s[r]
 * (the real quotient; ties to even), in [-127, 127]; value = q * s.  A row whose s is 0 gets codes 0; a row
 * that holds an infinity or a NaN gets s = NaN and codes 0, so that everything made of it is NaN.  A weight
 * matrix [N, K] is quantized per channel by the same call (rows = N, or E * N).
 *   x [rows, K] of in_dtype MOE_IN_BF16, MOE_IN_F16 or MOE_IN_F32; q int8 [rows, K]; s fp32 [rows].
 * Shapes: 0 <= rows < 2^26, K a positive multiple of 16.  Alignment: x and q 16 bytes, s 4 bytes.
 */
moe_status_t moe_i8_quantize(const void* x, int32_t in_dtype, int32_t rows, int32_t K, int8_t* q, float* s, void* stream);

/*
 * Dense int8 product: G[m, n] = As[m] * Ws[n] * sum_k Aq[m, k] * Wq[n, k], the sum exact in int32, the
 * scales applied in fp32.  epilogue MOE_EPI_NONE: C = G [M, N]; MOE_EPI_SILU_MUL: C [M, N/2] as in
 * moe_grouped_gemm_w4a16.  out_dtype MOE_OUT_BF16, MOE_OUT_F16 or (NONE) MOE_OUT_F32.
 * Shapes: 0 <= M < 2^26, N >= 1 (even for SILU_MUL) and <= MOE_RAGGED_MAX_DIM, K a positive multiple of 16
 * and <= MOE_I8_MAX_K.  Alignment: Aq, Wq, C 16 bytes; As, Ws 4 bytes.
 */
moe_status_t moe_gemm_i8(const int8_t* Aq, const float* As, const int8_t* Wq, const float* Ws, int32_t M, int32_t N,
                         int32_t K, int32_t epilogue, void* C, int32_t out_dtype, void* stream);

/* Workspace bytes of moe_linear_i8 (host-only, pure; 0 on invalid sizes). */
size_t moe_linear_i8_workspace_bytes(int32_t T, int32_t K);

/*
 * Linear layer with int8 weights and activations quantized on the fly [ATOM, 8.2]: moe_i8_quantize of x
 * [T, K] (in_dtype as there), then moe_gemm_i8 of it, with the same results as these two calls.  workspace: at
 * least moe_linear_i8_workspace_bytes(T, K) bytes, 16-byte aligned (0 bytes, and NULL, where one launch does
 * both whatever N is: T <= 4 and T * K <= 8192).  Other arguments as for moe_gemm_i8.
 */
moe_status_t moe_linear_i8(const void* x, int32_t in_dtype, const int8_t* Wq, const float* Ws, int32_t T, int32_t N,
                           int32_t K, int32_t epilogue, void* y, int32_t out_dtype, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * Grouped int8 product: for row r of expert e, with activation row a of r,
 *   G[r, n] = As[a] * Ws[e, n] * sum_k Aq[a, k] * Wq[e, n, k].
 *   Aq int8 [*, K], As fp32 [*]; Wq int8 [E, N, K], Ws fp32 [E, N]; C [R, N], or [R, N/2] for SILU_MUL.
 * Shapes: 0 <= R < 2^26, 1 <= E <= MOE_MAX_EXPERTS, N, K, out_dtype and alignment as for moe_gemm_i8.
 */
moe_status_t moe_grouped_gemm_i8(const int8_t* Aq, const float* As, const int32_t* a_row_of, int32_t a_row_div,
                                 const int8_t* Wq, const float* Ws, const int32_t* expert_offsets, int32_t R, int32_t E,
                                 int32_t N, int32_t K, int32_t epilogue, void* C, int32_t out_dtype, void* stream);

/* Workspace bytes of moe_ffn_forward_i8 (host-only, pure; 0 on invalid sizes). */
size_t moe_ffn_i8_workspace_bytes(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k);

/*
 * The whole INT8 layer [ATOM, 6.1 and 8.1]: route -> permute -> x quantized -> gate_up (SiLU*mul, h in
 * bf16) -> h quantized -> down (fp32) -> combine, all enqueued on `stream`.
 *   x bf16 [T, H]; router_logits fp32 [T, E]; w13_q int8 [E, 2I, H], w13_s fp32 [E, 2I], w2_q int8 [E, H, I],
 *   w2_s fp32 [E, H]; y bf16 [T, H].  Optional routing copies as for moe_ffn_forward.
 *   workspace: at least moe_ffn_i8_workspace_bytes(T, H, I, E, k) bytes.
 * Shapes: as moe_ffn_forward, with H and I positive multiples of 16, <= MOE_I8_MAX_K.
 */
moe_status_t moe_ffn_forward_i8(const uint16_t* x, const float* router_logits, int32_t T, int32_t H, int32_t I,
                                int32_t E, int32_t k, const int8_t* w13_q, const float* w13_s, const int8_t* w2_q,
                                const float* w2_s, uint16_t* y, int32_t* topk_ids_out, float* topk_w_out,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * Grouped product with 16-bit expert weights: for row r of expert e, with activation row a of r,
 *   G[r, n] = sum_k A[a, k] * W[e, n, k]      (exact products, fp32 accumulation)
 *   MOE_EPI_NONE: C = G [R, N]; MOE_EPI_SILU_MUL: C [R, N/2] as in moe_grouped_gemm_w4a16.
 *   A [*, K] and W [E, N, K] both of dtype MOE_IN_BF16 or MOE_IN_F16; out_dtype MOE_OUT_BF16, MOE_OUT_F16 or
 *   (NONE) MOE_OUT_F32.
 * Shapes: 0 <= R < 2^26, 1 <= E <= MOE_MAX_EXPERTS, N >= 1 (even for SILU_MUL), K a positive multiple of 8,
 *         N and K <= MOE_RAGGED_MAX_DIM.  Alignment: A, W, C 16 bytes; a_row_of, expert_offsets 4 bytes.
 */
moe_status_t moe_grouped_gemm_w16(const uint16_t* A, const int32_t* a_row_of, int32_t a_row_div, const uint16_t* W,
                                  int32_t dtype, const int32_t* expert_offsets, int32_t R, int32_t E, int32_t N,
                                  int32_t K, int32_t epilogue, void* C, int32_t out_dtype, void* stream);

/*
 * Gradient of moe_grouped_gemm_w16 (NONE) with respect to its rows: dA[r, k] = sum_n dC[r, n] * W[e, n, k] for row r of
 * expert e, dC [R, N] of dtype, dA [R, K] of out_dtype.  Rows that share an activation row are added by
 * moe_combine (fp32 dA as its O, weights 1).  N and K multiples of 8; otherwise as moe_grouped_gemm_w16.
 */
moe_status_t moe_grouped_gemm_w16_dx(const uint16_t* dC, const uint16_t* W, int32_t dtype, const int32_t* expert_offsets,
                                     int32_t R, int32_t E, int32_t N, int32_t K, void* dA, int32_t out_dtype,
                                     void* stream);

/* Workspace bytes moe_grouped_gemm_w16_dw needs (host-only, pure; 0 where the rows are not cut into parts, and on
 * invalid sizes). */
size_t moe_grouped_gemm_w16_dw_workspace_bytes(int32_t R, int32_t E, int32_t N, int32_t K);

/*
 * Gradient of moe_grouped_gemm_w16 (NONE) with respect to its weights:
 *   dW[e, n, k] = sum over the rows r of expert e of dC[r, n] * A[a(r), k],
 * dC [R, N] and A [*, K] of dtype, dW [E, N, K] of out_dtype, every element written (zeros for an expert
 * without rows, also when R is 0).  Few weights with many rows a group are summed in parts of the rows, which are
 * then added in order: workspace of at least moe_grouped_gemm_w16_dw_workspace_bytes(R, E, N, K) bytes, 16-byte
 * aligned (NULL where that is 0).  N and K multiples of 8; otherwise as moe_grouped_gemm_w16.
 */
moe_status_t moe_grouped_gemm_w16_dw(const uint16_t* dC, const uint16_t* A, const int32_t* a_row_of, int32_t a_row_div,
                                     int32_t dtype, const int32_t* expert_offsets, int32_t R, int32_t E, int32_t N,
                                     int32_t K, void* dW, int32_t out_dtype, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * SiLU*mul of a stored gate_up result G [R, 2I] (columns [0, I) the gate g, [I, 2I) the up projection u), for
 * training, where the backward pass needs G: h = silu(g) * u [R, I]; and its gradient: with s = 1 / (1 + exp(-g)),
 *   dG = [dh * u * s * (1 + g * (1 - s)), dh * g * s]  [R, 2I].
 * All of dtype MOE_IN_BF16 or MOE_IN_F16, arithmetic in fp32, one rounding; s below 2^-126 (g < -87) counts as 0.
 * Finite operands give a finite result unless the result itself passes the type.  An infinite g has no defined
 * result.  dG may be G.  Shapes: 0 <= R < 2^26, I a positive multiple of 8 and <= MOE_RAGGED_MAX_DIM.
 * Alignment: 16 bytes.
 */
moe_status_t moe_silu_mul(const uint16_t* G, int32_t dtype, int32_t R, int32_t I, uint16_t* h, void* stream);
moe_status_t moe_silu_mul_grad(const uint16_t* G, const uint16_t* dh, int32_t dtype, int32_t R, int32_t I, uint16_t* dG,
                               void* stream);

/* Workspace bytes of moe_ffn_forward_w16 (host-only, pure; 0 on invalid sizes). */
size_t moe_ffn_w16_workspace_bytes(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k);

/*
 * The whole layer with bf16 weights: route -> permute -> gate_up (SiLU*mul, h in bf16) -> down (fp32) ->
 * combine, all enqueued on `stream`.  x bf16 [T, H]; w13 bf16 [E, 2I, H]; w2 bf16 [E, H, I]; y bf16 [T, H].
 * workspace: at least moe_ffn_w16_workspace_bytes(T, H, I, E, k) bytes.  Shapes as moe_ffn_forward_i8.
 */
moe_status_t moe_ffn_forward_w16(const uint16_t* x, const float* router_logits, int32_t T, int32_t H, int32_t I,
                                 int32_t E, int32_t k, const uint16_t* w13, const uint16_t* w2, uint16_t* y,
                                 int32_t* topk_ids_out, float* topk_w_out, void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * ---- Root-mean-square norm in front of the experts -----------------------------------------------------
 * [ATOM, 8.2: dynamic activation quantization is part of a format's contract.]  For each row of x [T, H]:
 *   s = x + residual (fp32, rounded to the type; s = x where residual is NULL)
 *   r = 1 / sqrt(mean(s^2) + eps),  y = (s * r) * weight (fp32, rounded once; the same bits whatever quant is)
 * and, formed in the same pass, 8-bit codes and scales of y for the products that take them:
 *   MOE_QUANT_I8  one scale a row (moe_gemm_i8, moe_grouped_gemm_i8): scale = max |y| / 127, code = the integer
 *                 nearest to the real quotient 127 z / max |z|, z = s * weight (which y / scale is), ties to even.
 *   MOE_QUANT_F8  one scale per row and 128 columns (moe_grouped_gemm_f8): scale = max |y| / 448, code = the E4M3
 *                 value nearest to the real quotient 448 z / max |z|, ties to the even code.
 * The codes are those of the unrounded y.  Where a scale is 0 its codes are 0.  A row in which s or z holds an
 * infinity or a NaN gets scales NaN and codes 0; its y follows the formula (r = 0 beside an infinity).
 *   dtype      MOE_IN_BF16 or MOE_IN_F16: the type of x, residual, s and y; weight [H] of weight_dtype (dtype or
 *              MOE_IN_F32).  eps finite and > 0.
 *   s          [T, H], written where residual is given (it may be x or residual); ignored (NULL) without one.
 *   y          [T, H] or NULL (only with codes); may be x without a residual, and residual with one.
 *   q, q_scale codes [T, H] (int8, or E4M3 bytes) and fp32 scales [T] or [T, H / 128]; NULL for MOE_QUANT_NONE.
 * Shapes: 0 <= T < 2^26; H a positive multiple of 8 (I8: 16, F8: 128) and <= MOE_NORM_MAX_H.
 * Alignment: q_scale 4 bytes, all other pointers 16.
 */
#define MOE_QUANT_NONE 0
#define MOE_QUANT_I8 1
#define MOE_QUANT_F8 2
#define MOE_NORM_MAX_H 16384
moe_status_t moe_rmsnorm_add(const void* x, const void* residual, int32_t dtype, const void* weight, int32_t weight_dtype,
                             float eps, int32_t T, int32_t H, void* s, void* y, int32_t quant, void* q, float* q_scale,
                             void* stream);

/* Workspace bytes of moe_rmsnorm_add_grad (host-only, pure; 0 on invalid sizes, and where T is 0). */
size_t moe_rmsnorm_add_grad_workspace_bytes(int32_t T, int32_t H);

/*
 * Gradient of moe_rmsnorm_add: dy [T, H] (gradient of y), the s of the forward pass (x where it had no residual),
 * ds [T, H] (gradient that reaches s by other paths, such as the residual stream's, or NULL):
 *   dx = r * (dy * weight - s * r^2 * mean(dy * weight * s)) + ds     [T, H], of x and of the residual alike
 *   dweight = sum over the rows of dy * s * r                         [H], of dweight_dtype MOE_OUT_BF16, _F16 or _F32
 * Sums over a row in 64 bits, everything else in fp32 (dy * weight within its range), one rounding.  dweight is summed
 * in parts of at most 256 rows one after the other, which are added in order in 64 bits (zeros where T is 0).  workspace: at least
 * moe_rmsnorm_add_grad_workspace_bytes(T, H) bytes.
 * dx may be dy, s or ds.  Types, shapes and alignment as for moe_rmsnorm_add.
 */
moe_status_t moe_rmsnorm_add_grad(const void* dy, const void* s, int32_t dtype, const void* weight, int32_t weight_dtype,
                                  float eps, const void* ds, int32_t T, int32_t H, void* dx, void* dweight,
                                  int32_t dweight_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * ---- The layer for a few tokens, in two launches --------------------------------------------------------
 * [ATOM, 8.1.]  What moe_ffn_forward_w16 and moe_ffn_forward_i8 compute in five to seven launches, for decode steps of
 * at most MOE_FEW_MAX_TOKENS tokens: routing, gate_up and SiLU*mul in one launch, down and the weighted sum in another.
 *   y[t] = sum_s w[t,s] * W2_e(s) ( silu(W1_e(s) x[t]) * (W3_e(s) x[t]) ),  e(s) = topk_ids[t, s]  (moe_route_topk)
 *   moe_ffn_few_w16:   w13 bf16 [E, 2I, H], w2 bf16 [E, H, I].
 *   moe_ffn_few_w8a16: the int8 weights and channel scales of moe_ffn_forward_i8; activations are not quantized (a few
 *                      tokens are bound by the weights' bytes).
 * x bf16 [T, H]; router_logits fp32 [T, E], finite or (an expert that is closed) -infinity, in each token at least one
 * finite; a slot whose weight is 0 adds nothing, whatever its expert holds.  y bf16 [T, H] out, rounded once: h keeps about
 * 16 significant bits and all sums are fp32.  topk_ids_out int32 [T, k], topk_w_out fp32 [T, k]: optional copies of the
 * routing (NULL = skip).  workspace: at least moe_ffn_few_workspace_bytes(T, H, I, E, k) bytes, of one call at a time.
 * (Where H <= 1024 and the experts' contraction is long, a third, small launch adds what workgroups share.)
 * Where T * H passes 65536 the tokens are taken in groups that do not, each with its own launches (and its own reading
 * of the weights: the layers of any size are faster there).
 * Shapes: 0 <= T <= MOE_FEW_MAX_TOKENS, 1 <= k <= min(E, MOE_FEW_MAX_K), E <= MOE_MAX_EXPERTS, H and I multiples of
 * 16, 16 <= H <= 65536, 16 <= I <= MOE_I8_MAX_K, one expert's gate_up weights below 4 GiB.  Alignment: x, weights, y and
 * workspace 16 bytes, the others 4.
 */
#define MOE_FEW_MAX_TOKENS 16
#define MOE_FEW_MAX_K 16
/* Workspace bytes of both (host-only, pure; 0 on sizes that both refuse, and where T is 0). */
size_t moe_ffn_few_workspace_bytes(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k);
moe_status_t moe_ffn_few_w16(const uint16_t* x, const float* router_logits, int32_t T, int32_t H, int32_t I, int32_t E,
                             int32_t k, const uint16_t* w13, const uint16_t* w2, uint16_t* y, int32_t* topk_ids_out,
                             float* topk_w_out, void* workspace, size_t workspace_bytes, void* stream);
moe_status_t moe_ffn_few_w8a16(const uint16_t* x, const float* router_logits, int32_t T, int32_t H, int32_t I, int32_t E,
                               int32_t k, const int8_t* w13_q, const float* w13_s, const int8_t* w2_q, const float* w2_s,
                               uint16_t* y, int32_t* topk_ids_out, float* topk_w_out, void* workspace,
                               size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_W4A16_H */
