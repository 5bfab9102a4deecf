/*
 * nvfp4_w4a16.h -- C ABI of the MI355X (gfx950) W4A16 NVFP4 GEMM library.
 *
 * The operation (dense form):
 *
 *     Y[M,N] = g * (X[M,K] (.) s_pre[K]) . dequant(W)^T,
 *     dequant(W)[n,k] = e2m1(code(n,k)) * e4m3(S[n, k/16])
 *
 * W is packed FP4 (E2M1, two codes per byte along K) with one FP8 (E4M3)
 * scale per 16 consecutive K of a row and one fp32 global scale g; the
 * activation X and the output Y stay bf16 (fp16 in the *_f16 calls at the
 * end of this file).  Where the operation is defined:
 *   - packed FP4 weights + per-group FP8 scales + bf16/fp16 activations:
 *     "Support nvfp4 w4a16 on sm120", Summary;
 *   - E2M1 codebook lookup times a per-block FP8 scale and a per-tensor
 *     global scale (linear and active-expert-only MoE dequant):
 *     "Support Nemotron-H nvfp4 ckpt on Hopper", Walkthrough, Changes table;
 *   - group size 16 with E4M3 group scales and a real global scale, and the
 *     divisor-stored global scale that must be inverted: SGLang
 *     compressed-tensors NVFP4 weight-only page, Motivation and Modifications;
 *   - the per-channel pre-quant scale multiplies the bf16 activation before
 *     the GEMM (product kept in bf16), and a zero-token call launches no
 *     kernel: "Apply the NVFP4_AWQ pre-quant scale in MegaMoE CuteDSL",
 *     Description.
 * The E2M1 values and the low-nibble-is-even-k order follow the OCP MX
 * format; E4M3 is the OCP E4M3FN encoding (bias 7, max 448, NaN = 0x7F/0xFF).
 *
 * Conventions for every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the
 *     library allocates nothing and keeps no pointer after it returns.
 *   - `stream` is a hipStream_t passed as void* (NULL = default stream).
 *     Every call is asynchronous on that stream and never synchronises the
 *     host, so it can be captured into a HIP graph.
 *   - Arguments are checked on the host before anything is launched; on an
 *     error nothing has been enqueued and nvfp4_last_error() (thread-local)
 *     names the argument and the violated constraint.
 *   - Device-resident values (global scales, expert offsets) are not read by
 *     the host and are not checked: offsets that are not a non-decreasing
 *     sequence from 0 to R are undefined behaviour; a stored divisor of 0
 *     gives non-finite outputs.
 *   - bf16 values are IEEE binary32 upper halves; all rounding to bf16 is
 *     round-to-nearest-even.
 */
#ifndef NVFP4_W4A16_H
#define NVFP4_W4A16_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NVFP4_OK = 0,
    NVFP4_ERR_INVALID_ARG = 1,     /* a size, pointer or flag is invalid */
    NVFP4_ERR_ALIGNMENT = 2,       /* a pointer or leading dimension is misaligned */
    NVFP4_ERR_BUFFER_TOO_SMALL = 3,/* out_bytes / workspace_bytes below the size query */
    NVFP4_ERR_HIP = 4              /* the HIP runtime reported an error at launch */
} nvfp4_status;

/* Message of the last failed call on this thread ("" if none). */
const char* nvfp4_last_error(void);

/* Zero sizes: a call with no rows (M, R or T == 0) or no output columns
 * (N == 0) checks its other arguments, returns NVFP4_OK and launches nothing
 * (a zero-token chunk launches no kernel: "Apply the NVFP4_AWQ pre-quant
 * scale in MegaMoE CuteDSL", Description). */

/* ---------------------------------------------------------------- repack --
 * One-time re-tiling of canonical weights into the layout the GEMM kernels
 * stream (a step the pages perform as the Marlin weight transformation with
 * K/N padding: "Support nvfp4 w4a16 on sm120", Changes, Linear).
 *
 * Canonical input, E experts (E = 1 for a dense layer):
 *   w_packed : uint8 [E][N][ld_w], row (e,n) at w_packed + (e*N + n)*ld_w;
 *              byte j holds codes k = 2j (low nibble) and k = 2j+1 (high
 *              nibble); ld_w >= K/2.
 *   w_scale  : uint8 [E][N][ld_s] E4M3 bytes, row (e,n) at w_scale +
 *              (e*N + n)*ld_s; byte b scales k in [16b, 16b+16); ld_s >= K/16.
 * Output: `out`, nvfp4_repack_bytes(E,N,K) bytes, 16-byte aligned.  The blob
 * is pure derived state: repacking the same input again gives the same bytes,
 * and the canonical input is never modified.  N is padded to a multiple of
 * 16 and K to a multiple of 128 with zero codes and zero scales.  N == 0
 * needs 0 bytes and launches nothing.
 * Errors: E < 1, N < 0, K < 16, K % 16 != 0, ld_w < K/2, ld_s < K/16, NULL
 * pointer (N > 0) -> INVALID_ARG; out not 16-byte aligned -> ALIGNMENT;
 * out_bytes too small -> BUFFER_TOO_SMALL. */
int64_t nvfp4_repack_bytes(int64_t E, int64_t N, int64_t K); /* < 0 if invalid */
nvfp4_status nvfp4_repack(const uint8_t* w_packed, int64_t ld_w, const uint8_t* w_scale, int64_t ld_s,
                          int64_t E, int64_t N, int64_t K, void* out, int64_t out_bytes, void* stream);

/* ------------------------------------------------------------ dense GEMM --
 * Y = RNE_bf16(g * sum_k X'[m,k] * dequant(W)[n,k]) with
 *   X'[m,k] = pre_scale ? RNE_bf16(X[m,k] * pre_scale[k]) : X[m,k]
 *   g       = global_scale_is_divisor ? fp32(1 / *global_scale) : *global_scale
 * (the inversion happens at use, in the epilogue; *global_scale is never
 * rewritten).  The pre-quant scale is applied where the kernels load the
 * activation; X' is never written to memory.  Accumulation is fp32; the
 * summation order is fixed, so results are bitwise reproducible run to run.
 *   x         : bf16 [M][ld_x] (16-byte aligned, K <= ld_x <= 2^23, ld_x % 8 == 0)
 *   pre_scale : bf16 [K] (16-byte aligned) or NULL
 *   w_repacked: output of nvfp4_repack with E = 1 and the same N, K
 *   global_scale: device pointer to one fp32
 *   y         : bf16 [M][ld_y] (2-byte aligned, ld_y >= N)
 *   workspace : device scratch of nvfp4_w4a16_gemm_workspace_bytes(M,N,K)
 *               bytes, 256-byte aligned (may be NULL when that is 0; it is 0
 *               unless the call's kernel splits K across workgroups).  It
 *               holds split-K partial sums and arrival counters; it must be
 *               zero-filled before its first use; every call leaves the
 *               counters zero again, so one workspace can serve any number
 *               of calls issued one after another.  Calls that may overlap
 *               in time (other streams) need their own workspace.  The size
 *               covers every kernel variant that takes the shape.
 * M == 0 or N == 0 returns NVFP4_OK without launching anything.
 * Errors: M < 0, N < 0, K < 16, K % 16 != 0, ld_x < K, ld_x > 2^23, ld_y < N, NULL
 * x / w_repacked / global_scale / y (x and y may be NULL when M == 0) ->
 * INVALID_ARG; misaligned x, pre_scale, w_repacked, y or workspace, or
 * ld_x % 8 != 0 -> ALIGNMENT; workspace smaller than this call needs ->
 * BUFFER_TOO_SMALL. */
int64_t nvfp4_w4a16_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
nvfp4_status nvfp4_w4a16_gemm(const void* x, int64_t ld_x, const void* pre_scale, const void* w_repacked,
                              const float* global_scale, int global_scale_is_divisor,
                              void* y, int64_t ld_y, int64_t M, int64_t N, int64_t K,
                              void* workspace, int64_t workspace_bytes, void* stream);

/* ---------------------------------------------------------- grouped GEMM --
 * Active-expert-only MoE form ("Support Nemotron-H nvfp4 ckpt on Hopper",
 * Walkthrough, Changes table, MoE rows: only experts that received tokens
 * are dequantised).  Rows of x are grouped by expert: rows
 * [expert_offsets[e], expert_offsets[e+1]) use expert e's weights and global
 * scale; every other row of y is left untouched.  Experts with no rows read
 * no weight bytes.  The tile schedule is built on the device from
 * expert_offsets, with no host synchronisation.
 *   x             : bf16 [R][ld_x] (same alignment rules as the dense form)
 *   expert_offsets: device int32 [E+1], offsets[0] = 0, non-decreasing, offsets[E] = R
 *   pre_scale     : bf16 [K] shared by all experts, or NULL
 *   w_repacked    : output of nvfp4_repack with this E, N, K
 *   global_scales : device fp32 [E]
 *   y             : bf16 [R][ld_y]
 *   workspace     : as for the dense form, nvfp4_w4a16_grouped_gemm_workspace_bytes
 *                   bytes (0: the grouped kernels never split K)
 * R == 0 or N == 0 returns NVFP4_OK without launching anything.
 * Errors as for the dense form, plus E < 1 -> INVALID_ARG. */
int64_t nvfp4_w4a16_grouped_gemm_workspace_bytes(int64_t R, int64_t E, int64_t N, int64_t K);
nvfp4_status nvfp4_w4a16_grouped_gemm(const void* x, int64_t ld_x, const int32_t* expert_offsets,
                                      const void* pre_scale, const void* w_repacked,
                                      const float* global_scales, int global_scale_is_divisor,
                                      void* y, int64_t ld_y, int64_t R, int64_t E, int64_t N, int64_t K,
                                      void* workspace, int64_t workspace_bytes, void* stream);

/* ------------------------------------------------------------ MoE glue --
 * The steps either side of the grouped GEMM in a mixture-of-experts layer
 * whose experts take only the tokens routed to them ("Support Nemotron-H
 * nvfp4 ckpt on Hopper", Changes table, MoE W4A16 execution path: the layer
 * dispatches tokens to their active experts and runs a fused MoE over them;
 * the gated FC1 holds the gate and up projections together, the SGLang
 * compressed-tensors NVFP4 weight-only page, review discussion of the w13
 * sizing for gated and non-gated experts).  A layer of T tokens, top-k
 * routing over E experts, hidden size Hd and expert width I runs as
 *   nvfp4_moe_route -> nvfp4_w4a16_grouped_gemm_gather (FC1, N = 2 I)
 *   -> nvfp4_moe_silu_mul -> nvfp4_w4a16_grouped_gemm (FC2, K = I, N = Hd)
 *   -> nvfp4_moe_combine,
 * or with the activation in FC1's epilogue (one step fewer, and FC1 writes
 * I columns instead of 2 I):
 *   nvfp4_moe_route -> nvfp4_moe_fc1 (gated weights from nvfp4_repack_gated)
 *   -> nvfp4_w4a16_grouped_gemm (FC2) -> nvfp4_moe_combine,
 * every step stream-ordered, with no host synchronisation.
 *
 * Routing: topk_ids is device int32 [T][k] (row t: the k experts of token
 * t, values in [0, E); the caller keeps them distinct per token).  The
 * (token, slot) pairs p = t*k + j are ordered by expert, ties in pair order
 * (a stable sort), which defines the grouped rows:
 *   expert_offsets[e] : first grouped row of expert e; [E] = T*k,
 *   row_token[r]      : token of grouped row r,              [T*k]
 *   token_row[p]      : grouped row of pair p = t*k + j,     [T*k]
 * all device int32, 4-byte aligned.  The result does not depend on timing.
 * workspace: nvfp4_moe_route_workspace_bytes(T, k, E) bytes of device
 * scratch (4-byte aligned, no initial contents needed; calls that may
 * overlap in time need their own).  Ids outside [0, E) give undefined (but
 * in-bounds) results.  T == 0 returns NVFP4_OK without launching anything
 * (the outputs are not written).
 * Errors: T < 0, E < 1 or E > 1024, k < 1 or k > E, T*k >= 2^31, a NULL
 * array -> INVALID_ARG; misaligned array or workspace -> ALIGNMENT;
 * workspace too small -> BUFFER_TOO_SMALL. */
int64_t nvfp4_moe_route_workspace_bytes(int64_t T, int64_t k, int64_t E);   /* < 0 if invalid */
nvfp4_status nvfp4_moe_route(const int32_t* topk_ids, int64_t T, int64_t k, int64_t E, int32_t* expert_offsets,
                             int32_t* row_token, int32_t* token_row, void* workspace, int64_t workspace_bytes,
                             void* stream);

/* Grouped GEMM whose activation rows are gathered on the fly: grouped row r
 * reads row row_token[r] of x (bf16 [T][ld_x], the tokens in their own
 * order), so the expert-ordered copy of the activation is never written.
 * Otherwise as nvfp4_w4a16_grouped_gemm (y is in grouped row order; the
 * pre-scale, if any, applies to the T token rows).  row_token values must be
 * in [0, T) (device data, not checked: undefined behaviour otherwise).
 * Errors: as for nvfp4_w4a16_grouped_gemm, plus T < 0, R > 0 with T == 0,
 * T * ld_x >= 2^31, row_token NULL (R > 0) -> INVALID_ARG; row_token not
 * 4-byte aligned -> ALIGNMENT. */
int64_t nvfp4_w4a16_grouped_gemm_gather_workspace_bytes(int64_t T, int64_t R, int64_t E, int64_t N, int64_t K);
nvfp4_status nvfp4_w4a16_grouped_gemm_gather(const void* x, int64_t ld_x, int64_t T, const int32_t* row_token,
                                             const int32_t* expert_offsets, const void* pre_scale,
                                             const void* w_repacked, const float* global_scales,
                                             int global_scale_is_divisor, void* y, int64_t ld_y, int64_t R,
                                             int64_t E, int64_t N, int64_t K, void* workspace,
                                             int64_t workspace_bytes, void* stream);

/* Gated SiLU between FC1 and FC2: h is bf16 [R][ld_h] holding the gate
 * projection in columns [0, I) and the up projection in [I, 2I) (the w13
 * order, gate first); a[r][i] = RNE_bf16(silu(h[r][i]) * h[r][I + i]) with
 * silu(v) = v / (1 + exp(-v)) evaluated in fp32.  a is bf16 [R][ld_a].
 * Errors: R < 0, I < 1, ld_h < 2I, ld_a < I, NULL (R > 0) -> INVALID_ARG;
 * odd addresses -> ALIGNMENT. */
nvfp4_status nvfp4_moe_silu_mul(const void* h, int64_t ld_h, int64_t R, int64_t I, void* a, int64_t ld_a,
                                void* stream);

/* Non-gated squared ReLU for experts without a gate projection (the SGLang
 * compressed-tensors NVFP4 weight-only page, review discussion: non-gated
 * relu2 experts hold one FC1 projection): a[r][i] = RNE_bf16(max(h[r][i], 0)^2)
 * evaluated in fp32; h is bf16 [R][ld_h] with I columns, a bf16 [R][ld_a].
 * Errors: R < 0, I < 1, ld_h < I, ld_a < I, NULL (R > 0) -> INVALID_ARG; odd
 * addresses -> ALIGNMENT. */
nvfp4_status nvfp4_moe_relu2(const void* h, int64_t ld_h, int64_t R, int64_t I, void* a, int64_t ld_a, void* stream);

/* Gated FC1 weights in the layout the fused FC1 reads.  The pages name two
 * orders for the fused gate / up weight: gate first (SGLang's w13, the w1
 * rows then the w3 rows: the SGLang compressed-tensors NVFP4 weight-only page,
 * review discussion) and up first (TensorRT-LLM's w3_w1 / fc31: the inline
 * review comments on "Support Nemotron-H nvfp4 ckpt on Hopper" and the
 * Description of "Apply the NVFP4_AWQ pre-quant scale in MegaMoE CuteDSL").
 * Input: canonical NVFP4 weights of E experts with 2 I rows each (as
 * nvfp4_repack, N = 2 I), rows [0, I) the gate projection and [I, 2 I) the
 * up projection when up_first = 0, the other way round when up_first = 1.
 * Output: nvfp4_repack_gated_bytes(E, I, K) bytes (= nvfp4_repack_bytes(E,
 * 2 I, K)), 16-byte aligned, whose 16-row units alternate gate / up: unit 2 j
 * holds gate rows 16 j .. 16 j + 15 and unit 2 j + 1 the up rows of the same
 * columns.  It is meant for nvfp4_moe_fc1 only.
 * Errors: as nvfp4_repack, plus I < 0 or I not a multiple of 16, up_first not
 * 0 or 1 -> INVALID_ARG. */
int64_t nvfp4_repack_gated_bytes(int64_t E, int64_t I, int64_t K); /* < 0 if invalid */
nvfp4_status nvfp4_repack_gated(const uint8_t* w_packed, int64_t ld_w, const uint8_t* w_scale, int64_t ld_s,
                                int64_t E, int64_t I, int64_t K, int up_first, void* out, int64_t out_bytes,
                                void* stream);

/* FC1 with its activation applied in the GEMM's epilogue, so the 2 I-wide
 * FC1 output is never written:
 *   NVFP4_MOE_SILU_GLU: w_fc1 from nvfp4_repack_gated (E experts, I, K);
 *     a[r][i] = RNE_bf16(silu(h_gate) * h_up) with h = RNE_bf16(g_e * acc)
 *     of the gate and up columns i: bitwise what nvfp4_w4a16_grouped_gemm
 *     (gather) followed by nvfp4_moe_silu_mul gives on the canonical weights;
 *   NVFP4_MOE_RELU2: w_fc1 from nvfp4_repack (E, N = I, K); a[r][i] =
 *     RNE_bf16(max(h, 0)^2), h = RNE_bf16(g_e * acc): bitwise the grouped GEMM
 *     followed by nvfp4_moe_relu2.
 * Rows: with row_token, grouped row r reads token row row_token[r] of x
 * (bf16 [T][ld_x]) as in nvfp4_w4a16_grouped_gemm_gather; with row_token
 * NULL, x holds the R grouped rows (T must equal R).  a is bf16 [R][ld_a] in
 * grouped row order; expert_offsets, pre_scale, global_scales and the
 * divisor flag as in nvfp4_w4a16_grouped_gemm.  No workspace.
 * Errors: as nvfp4_w4a16_grouped_gemm_gather (with N = 2 I or I), plus an
 * unknown activation, I < 0, I not a multiple of 16 (gated), ld_a < I,
 * row_token NULL with T != R -> INVALID_ARG. */
enum { NVFP4_MOE_SILU_GLU = 1, NVFP4_MOE_RELU2 = 2 };
nvfp4_status nvfp4_moe_fc1(const void* x, int64_t ld_x, int64_t T, const int32_t* row_token,
                           const int32_t* expert_offsets, const void* pre_scale, const void* w_fc1,
                           const float* global_scales, int global_scale_is_divisor, int activation, void* a,
                           int64_t ld_a, int64_t R, int64_t E, int64_t I, int64_t K, void* stream);

/* Test export: one grouped GEMM (activation 0: plain output, N columns) or
 * fused FC1 (activation NVFP4_MOE_SILU_GLU on a gated blob, N = 2 I and I
 * output columns; NVFP4_MOE_RELU2) on a chosen kernel, so that the kernels
 * can be checked against each other on the same inputs: variant 0 the
 * automatic choice, 1 the small-M kernel, 2 the tile kernel (64-row tiles),
 * 3 the MFMA-bound kernel (256-row tiles per expert).  Rows as in
 * nvfp4_moe_fc1 (row_token NULL: x holds the R grouped rows, T = R); f16:
 * fp16 activations and output; mx: an MXFP4 blob (mxfp4_repack; the global
 * scales are then not read and may be NULL); no workspace.  Errors: as the grouped GEMM,
 * plus an unknown activation or variant, N not a multiple of 32 with the
 * gated activation, mx not 0 or 1, and for variant 3 a blob of 2 GiB of
 * codes or more or NVFP4_MOE_RELU2 (the tile kernel serves it) -> INVALID_ARG. */
nvfp4_status nvfp4_w4a16_grouped_gemm_variant(const void* x, int64_t ld_x, int64_t T, const int32_t* row_token,
                                              const int32_t* expert_offsets, const void* pre_scale, const void* w,
                                              const float* global_scales, int global_scale_is_divisor, int activation,
                                              void* y, int64_t ld_y, int64_t R, int64_t E, int64_t N, int64_t K,
                                              int variant, int f16, int mx, void* stream);

/* Top-k weighted combine back to token order: out[t][c] =
 * RNE_bf16(sum_{j=0..k-1} topk_weights[t*k + j] * y[token_row[t*k + j]][c]),
 * accumulated in fp32 in slot order.  y: bf16 [R][ld_y] (FC2 output in
 * grouped row order), token_row: from nvfp4_moe_route, topk_weights: device
 * fp32 [T][k], out: bf16 [T][ld_o].
 * Errors: T < 0, k < 1, H < 1, ld_y < H, ld_o < H, NULL (T > 0) ->
 * INVALID_ARG; misaligned pointer -> ALIGNMENT. */
nvfp4_status nvfp4_moe_combine(const void* y, int64_t ld_y, const int32_t* token_row, const float* topk_weights,
                               int64_t T, int64_t k, int64_t H, void* out, int64_t ld_o, void* stream);

/* --------------------------------------------------------- test exports --
 * Decode a repacked blob back to bf16 [E][N][ld_out] in canonical order with
 * the same device decode the GEMM kernels use (no global scale applied):
 * out[e][n][k] = RNE_bf16(e2m1(code) * e4m3(scale)), which is exact.
 * Errors: as for repack, ld_out < K -> INVALID_ARG. */
nvfp4_status nvfp4_dequant_bf16(const void* w_repacked, int64_t E, int64_t N, int64_t K,
                                void* out, int64_t ld_out, void* stream);

/* Dense GEMM with the kernel variant forced instead of chosen from M:
 *   variant 0 = automatic (same as nvfp4_w4a16_gemm),
 *   variant 1 = small-M kernel (M <= 16 only; larger M -> INVALID_ARG),
 *   variant 2 = tile kernel (any M),
 *   variant 3 = MFMA-bound kernel (any M; launched as one or two kernels),
 *   variant 4 = activation-resident kernel: M <= 16, K <= 32768 (K split
 *               across workgroups beyond 4096) and
 *               ceil(N / 16) * ceil(K / 4096) <= 2048; otherwise INVALID_ARG,
 *   variant 5 = MFMA-bound kernel with every 256 x 256 tile run as four
 *               64-row workgroups (several then share a compute unit).
 * The automatic choice takes the small-M kernel up to 4 rows, the
 * activation-resident kernel for 5..16 rows where it applies, the MFMA-bound
 * kernel for large M and the tile kernel otherwise (nvfp4_w4a16_gemm_plan).
 * Used to check that the variants agree on the same inputs. */
nvfp4_status nvfp4_w4a16_gemm_variant(const void* x, int64_t ld_x, const void* pre_scale, const void* w_repacked,
                                      const float* global_scale, int global_scale_is_divisor,
                                      void* y, int64_t ld_y, int64_t M, int64_t N, int64_t K,
                                      void* workspace, int64_t workspace_bytes, int variant, void* stream);

/* The variant (1..4 above) that nvfp4_w4a16_gemm runs for an M x N x K call,
 * 0 when it launches nothing (M == 0 or N == 0), -1 for invalid sizes.  A
 * pure host function of the sizes (bf16 and fp16 calls choose alike). */
int nvfp4_w4a16_gemm_plan(int64_t M, int64_t N, int64_t K);

/* 1 if nvfp4_w4a16_gemm_variant accepts `variant` for an M x N x K call, 0 if
 * it rejects the shape (INVALID_ARG), -1 for invalid sizes or variants.  A
 * pure host function of the sizes. */
int nvfp4_w4a16_gemm_variant_takes(int64_t M, int64_t N, int64_t K, int variant);

/* ------------------------------------------------- no-allocation entry --
 * For callers that cannot allocate device memory or pass a workspace: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation.  nvfp4_w4a16_gemm without the workspace arguments: the split-K
 * partial sums and arrival counters that some shapes need live in a static
 * device array of the library, nvfp4_w4a16_gemm_noalloc_max_scratch_bytes()
 * bytes (4 MiB) on every GPU the library runs on, held until the process
 * ends.  The call allocates nothing (no hipMalloc, no allocating library
 * routine); the caller still passes the inputs and the output.  The first
 * call on a device looks up the array's device address and clears its
 * counters on `stream` (a fill kernel); every call leaves the counters it
 * used at zero.  All calls on one GPU share that GPU's array: calls that may
 * overlap in time on one GPU (other streams, other threads) race and give
 * undefined results; issue them one after another.
 * Arguments, kernel choice, results (bitwise those of nvfp4_w4a16_gemm) and
 * errors as for nvfp4_w4a16_gemm, plus: a call whose kernel needs more
 * scratch than the array holds (nvfp4_w4a16_gemm_workspace_bytes above the
 * maximum) -> BUFFER_TOO_SMALL, before anything is launched; the address
 * lookup failing -> HIP. */
int64_t nvfp4_w4a16_gemm_noalloc_max_scratch_bytes(void);
nvfp4_status nvfp4_w4a16_gemm_noalloc(const void* x, int64_t ld_x, const void* pre_scale, const void* w_repacked,
                                      const float* global_scale, int global_scale_is_divisor, void* y, int64_t ld_y,
                                      int64_t M, int64_t N, int64_t K, void* stream);

/* Measurement export: a plain read of `bytes` (a multiple of 16) at p
 * (16-byte aligned), the bandwidth reference the GEMMs are measured against.
 * `workgroups` workgroups of 256 threads each read a contiguous share with
 * non-temporal 16-byte loads, `unroll` (1, 2, 4 or 8) loads per thread in
 * flight; out (uint32 [workgroups], 4-byte aligned) is written only in the
 * practically impossible case that a workgroup's data folds to a fixed value
 * (it keeps the loads alive).  Errors: bad sizes or unroll -> INVALID_ARG,
 * misaligned pointers -> ALIGNMENT. */
nvfp4_status nvfp4_bench_stream_read(const void* p, int64_t bytes, uint32_t* out, int64_t workgroups, int unroll,
                                     void* stream);

/* ---- MXFP4 weights -----------------------------------------------------------
 *
 * Weight-only MXFP4: the same packed E2M1 codes with one E8M0 scale per 32
 * consecutive K of a row and no global scale (SGLang compressed-tensors
 * NVFP4 weight-only page, Modifications: the paragraph on MXFP4 names group
 * size 32 (group_blocks == 2), E8M0 scales and the missing global scale as
 * what sets it apart from NVFP4).  E8M0 is the OCP MX scale: byte e decodes
 * to 2^(e-127), 0xFF is NaN.
 *
 *     Y = RNE(sum_k X'[m,k] * e2m1(code(n,k)) * e8m0(S[n, k/32]))
 *
 *   w_scale : uint8 E8M0 [E][N][ld_s], ld_s >= K/32; K must be a multiple of
 *             32 (INVALID_ARG otherwise).
 * The repacked blob has the size mxfp4_repack_bytes(E,N,K) (equal to
 * nvfp4_repack_bytes) and may only be passed to the mxfp4_* calls.  The
 * GEMMs take the arguments, kernel choice, workspace sizes
 * (nvfp4_w4a16_gemm_workspace_bytes, nvfp4_w4a16_grouped_gemm_workspace_bytes),
 * pre-quant scale, ownership, zero sizes and errors of the NVFP4 calls, minus
 * the global scale; the _f16 forms take fp16 activations and outputs.
 * Decoded weights are exact in bf16 while |e2m1 * 2^(e-127)| stays in bf16's
 * normal range (scale bytes 2..252; the kernels may flush smaller ones to
 * zero and larger ones overflow to infinity), in fp16 while it stays in
 * fp16's (bytes 114..140 for every code). */
int64_t mxfp4_repack_bytes(int64_t E, int64_t N, int64_t K); /* < 0 if invalid */
nvfp4_status mxfp4_repack(const uint8_t* w_packed, int64_t ld_w, const uint8_t* w_scale, int64_t ld_s,
                          int64_t E, int64_t N, int64_t K, void* out, int64_t out_bytes, void* stream);
nvfp4_status mxfp4_w4a16_gemm(const void* x, int64_t ld_x, const void* pre_scale, const void* w_repacked, void* y,
                              int64_t ld_y, int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                              void* stream);
nvfp4_status mxfp4_w4a16_gemm_f16(const void* x, int64_t ld_x, const void* pre_scale, const void* w_repacked, void* y,
                                  int64_t ld_y, int64_t M, int64_t N, int64_t K, void* workspace,
                                  int64_t workspace_bytes, void* stream);
nvfp4_status mxfp4_w4a16_grouped_gemm(const void* x, int64_t ld_x, const int32_t* expert_offsets, const void* pre_scale,
                                      const void* w_repacked, void* y, int64_t ld_y, int64_t R, int64_t E, int64_t N,
                                      int64_t K, void* workspace, int64_t workspace_bytes, void* stream);
nvfp4_status mxfp4_w4a16_grouped_gemm_f16(const void* x, int64_t ld_x, const int32_t* expert_offsets,
                                          const void* pre_scale, const void* w_repacked, void* y, int64_t ld_y,
                                          int64_t R, int64_t E, int64_t N, int64_t K, void* workspace,
                                          int64_t workspace_bytes, void* stream);
/* The fused MoE FC1 on MXFP4 weights (the weight format of the section above,
 * in the MoE FC1 that nvfp4_moe_fc1 cites): mxfp4_repack_gated is
 * nvfp4_repack_gated with E8M0 scales [E][2 I][ld_s], ld_s >= K/32 (K a
 * multiple of 32), and mxfp4_moe_fc1 is nvfp4_moe_fc1 without global scales,
 * on a blob from mxfp4_repack_gated (NVFP4_MOE_SILU_GLU) or mxfp4_repack
 * (NVFP4_MOE_RELU2): bitwise mxfp4_w4a16_grouped_gemm (with the row gather)
 * followed by nvfp4_moe_silu_mul or nvfp4_moe_relu2.  Errors as those calls. */
int64_t mxfp4_repack_gated_bytes(int64_t E, int64_t I, int64_t K); /* < 0 if invalid */
nvfp4_status mxfp4_repack_gated(const uint8_t* w_packed, int64_t ld_w, const uint8_t* w_scale, int64_t ld_s,
                                int64_t E, int64_t I, int64_t K, int up_first, void* out, int64_t out_bytes,
                                void* stream);
nvfp4_status mxfp4_moe_fc1(const void* x, int64_t ld_x, int64_t T, const int32_t* row_token,
                           const int32_t* expert_offsets, const void* pre_scale, const void* w_fc1, int activation,
                           void* a, int64_t ld_a, int64_t R, int64_t E, int64_t I, int64_t K, void* stream);
nvfp4_status mxfp4_moe_fc1_f16(const void* x, int64_t ld_x, int64_t T, const int32_t* row_token,
                               const int32_t* expert_offsets, const void* pre_scale, const void* w_fc1, int activation,
                               void* a, int64_t ld_a, int64_t R, int64_t E, int64_t I, int64_t K, void* stream);
/* Test exports: the decoded tile (as nvfp4_dequant_bf16, E8M0 scales) and the
 * dense GEMM with a forced kernel variant (as nvfp4_w4a16_gemm_variant; f16
 * selects fp16 activations and outputs). */
nvfp4_status mxfp4_dequant_bf16(const void* w_repacked, int64_t E, int64_t N, int64_t K, void* out, int64_t ld_out,
                                void* stream);
nvfp4_status mxfp4_w4a16_gemm_variant(const void* x, int64_t ld_x, const void* pre_scale, const void* w_repacked,
                                      void* y, int64_t ld_y, int64_t M, int64_t N, int64_t K, void* workspace,
                                      int64_t workspace_bytes, int variant, int f16, void* stream);

/* ---- FP16 activations and outputs ------------------------------------------
 *
 * The same operations with X, the pre-quant scale and Y in IEEE binary16
 * instead of bf16 (weight-only FP4 serves bf16 or fp16 activations: "Support
 * nvfp4 w4a16 on sm120", Summary; SGLang compressed-tensors NVFP4
 * weight-only page, Motivation).  Arguments, layouts, workspace sizes
 * (nvfp4_w4a16_gemm_workspace_bytes / nvfp4_w4a16_grouped_gemm_workspace_bytes),
 * kernel choice, ownership and errors are those of the bf16 calls above.
 * The decoded weights are exact in fp16 (e2m1 * e4m3 lies in [2^-10, 2688]
 * with at most 6 significant bits), the MFMAs take fp16 with fp32
 * accumulation, the pre-scaled activation is RNE_fp16(X * s) and
 * Y = RNE_fp16(g * acc); outputs beyond the fp16 range become +-infinity. */
nvfp4_status nvfp4_w4a16_gemm_f16(const void* x, int64_t ld_x, const void* pre_scale, const void* w_repacked,
                                  const float* global_scale, int global_scale_is_divisor, void* y, int64_t ld_y,
                                  int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                                  void* stream);

/* nvfp4_w4a16_gemm_variant with fp16 activations and outputs. */
nvfp4_status nvfp4_w4a16_gemm_variant_f16(const void* x, int64_t ld_x, const void* pre_scale, const void* w_repacked,
                                          const float* global_scale, int global_scale_is_divisor, void* y,
                                          int64_t ld_y, int64_t M, int64_t N, int64_t K, void* workspace,
                                          int64_t workspace_bytes, int variant, void* stream);

/* nvfp4_w4a16_grouped_gemm with fp16 activations and outputs. */
nvfp4_status nvfp4_w4a16_grouped_gemm_f16(const void* x, int64_t ld_x, const int32_t* expert_offsets,
                                          const void* pre_scale, const void* w_repacked, const float* global_scales,
                                          int global_scale_is_divisor, void* y, int64_t ld_y, int64_t R, int64_t E,
                                          int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                                          void* stream);

/* The MoE glue steps with fp16 activations (the routing is type-free): the
 * gathering grouped GEMM, the gated SiLU, the squared ReLU and the top-k
 * combine, each as its bf16 form above with every 16-bit array in IEEE
 * binary16 and every rounding RNE to fp16 (overflow to +-infinity). */
nvfp4_status nvfp4_w4a16_grouped_gemm_gather_f16(const void* x, int64_t ld_x, int64_t T, const int32_t* row_token,
                                                 const int32_t* expert_offsets, const void* pre_scale,
                                                 const void* w_repacked, const float* global_scales,
                                                 int global_scale_is_divisor, void* y, int64_t ld_y, int64_t R,
                                                 int64_t E, int64_t N, int64_t K, void* workspace,
                                                 int64_t workspace_bytes, void* stream);
nvfp4_status nvfp4_moe_silu_mul_f16(const void* h, int64_t ld_h, int64_t R, int64_t I, void* a, int64_t ld_a,
                                    void* stream);
nvfp4_status nvfp4_moe_relu2_f16(const void* h, int64_t ld_h, int64_t R, int64_t I, void* a, int64_t ld_a,
                                 void* stream);
nvfp4_status nvfp4_moe_combine_f16(const void* y, int64_t ld_y, const int32_t* token_row, const float* topk_weights,
                                   int64_t T, int64_t k, int64_t H, void* out, int64_t ld_o, void* stream);
/* nvfp4_moe_fc1 with fp16 activations and output (RNE to fp16 throughout). */
nvfp4_status nvfp4_moe_fc1_f16(const void* x, int64_t ld_x, int64_t T, const int32_t* row_token,
                               const int32_t* expert_offsets, const void* pre_scale, const void* w_fc1,
                               const float* global_scales, int global_scale_is_divisor, int activation, void* a,
                               int64_t ld_a, int64_t R, int64_t E, int64_t I, int64_t K, void* stream);

/* ---- The attention half of a decoder layer -----------------------------------
 *
 * What a decoder layer runs around its FP4 linears when it serves one new
 * token per sequence (or writes a prompt's tokens into its cache): the norm
 * with the residual's addition, rotary positions, the paged key-value cache
 * and the attention over it.  f16 selects fp16 activations (0: bf16); every
 * 16-bit array of a call has that type.  Strides are in elements of the array
 * unless a byte stride is named.  All rows start 16-byte aligned and are
 * contiguous, except where stated.  Rows that are written share no memory. */

/* Root-mean-square norm.  Row t of T, N values:
 *   h = residual ? RNE16(x + residual) : x          (stored to h if given)
 *   v = h * rsqrt(mean(h^2) + eps) * weight         (fp32, over h as rounded)
 *   scales == NULL: y[t] = RNE16(v);
 *   scales != NULL: y[t] = e4m3(v * fp32(1 / s)), scales[t] = s = max(fp32(max |v| / 448), 2^-126)
 *                   (bytes; the value a byte stands for is e4m3 * s).
 *   x [T][ld_x], residual [T][ld_r] or NULL, weight [N], y [T][ld_y] of 16-bit
 *   values or bytes, scales fp32 [T] or NULL, h [T][ld_h] or NULL (needs a
 *   residual).  h may be residual's or x's memory with the same leading
 *   dimension, and y x's if it is 16 bits wide and h does not take it; no other
 *   overlap.  2-byte alignment of rows suffices (1-byte for 8-bit y, 4-byte
 *   for scales); rows and leading dimensions of 16 bytes (8 for 8-bit y) and N
 *   a multiple of 8 up to 32768 take the one-pass kernel.
 * T == 0 launches nothing.  Errors: T < 0, T rows that take 2^32 threads or
 * more (from T = 2^22 on), N < 1 or N > 2^31 - 256, a leading dimension < N, eps
 * negative or not finite, h without residual, NULL x / weight / y ->
 * INVALID_ARG; misaligned -> ALIGNMENT. */
nvfp4_status nvfp4_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, const void* weight,
                            float eps, void* y, int64_t ld_y, float* scales, void* h, int64_t ld_h, int64_t T,
                            int64_t N, int f16, void* stream);

/* Rotary positions.  The first R columns of each head are turned in R / 2
 * pairs, columns (i, i + R / 2), or (2 i, 2 i + 1) with neighbours; the rest
 * pass.  Pair i of token t turns by
 *   angle = positions[axis(i)][t] * inv_freq[i]     (in 64 bits),
 *   (x0, x1) -> RNE16(x0 c - x1 s), RNE16(x1 c + x0 s),
 * c and s the cosine and sine rounded to fp32, each product and sum rounded to
 * fp32.  axis(i) = pair_axis[i], or 0 with pair_axis NULL; several axes serve
 * positions of images and video (time, height, width).
 *   inv_freq fp32 [R / 2]; positions int32 [axes][ld_pos], negative ones too;
 *   pair_axis int32 [R / 2] or NULL (values outside [0, axes) are clamped). */
typedef struct {
    const float* inv_freq;
    const int32_t* positions;
    const int32_t* pair_axis;
    int64_t ld_pos;
    int32_t axes;
    int32_t rotary;      /* R: even columns turned, a multiple of 16 */
    int32_t neighbours;  /* pairs (2 i, 2 i + 1) instead of (i, i + R / 2) */
    int32_t reserved;    /* 0 */
} nvfp4_rope;

/* The paged key-value cache: `pages` pages of `page_size` tokens, `heads`
 * key-value heads of head_dim = D columns.  The block of a (page, head) starts
 * at page * stride[0] + head * stride[1] bytes:
 *   NVFP4_KV_16BIT  values of the activation type, row i of the page stride[2]
 *                   bytes after row i - 1; no scales;
 *   NVFP4_KV_E4M3   E4M3 bytes, rows likewise; the stored value of x in head h
 *                   is e4m3(sat448(fp32(x * fp32(1 / scale[h]))));
 *   NVFP4_KV_NVFP4  page_size * D / 2 code bytes (token-major, two E2M1 codes a
 *                   byte, the even column in the low nibble), then page_size *
 *                   D / 16 E4M3 group scales (token-major, one per 16 columns);
 *                   stride[2] is not used.  A group with the largest absolute
 *                   value a gets the scale S = e4m3(sat448(fp32(fp32(a * r) *
 *                   fp32(1 / 6)))), r = fp32(1 / scale[h]), and the codes
 *                   e2m1(sat6(fp32(x * fp32(r / S)))), all 0 where S is 0.  A
 *                   NaN in the group makes S and so the group NaN.
 * Values read back as code (* S) * scale[h].  Roundings are to nearest, ties to
 * even.  k_scale / v_scale: device fp32 [heads], positive, or NULL for 1 (must
 * be NULL for NVFP4_KV_16BIT).
 * D: a multiple of 16 in [16, 256] (of 32 for NVFP4_KV_NVFP4); page_size >= 1,
 * any size (NVFP4: page_size * 9 * D / 16 a multiple of 16); strides multiples
 * of 16 bytes, non-negative; at most 64 GB from the first to the last block of
 * each side; pages * page_size < 2^31. */
enum { NVFP4_KV_16BIT = 0, NVFP4_KV_E4M3 = 1, NVFP4_KV_NVFP4 = 2 };
typedef struct {
    void* k;
    void* v;
    const float* k_scale;
    const float* v_scale;
    int64_t k_stride[3];   /* bytes: page, head, token */
    int64_t v_stride[3];
    int64_t pages;
    int32_t page_size;
    int32_t heads;
    int32_t head_dim;
    int32_t format;
} nvfp4_kv_cache;

/* Rotates x [T][H][D] (strides x_t, x_h) into out (strides o_t, o_h), which may
 * be x itself with the same strides.  D a multiple of 16 in [16, 1024], R <=
 * min(D, 256).  T == 0 or H == 0 launches nothing.  Errors: sizes (T < 2^24), NULL
 * pointers -> INVALID_ARG; rows or strides not multiples of 16 bytes,
 * misaligned arrays -> ALIGNMENT. */
nvfp4_status nvfp4_rope_apply(const nvfp4_rope* rope, const void* x, int64_t x_t, int64_t x_h, void* out, int64_t o_t,
                              int64_t o_h, int64_t T, int64_t H, int64_t D, int f16, void* stream);

/* Appends T tokens to the cache: keys k [T][heads][D] (strides k_t, k_h) and
 * values v go to row slots[t] % page_size of page slots[t] / page_size; tokens
 * whose slot is negative or past the cache are skipped (padding).  Two tokens
 * with one slot leave a row made of pieces of both (16 columns at a time are
 * written together, and an NVFP4 group's scale apart from its codes): a call's
 * slots are distinct.  With rope the keys are rotated first
 * and rounded to 16 bits (R a multiple of 32 for NVFP4_KV_NVFP4, at most 256),
 * and queries q [T][Hq][D] are rotated into q_out in the same launch, padding
 * included (q_out may be q; Hq = 0 and NULL without queries).
 * Errors as above, plus an invalid cache description -> INVALID_ARG /
 * ALIGNMENT, queries without rope -> INVALID_ARG. */
nvfp4_status nvfp4_kv_append(const nvfp4_kv_cache* cache, const nvfp4_rope* rope, const void* q, int64_t q_t,
                             int64_t q_h, void* q_out, int64_t qo_t, int64_t qo_h, int64_t Hq, const void* k,
                             int64_t k_t, int64_t k_h, const void* v, int64_t v_t, int64_t v_h, const int32_t* slots,
                             int64_t T, int f16, void* stream);

/* Reads rows back in 16 bits: k[t] and v[t] (16-bit [T][heads][D]) = RNE16 of
 * the values of slot slots[t], zeros for a slot outside the cache. */
nvfp4_status nvfp4_kv_read(const nvfp4_kv_cache* cache, const int32_t* slots, void* k, int64_t k_t, int64_t k_h,
                           void* v, int64_t v_t, int64_t v_h, int64_t T, int f16, void* stream);

/* Attention of one new token per sequence.  Sequence b of B has lengths[b]
 * cached tokens (the new one's own key and value among them); token t is row
 * t % page_size of page page_table[b][t / page_size].  Query head j reads
 * key-value head j / (Hq / heads):
 *   w_t = exp(softmax_scale * q . k_t),  t in [max(0, L - window), L)
 *   out = sum_t w_t v_t / sum_t w_t,     lse = ln sum_t w_t
 * (window 0: every token).  With no tokens, or only tokens of weight 0, out is
 * 0 and lse -inf.  Lengths are clamped to [0, max_pages * page_size]; the
 * tokens of a page whose table entry is outside [0, pages) are left out.
 *   q [B][Hq][D] and out [B][Hq][D] of the activation type (strides q_b, q_h,
 *   o_b, o_h; out may be q with the same strides), lse fp32 [B][Hq] or NULL, page_table int32
 *   [B][ld_table] (max_pages entries used), lengths int32 [B].
 * Products are fp32-accumulated MFMAs on bf16 (bf16 cache) or fp16 values, in
 * which a weight w_t has 16 (bf16), 22 (fp16, E4M3 cache) or 11 bits (NVFP4
 * cache); softmax statistics and sums are fp32; results are bitwise reproducible.
 *   workspace: nvfp4_paged_attention_workspace_bytes(B, Hq, heads, D,
 *   max_pages * page_size) bytes, 256-byte aligned, its first
 *   NVFP4_ATTENTION_COUNTER_BYTES zero before its first use; every call
 *   leaves the counters in them zero, so one workspace serves any
 *   number of calls of any sizes one after another (not calls that may overlap
 *   in time, and not the GEMMs: theirs has another layout).
 * Calls of up to 2048 sequences are split over the lengths.  With more, each
 * (sequence, key-value head, 16 query heads) is one workgroup's, so that the
 * longest sequence alone can decide how long a call takes (one of 131072 tokens
 * among 2048 of 40, 8 key-value heads of 128, bf16: 1.7 ms; among 2047, split,
 * 0.33): calls with such sequences are better made of 2048 at a time.
 * B == 0 launches nothing.  Errors: sizes, B > 65535, heads * ceil(Hq / heads / 16) >
 * 65535, Hq not a multiple of heads, max_pages < 0, max_pages * page_size >=
 * 2^30, softmax_scale not finite, window < 0, NULL pointers -> INVALID_ARG;
 * misaligned -> ALIGNMENT; workspace too small -> BUFFER_TOO_SMALL. */
#define NVFP4_ATTENTION_COUNTER_BYTES 2048
int64_t nvfp4_paged_attention_workspace_bytes(int64_t B, int64_t Hq, int64_t heads, int64_t D, int64_t max_tokens);
nvfp4_status nvfp4_paged_attention(const nvfp4_kv_cache* cache, const void* q, int64_t q_b, int64_t q_h,
                                   const int32_t* page_table, int64_t ld_table, int64_t max_pages,
                                   const int32_t* lengths, int64_t B, int64_t Hq, float softmax_scale, int64_t window,
                                   void* out, int64_t o_b, int64_t o_h, float* lse, void* workspace,
                                   int64_t workspace_bytes, int f16, void* stream);

/* ---- Around the layers of a decode step ----------------------------------------
 *
 * What a step runs before, beside and after the operators above: page tables
 * and slots from the requests' lengths, low-rank adapters beside a shared
 * projection, the expert layer of a few tokens in one call, and the next token
 * from its logits.  Alignment, strides, f16 and asynchrony as above. */

/* Page tables, slots and positions of a step's new tokens.  Request b of B has
 * cached[b] tokens in the cache and brings fresh[b] more; its pages of
 * page_size tokens are page_table[b][0 .. ceil(cached[b] / page_size)).  The
 * step's T rows hold the requests' new tokens one request after another:
 *   offsets[b] = min(T, sum_{a<b} max(0, fresh[a])),  b in [0, B],
 *   row offsets[b] + i is token cached[b] + i of request b:
 *     requests[row] = b, positions[row] = cached[b] + i,
 *     slots[row] = page_table[b][position / page_size] * page_size + position % page_size,
 * and requests take the pages that they need further from free_pages [F],
 * from place head[0] on, in their order; those are entered into page_table.
 *   lengths[b] = cached[b] + fresh[b],  head_out[0] = head[0] + the pages taken.
 * A request is refused, which leaves its row of page_table as it was, when a
 * length is negative, its pages do not fit the max_pages entries of a row, its
 * rows do not fit T, or its pages and those of the requests before it (refused
 * for this reason among them) do not fit the list: lengths[b] is then
 * max(0, cached[b]).  Rows of refused requests and rows behind the last one
 * have slot -1, position 0, request -1.  An entry or page outside [0, 2^31 /
 * page_size) gives slot -1.  Pages in the list are not checked for being used.
 *   Every array is int32 on the device: cached, fresh, lengths [B], page_table
 *   [B][ld_table], offsets [B + 1], head, head_out [1], slots, positions,
 *   requests [T].  lengths may be cached's memory and head_out head's, so that a
 *   captured step advances by itself; no other overlap.
 *   workspace: nvfp4_kv_plan_workspace_bytes(B, T) bytes (0 for small calls), 8-byte
 *   aligned, any contents.
 * Errors: sizes (B, T, max_pages * page_size and F < 2^30, ld_table), NULL
 * pointers -> INVALID_ARG; misaligned -> ALIGNMENT; workspace too small ->
 * BUFFER_TOO_SMALL. */
int64_t nvfp4_kv_plan_workspace_bytes(int64_t B, int64_t T); /* < 0 if invalid */
nvfp4_status nvfp4_kv_plan(const int32_t* cached, const int32_t* fresh, int64_t B, int32_t* page_table, int64_t ld_table,
                           int64_t max_pages, int64_t page_size, const int32_t* free_pages, int64_t F, const int32_t* head,
                           int64_t T, int32_t* slots, int32_t* positions, int32_t* requests, int32_t* lengths,
                           int32_t* offsets, int32_t* head_out, void* workspace, int64_t workspace_bytes, void* stream);

/* Low-rank adapters beside a shared projection: with a = adapter[t],
 *   out[t] = RNE16(y[t] + scale[a] * (x[t] A_a^T) B_a^T),
 * or y[t] unchanged where a is outside [0, L).  Sums are fp32; x A_a^T enters
 * the second product with 16 (bf16) or 22 (fp16) bits, in two parts (in fp16 on a
 * scale of its row: values below 2^-16 of the row's largest have fewer), so that
 * an infinite value of B gives an infinity or NaN.  A row depends on no other
 * row's values or adapter; where its sum over K is cut depends on T, K and L, so
 * the last bits may differ between calls of different sizes.
 *   x [T][ld_x] of K values, y and out [T][ld_y], [T][ld_o] of N (out may be y
 *   with the same leading dimension; no other overlap), a [L] matrices [R][K]
 *   (strides a_l, a_r), b [L] matrices [N][R] (strides b_l, b_n), adapter int32
 *   [T], scale fp32 [L] or NULL for 1.  Rows of x, a and b are 16-byte aligned;
 *   y and out need 2 bytes.
 *   workspace: nvfp4_lora_workspace_bytes(T, K, N, R) bytes, 16-byte aligned,
 *   any contents.
 * R a multiple of 8 in [8, 128], K a multiple of 8 (rows of a and b in 16-byte
 * pieces): a lower rank is padded, once, with rows of zeros in a and columns of
 * zeros in b, a higher one goes in parts (out as the next call's y, which rounds
 * it).  T == 0 or N == 0 launches nothing.  Errors: sizes (T <= 1048560, K and N < 2^24), NULL pointers ->
 * INVALID_ARG; misaligned -> ALIGNMENT; workspace too small -> BUFFER_TOO_SMALL. */
int64_t nvfp4_lora_workspace_bytes(int64_t T, int64_t K, int64_t N, int64_t R); /* < 0 if invalid */
nvfp4_status nvfp4_lora_add(const void* x, int64_t ld_x, const void* a, int64_t a_l, int64_t a_r, const void* b, int64_t b_l,
                            int64_t b_n, const int32_t* adapter, const float* scale, const void* y, int64_t ld_y, void* out,
                            int64_t ld_o, int64_t T, int64_t K, int64_t N, int64_t R, int64_t L, void* workspace,
                            int64_t workspace_bytes, int f16, void* stream);

/* A whole mixture-of-experts layer for a few tokens, T <= 64 and T * k <= 512:
 *   h = g1[e] * (X'[t] W1_e^T),  a = silu(h_gate) * h_up or max(h, 0)^2, times pre_scale2 if given,
 *   out[t] = RNE16(sum_j topk_weights[t][j] * g2[e] * (a W2_e^T)),  e = topk_ids[t][j],
 * X' = RNE16(x * pre_scale1) if that is given (pre_scale1 [H], pre_scale2 [I]).
 * Unlike the separate calls (nvfp4_moe_fc1, the grouped GEMM, nvfp4_moe_combine),
 * which round h, a and the experts' outputs to 16 bits, nothing is on the way:
 * sums are fp32, and a enters the second product with fp32's range and 24 bits
 * (below 2^-110 with fewer).  Results are bitwise reproducible; a token's last
 * bits may depend on the other tokens' number and experts, which decide where
 * sums are cut.  A pair whose id is outside [0, E) adds nothing; a token may name
 * an expert twice.
 * With many rows an expert the separate calls are faster (128 experts, top-8,
 * 2048 x 768: 16 tokens 46 us here and 49 by them, 24 60 and 60, 32 74 and 64, 64
 * 147 and 88; 8 experts, top-2, 4096 x 14336: 1 token 44 and 48, 5 100 and 92).
 *   x [T][ld_x] of H values, topk_ids int32 and topk_weights fp32 [T][k], w_fc1 a
 *   blob of nvfp4_repack_gated (NVFP4_MOE_SILU_GLU) or nvfp4_repack
 *   (NVFP4_MOE_RELU2) of E experts, I and H; w_fc2 of nvfp4_repack (E, H, I);
 *   global scales fp32 [E], or NULL with mx (blobs of mxfp4_repack_gated /
 *   mxfp4_repack); out [T][ld_o] of H values (may be x).
 *   workspace: nvfp4_moe_layer_workspace_bytes(T, k, E, H, I) bytes, 256-byte
 *   aligned, its first NVFP4_MOE_LAYER_COUNTER_BYTES zero before its first use;
 *   every call leaves them zero, so one workspace serves any number of these
 *   calls of any sizes one after another (not calls that may overlap in time,
 *   and no other operator's).
 * T == 0 launches nothing.  Errors: sizes (H and I multiples of 16, with mx of
 * 32, below 2^21), activation, mx, NULL pointers, global scales with mx ->
 * INVALID_ARG; misaligned -> ALIGNMENT; workspace too small -> BUFFER_TOO_SMALL. */
#define NVFP4_MOE_LAYER_COUNTER_BYTES 4096
int64_t nvfp4_moe_layer_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I); /* < 0 if invalid */
nvfp4_status nvfp4_moe_layer(const void* x, int64_t ld_x, const int32_t* topk_ids, const float* topk_weights, int64_t T,
                             int64_t k, const void* pre_scale1, const void* w_fc1, const float* global_scales1,
                             const void* pre_scale2, const void* w_fc2, const float* global_scales2,
                             int global_scale_is_divisor, int activation, void* out, int64_t ld_o, int64_t E, int64_t H,
                             int64_t I, void* workspace, int64_t workspace_bytes, int f16, int mx, void* stream);

/* The next token of each row from its logits l [B][ld] of V values (type: one
 * of NVFP4_LOGITS_*; NaN counts as -infinity).  With m the row's largest
 * logit, t = temperature[b] and w_i = exp((l_i - m) / t), tokens ordered by (l
 * descending, i ascending), these are kept:
 *   the first top_k[b] (all if top_k[b] < 1);
 *   of those, the ones before which the sum of w is < top_p[b] times the sum of
 *   w of those, the first always (all if top_p[b] >= 1 or NaN);
 *   of those, the ones with w >= min_p[b], the largest always.
 * tokens[b] is the kept token, in the order of i, at which the cumulative sum of
 * w first exceeds u[b] times its total (u in [0, 1); below it, or NaN, counts as
 * 0, above it as the last), and logprobs[b] = ln(w / total).  t <= 0 or NaN: the
 * first largest, logprob 0.  A row of -infinities: token -1, logprob -infinity.
 * A largest logit of +infinity leaves only those that equal it.
 * The weights are computed in fp64 and rounded to multiples of 2^-s, s = min(45,
 * 62 - ceil(log2 V)), or of less; sums do not depend on timing.
 *   u fp32 [B]; temperature (NULL: 1), top_p, min_p fp32 [B], top_k int32 [B]
 *   (NULL: off); tokens int32 [B]; logprobs fp32 [B] or NULL.  Rows of logits
 *   need only their type's alignment, and may share memory (ld below V).
 *   workspace: nvfp4_sample_workspace_bytes(B, V) bytes, 256-byte aligned, any
 *   contents.
 * B == 0 launches nothing.  Errors: sizes (B <= 65535, V in [1, 2^23], ld < 0),
 * NULL pointers -> INVALID_ARG; misaligned -> ALIGNMENT; workspace too small ->
 * BUFFER_TOO_SMALL. */
enum { NVFP4_LOGITS_BF16 = 0, NVFP4_LOGITS_F16 = 1, NVFP4_LOGITS_F32 = 2 };
int64_t nvfp4_sample_workspace_bytes(int64_t B, int64_t V); /* < 0 if invalid */
nvfp4_status nvfp4_sample(const void* logits, int64_t ld, int type, int64_t B, int64_t V, const float* u,
                          const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                          int32_t* tokens, float* logprobs, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_W4A16_H */
