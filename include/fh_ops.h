/*
 * fh_ops.h - operator-level entry points of the FlashHead DiT library, for unit
 * parity tests of single kernels. Same conventions as fh.h (return codes,
 * fh_last_error, caller-owned 16-byte-aligned device pointers, asynchronous on
 * `stream`). They allocate no device memory, and nothing else but one word of mapped host memory per
 * device, at the first fh_op_linear_mx or fh_op_probe_wait_timeout there (also while a stream captures),
 * kept for the process: the error word that fh_op_sync reports.
 *
 * Microscaled tensors (types FH_MXFP8 and FH_MXFP4) of M rows x K columns, K % 32 == 0, hold a
 * number as an element times its block's scale; a block is 32 consecutive values of a row.
 *   data    FH_MXFP8: e4m3 (largest value 448), one byte each, row-major [M][K]
 *           FH_MXFP4: e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte, the
 *           even column in the low four bits, row-major [M][K / 2]
 *   scales  e8m0, one byte per block: 2^(byte - 127), 255 is NaN. In tiles of 128 rows x 4
 *           blocks: row r, block k at ((r / 128) * ceil(K / 128) + k / 4) * 512 + (r % 32) * 16 +
 *           ((r % 128) / 32) * 4 + k % 4 (the order in which the tensor core takes them);
 *           fh_mx_scale_bytes(M, K) bytes, those past the tensor 0
 * Every operator that writes one chooses each block's scale as the smallest power of two,
 * 2^-127 or more, under which the block's largest magnitude is an element, and rounds each
 * value / scale to the nearest element, ties to the even code. A block with an infinity or a
 * NaN gets the scale byte 255 and zero codes: all its values read back as NaN.
 * M <= 2^27, K and N <= 2^20.
 */
#ifndef FH_OPS_H_
#define FH_OPS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* out[M, N] (float32) = A[M, K] * W[N, K]^T + bias[N]: the dense contraction every
 * Linear of the DiT uses (gizai:flashhead, Types > FlashHead: `patch`, `head` and the
 * blocks' projections are Linear layers). dtype FH_BF16: A, W bfloat16, tensor-core
 * (tcgen05) path, requires N % 128 == 0, K % 64 == 0; FH_F32: A, W float32, CUDA-core
 * path, requires N % 128 == 0, K % 32 == 0. Errors: FH_ERR_ARG, FH_ERR_SHAPE,
 * FH_ERR_CUDA. */
int fh_op_linear(const void* A, const void* W, const float* bias, float* out, int M, int N, int K, int dtype,
                 void* stream);

/* Non-causal self-attention over L tokens per (stream, head), as inside a block
 * (gizai:flashhead, opening paragraph; readings R4-R6): q, k, v [batch, heads, L,
 * 128] in dtype, except that with FH_BF16 v is float16 (as the QKV projection stores it:
 * the kernel multiplies v by float16 softmax weights); ssq float32 [batch*L, 2*heads] with the per-head partial sums of
 * squares of q (first heads columns) and k (last heads columns), whose sum over
 * heads divided by heads*128, plus eps, gives each token's RMS factor r^-2; scores
 * are r_i r_j (q_i . k_j) / sqrt(128). out [batch*L, heads*128] in dtype. */
int fh_op_attention(const void* q, const void* k, const void* v, const float* ssq, void* out, int batch,
                    int heads, int L, float eps, int dtype, void* stream);

/* Per-frame audio cross-attention, as inside a block (gizai:flashhead, opening paragraph:
 * each slice's audio becomes 5 latent frames of 32 audio tokens; readings R4-R6): token n
 * of latent frame f = n / hw of stream b attends to the audio_tokens (= 32, else
 * FH_ERR_SHAPE) keys of that frame only,
 *   out_n = sum_a softmax_a(r_n r_a (q_n . k_a) / sqrt(128)) v_a   per head.
 * q [batch*frames*hw, heads*128] (token-major, frame-major within a stream) in dtype;
 * ssq_q float32 [batch*frames*hw, heads] per-head partial sums of squares of the query
 * row, whose sum over heads divided by heads*128, plus eps, gives r_n^-2; kv
 * [batch*frames*32, 2*heads*128] in dtype: row (b*frames + f)*32 + a holds key a of that
 * frame in its first heads*128 columns and its value in the rest; ssq_k float32
 * [batch*frames*32, heads] the keys' partial sums. out like q. dtype FH_BF16: the
 * tensor-core kernel (TMA over 3D [frame][hw][D] views: hw need not be a multiple of
 * 128, rows past a frame are neither read nor written); FH_F32: CUDA cores. */
int fh_op_cross_attention(const void* q, const float* ssq_q, const void* kv, const float* ssq_k, void* out,
                          int batch, int heads, int frames, int hw, int audio_tokens, float eps, int dtype,
                          void* stream);

/* One norm and modulation per row, as before the block's projections (gizai:flashhead,
 * opening paragraph, "Wan-style"; readings R1, R2, R7, R9): x float32 [M, D] (D / 128 in
 * {1, 2, 3, 4, 6, 8, 12, 16}, else FH_ERR_SHAPE), out [M, D] in dtype.
 *   mode 0: LayerNorm(x) * (1 + a) + c    mode 2: RMSNorm(x) * (1 + a) + c
 *     (a = scale, c = shift: float32 vectors of D, the stream's own at a + (row /
 *      rows_per_batch) * bstride)
 *   mode 1: LayerNorm(x) * a + c            (a = weight, c = bias; bstride ignored)
 * LayerNorm with the biased variance, no gain of its own; eps inside the root. */
int fh_op_row_norm(const float* x, void* out, int M, int D, int mode, const float* a, const float* c, long bstride,
                   int rows_per_batch, float eps, int dtype, void* stream);

/* Bytes of a microscaled tensor's two parts; 0 for a type or a size that has none. */
size_t fh_mx_data_bytes(int M, int K, int mxtype);
size_t fh_mx_scale_bytes(int M, int K);

/* x [M][K] in dtype (FH_F32 or FH_BF16), rows ldx elements apart (ldx >= K, a multiple of 16
 * bytes), to the microscaled type mxtype. Errors: FH_ERR_ARG (pointers, types), FH_ERR_SHAPE. */
int fh_op_quantize(const void* x, long ldx, int M, int K, int dtype, int mxtype, void* data, void* scales,
                   void* stream);

/* The values of a microscaled tensor, out [M][K] in dtype: exact, but that values of 2^128 and
 * above (which scales of 2^118 and more can make) become infinite, and that FH_BF16 rounds
 * what is no multiple of 2^-133. */
int fh_op_dequantize(const void* data, const void* scales, int M, int K, int mxtype, void* out, int dtype,
                     void* stream);

/* The residual's addition and the RMS norm after it, with the result in the type that the next
 * Linear takes: sum = x + res in x's type, and with n = sum / sqrt(mean(sum^2) + eps) per row (of
 * the sum as it is kept), out = n * a where c is null, n * (1 + a) + c elsewhere. x, sum [M][D] in
 * x_dtype, res [M][D] in res_dtype (FH_F32 or FH_BF16); D % 32 == 0, D <= 16384; a, c float32
 * vectors of D, row r's at a + (r / rows_per_batch) * bstride (bstride % 4 == 0). out_type any
 * of fh_dtype; out_scales for the microscaled ones, else null. sum may be x, or res where its
 * type is x's; it may not overlap them otherwise, nor a or c, nor out anything. */
int fh_op_add_rms_norm(const void* x, int x_dtype, const void* res, int res_dtype, void* sum, const float* a,
                       const float* c, long bstride, int rows_per_batch, int M, int D, float eps, int out_type,
                       void* out, void* out_scales, void* stream);

enum fh_act { FH_ACT_NONE = 0, FH_ACT_GELU = 1 };

/* out [M][N] = act(A [M][K] * W [N][K]^T + bias [N]) of two microscaled operands of one type, on
 * the block-scaled tensor core, accumulated in fp32 (it cuts off what does not fit an addition: the
 * result's norm is off by 1e-7 at K = 1536, 3e-7 at 8960); bias float32 or null; act FH_ACT_GELU: the
 * tanh form of GELU (-2.7e-9 for arguments below -5.6, which is off by up to that). K % 32 == 0; N any,
 * but a multiple of 32 for a microscaled out. out_type any of fh_dtype; out_scales for the
 * microscaled ones, else null. A row or column with a NaN scale gives NaN results. out may not overlap
 * the operands. FH_ERR_TIMEOUT: a kernel-side wait of an earlier call on this device ran out; reported
 * once, nothing is launched. */
int fh_op_linear_mx(const void* A, const void* A_scales, const void* W, const void* W_scales, const float* bias,
                    int M, int N, int K, int mxtype, int act, int out_type, void* out, void* out_scales,
                    void* stream);

/* Wait for `stream`, then report (FH_ERR_TIMEOUT) and clear what the microscaled product latched on the
 * current device: a bounded kernel-side wait that ran out, so that a result since the last report is not
 * valid. The next fh_op_linear_mx reports it too. */
int fh_op_sync(void* stream);

/* Make one such wait run out, as fh_dit_probe_wait_timeout below does for a model. */
int fh_op_probe_wait_timeout(void* stream);

/* Failure-detection check (no counterpart on the pages; reading of the pages'
 * reject-don't-hang stance): launches one CTA whose mbarrier wait has no arriving
 * party. The kernel's bounded wait (the same one every production kernel uses, about
 * one second of %globaltimer) runs out, latches the timeout bit into the model's
 * device-visible error word and the kernel returns; nothing faults or hangs. The next
 * fh_dit_sync on `stream` reports FH_ERR_TIMEOUT once and clears the word. */
struct fh_dit;
int fh_dit_probe_wait_timeout(struct fh_dit* m, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FH_OPS_H_ */
