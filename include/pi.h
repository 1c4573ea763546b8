/*
 * pi.h -- C ABI of the neuron-aware sparse FFN library (libpi.so) for AMD MI355X (gfx950).
 *
 * The library computes the FFN of a ReLU / ReGLU transformer layer by predicting which
 * FFN neurons fire for the current token(s), compacting their indices, and reading and
 * multiplying only those neurons' up/gate rows and down columns. This is the hot path of
 * PowerInfer as described on the pages
 *   P1 "Tüketici sınıfı GPU takılı PC'lerde yüksek hızlı büyük dil modeli serving",
 *   P2 "PowerInfer: Fast Large Language Model Serving with a Consumer-grade GPU" (КПД),
 *   P3 "PowerInfer: Mesin Inferensi LLM Cepat dengan GPU Konsumen" (unite.ai).
 *
 * Conventions shared by every entry point:
 *  - Tensor pointers are DEVICE pointers owned by the caller, 16-byte aligned, row-major.
 *    The library never frees them. A pi_ffn borrows its weight pointers until destroyed.
 *  - Compute entry points enqueue work on the context's HIP stream and return without
 *    host synchronisation. Device faults surface at the caller's next synchronisation.
 *  - Argument errors are detected on the host before anything is enqueued: the call
 *    returns PI_ERR_INVALID (or PI_ERR_UNSUPPORTED) and enqueues nothing. HIP launch
 *    failures return PI_ERR_HIP. pi_last_error(ctx) gives a human-readable reason.
 *  - Compute entry points allocate nothing: every scratch buffer (activations, partial
 *    sums, mask words, staging) belongs to the pi_ctx and is sized at pi_ctx_create.
 *  - No C++ exception crosses this boundary. A pi_ctx is used by one host thread at a time,
 *    and the work of one context must not run concurrently with itself (its scratch is
 *    shared between calls): keep a context's calls on one stream, or order them.
 *  - Neuron index space: the "stored" order of the layer's rows. With a hot-first layout
 *    (pi_permute_rows), neuron_table[k] maps stored row k back to its original neuron.
 */
#ifndef PI_H
#define PI_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PI_ABI_VERSION 2

typedef enum {
  PI_OK = 0,
  PI_ERR_INVALID = 1,      /* bad argument: null pointer, bad shape, misalignment, too large */
  PI_ERR_UNSUPPORTED = 2,  /* valid but not implemented (e.g. batch size outside a path)     */
  PI_ERR_OOM = 3,          /* device allocation failed in pi_ctx_create                      */
  PI_ERR_HIP = 4           /* a HIP runtime call failed; see pi_last_error                    */
} pi_status;

/* Activation families the method supports (P1 header bullets, «Kısıtlar ve SSS»):
 * ReLU a = max(h, 0); ReGLU a = max(g, 0) * u; Squared-ReLU a = max(h, 0)^2. ReLU and
 * Squared-ReLU read one row per neuron (w_up, masked on h > 0); ReGLU reads two (w_gate,
 * masked on g > 0, and w_up). */
typedef enum { PI_ACT_RELU = 0, PI_ACT_REGLU = 1, PI_ACT_SQRELU = 2 } pi_act;

/* Weight storage. PI_W_Q4_0: each block of 32 consecutive elements of a row stores an fp16
 * scale s and 32 4-bit codes q; the weight is (q - 8) * s (P1 «Kuantizasyon ve uyumluluk»).
 * Layout is struct-of-arrays: codes uint8 [rows][d/32][16], byte j of a block holding
 * element j in its low nibble and element j+16 in its high nibble; scales fp16 [rows][d/32]. */
typedef enum { PI_W_F32 = 0, PI_W_F16 = 1, PI_W_Q4_0 = 2 } pi_wtype;

typedef struct pi_ctx pi_ctx;
typedef struct pi_ffn pi_ffn;

/* One FFN layer (borrowed device pointers). Neuron-major layout: row i of w_up / w_gate is
 * neuron i's input row, row i of w_down_t is neuron i's output column (W_down transposed),
 * so an active neuron's weights are contiguous rows (P3 «Operator yang Sadar Neuron»).
 *   d        model width, multiple of 8 (of 32 for Q4_0)
 *   ffn      number of FFN neurons, multiple of 64
 *   rank     predictor rank r (multiple of 8, at most 1024; fp16 / Q4_0 layers only), or 0:
 *            no predictor, the mask is the true pre-activation of the masked projection
 *            (> threshold)
 *   act      pi_act. ReLU and Squared-ReLU mask the up projection; ReGLU masks the gate.
 *   wtype    pi_wtype of w_up / w_gate / w_down_t
 *   threshold decision threshold on the predictor logit (0 == "sigmoid > 0.5")
 *   w_up, w_gate, w_down_t   [ffn][d] (fp32 / fp16) or Q4_0 codes; w_gate NULL unless ReGLU
 *   s_up, s_gate, s_down     Q4_0 fp16 scales [ffn][d/32]; NULL otherwise
 *   b        fp32 [ffn] bias of the masked projection (gate for ReGLU, else up)
 *   p_w1     fp16 [rank][d], p_w2 fp16 [ffn][rank], p_b fp32 [ffn]: the low-rank predictor
 *            logit = p_w2 (p_w1 x) + p_b (P3 «Prediktor Kepadatan Adaptif»); NULL if rank 0
 *   neuron_table  int32 [ffn] stored row -> original neuron id, or NULL (identity).
 *            Informational: outputs are in stored order.
 *   hot_prefix  H in [0, ffn]: the first H stored neurons are taken for every token without
 *            a prediction (their predictor rows are not read, their decision value is +inf)
 *            and the activation itself zeroes those that do not fire: the hot neurons
 *            PowerInfer keeps resident and always computes (P1 header bullets and «CPU/GPU
 *            hibrit çıkarım yöntemi»; P3 «Penempatan dan Pengelolaan Neuron»), on a hot-first
 *            layout. Predictor layers only (rank > 0); 0 for none.
 *   y_center fp32 [d] or NULL: this layer's expected output, subtracted from its y before the
 *            normalisation that feeds the next layer of a stack (pi_stack_run, pi_glue). */
typedef struct pi_ffn_desc {
  int32_t d, ffn, rank;
  int32_t act;
  int32_t wtype;
  float threshold;
  const void *w_up, *w_gate, *w_down_t;
  const uint16_t *s_up, *s_gate, *s_down;
  const float *b;
  const uint16_t *p_w1, *p_w2;
  const float *p_b;
  const int32_t *neuron_table;
  int32_t hot_prefix;
  const float *y_center;
} pi_ffn_desc;

int32_t pi_abi_version(void);
const char *pi_status_str(pi_status s);
/* Reason of the last failed call on ctx (empty string if none). Valid until the next call. */
const char *pi_last_error(const pi_ctx *ctx);

/* Create a context bound to `device` and the HIP stream `hip_stream` (hipStream_t, may be
 * NULL for the default stream). Sizes the scratch for batches up to max_batch tokens and
 * layers up to max_d x max_ffn with predictor rank up to max_rank. Allocates device memory.
 * A context and its handles may be destroyed in any order; no call takes a handle once its
 * context is destroyed. */
pi_status pi_ctx_create(int32_t device, void *hip_stream, int32_t max_batch, int32_t max_d,
                        int32_t max_ffn, int32_t max_rank, pi_ctx **out);
void pi_ctx_destroy(pi_ctx *ctx);
/* Rebind the context to another stream on the same device. */
pi_status pi_ctx_set_stream(pi_ctx *ctx, void *hip_stream);

/* Validate a layer description against the context and wrap it. Copies the descriptor,
 * not the weights. */
pi_status pi_ffn_create(pi_ctx *ctx, const pi_ffn_desc *desc, pi_ffn **out);
void pi_ffn_destroy(pi_ffn *ffn);

/* Masking of a batch of B > 1 tokens in pi_layer, pi_stack_run and pi_stack_profile:
 *  PI_MASK_UNION      (default) every token gets the activations of every neuron in the
 *                     union of the batch's masks (ReLU zeroes the neurons it does not
 *                     itself activate)
 *  PI_MASK_PER_TOKEN  each token gets only its own predicted neurons, a_t,i = 0 where bit i
 *                     of token t's mask is clear: the operator of P3 «Operator yang Sadar
 *                     Neuron» applied one token at a time with the mask P3 «Prediktor
 *                     Kepadatan Adaptif» gives that token.
 * The same rows are read either way (those of the union). The mode is a property of the
 * context; pi_sparse_ffn (one list for all tokens) does not depend on it. */
typedef enum { PI_MASK_UNION = 0, PI_MASK_PER_TOKEN = 1 } pi_mask_mode;

/* Set the context's masking of batches; PI_ERR_INVALID for another value. Work already
 * enqueued keeps the mode it was enqueued with. */
pi_status pi_ctx_set_mask_mode(pi_ctx *ctx, int32_t mode);

/* Predict the active neurons of B tokens (P3 «Fase Online», «Prediktor Kepadatan Adaptif»).
 *   x         [B][d] fp16 (fp32 when wtype == PI_W_F32)
 *   mask      [B][ffn/64] uint64 per-token bits: bit j of word w is neuron 64w+j, set when
 *             the decision value (predictor logit, or true pre-activation if rank 0) is
 *             strictly above the threshold
 *   idx       [ffn] int32: ascending indices of the UNION of the B masks (the token's own
 *             list when B == 1); entries at and beyond n_active are unspecified
 *   n_active  device int32 scalar: length of idx
 *   logits_out nullable fp32 [B][ffn]: the decision values themselves (for checking)
 *   B         1..max_batch (at most 64); 1..8 run on the vector units, 9..64 on the
 *             matrix cores (fp16 weights, d and rank multiples of 16); mask words are then
 *             written as 32-bit halves (same bit layout) */
pi_status pi_predict(pi_ctx *ctx, const pi_ffn *ffn, const void *x, int32_t B, uint64_t *mask,
                     int32_t *idx, int32_t *n_active, float *logits_out);

/* The neuron-aware sparse FFN on a given index list (P3 «Operator yang Sadar Neuron»): for
 * every listed neuron i, a_t,i = relu(w_up[i].x_t + b_i) (ReLU), its square (Squared-ReLU)
 * or relu(w_gate[i].x_t + b_i) * (w_up[i].x_t) (ReGLU), and y_t = sum_i a_t,i w_down_t[i].
 * The one list applies to all B tokens.
 *   idx, n_active  device [ffn] int32 (each entry < ffn, no duplicates) and device int32
 *   y         [B][d] fp32 output (overwritten) */
pi_status pi_sparse_ffn(pi_ctx *ctx, const pi_ffn *ffn, const void *x, int32_t B,
                        const int32_t *idx, const int32_t *n_active, float *y);

/* One FFN layer for B tokens (P3 «Fase Online»: the predictor marks the neurons likely to
 * fire, inactive ones are skipped, active ones computed): pi_predict followed by
 * pi_sparse_ffn on its union list, as three or four fused kernels. mask, idx and n_active
 * are nullable outputs (context scratch is used when NULL). */
pi_status pi_layer(pi_ctx *ctx, const pi_ffn *ffn, const void *x, int32_t B, float *y,
                   uint64_t *mask, int32_t *idx, int32_t *n_active);

/* pi_layer for callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): no pi_ctx, and no allocation at
 * all. Its scratch (predictor stage 1 output, mask words, index list, activations, partial
 * sums) is one fixed device array of the library, 26.1 MiB, which each GPU it runs on
 * holds until the process ends. Every call on a GPU shares that GPU's array: calls that
 * overlap on one GPU (several streams or threads) race; order them. No part of the array
 * needs to start at zero. Limits: B <= 8 tokens, d <= 12288, ffn <= 49152, rank <= 1024
 * (PI_ERR_UNSUPPORTED beyond them); otherwise the arguments, outputs, errors and kernels are
 * those of pi_layer on a context of the same stream in union masking (the result is bitwise
 * the same). PI_ERR_INVALID for a bad argument or description (no reason is kept: there is
 * no context). Work is enqueued on hip_stream (NULL: the default stream) of `device`, which
 * becomes the current device. */
pi_status pi_layer_noalloc(int32_t device, void *hip_stream, const pi_ffn_desc *desc, const void *x,
                           int32_t B, float *y, uint64_t *mask, int32_t *idx, int32_t *n_active);

/* Threshold + compaction alone, on caller-provided decision values v [B][ffn] fp32:
 * the same device code pi_predict uses after computing v (P3 «Prediktor Kepadatan Adaptif»:
 * neurons predicted active are processed; P3 «Operator yang Sadar Neuron»: they are then
 * addressed directly, with no dense conversion). B is 1..8. */
pi_status pi_compact(pi_ctx *ctx, const float *v, int32_t B, int32_t ffn, float threshold,
                     uint64_t *mask, int32_t *idx, int32_t *n_active);

/* Chain between stacked layers, so that each token passes through every layer before the
 * next token (P3 introduction). The pages define no layer between FFNs; this one keeps every
 * layer's input at the scale its calibration assumes: u_t = y_t - c, x_out_t = round(u_t /
 * sqrt(mean(u_t^2))) to x's storage type (fp16, or fp32 when x_is_f32), or x_prev_t
 * unchanged when y_t (or u_t) is all zero.
 *   y [B][d] fp32, center c fp32 [d] or NULL (zero), x_prev [B][d], x_out [B][d] */
pi_status pi_glue(pi_ctx *ctx, const float *y, const float *center, const void *x_prev, int32_t B,
                  int32_t d, int32_t x_is_f32, void *x_out);

/* Run L layers over T tokens, B tokens per step (T % B == 0), one step at a time: step s
 * feeds x_tokens[s*B..s*B+B) to layer 0, each layer's y (through pi_glue, with that layer's
 * y_center) to the next, and writes the last layer's y to y_out[s*B..]. Token-by-token
 * decode (P3 intro) at B == 1.
 *   layers     host array of L layer handles with equal d and activation/weight types
 *   x_tokens   [T][d] fp16 (fp32 for PI_W_F32 stacks); y_out [T][d] fp32
 *   n_active_log nullable device int32 [T/B][L]: n_active of every (step, layer)
 *   use_graph  nonzero: each step's L layers run as one captured HIP graph */
pi_status pi_stack_run(pi_ctx *ctx, const pi_ffn *const *layers, int32_t L, const void *x_tokens,
                       int32_t T, int32_t B, float *y_out, int32_t *n_active_log, int32_t use_graph);

/* What pi_stack_run_dump records of every (step, layer); each pointer is DEVICE memory or
 * NULL (not recorded). With S = T/B steps, slot (s, l) is at index s*L + l:
 *   x     [S][L][B][d] in x's storage type: the layer's input as its kernels read it
 *   mask  [S][L][B][ffn_stride/64] uint64: the tokens' predicted mask words
 *   idx   [S][L][ffn_stride] int32: the ascending union list (entries past n unspecified)
 *   n     [S][L] int32: the union count
 *   y     [S][L][B][d] fp32: the layer's output (its partial sums added)
 *   ffn_stride  >= every layer's ffn, a multiple of 64 */
typedef struct pi_stack_dump {
  void *x;
  uint64_t *mask;
  int32_t *idx;
  int32_t *n;
  float *y;
  int32_t ffn_stride;
} pi_stack_dump;

/* pi_stack_run with every layer's input, mask, index list, count and output recorded, for
 * checking a whole stack layer by layer against a reference that takes each layer's
 * recorded input (P3 «Fase Online»: per layer, predict, skip the inactive, compute the
 * active). Runs the same kernels in the same order as pi_stack_run, eagerly (no graph),
 * with copies and sums of partials into the dump between layers; y_out and n_active_log are
 * therefore bitwise those of pi_stack_run. Other arguments as for pi_stack_run. */
pi_status pi_stack_run_dump(pi_ctx *ctx, const pi_ffn *const *layers, int32_t L, const void *x_tokens,
                            int32_t T, int32_t B, float *y_out, int32_t *n_active_log,
                            const pi_stack_dump *dump);

/* Kernel classes of pi_stack_profile's outputs, in this order:
 * predictor stage 1 (with the glue); predictor stage 2 + threshold + the activations of the
 * workgroup's active neurons; true-mask threshold GEMV + activations; gathered up/gate GEMV
 * (index-list entry point; the separate, column-sliced GEMV that 1..8 tokens take instead
 * of stage 2's activations when x is above 64 KiB, for Q4_0, d >= 8192 or 5..8 tokens; the
 * matrix-core path's gathered GEMM);
 * down projection (with the index scan) into partial sums; the small kernels: sum of
 * partial sums into y, activations from the column slices' partial sums, glue between
 * layers of several tokens, compaction and predictor hi/lo split of the matrix-core path. */
#define PI_KERNEL_CLASSES 6

/* pi_stack_run without a graph, every kernel dispatched with a pair of hipEvents
 * (hipExtLaunchKernelGGL) on the context's stream, so each pair times that kernel's own
 * execution: the per-kernel time of the generation speed the pages measure end to end
 * in tokens/s (P1 «Performans değerlendirmesi ve demo»). Blocks until the work is done,
 * then writes the summed event time in milliseconds (ms_out[PI_KERNEL_CLASSES], host) and
 * the number of launches (launches_out[PI_KERNEL_CLASSES], host) of each kernel class.
 * Other arguments as for pi_stack_run. For measurement. */
pi_status pi_stack_profile(pi_ctx *ctx, const pi_ffn *const *layers, int32_t L, const void *x_tokens,
                           int32_t T, int32_t B, float *y_out, int32_t *n_active_log, double *ms_out,
                           int64_t *launches_out);

/* Q4_0 rows to fp32 with the kernels' own in-register unpacking (P1 «Kuantizasyon ve
 * uyumluluk»: 4-bit weights in 32-element blocks with a 16-bit scale): out[i][c] =
 * (q - 8) * s for every row i < rows and column c < d, where block b of row i is the 16
 * code bytes codes[(i * d/32 + b) * 16 ...] (byte j: element j in the low nibble, element
 * j + 16 in the high nibble) and its scale is the fp16 scales[i * d/32 + b]. (q - 8) is
 * rebuilt exactly in fp16 and multiplied by the scale in fp32, which is exact (a 4-bit by an
 * 11-bit significand), so the result is bitwise the dequantised weight. Device pointers:
 * codes [rows][d/2] bytes, scales [rows][d/32] fp16, out [rows][d] fp32. d % 32 == 0. For
 * checking the dequantisation against a plain implementation. */
pi_status pi_q4_dequant(pi_ctx *ctx, const uint8_t *codes, const uint16_t *scales, int32_t rows, int32_t d,
                        float *out);

/* Hot-first neuron order (P3 «Penempatan dan Pengelolaan Neuron»): perm[k] = the neuron
 * with the k-th largest activation probability, ties in ascending neuron order. HOST
 * pointers: p double [ffn], perm int32 [ffn]. */
pi_status pi_hot_first_order(const double *p, int32_t ffn, int32_t *perm);

/* Gather rows on the device: dst[k] = src[perm[k]] for k < rows, each row_bytes long
 * (a multiple of 4). Used to store a layer's neuron-indexed arrays in hot-first order
 * (P3 «Penempatan dan Pengelolaan Neuron»: neurons placed by hotness, with a table back to
 * their original positions).
 * perm is a device int32 [rows] permutation; src and dst must not overlap. */
pi_status pi_permute_rows(pi_ctx *ctx, const void *src, void *dst, const int32_t *perm,
                          int32_t rows, int64_t row_bytes);

/* ---------------------------------------------------------------- the decoder around the FFN
 *
 * The dense operators a decoder layer needs next to the sparse FFN when it serves drafted
 * tokens: attention of a tree of tokens over a paged key/value cache, the append of the
 * accepted tokens to that cache, the check of drafted tokens against the target's
 * distribution, the residual's RMS norm with an 8-bit output, and the 8-bit matrix product; and for
 * prompts and long caches the norm and rotary positions of query and key heads, causal attention of
 * packed prompts, and the cache held in 4 bits.
 * They follow the conventions above. Tensors of these calls may be views: strides are given
 * in elements, the last axis is contiguous, and rows start at a multiple of 16 bytes unless a
 * call says otherwise. A pi_attn, a pi_prompt and a pi_verifier keep their own scratch, sized when they are
 * created. The product's scratch is the context's, one buffer of 33.5 MB that all its pi_linear
 * share: as for the FFN's calls, they and the replays of graphs that hold them must be ordered.
 * Every handle borrows the pointers of its description; a pi_attn keeps its cache's description
 * and pointers, not the pi_kv. */

typedef enum { PI_T_F32 = 0, PI_T_F16 = 1, PI_T_BF16 = 2 } pi_dtype;

typedef struct pi_kv pi_kv;
typedef struct pi_attn pi_attn;
typedef struct pi_verifier pi_verifier;
typedef struct pi_linear pi_linear;

/* A key/value cache of one layer: `pages` pages of page_tokens tokens each, k and v alike.
 * Token t of page p, head h is head_dim contiguous elements at p*page_stride + t*token_stride +
 * h*head_stride.
 *   dtype      PI_T_F16 or PI_T_BF16
 *   heads      key/value heads; head_dim a multiple of 8 up to 256
 *   strides    in elements, multiples of 8 below 2^35
 * Which pages a sequence has is an argument of the calls: table, int32 [B][table_width] with
 * table_stride elements between sequences, names page table[b][i] for the positions from
 * i*page_tokens on. A NULL table stands for one page each, page b for sequence b. Positions
 * are below table_width*page_tokens, which must be below 2^31 - 64. Tokens of a page number
 * outside the cache count as zeros where they are read and are dropped where they are written. */
typedef struct pi_kv_desc {
  int32_t dtype;
  int32_t heads, head_dim, pages, page_tokens;
  void *k, *v;
  int64_t page_stride, token_stride, head_stride;
} pi_kv_desc;

pi_status pi_kv_create(pi_ctx *ctx, const pi_kv_desc *desc, pi_kv **out);
void pi_kv_destroy(pi_kv *kv);

/* A key/value cache of one layer in 4 bits: 4.5 bits per element. Token t of page p, head h has
 * head_dim/2 bytes of codes at p*page_stride + t*token_stride + h*head_stride and head_dim/32 fp16
 * scales at p*scale_page_stride + t*scale_token_stride + h*scale_head_stride, k and v alike. Each block
 * of 32 elements along the head has one scale and 16 bytes, byte j holding element j in its low half and
 * element j + 16 in its high half; an element's value is (code - 8) * scale (the layout of PI_W_Q4_0).
 *   dtype      PI_T_F16 or PI_T_BF16: the type of the tokens appended, read and attended with
 *   head_dim   a multiple of 32 up to 256
 *   strides    of the codes in bytes, multiples of 16 below 2^35; of the scales in elements below 2^32,
 *              even where head_dim is a multiple of 64
 * pi_kv_append writes a block so: m is its element of the largest magnitude (of two alike the positive
 * one), scale = -m/8 rounded to bf16's 8 significant bits, at most 8160, then to fp16; code =
 * round(x/scale) + 8 within 0..15. Every value is then an fp16 number exactly. A block with an
 * infinity or a NaN has the scale NaN; one whose scale is 0 reads as zeros. Scales from elsewhere may be any
 * fp16 number up to 8188 in magnitude; values are then rounded to fp16 where attention uses them.
 * The handle is a pi_kv: pi_kv_append, pi_kv_read, pi_attn_create and pi_kv_destroy take it. A
 * head's tokens of a page next to each other (head_stride above token_stride) read fastest. */
typedef struct pi_kv4_desc {
  int32_t dtype;
  int32_t heads, head_dim, pages, page_tokens;
  uint8_t *k, *v;
  int64_t page_stride, token_stride, head_stride;
  uint16_t *k_scale, *v_scale;
  int64_t scale_page_stride, scale_token_stride, scale_head_stride;
} pi_kv4_desc;

pi_status pi_kv4_create(pi_ctx *ctx, const pi_kv4_desc *desc, pi_kv **out);

/* Append tokens to the cache: token nodes[b][j] (j itself when nodes is NULL) of sequence b's N
 * new tokens goes to position ctx_len[b] + j, for j < n[b] (all N when n is NULL).
 *   k_new, v_new  [B][N][heads][head_dim] of the cache's type, strides for both
 *   ctx_len    device int32 [B]: tokens held before the call (negative: 0)
 *   nodes, n   device int32 [B][N] and [B], nullable; an entry outside [0, N) writes nothing
 *   len_out    device int32 [B], nullable: ctx_len + n, at most the table's positions. It may be
 *              ctx_len itself.
 * Positions beyond the table are dropped. Two sequences must not share the pages written. */
typedef struct pi_append_args {
  const void *k_new, *v_new;
  int64_t kv_batch, kv_node, kv_head;
  const int32_t *table;
  int64_t table_stride;
  int32_t table_width;
  const int32_t *ctx_len;
  const int32_t *nodes, *n;
  int32_t *len_out;
  int32_t B, N;
} pi_append_args;

pi_status pi_kv_append(pi_ctx *ctx, const pi_kv *kv, const pi_append_args *args);

/* Read positions of a cache of either kind into packed rows: row cu[b] + i, for i below cu[b+1] -
 * cu[b], gets the keys and values of sequence b's position start[b] + i. Rows of positions at or beyond
 * ctx_len[b], and rows of no sequence, stay as they are; positions of pages outside the cache read as
 * zeros. Values of a 4-bit cache are rounded to its dtype (fp16 holds them exactly).
 *   cu         device int32 [B+1], ascending; rows outside [0, rows) are not written
 *   start      device int32 [B] (negative: 0), or NULL: 0
 *   ctx_len    device int32 [B], taken as 0 below 0 and as the table's positions above them
 *   k_out, v_out  [rows][heads][head_dim] of the cache's dtype, strides for both; rows up to 2^27 */
typedef struct pi_read_args {
  const int32_t *table;
  int64_t table_stride;
  int32_t table_width;
  const int32_t *ctx_len, *start, *cu;
  void *k_out, *v_out;
  int64_t out_row, out_head;
  int32_t B, rows;
} pi_read_args;

pi_status pi_kv_read(pi_ctx *ctx, const pi_kv *kv, const pi_read_args *args);

/* Attention of drafted trees over the cache. Node i of sequence b sees every cached position
 * below ctx_len[b] and the new nodes j whose bit j is set in tree[b][i]:
 *   out[b][i][h] = sum_p w_p v_p,  w = softmax over the seen p of scale * q[b][i][h] . k_p,
 * with key/value head h * kv_heads / heads. A node that sees nothing gets zeros; what is not
 * seen does not enter the result, whatever it holds. Over a 4-bit cache the cached keys and values are its
 * values, the new nodes' are given in its dtype; of a bf16 query, elements more than 2^31 times smaller than the
 * head's largest lose bits there, more than 2^39 times smaller ones count as zeros. Sums are in fp32: over a plain
 * bf16 cache, values above 2^128 / (ctx_len + N) may leave its range.
 *   heads      query heads, a multiple of the cache's heads
 *   scale      above 0, at most 2^127
 *   max_batch, max_nodes (1..64)   limits of B and N, which size the scratch
 * Over a 4-bit cache B times the table's positions is below 2^37. */
pi_status pi_attn_create(pi_ctx *ctx, const pi_kv *kv, int32_t heads, int32_t max_batch, int32_t max_nodes,
                         float scale, pi_attn **out);
void pi_attn_destroy(pi_attn *attn);

/*   q, out     [B][N][heads][head_dim] of the cache's type
 *   k_new, v_new  [B][N][kv heads][head_dim], the new nodes' keys and values (strides for both)
 *   tree       device uint64 [B][N], or NULL: node i sees nodes 0..i (a chain)
 *   ctx_len    device int32 [B], taken as 0 below 0 and as the table's positions above them */
typedef struct pi_attn_args {
  const void *q;
  int64_t q_batch, q_node, q_head;
  const void *k_new, *v_new;
  int64_t kv_batch, kv_node, kv_head;
  const uint64_t *tree;
  const int32_t *table;
  int64_t table_stride;
  int32_t table_width;
  const int32_t *ctx_len;
  void *out;
  int64_t out_batch, out_node, out_head;
  int32_t B, N;
} pi_attn_args;

pi_status pi_tree_attention(pi_ctx *ctx, pi_attn *attn, const pi_attn_args *args);

/* Check of drafted tokens against the target's distribution by rejection sampling, so that the
 * tokens kept are distributed as the target's own. Node 0 is the last token already kept; node
 * i > 0 has parent parents[b][i] < i and token tokens[b][i]; logits[b][i] is the target's row
 * after node i. With p = softmax(logits[cur] / temperature) (all weight on the lowest index of
 * the largest logit where the temperature is not above 0), the children of the current node
 * are tried in index order, starting from r = p:
 *   with q:     child t is taken where u[b][i] * q[b][cur][t] < r[t]; else r becomes
 *               max(r - q[b][cur], 0), normalised
 *   without q:  child t is taken where u[b][i] < r[t]; else r[t] becomes 0 and r is normalised
 * until a node has no child that is taken. The next token is then drawn from r (from p where r
 * has no weight left) at u_next[b]: the first whose running sum is above u_next * the total.
 * An infinite temperature weighs all logits but -inf alike. NaN logits count as -inf, +inf as the
 * largest finite value; a row of nothing else but -inf gives the next token -1. Sums are in
 * 64 bits and in a fixed order.
 *   logits     [B][N][vocab], rows need no alignment beyond the element's
 *   q          fp32 [B][N][vocab] or NULL: the draft's probabilities after each node
 *   tokens, parents  device int32 [B][N]; a parent outside [0, i) keeps node i off every path
 *   u, u_next, temperature  device fp32 [B][N], [B], [B] (NULL: 1)
 *   nodes, out device int32 [B][N]: the path's nodes from node 0 on; their tokens without node
 *              0's, then the next token; both filled up with -1
 *   n          device int32 [B]: the path's length */
pi_status pi_verifier_create(pi_ctx *ctx, int32_t vocab, int32_t max_batch, int32_t max_nodes, pi_verifier **out);
void pi_verifier_destroy(pi_verifier *ver);

typedef struct pi_verify_args {
  const void *logits;
  int32_t dtype;
  int64_t logits_batch, logits_node;
  const float *q;
  int64_t q_batch, q_node;
  const int32_t *tokens, *parents;
  const float *u, *u_next, *temperature;
  int32_t *nodes, *out, *n;
  int32_t B, N;
} pi_verify_args;

pi_status pi_verify(pi_ctx *ctx, pi_verifier *ver, const pi_verify_args *args);

/* The residual's addition and RMS norm, with the norm in 8 bits, for T rows of d:
 *   res_out = round(x + res)            to res's type (x's, where res is NULL)
 *   y       = res_out / sqrt(mean(res_out^2) + eps) * w      in fp32
 *   scale   = max |y| / 127,  q = round(y / scale)           (0 and 0 for a row of zeros, NaN and 0
 *             for one with an infinity or a NaN)
 *   x, res, res_out  any pi_dtype (res_out has res's; it may be x or res itself, of its own type)
 *   w          fp32 [d]; d a multiple of 8 up to 32768
 *   q, scale   int8 [T][d] (rows 8-byte aligned) and fp32 [T], both or neither
 *   y          [T][d] of y_dtype, nullable
 * Strides are between rows. */
typedef struct pi_norm_args {
  const void *x, *res;
  void *res_out;
  int32_t x_dtype, res_dtype;
  int64_t x_stride, res_stride, res_out_stride;
  const float *w;
  float eps;
  int8_t *q;
  int64_t q_stride;
  float *scale;
  void *y;
  int32_t y_dtype;
  int64_t y_stride;
  int32_t T, d;
} pi_norm_args;

pi_status pi_add_rmsnorm(pi_ctx *ctx, const pi_norm_args *args);

/* A weight of N x K 8-bit integers with one scale per output channel.
 *   w          int8 [N][K], w_stride elements between rows (a multiple of 16 below 2^22); K a multiple of
 *              16 below 131072 (the sums are exact in 32 bits)
 *   w_scale    fp32 [N]; bias fp32 [N] or NULL
 *   max_tokens limit of M; above 1 the context's scratch for sums of ranges of K is allocated
 *              (once, of a size that serves every M, N and K) */
typedef struct pi_linear_desc {
  int32_t N, K;
  const int8_t *w;
  int64_t w_stride;
  const float *w_scale, *bias;
  int32_t max_tokens;
} pi_linear_desc;

pi_status pi_linear_create(pi_ctx *ctx, const pi_linear_desc *desc, pi_linear **out);
void pi_linear_destroy(pi_linear *lin);

/* y[m][n] = x_scale[m] * w_scale[n] * sum_k x[m][k] w[n][k] + bias[n] for M tokens, the sum in
 * whole numbers.
 *   x          int8 [M][K], x_stride a multiple of 16 below 2^22; x_scale fp32 [M]
 *   y          [M][N] of y_dtype; rows need no alignment beyond the element's */
pi_status pi_linear_q8(pi_ctx *ctx, pi_linear *lin, const int8_t *x, int64_t x_stride, const float *x_scale, int32_t M,
                       void *y, int32_t y_dtype, int64_t y_stride);

/* Causal attention of whole prompts, packed one after another, with grouped heads. Sequence b has the
 * queries cu_q[b]..cu_q[b+1] and the keys cu_k[b]..cu_k[b+1]; its queries are the last ones of its keys
 * (a prompt continued after tokens held before has more keys than queries). With n queries and m keys,
 *   out[i][h] = sum_j w_j v_j,  w = softmax over j <= i + m - n of scale * q[i][h] . k_j
 * with key/value head h * kv_heads / heads. A query that sees no key (m < n) gets zeros; what is not
 * seen does not enter the result, whatever it holds. Rows of no sequence stay as they are. The handle
 * keeps its own scratch: calls that share it, and the replays of graphs that hold them, are ordered.
 *   heads      a multiple of kv_heads;  head_dim a multiple of 8 up to 256
 *   dtype      PI_T_F16 or PI_T_BF16;  scale above 0, at most 2^127
 *   max_tokens, max_batch   limits of rows of q and of sequences */
typedef struct pi_prompt pi_prompt;

pi_status pi_prompt_create(pi_ctx *ctx, int32_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim,
                           int32_t max_tokens, int32_t max_batch, float scale, pi_prompt **out);
void pi_prompt_destroy(pi_prompt *prompt);

/*   q, out     [q_rows][heads][head_dim];  k, v [k_rows][kv_heads][head_dim]
 *   cu_q, cu_k device int32 [B+1], ascending, cu_k NULL: cu_q; offsets are taken into [0, q_rows] and
 *              [0, k_rows]
 *   k_row, v_row  below 2^24
 *   out may not share memory with q, k or v */
typedef struct pi_prompt_args {
  const void *q;
  int64_t q_row, q_head;
  const void *k;
  int64_t k_row, k_head;
  const void *v;
  int64_t v_row, v_head;
  void *out;
  int64_t out_row, out_head;
  const int32_t *cu_q, *cu_k;
  int32_t B, q_rows, k_rows;
} pi_prompt_args;

pi_status pi_prompt_attention(pi_ctx *ctx, pi_prompt *prompt, const pi_prompt_args *args);

/* RMS norm of every query and key head, and rotary positions, in one pass over T tokens:
 *   y = x / sqrt(mean(x^2) + eps) * w      per head of head_dim elements (y = x without w; zeros
 *                                          for a head of zeros where eps is 0)
 *   out = y with pair i of its first `rot` elements turned by the angle pos[t] * inv_freq[i]:
 *         (a, b) becomes (a cos - b sin, b cos + a sin)
 * Pair i is elements i and i + rot/2, or 2i and 2i + 1 where `interleaved`. Angles are formed and
 * reduced in 64 bits, everything else is in fp32, rounded once.
 *   q, k       [T][heads][head_dim] and [T][kv_heads][head_dim] of x_dtype; heads or kv_heads may be 0
 *              (q or k is not looked at); head_dim a multiple of 8 up to 512; T up to 2^23
 *   q_out, k_out  of y_dtype; each may be its input itself, of the same type and strides
 *   q_w, k_w   fp32 [head_dim], or NULL: no norm of these heads
 *   pos        device int32 [T];  inv_freq device fp32 [rot/2]
 *   rot        a multiple of 4 up to head_dim (of 8 where heads are above 256), or 0: no rotation (pos and
 *              inv_freq are not looked at) */
typedef struct pi_rope_args {
  const void *q, *k;
  int64_t q_row, q_head, k_row, k_head;
  void *q_out, *k_out;
  int64_t q_out_row, q_out_head, k_out_row, k_out_head;
  int32_t x_dtype, y_dtype;
  const float *q_w, *k_w;
  float eps;
  const int32_t *pos;
  const float *inv_freq;
  int32_t rot, interleaved;
  int32_t T, heads, kv_heads, head_dim;
} pi_rope_args;

pi_status pi_qk_norm_rope(pi_ctx *ctx, const pi_rope_args *args);

#ifdef __cplusplus
}
#endif

#endif /* PI_H */
