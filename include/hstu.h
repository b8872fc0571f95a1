/*
 * hstu.h — C ABI of libhstu.so: the forward pass of an HSTU layer stack over
 * jagged (unpadded) user sequences, and M-FALCON candidate ranking, on one
 * NVIDIA B200 (sm_100a).
 *
 * Source of the operations: the page 'HSTUとGenerative Recommenders――行動履歴から
 * 1.5兆parameterの推薦モデルへ' (koktn.github.io, an explainer of Zhai et al.,
 * "Actions Speak Louder than Words", ICML 2024):
 *   - section 'HSTUはTransformerと何が違うのか', subsections
 *     '1. U、V、Q、Kは同じ入力を見る4つの役割' (f1 + SiLU, split U,V,Q,K),
 *     '2. QKᵀで「どの履歴を見るか」を決める' (score = Q_i.K_j + position bias +
 *     time bias, causal, pointwise SiLU weights without softmax),
 *     '3. Uでcontextをgateし、次のlayerへ渡す' (LayerNorm(context) * U, f2,
 *     residual connection);
 *   - section '長い履歴を現実の計算量へ収める4つの工夫', subsections
 *     '1. 長さの異なるsequenceをpaddingせず処理する' (ragged batches without
 *     padding) and '4. M-FALCONで候補間の履歴計算を共有する' (candidates in
 *     microbatches appended after the history, mask and relative bias
 *     adjusted, history K/V cache shared across microbatches).
 *
 * Per user b (rows i, j of that user, n_b rows) one layer computes
 *   G = SiLU(X W1^T + b1) = [U | V | Q | K]   (head-major inside each part)
 *   s_ij = Q_i.K_j + rab_pos[h][pb(i-j)] + rab_time[h][tb(max(0, t_i - t_j))],  j <= i
 *   O_i  = (1/n_b) sum_{j<=i} SiLU(s_ij) V_j
 *   Y_i  = X_i + (LayerNorm(O_i) * U_i) W2^T + b2
 * where pb/tb are log-linear buckets: x < 2^S -> x; otherwise, with
 * e = floor(log2 x), (e-S+1)*2^S + (x >> (e-S)) - 2^S; clamped to N-1.
 * LayerNorm runs over all h*d_v features of a row (biased variance, eps from
 * the descriptor), then gamma, beta.
 *
 * Conventions for every entry point
 *   Ownership   The caller owns every buffer.  The library never allocates,
 *               frees or synchronises device memory, except that
 *               hstu_read_status synchronises the given stream.
 *   Execution   Asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *               default stream).  Returning HSTU_OK means the work was
 *               enqueued; device-detected errors are read with hstu_read_status.
 *   Layout      Row-major.  Activations [rows, d_model]; weights in [out, in]
 *               layout: W1 [F, d_model] with F = 2*h*d_v + 2*h*d_qk in the
 *               column order U, V, Q, K; W2 [d_model, h*d_v]; b1 [F]; b2
 *               [d_model]; ln_gamma, ln_beta [h*d_v]; rab_pos [h, n_pos_buckets]
 *               and rab_time [h, n_time_buckets] always fp32.  Element type of
 *               everything else is the descriptor's dtype (bf16 or fp32).
 *               Every device pointer must be 16-byte aligned.  Inputs and
 *               outputs must not alias each other or the workspace.
 *   Offsets     int64 [B+1], offsets[0] = 0, non-decreasing, offsets[B] =
 *               total rows; every length <= max_len.
 *   Timestamps  int64 seconds, one per row; within one user every timestamp
 *               must lie within 2^30 s of that user's first one.
 *   Errors      Host-detectable argument errors return at once and enqueue
 *               nothing.  Device-detected errors (bad offsets or timestamps,
 *               a wait that timed out) set a status word in the workspace; the
 *               remaining kernels of the call then exit early.  No entry
 *               point traps or asserts on the device.
 *   Precision   dtype HSTU_BF16 (inputs, weights, outputs bf16): the tensor
 *               cores take fp16 operands with fp32 accumulation.  bf16 values
 *               within [2^-14, 65504] in magnitude convert to fp16 exactly;
 *               the f1 output, P, Z and the residual stream between layers
 *               are stored in fp16 (saturating at +-65504), the attention
 *               output O and the LayerNorm statistics stay fp32 (M-FALCON's
 *               candidate rows also keep an fp32 residual), and only the final
 *               output is rounded to bf16.  fp16 keeps 3 more mantissa bits than
 *               bf16 at the same tensor-core rate; inputs, weights and layer
 *               outputs must lie within fp16 range (|x| <= 65504).  Weights
 *               below 2^-14 in magnitude become fp16 subnormals (absolute
 *               error up to 2^-25 each): against activations of order one
 *               they stay within the bf16 bound (tested: W2 drawn from
 *               N(0, 1e-5)); against activations in the thousands the error
 *               they add grows with the activations and can exceed it (Q and
 *               K rows of W1 near 1e-5 against activations of 8192 gave
 *               2.3e-2).  dtype HSTU_FP32: fp32 throughout (CUDA-core FMA).
 *   Supported   bf16: d_qk = d_v in {64, 128}; d_model and h*d_v multiples
 *               of 64; bucket counts in [1, 4096].  fp32: d_qk, d_v <= 128
 *               and multiples of 4; d_model multiple of 4.
 */
#ifndef HSTU_H_
#define HSTU_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  HSTU_OK = 0,
  HSTU_ERR_INVALID_ARG = 1,   /* host: null/misaligned pointer, bad size */
  HSTU_ERR_UNSUPPORTED = 2,   /* host: a shape or dtype the library does not run */
  HSTU_ERR_WORKSPACE = 3,     /* host: workspace smaller than hstu_workspace_size */
  HSTU_ERR_CUDA = 4,          /* host: a CUDA runtime call failed */
  HSTU_ERR_BAD_OFFSETS = 5,   /* device: offsets not monotone, wrong total, length > max */
  HSTU_ERR_TIMEOUT = 6,       /* device: an in-kernel wait gave up */
  HSTU_ERR_BAD_TIMESTAMPS = 7, /* device: a user's timestamps span 2^30 s or more */
  HSTU_ERR_BAD_IDS = 8         /* device: a token or row id outside its embedding table */
} hstu_status;

/* Layers are HSTU_BF16 or HSTU_FP32; the embedding and optimizer entry points
 * take all three. */
typedef enum { HSTU_BF16 = 0, HSTU_FP32 = 1, HSTU_FP16 = 2 } hstu_dtype;

/* Shape of one layer (all layers of a stack share it). */
typedef struct {
  int32_t d_model;         /* d */
  int32_t n_heads;         /* h */
  int32_t d_qk;            /* per-head query/key width */
  int32_t d_v;             /* per-head value/gate width */
  int32_t n_pos_buckets;   /* N_p: entries per head in rab_pos */
  int32_t n_time_buckets;  /* N_t: entries per head in rab_time */
  int32_t pos_sub_bits;    /* S_p of the position buckets, 0..20 */
  int32_t time_sub_bits;   /* S_t of the time-gap buckets, 0..20 */
  float ln_eps;            /* LayerNorm epsilon */
  int32_t dtype;           /* hstu_dtype of activations and dense weights */
} hstu_layer_desc;

/* Device pointers to one layer's parameters (layout above). */
typedef struct {
  const void* W1;
  const void* b1;
  const void* W2;
  const void* b2;
  const void* ln_gamma;
  const void* ln_beta;
  const float* rab_pos;
  const float* rab_time;
  /* Optional, bf16 layers only: fp16 copies of W1 and W2 (same layout),
   * e.g. made once with hstu_bf16_to_f16.  The tensor-core path multiplies
   * the fp16 residual stream and the fp16 gated Z by fp16 weights; when these
   * are null every call converts W1 (layers >= 1) and W2 into its workspace
   * first.  Must be 16-byte aligned when set; ignored for fp32 layers. */
  const void* W1_f16;
  const void* W2_f16;
} hstu_layer_weights;

/* Bytes of device workspace an entry point needs for these sizes.
 * For hstu_layer_fwd / hstu_stack_fwd pass total_cands = max_cands = 0 and
 * microbatch = 0.  Returns 0 if the arguments are invalid. */
size_t hstu_workspace_size(const hstu_layer_desc* desc, int32_t n_layers, int64_t B,
                           int64_t total_tokens, int64_t max_len, int64_t total_cands,
                           int64_t max_cands, int32_t microbatch);

/* One HSTU layer.  offsets: device int64 [B+1]; X: device [T, d]; weights:
 * host struct of device pointers; timestamps: device int64 [T]; out: device
 * [T, d] (must not alias X). */
hstu_status hstu_layer_fwd(const hstu_layer_desc* desc, int64_t B, int64_t total_tokens,
                           int64_t max_len, const int64_t* offsets, const void* X,
                           const hstu_layer_weights* weights, const int64_t* timestamps,
                           void* out, void* workspace, size_t workspace_bytes, void* stream);

/* n_layers layers, each layer's output the next one's input (section '3. U
 * でcontextをgateし、次のlayerへ渡す').  weights: host array [n_layers].  The
 * offsets are validated once and the tile schedule is shared by all layers. */
hstu_status hstu_stack_fwd(const hstu_layer_desc* desc, int32_t n_layers,
                           const hstu_layer_weights* weights, int64_t B, int64_t total_tokens,
                           int64_t max_len, const int64_t* offsets, const void* X,
                           const int64_t* timestamps, void* out, void* workspace,
                           size_t workspace_bytes, void* stream);

/* M-FALCON ranking (section '4. M-FALCONで候補間の履歴計算を共有する').
 * The histories run through n_layers layers once, keeping every layer's K/V;
 * then candidates, in microbatches of `microbatch` per user, run through the
 * layers attending to their user's whole history and to themselves only.
 * Every candidate sits at position n_b (distance n_b - j to history row j)
 * and at time request_ts[b] (NULL: the user's last history timestamp); its
 * normaliser is max(n_b, 1).  scores[c] = <y_c, head_vec> in fp32, where y_c
 * is candidate c's output of the last layer.
 * hist_offsets [B+1], history [T_hist, d], hist_timestamps [T_hist],
 * cand_offsets [B+1] (device), candidates [C, d], head_vec [d], scores fp32
 * [C].  Every user has at most max_cands candidates. */
hstu_status hstu_mfalcon_rank(const hstu_layer_desc* desc, int32_t n_layers,
                              const hstu_layer_weights* weights, int64_t B, int64_t total_hist,
                              int64_t max_len, const int64_t* hist_offsets, const void* history,
                              const int64_t* hist_timestamps, int64_t total_cands,
                              int64_t max_cands, const int64_t* cand_offsets,
                              const void* candidates, const int64_t* request_ts,
                              int32_t microbatch, const void* head_vec, float* scores,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of the fixed device scratch used by hstu_layer_fwd_noalloc. */
#define HSTU_NOALLOC_SCRATCH_BYTES (64u << 20)

/* hstu_layer_fwd without a workspace argument, for callers that cannot
 * allocate device memory (an allocator owned by another runtime, no
 * cudaMalloc allowed after start-up, a memory-capped sandbox).  It has no
 * counterpart on the pages: it is the same layer as hstu_layer_fwd, run in a
 * file-scope device array of HSTU_NOALLOC_SCRATCH_BYTES (64 MiB) that every
 * device loading this library holds until the process exits.  It allocates
 * nothing itself: no cudaMalloc, no cudaFree, no allocating library call.
 * The caller still passes the inputs and the output (as for hstu_layer_fwd).
 *   - Sizes whose workspace (hstu_workspace_size with n_layers = 1) exceeds
 *     HSTU_NOALLOC_SCRATCH_BYTES return HSTU_ERR_WORKSPACE and launch nothing;
 *     other argument errors are those of hstu_layer_fwd.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.  The address is kept for the life of the
 *     process: after a cudaDeviceReset (which releases the module's device
 *     memory) it is stale, so the function must not be called again in that
 *     process.
 *   - Every call shares the one array and leaves its contents behind; each
 *     call resets what must start at zero (the status word and counters).
 *     Calls whose execution overlaps on the GPU (other streams, other host
 *     threads) race on the array: serialise them.
 *   - The device status word lives in the array, so hstu_read_status cannot
 *     read it; check the output or use hstu_layer_fwd to diagnose. */
hstu_status hstu_layer_fwd_noalloc(const hstu_layer_desc* desc, int64_t B, int64_t total_tokens,
                                   int64_t max_len, const int64_t* offsets, const void* X,
                                   const hstu_layer_weights* weights, const int64_t* timestamps,
                                   void* out, void* stream);

/* Backward pass (gradients, for training) of hstu_layer_fwd / hstu_stack_fwd
 * ('HSTUとGenerative Recommenders', section 'HSTUはTransformerと何が違うのか': the
 * forward layer whose chain rule this is; section 'Production評価の12.4%をどう
 * 読むか': training is where the pages report the largest gain).  Given the
 * layers' input X and the gradient dY of a loss with respect to the stack's
 * output, computes dX (the gradient with respect to X) and, per layer, the
 * gradients of every parameter.  The call runs the stack's forward itself
 * first, keeping each layer's input, f1 output and pre-activation and
 * attention output in the workspace (about 2 T (d + 2F + h d_v) bytes per
 * layer), so nothing of an earlier forward call has to be kept.
 * Derivatives, per user (n = n_b) and head, written out by the chain rule:
 *   dZ = dY W2;  dW2 = dY^T Z;  db2 = sum_rows dY
 *   dL = dZ * U; dU = dZ * L (L = LayerNorm(O) before the gate); dgamma =
 *   sum_rows dL * xhat; dbeta = sum_rows dL; dO = (dxh - mean(dxh) - xhat
 *   mean(dxh xhat)) / sd with dxh = dL * gamma
 *   dA_ij = (1/n) dO_i . V_j; dV_j = (1/n) sum_i SiLU(s_ij) dO_i;
 *   dS_ij = dA_ij SiLU'(s_ij); dQ_i = sum_j dS_ij K_j; dK_j = sum_i dS_ij Q_i;
 *   drab_pos[h][b] / drab_time[h][b] = sum of dS_ij over the pairs (i, j) of
 *   bucket b
 *   dP = [dU | dV | dQ | dK] * SiLU'(P), P = X W1^T + b1;  dW1 = dP^T X;
 *   db1 = sum_rows dP;  dX = dY + dP W1.
 * dtype HSTU_BF16 only (HSTU_ERR_UNSUPPORTED otherwise), with the forward's
 * shape limits and n_time_buckets <= 256.  X and dY are bf16 [T, d] (device);
 * dX is bf16 [T, d]; every gradient is fp32, in its parameter's layout, and
 * is overwritten (not accumulated into).  The tensor cores take fp16
 * operands with fp32 accumulation (as in the forward; the gradients flowing
 * into them must lie within fp16 range); the gradient stream between layers
 * is fp32.  Every result is deterministic: the bias-table gradients are summed
 * in 64-bit fixed point (units of 2^-32, each partial sum clamped to
 * +-2^30), whose additions do not depend on their order, then rounded to fp32.
 * grads: host array [n_layers] of device pointers.  Workspace:
 * hstu_bwd_workspace_size() bytes, 256-byte aligned.  Asynchronous on
 * `stream`; device-detected errors (bad offsets or timestamps, a wait that
 * gave up) set the workspace's status word (hstu_read_status) and leave dX and
 * gradients unwritten or partly written (hstu_grad_norm_after tells an
 * optimizer step on the device). */
typedef struct {
  float* dW1;        /* [F, d_model] */
  float* db1;        /* [F] */
  float* dW2;        /* [d_model, h*d_v] */
  float* db2;        /* [d_model] */
  float* dln_gamma;  /* [h*d_v] */
  float* dln_beta;   /* [h*d_v] */
  float* drab_pos;   /* [h, n_pos_buckets] */
  float* drab_time;  /* [h, n_time_buckets] */
} hstu_layer_grads;
size_t hstu_bwd_workspace_size(const hstu_layer_desc* desc, int32_t n_layers, int64_t B,
                               int64_t total_tokens, int64_t max_len);
hstu_status hstu_layer_bwd(const hstu_layer_desc* desc, const hstu_layer_weights* weights,
                           int64_t B, int64_t total_tokens, int64_t max_len,
                           const int64_t* offsets, const void* X, const int64_t* timestamps,
                           const void* dY, void* dX, const hstu_layer_grads* grads,
                           void* workspace, size_t workspace_bytes, void* stream);
hstu_status hstu_stack_bwd(const hstu_layer_desc* desc, int32_t n_layers,
                           const hstu_layer_weights* weights, int64_t B, int64_t total_tokens,
                           int64_t max_len, const int64_t* offsets, const void* X,
                           const int64_t* timestamps, const void* dY, void* dX,
                           const hstu_layer_grads* grads, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Stochastic Length sampling and token embedding ('HSTUとGenerative
 * Recommenders', section '2. Stochastic Lengthで学習時の履歴を間引く': a long
 * history is shortened to a random subset of its positions; 4096 tokens keep
 * 776).  For each user b with a raw sequence of n_b tokens, keeps
 * k_b = min(n_b, floor(n_b^0.8)) (at least 1) positions: those whose keys are
 * smallest, the key of position p being output number b * 2^32 + p + 1 of the
 * SplitMix64 generator started from state `seed`, ties by position; the kept
 * tokens stay in their original order.  A kept token at an even original
 * position is a content item (row raw_ids[.] of content_table), at an odd
 * position an action (row of action_table).
 *   raw_offsets     device int64 [B+1], raw_offsets[0] = 0, [B] = raw_total,
 *                   each length at most max_raw_len (<= 32767)
 *   raw_ids         device int64 [raw_total] (row indices into the tables)
 *   raw_timestamps  device int64 [raw_total]
 *   content_table   device bf16 [n_content, d_model], 16-byte aligned
 *   action_table    device bf16 [n_action, d_model], 16-byte aligned
 *   out_offsets     device int64 [B+1]: the kept sequences' offsets
 *   out_X           device bf16 [sum k_b, d_model] (at most raw_total rows)
 *   out_timestamps  device int64 [sum k_b]
 *   workspace       hstu_sl_embed_workspace_size() bytes, 256-byte aligned
 *                   (holds the device status word)
 * d_model must be a multiple of 8.  Host-detectable errors return at once;
 * bad offsets or an id outside its table set the status word
 * (HSTU_ERR_BAD_OFFSETS: all out_offsets are 0; HSTU_ERR_BAD_IDS: that row is
 * zero), read back with hstu_read_status.  Asynchronous on `stream`. */
size_t hstu_sl_embed_workspace_size(void);
/* Full-catalog retrieval ('NetflixのGenRec解説――LLMを生成させず推薦rankerとして使う',
 * section '全体像：LLMは入力を読み、ranking headが作品を採点する'; the GenRec
 * explainer on techistory.net, s = E^T h): every one of n_items catalog
 * items is scored against every user vector, s[u, m] = <E_m, h_u>, in fp32
 * on the tensor cores, and the K highest scores per user are returned in
 * descending order, equal scores ordered by ascending item id.
 *   H             device bf16: the user vectors [n_users, d], or, when
 *                 user_offsets is given, the encoder output [total_rows, d]
 *                 whose row user_offsets[u+1]-1 is user u's vector (a user
 *                 without rows scores every item 0)
 *   user_offsets  device int64 [n_users+1] or null
 *   E             device bf16 [n_items, d] item embeddings
 *   out_scores    device fp32 [n_users, K]; out_ids device int64 [n_users, K]
 *   workspace     hstu_retrieval_workspace_size(...) bytes, 256-byte aligned
 *                 (from_rows = 1 when user_offsets will be given); it holds
 *                 the status word and the [n_users, n_items] score matrix
 * Requires d % 64 == 0, 1 <= K <= min(n_items, 1024), n_users <= 65535,
 * n_items < 2^31 - 256, H and E 16-byte aligned.  Offsets that are not
 * monotone or pass total_rows set HSTU_ERR_BAD_OFFSETS in the status word
 * (outputs then unspecified).  Asynchronous on `stream`. */
size_t hstu_retrieval_workspace_size(int64_t n_users, int64_t n_items, int32_t d, int32_t K,
                                     int32_t from_rows);
hstu_status hstu_retrieval_topk(int64_t n_users, int64_t n_items, int32_t d, const void* H,
                                const int64_t* user_offsets, int64_t total_rows, const void* E,
                                int32_t K, float* out_scores, int64_t* out_ids, void* workspace,
                                size_t workspace_bytes, void* stream);
/* Catalogs of 65,536 items or more are first scored on a 1-in-16 strided
 * sample to find a per-user score threshold, and the full pass keeps only
 * the items at or above it (the score matrix is never written); a user left
 * with fewer than K such items (or too many) makes the call fall back to
 * scoring and selecting over every item, with the same result.  After a call
 * (and a synchronisation of `stream`), *taken = 1 if that fallback ran. */
hstu_status hstu_retrieval_fallback_taken(const void* workspace, size_t workspace_bytes,
                                          int32_t* taken, void* stream);

/* Softmax-Transformer encoder layer: the comparator of the HSTU layer on the
 * same jagged batches ('HSTUとGenerative Recommenders', section 'Production評価の
 * 12.4%をどう読むか': HSTU against a FlashAttention-2 Transformer at 8,192
 * tokens, d = 512, 8 heads; attention as in the GenRec explainer on
 * techistory.net, softmax(QK^T / sqrt(d_k)) V).  Pre-LayerNorm, causal per
 * user:  A = LN1(X); [Q|K|V] = A W_qkv^T; ctx = per-head causal softmax
 * attention; X1 = X + ctx W_o^T; Y = X1 + SiLU(LN2(X1) W_1^T + b_1) W_2^T + b_2.
 * Dense weights are fp16 ([out, in] row-major: W_qkv [3d, d] with Q, K, V
 * row blocks, W_o [d, d], W_1 [d_ff, d], W_2 [d, d_ff]); LayerNorm gamma/beta
 * and the biases are bf16.  X and out are bf16 [T, d]; intermediates fp16.
 * Requires d % 256 == 0, d <= 1024, head dim d/h of 64 or 128, d_ff % 256 == 0;
 * every pointer 16-byte aligned.  Offsets are checked on the device
 * (HSTU_ERR_BAD_OFFSETS in the status word). */
typedef struct {
  const void* ln1_gamma;
  const void* ln1_beta;
  const void* W_qkv;
  const void* W_o;
  const void* ln2_gamma;
  const void* ln2_beta;
  const void* W_1;
  const void* b_1;
  const void* W_2;
  const void* b_2;
} hstu_transformer_weights;
size_t hstu_transformer_workspace_size(int32_t d_model, int32_t n_heads, int32_t d_ff, int64_t B,
                                       int64_t total_tokens);
hstu_status hstu_transformer_layer_fwd(int32_t d_model, int32_t n_heads, int32_t d_ff,
                                       float ln_eps, const hstu_transformer_weights* weights,
                                       int64_t B, int64_t total_tokens, int64_t max_len,
                                       const int64_t* offsets, const void* X, void* out,
                                       void* workspace, size_t workspace_bytes, void* stream);

/* Round-to-nearest conversion of n bf16 values to fp16 (device to device,
 * asynchronous on `stream`), for the optional W1_f16 / W2_f16 weight copies.
 * n must be a multiple of 8 and both pointers 16-byte aligned. */
hstu_status hstu_bf16_to_f16(const void* src, void* dst, int64_t n, void* stream);

/* The keep count k(n) = min(n, floor(n^0.8)) (at least 1 for n >= 1) that
 * hstu_sl_embed applies to a raw stream of n tokens, computed on the host
 * with the same integer definition (the largest k with k^5 <= n^4), so a
 * caller can size the kept batch (sum and max of k) without reading the
 * device.  Returns -1 for n < 0 or n > 32767. */
int64_t hstu_sl_keep_count(int64_t n);
hstu_status hstu_sl_embed(int64_t B, int64_t raw_total, int64_t max_raw_len,
                          const int64_t* raw_offsets, const int64_t* raw_ids,
                          const int64_t* raw_timestamps, uint64_t seed,
                          const void* content_table, int64_t n_content,
                          const void* action_table, int64_t n_action, int32_t d_model,
                          int64_t* out_offsets, void* out_X, int64_t* out_timestamps,
                          void* workspace, size_t workspace_bytes, void* stream);

/* hstu_sl_embed that also writes, for every kept token, the row it was copied
 * from: out_ids (device int64 [sum k_b], 16-byte aligned) holds a content
 * item's row of content_table, and n_content + the row of action_table for an
 * action, i.e. rows of the two tables taken as one table with the actions
 * behind the content (-1 for an id outside its table).  Those are the ids
 * that hstu_embed_bwd takes for the gradient of such a table. */
hstu_status hstu_sl_embed_ids(int64_t B, int64_t raw_total, int64_t max_raw_len,
                              const int64_t* raw_offsets, const int64_t* raw_ids,
                              const int64_t* raw_timestamps, uint64_t seed,
                              const void* content_table, int64_t n_content,
                              const void* action_table, int64_t n_action, int32_t d_model,
                              int64_t* out_offsets, void* out_X, int64_t* out_timestamps,
                              int64_t* out_ids, void* workspace, size_t workspace_bytes,
                              void* stream);

/* Embedding lookup with scaling: out[t, :] = scale * table[ids[t], :], the
 * product in fp32 and rounded once to out_dtype.
 *   ids     device int64 [n_tokens]; a token whose id is pad_id gets a zero
 *           row.  pad_id may be a row of the table or any number outside it
 *           (the binding's default is -1: hstu_sl_embed_ids's mark of a bad id)
 *   table   device [n_rows, d] of table_dtype, ld_table elements apart
 *   out     device [n_tokens, d] of out_dtype, ld_out elements apart; the gap
 *           behind each row is left as it was
 * Any d up to 2^20 and any strides up to 2^31; rows are moved 16 bytes at a time where d
 * and both strides are multiples of 8, else element by element.  n_tokens and
 * n_rows below 2^31 - 8192.  An id outside the table that is not pad_id gets a
 * zero row and sets HSTU_ERR_BAD_IDS in the workspace's status word
 * (hstu_embed_workspace_size() bytes, 256-byte aligned).  Asynchronous on
 * `stream`. */
size_t hstu_embed_workspace_size(void);
hstu_status hstu_embed_fwd(int64_t n_tokens, const int64_t* ids, const void* table,
                           int32_t table_dtype, int64_t n_rows, int32_t d, int64_t ld_table,
                           int64_t pad_id, float scale, void* out, int32_t out_dtype,
                           int64_t ld_out, void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of the lookup: row r of the table's gradient is scale * the sum of
 * dY[t, :] over the tokens with ids[t] = r, summed in fp32 and rounded once.
 * The tokens are sorted by (id, t) first, so every sum has one order and the
 * result is the same bit for bit on every run.  Tokens of pad_id and of ids
 * outside the table take no part (the latter set HSTU_ERR_BAD_IDS).
 * hstu_embed_bwd writes the whole gradient dE [n_rows, d] (rows without
 * tokens become zero), or with accumulate = 1 adds into it (rows without
 * tokens are not touched).  hstu_embed_bwd_rows writes the touched rows only:
 *   n_unique  device int64 [1]: their number U
 *   row_ids   device int64 [min(n_tokens, n_rows)]: the first U entries are
 *             the touched rows, ascending
 *   rows      device [min(n_tokens, n_rows), d] of rows_dtype, ld_rows
 *             elements apart: the first U rows are their gradients
 * What lies behind the first U entries and rows is left as it was.  This is
 * the form that hstu_adamw_step and hstu_grad_norm take.  Workspace:
 * hstu_embed_bwd_workspace_size() bytes (0 if the arguments are invalid),
 * 256-byte aligned; limits and strides as for hstu_embed_fwd. */
size_t hstu_embed_bwd_workspace_size(int64_t n_tokens, int64_t n_rows, int32_t d);
hstu_status hstu_embed_bwd(int64_t n_tokens, const int64_t* ids, const void* dY, int32_t dy_dtype,
                           int64_t ld_dy, int64_t n_rows, int32_t d, int64_t pad_id, float scale,
                           int32_t accumulate, void* dE, int32_t de_dtype, int64_t ld_de,
                           void* workspace, size_t workspace_bytes, void* stream);
hstu_status hstu_embed_bwd_rows(int64_t n_tokens, const int64_t* ids, const void* dY,
                                int32_t dy_dtype, int64_t ld_dy, int64_t n_rows, int32_t d,
                                int64_t pad_id, float scale, int64_t* row_ids, void* rows,
                                int32_t rows_dtype, int64_t ld_rows, int64_t* n_unique,
                                void* workspace, size_t workspace_bytes, void* stream);

/* One tensor of an optimizer step (all pointers but the struct itself are
 * device pointers, 16-byte aligned except where noted).  Dense: row_ids and
 * n_rows null; `grad`, `param` and the states hold n elements.  Row-sparse (an
 * embedding table with the gradient of hstu_embed_bwd_rows): the parameter and
 * its states are [n / row_len, row_len], contiguous; `grad` holds up to
 * max_rows rows, of which the first *n_rows belong to the table rows
 * row_ids[0 .. *n_rows), strictly ascending; row_ids is not null even if
 * max_rows is 0.  Rows without a gradient, their states and the weight decay
 * on them are not touched. */
#define HSTU_STATE_BLOCK 256  /* elements that share a scale in 8-bit states */
#define HSTU_MAX_TENSORS 4096
typedef struct {
  int64_t n;               /* elements of the parameter */
  int64_t row_len;         /* row-sparse only: elements of a row */
  int64_t max_rows;        /* row-sparse only: rows allocated in grad and row_ids */
  const int64_t* row_ids;  /* row-sparse only */
  const int64_t* n_rows;   /* row-sparse only: number of rows in use (8-byte aligned) */
  const void* grad;        /* of grad_dtype */
  void* param;             /* of param_dtype, updated */
  float* master;           /* optional fp32 copy of a 16-bit param: read and updated in its
                            * place; param then receives the rounded result.  Without one a
                            * 16-bit param is rounded to nearest after every step, and what is
                            * less than half a step of its type is lost: in bf16 a change below
                            * |p| / 512 to |p| / 256, so weight decay as a rule, and updates of
                            * the size of lr where |p| > 512 lr */
  void* copy_f16;          /* optional: receives the new (rounded) param as fp16, saturating at
                            * +-65504, as hstu_bf16_to_f16 does (W1_f16, W2_f16) */
  void* m;                 /* first moment: fp32, or e4m3 codes */
  void* v;                 /* second moment: fp32; 8-bit: e4m3 codes of its square root */
  uint8_t* m_scale;        /* 8-bit states: one byte per block of 256 elements (any alignment) */
  uint8_t* v_scale;
  double weight_decay;
  int32_t grad_dtype;      /* hstu_dtype */
  int32_t param_dtype;     /* hstu_dtype */
  int32_t state_bits;      /* 32 or 8 */
} hstu_adamw_tensor;

/* Global gradient norm over a list of tensors, one reading of every gradient:
 * out[0] = sqrt(sum of all squares) (squares and sums in fp64) and out[1] =
 * the factor that clips it, min(1, max_norm / norm), or NaN when the norm is
 * not finite; out: device fp32 [2], 16-byte aligned.  Only the gradient's
 * fields of each tensor are read (n, grad, grad_dtype, and for a row-sparse
 * one row_len, max_rows, n_rows; a row count outside [0, max_rows] is cut to
 * it).  max_norm > 0 (infinity: never clips).  At
 * most HSTU_MAX_TENSORS tensors (host array).  Deterministic on one device. */
size_t hstu_grad_norm_workspace_size(void);
hstu_status hstu_grad_norm(const hstu_adamw_tensor* tensors, int32_t n_tensors, double max_norm,
                           float* out, void* workspace, size_t workspace_bytes, void* stream);
/* hstu_grad_norm of gradients that an earlier call on the stream made:
 * `after` is that call's workspace (hstu_layer_bwd, hstu_stack_bwd; null: as
 * hstu_grad_norm).  If its status word is not HSTU_OK, the gradients were not
 * (all) written, and out[0] and out[1] are NaN, so that an AdamW step with
 * out[1] as its grad_scale changes nothing. */
hstu_status hstu_grad_norm_after(const hstu_adamw_tensor* tensors, int32_t n_tensors,
                                 double max_norm, const void* after, float* out, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* One AdamW step (decoupled weight decay) of a list of tensors.  With
 * g = grad_scale * grad and t = step, per element
 *   m = beta1 m + (1 - beta1) g;   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * in fp32 (the constants from doubles); p is the master where there is one.
 * 8-bit states: m and r = sqrt(v) are held as e4m3 codes (4 exponent and 3
 * significand bits) times a power of two per block of 256 consecutive
 * elements (of one row, in a row-sparse tensor, which then has
 * ceil(row_len / 256) blocks per row): scale byte s stands for 2^(s - 127),
 * chosen so that the block's largest finite magnitude lies in [2^7, 2^8).
 * The update uses the unrounded moments; what is stored is rounded up or down
 * to a neighbouring code at random, with the probability that makes the mean
 * (of m and of r) right, because v moves by 1 - beta2 of itself per step, far
 * less than half a code, and would stand still under rounding to nearest.  The random number
 * is a function of (seed, step, position of the tensor in the list, element)
 * alone.  Moments that are not finite are stored as NaN.  Buffers of zeros are
 * valid initial states in either form.
 *   grad_scale  optional device fp32: e.g. out[1] of hstu_grad_norm.  If it is
 *               not finite the step changes nothing.
 *   step_dev    optional device int64, read instead of `step` (for a step
 *               captured into a graph; advance it between replays); a value
 *               below 1 sets HSTU_ERR_INVALID_ARG and changes nothing
 *   lr_dev      optional device fp32, read instead of `lr`
 * Row ids out of range or not ascending, and a row count above max_rows or
 * below 0, set HSTU_ERR_BAD_IDS; such rows are skipped (rows given twice
 * without being adjacent have an unspecified result).  No two tensors may
 * share memory.  Workspace: hstu_adamw_workspace_size() bytes, 256-byte
 * aligned (the status word).  Asynchronous on `stream`. */
typedef struct {
  double lr;
  double beta1;            /* [0, 1) */
  double beta2;            /* [0, 1) */
  double eps;              /* >= 2^-126 */
  int64_t step;            /* >= 1 */
  const int64_t* step_dev;
  const float* lr_dev;
  const float* grad_scale;
  uint64_t seed;           /* of the 8-bit states' rounding */
} hstu_adamw_args;
size_t hstu_adamw_workspace_size(void);
hstu_status hstu_adamw_step(const hstu_adamw_args* args, const hstu_adamw_tensor* tensors,
                            int32_t n_tensors, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Synchronises `stream`, then returns the device status word that the last
 * call using this workspace left (HSTU_OK if none of its checks failed). */
hstu_status hstu_read_status(const void* workspace, size_t workspace_bytes, void* stream);

/* Test hook: byte offsets inside the workspace where hstu_layer_fwd (and the
 * last layer of hstu_stack_fwd) leaves its intermediates: the f1 output
 * [T, F] (U|V|Q|K after SiLU), the pre-LayerNorm attention output O [T, h*d_v]
 * (already scaled by 1/n_b) and the gated Z [T, h*d_v].
 * dtype HSTU_FP32: O and Z are fp32.  dtype HSTU_BF16: the f1 output is fp16;
 * O is stored per (row, head) as its mean m and standard deviation s over
 * the head's d_v values and the normalised values (O - m) / s: the fp16
 * values [T, h*d_v] at o_offset, then, at the next multiple of 256 bytes,
 * the (m, s) pairs as fp32 [T, h, 2]; Z (fp16) is formed inside the output
 * projection and written at z_offset only while hstu_debug_keep_z(1) is in
 * effect. */
hstu_status hstu_debug_offsets(const hstu_layer_desc* desc, int64_t B, int64_t total_tokens,
                               int64_t max_len, size_t* f1_offset, size_t* o_offset,
                               size_t* z_offset);

/* Tracing.  hstu_trace_enable(n) records a CUDA event pair around each of
 * the next n kernel launches (n = 0 turns tracing off); hstu_trace_only(id)
 * restricts the recording to launches of one kernel id (-1, the default:
 * every kernel; HSTU_ERR_INVALID_ARG for an unknown id); hstu_trace_read
 * synchronises and returns, per traced launch, the kernel id and the device
 * time in ms.  hstu_kernel_name maps an id to a name.  hstu_launch_count
 * counts every kernel this library has launched in this process. */
hstu_status hstu_trace_enable(int32_t max_records);
hstu_status hstu_trace_only(int32_t kernel_id);
int32_t hstu_trace_read(int32_t* kernel_ids, float* ms, int32_t capacity);
const char* hstu_kernel_name(int32_t kernel_id);
int64_t hstu_launch_count(void);

/* Test hook: with on = 1, later layer calls on the tensor-core path also
 * write the gated Z = LayerNorm(O) * U into the workspace (at the z offset
 * of hstu_debug_offsets) when the output projection forms it in its shared
 * memory (see the "ln_fusion" option); with on = 0 (the default) Z is in the
 * workspace only when the separate LayerNorm * U kernel formed it.
 * Process-wide.  Returns HSTU_ERR_INVALID_ARG for other values. */
hstu_status hstu_debug_keep_z(int32_t on);

/* Test hook for the failure detection of the in-kernel waits.  Every wait
 * inside the attention kernel is bounded: after wait_limit_us microseconds
 * (default 1 s) it gives up, the call's status word becomes HSTU_ERR_TIMEOUT,
 * and the kernel winds down (loads in flight land, tensor memory is freed)
 * and returns, so the context stays usable and the next call on the same
 * workspace runs normally.  hstu_debug_wait_test sets, for the NEXT attention
 * launch only (of any call, on any stream), the wait bound (0 = the default)
 * and, with inject_stall = 1, makes that launch's first CTA stop handing out
 * work after two items without telling its other roles, which then wait
 * until the bound runs out.  It touches no memory and issues no load; the
 * launch after that one uses the defaults again.  Not a page operation: the
 * pages describe no failure handling.  Returns HSTU_ERR_INVALID_ARG for an
 * inject_stall other than 0 or 1. */
hstu_status hstu_debug_wait_test(uint32_t wait_limit_us, int32_t inject_stall);

/* Process-wide options.  "ln_fusion": 1 forms LayerNorm(O) * U inside the
 * output projection's operand stage (Z never reaches memory), 0 writes Z with
 * a separate kernel that f2 then reads, 2 (default) chooses per layer: inside
 * f2 when d_model <= 512 (f2 then has at most two 256-column output tiles,
 * each of which forms Z again), the separate kernel otherwise.  All give the
 * same layer within the bf16 bound.  "gemm_pair": where a projection (f1 with
 * SiLU, f2 with its 16-bit residual, a plain-bias product) takes 256-column
 * output tiles, 1 (default) runs it on clusters of two CTAs sharing each
 * 256 x 256 tile through the pair MMA when its inner dimension is at least
 * 1024, 2 does so at any inner dimension, 0 never; all give bitwise the same
 * result.  Returns HSTU_ERR_INVALID_ARG for
 * an unknown name or value. */
hstu_status hstu_set_option(const char* name, int64_t value);

/* After an entry point returned HSTU_ERR_CUDA: the failing CUDA runtime
 * call's error and the step it belonged to, as text (per host thread; ""
 * if none). */
const char* hstu_last_error(void);

const char* hstu_status_string(hstu_status s);
int32_t hstu_version(void);

#ifdef __cplusplus
}
#endif

#endif /* HSTU_H_ */
