/*
 * gptlayer_parts.h — the building blocks of the layer step, exported one by
 * one so that each kernel can be checked on its own.  Same conventions as
 * gptlayer.h: caller-owned 16-byte-aligned device pointers, asynchronous on
 * `stream`, 0 or a negative GPTL_E_* code, validation before any launch.
 */
#ifndef GPTLAYER_PARTS_H
#define GPTLAYER_PARTS_H

#include "gptlayer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One operand of gptl_gemm, seen through a 3-D view of a 16-bit tensor:
 * element (x, row, g) lives at ptr + g*g_pitch + row*row_pitch + x
 * (pitches in elements, multiples of 8).
 *   mn_major = 0: `row` indexes M (operand A) or N (operand B) and `x` the
 *                 reduction index k  ("K-major");
 *   mn_major = 1: `row` is k and `x` is the M/N index ("MN-major": the
 *                 tensor core reads it transposed, no copy is made).
 * For group G and k-shard ks the operand's x offset is
 *   (G % x_mod) * x_mul + x_off   and its g coordinate is
 *   G / g_div + (k_shard ? ks : 0).
 * Reads outside the view's extents return zeros. */
typedef struct {
  const void *ptr;
  long long x_ext, rows_ext, g_ext;
  long long row_pitch, g_pitch;
  int mn_major;
  int x_mod, x_mul, x_off;
  int g_div;
  int k_shard;
} gptl_operand;

enum {
  GPTL_ACT_NONE = 0,
  GPTL_ACT_GELU = 1,     /* out = value, out2 = GeLU(value)                   */
  GPTL_ACT_DGELU = 2     /* out = value * GeLU'(aux); out2 (optional) = GeLU(aux) */
};

/* out[G](m, n) = epilogue( sum over ks < k_shards, k < K of A(m,k) * B(n,k) )
 * for m < M, n < N, G < groups, with fp32 accumulation in tensor memory.
 * Output element (m, n) of group G is at
 *   out + (G % o_mod)*o_str_mod + (G / o_mod)*o_str_div + m*ldo + n.
 * Epilogue, in order: + bias[G*bias_g_stride + n] (if bias, 16-bit),
 * + resid[m*ld_resid + n] (if resid; fp32 when resid_f32, else 16-bit), then
 * act: GELU writes the value to out and GeLU(value) to out2; DGELU multiplies
 * by GeLU'(aux at the output's index) and, if out2 is not NULL, also writes
 * GeLU(aux) to out2 (the activation recomputed from its stored argument; with
 * the GELU epilogue's rounding, bit-identical to what GELU wrote for the same
 * 16-bit argument).  out_f32 = 1 stores the fp32 value
 * (act must be GPTL_ACT_NONE); otherwise out is 16-bit, rounded to nearest
 * even.  resid and DGELU do not combine.  Requirements: K % 16 == 0,
 * N % 16 == 0, all offsets/pitches multiples of 8 elements, out (and out2,
 * ws) 16-byte aligned.  The outputs are written by tensor stores of whole
 * 32-row boxes clipped to M x N: nothing outside the M x N window of each
 * group is written, but the groups' windows must not overlap.  causal is
 * reserved and must be 0.
 * Split-K: when out_f32 is set with no bias, resid or act, and ws (16-byte
 * aligned device memory of ws_bytes) is given, the library may cut the K
 * loop of each output tile into slices computed by different SMs; each slice
 * writes fp32 partial sums to ws and a second kernel adds them in slice
 * order (the result is deterministic).  It does so only when the output has
 * too few tiles to fill the GPU and the partials fit in ws_bytes.  ws may be
 * NULL (no split).
 * Column sums: when colsum is not NULL (16-byte aligned fp32 device memory of
 * ceil(M/32) * groups * N floats), the epilogue also writes, for every group
 * G, column n and r < ceil(M/32),
 *   colsum[(r*groups + G)*N + n] = sum over m in [32r, min(32r+32, M)) of
 *                                  out[G](m, n) as stored (16-bit),
 * each added in a fixed order; the caller adds the ceil(M/32) partial rows
 * (a bias gradient).  It needs a 16-bit output (out_f32 = 0) and act other
 * than GELU, and it rules out split-K. */
typedef struct {
  int M, N, K, groups, k_shards, causal;
  gptl_operand a, b;
  void *out;
  int out_f32;
  long long ldo;
  int o_mod;
  long long o_str_mod, o_str_div;
  const void *bias;
  long long bias_g_stride;
  const void *resid;
  long long ld_resid;
  const void *aux;
  void *out2;
  int act;
  int resid_f32;
  void *ws;
  long long ws_bytes;
  float *colsum;
} gptl_gemm_desc;

int gptl_gemm(const gptl_gemm_desc *d, gptl_dtype dtype, gptl_stream_t stream);

/* How gptl_gemm would run *d on the current device (no device work, same
 * argument checks and error codes as gptl_gemm): the tile width bn, the
 * split-K slice count (1 = none) and the use of each SM's two MMA pipelines:
 *   GPTL_GEMM_ALTERNATE  128 x bn tiles alternate between the pipelines;
 *   GPTL_GEMM_K_HALVES   both pipelines on each 128 x bn tile, one half of its
 *                        K range each, summed in a fixed order;
 *   GPTL_GEMM_M256       256 x bn tiles, one 128-row half per pipeline.
 * Results do not depend on the choice beyond fp32 summation order, and are
 * deterministic for a given choice. */
enum { GPTL_GEMM_ALTERNATE = 0, GPTL_GEMM_K_HALVES = 1, GPTL_GEMM_M256 = 2 };
int gptl_gemm_plan(const gptl_gemm_desc *d, gptl_dtype dtype, int *bn, int *split, int *mode);

/* Fused causal attention forward ("Training GPT-2 with Megatron-LM" §6.2
 * fused softmax; scores never leave the chip).  qkv: [tp][batch*seq][3h/tp],
 * shard i's columns [Q_i | K_i | V_i], each head_dim = hidden/heads columns
 * per head.  For every shard, batch element and head:
 *   O = softmax_{q <= p}(Q K^T / sqrt(head_dim)) V   -> o [tp][batch*seq][h/tp]
 *   lse[g][p] = log2 sum_{q <= p} exp2(Q_p.K_q log2(e)/sqrt(head_dim))
 * with g = (shard*batch + batch index)*(heads/tp) + head, lse [g][seq] fp32.
 * head_dim % 16 == 0 and <= 128, seq % 16 == 0. */
int gptl_attention_fwd(int batch, int seq, int hidden, int heads, int tp, gptl_dtype dtype,
                       const void *qkv, void *o, float *lse, gptl_stream_t stream);

/* Fused causal attention backward, the counterpart of gptl_attention_fwd.
 * Given qkv, o and lse of the forward and dout ([tp][batch*seq][h/tp], the
 * gradient with respect to o), writes dQ, dK and dV into the Q, K and V
 * columns of dqkv (same layout as qkv); dvec ([g][seq] fp32, caller scratch)
 * receives D = dO . O per row.  With P = softmax(Q K^T / sqrt(d)) (causal):
 *   dV = P^T dO,  dS = P (dO V^T - D) / sqrt(d),  dQ = dS K,  dK = dS^T Q,
 * P taken in the 16-bit type.  Same size limits as gptl_attention_fwd.
 * dbias (optional, with dbias_part): the QKV bias gradient, [tp][3h/tp] fp32,
 * the column sums of each shard's dqkv over its batch*seq rows, of the values
 * as stored; the kernels that write dQ, dK and dV sum every 32 rows into
 * dbias_part (caller scratch of batch * ceil(seq/32) * 3 * hidden floats) and
 * a second pass adds those in a fixed order.  Both NULL: no bias gradient;
 * only one NULL: GPTL_E_NULL. */
int gptl_attention_bwd(int batch, int seq, int hidden, int heads, int tp, gptl_dtype dtype,
                       const void *qkv, const void *o, const void *dout, const float *lse,
                       float *dvec, void *dqkv, float *dbias_part, float *dbias,
                       gptl_stream_t stream);

/* LayerNorm forward over `rows` rows of width h: y = g*(x-mu)*rstd + b with the
 * biased variance; mu and rstd ([rows] fp32) are saved for the backward.
 * h must split as h/8 = TPR*VPT with TPR a power of two in [16, 256], VPT <= 8. */
int gptl_layernorm_fwd(int rows, int h, gptl_dtype dtype, const void *x, const void *g,
                       const void *b, float eps, void *y, float *mu, float *rstd,
                       gptl_stream_t stream);

/* Scratch bytes gptl_layernorm_bwd needs. */
size_t gptl_layernorm_bwd_scratch_bytes(int rows, int h);

/* LayerNorm backward: dx = resid + LNbwd(gy); dg = sum_rows gy*xhat,
 * db = sum_rows gy (fp32, overwritten); dx_sum (optional, may be NULL) =
 * sum_rows dx.  resid may alias nothing that is written. */
int gptl_layernorm_bwd(int rows, int h, gptl_dtype dtype, const void *gy, const void *x,
                       const float *mu, const float *rstd, const void *g, const void *resid,
                       void *dx, float *dg, float *db, float *dx_sum, void *scratch,
                       gptl_stream_t stream);

/* Scratch bytes gptl_colsum needs. */
size_t gptl_colsum_scratch_bytes(int n, int groups);

/* out[G*n + c] = sum over r < rows of a[G*gstride + r*ld + c] (fp32). */
int gptl_colsum(int rows, int n, int groups, long long ld, long long gstride, gptl_dtype dtype,
                const void *a, float *out, void *scratch, gptl_stream_t stream);

/* The same column sums as gptl_colsum, for callers that cannot hand the
 * library any temporary device memory.  A plug-in or custom operator inside a
 * host framework that owns and pre-plans every device allocation may not call
 * cudaMalloc (nor ask the framework for memory) in the middle of its work, and
 * some deployments forbid device allocation after start-up altogether.  This
 * entry point allocates nothing: its partial sums live in one fixed array of
 * 64 * 16384 floats (4 MiB) in the library's device memory, which every GPU
 * that loads the library holds until the process exits.  (The Megatron-LM
 * pages have no counterpart to this; it is a property of this library.)
 *   - n * groups must be at most 16384, else GPTL_E_TOO_LARGE and nothing is
 *     launched; the other arguments and results are those of gptl_colsum,
 *     summed in the same order.
 *   - The first call on each device looks up the array's device address (with
 *     that device current); make that first call before any stream capture.
 *     The address is kept with the id of the CUDA context it came from: after
 *     a device reset the next call (again outside any capture) looks it up
 *     anew.  Host threads may call concurrently; a mutex guards the lookup.
 *   - All calls share the one array: calls whose kernels may overlap on the
 *     GPU (different streams, or different host threads, on one device) race
 *     and give wrong sums.  Calls in order on one stream are safe.  The array
 *     keeps the last call's partial sums; each call writes every partial it
 *     reads before reading it, so nothing needs clearing in between. */
int gptl_colsum_noalloc(int rows, int n, int groups, long long ld, long long gstride,
                        gptl_dtype dtype, const void *a, float *out, gptl_stream_t stream);

/* ------------------------------------------------------------------------
 * Norm and rotation of queries and keys, between the QKV product and
 * attention.  (The Megatron-LM pages give the layer no positions; these
 * calls, dropout and the token log probabilities below have no counterpart
 * there.)
 *
 * A packed row holds q_heads query heads, then k_heads key heads, then
 * v_heads value heads, head_dim elements each: the [Q_i | K_i | V_i] rows that
 * gptl_attention_fwd reads, with groups = tp.  For every query and key head x
 * of every token:
 *   n = x * g / sqrt(mean(x^2) + eps)       g = gq for queries, gk for keys
 *                                           (n = x when both are NULL)
 *   for each pair j < rot_dim/2 of elements (a, b) of n's first rot_dim:
 *     phi = 2 pi * pos[axis_j][token] * turns_j
 *     y_a = n_a cos(phi) - n_b sin(phi),   y_b = n_b cos(phi) + n_a sin(phi)
 *   the other elements of y are those of n.
 * Statistics and rotation are fp32, the angle's turns are reduced in fixed point
 * (exact to fp32 for every int position where turns < 1/4, as of every base >= 1),
 * and y is rounded once.  (A bf16 head whose squares leave fp32, beyond
 * 1e18, comes out as 0, and so do its gradients where their products stay in fp32.)
 * interleaved = 0 pairs elements (j, j + rot_dim/2), 1 pairs (2j, 2j + 1). */
typedef struct {
  int tokens, groups;              /* rows of a group, groups (tp shards);    */
                                   /* tokens * groups < 2^30                  */
  int q_heads, k_heads, v_heads;   /* of one group; v_heads may be 0; their   */
                                   /* sum times groups at most 2^20           */
  int head_dim;                    /* multiple of 16, at most 256             */
  int rot_dim;                     /* multiple of 16, 0 .. head_dim           */
  int interleaved;                 /* 0 or 1                                  */
  int axes;                        /* position axes, 1 .. 4                   */
  int seq;                         /* pos NULL: every axis is token % seq     */
  float eps;                       /* > 0 when there are gains                */
  /* element (group, token, c) of x is at x + group*x_gstride + token*x_ld + c,
   * of y at y + group*y_gstride + token*y_ld + c: multiples of 8, 0 for dense
   * (ld = row width, gstride = tokens*ld); each below 2^40, and tokens*ld and
   * groups*gstride below 2^56 */
  long long x_ld, x_gstride, y_ld, y_gstride;
} gptl_qk_desc;

/* One rotated pair: its turns (radians / 2 pi) for one step of its axis, and
 * the axis.  A program lays a table of rot_dim/2 of them out once, in DEVICE
 * memory, 16-byte aligned. */
typedef struct {
  double turns;
  int axis;
  int reserved;                    /* 0 */
} gptl_rope_pair;

/* Fills the host array table[rot_dim/2] for rotary positions with `base`:
 * axis a takes the next axis_pairs[a] pairs (their sum is rot_dim/2; NULL with
 * axes = 1).  per_axis = 0: turns_j = base^(-2j/rot_dim) / 2 pi over the whole
 * table, as for text with (time, height, width) positions; 1: each axis has a
 * ladder of its own, base^(-i/axis_pairs[a]) / 2 pi for its i-th pair, as for
 * the rows and columns of an image.  No device work.  GPTL_E_SHAPE for sizes
 * that do not fit, GPTL_E_ARG unless base > 0 is finite. */
int gptl_rope_table(int rot_dim, int axes, const int *axis_pairs, int per_axis, double base,
                    gptl_rope_pair *table);

/* Forward: x -> y.  y is x itself (same strides: in place; V columns are left
 * alone) or does not overlap it (V columns are copied, so that y is the whole
 * buffer that attention reads; training keeps x for the backward).  Columns
 * between the row width and ld are not touched; y may lie in those of x, or x
 * in those of y, where the two have the same strides (with other strides the
 * whole ranges, first to last element, have to be apart).
 * gq, gk: [head_dim] (cdt), both or neither.  pos: int32 [axes][tokens] or
 * NULL.  table: [rot_dim/2], may be NULL when rot_dim is 0; an axis outside
 * [0, axes) sets bit 2 of the device error word and counts as axis 0.
 * GPTL_E_SHAPE for sizes or strides outside the limits above, rows that
 * overlap or seq < 1 without pos; GPTL_E_ARG for eps, interleaved or an overlap
 * of x and y. */
int gptl_qk_norm_rope_fwd(const gptl_qk_desc *d, gptl_dtype dtype, const void *x, void *y,
                          const void *gq, const void *gk, const int *pos,
                          const gptl_rope_pair *table, gptl_stream_t stream);

/* Scratch bytes gptl_qk_norm_rope_bwd needs when there are gains (0 for a
 * descriptor outside the limits). */
size_t gptl_qk_norm_rope_scratch_bytes(const gptl_qk_desc *d);

/* Backward: dx from the forward's x (x strides) and dy, the gradient of y.  dy
 * and dx have the y strides; dx is dy itself (V columns are left alone) or
 * overlaps neither dy nor x, in the sense above (V columns are copied).  dgq, dgk: fp32
 * [head_dim], overwritten with the sums over all tokens, groups and heads, in
 * a fixed order; given exactly when gq and gk are, and scratch with them.
 * Without gains the kernel does not read x, which has to be a valid address all
 * the same (after a forward in place, that of y will do).  Calls that share
 * scratch, those of two captured graphs among them, must be ordered on the
 * device: each writes all the sums that it reads. */
int gptl_qk_norm_rope_bwd(const gptl_qk_desc *d, gptl_dtype dtype, const void *x, const void *dy,
                          void *dx, const void *gq, const void *gk, const int *pos,
                          const gptl_rope_pair *table, float *dgq, float *dgk, void *scratch,
                          gptl_stream_t stream);

/* ------------------------------------------------------------------------
 * Dropout from a counter-based generator: the mask is a function of the state
 * below, the call's site and the element's place, so it is never stored and
 * the backward makes it again.
 *
 * Element e of the 8-element block v (v = (row*h + column) / 8) of a call is
 * dropped when the 16-bit number u_e < D, D = floor(p * 65536 + 1/2), where
 * u_e is half e % 2 (low first) of word e / 2 of Philox4x32-10 (Salmon et al.,
 * SC 2011) with key = seed and counter words (v, site, offset low, offset
 * high).  A kept element is multiplied by 65536 / (65536 - D), the inverse of
 * the exact probability of keeping it. */
typedef struct {
  unsigned long long seed, offset;
} gptl_rng_state;                  /* DEVICE memory, caller-initialised       */

/* offset += n on the device (one thread), once per training step: a captured
 * step then draws new masks at each replay.  Within a step, give every call
 * (layer and place) a `site` of its own; a backward takes its forward's site
 * and runs before the state is advanced. */
int gptl_rng_advance(gptl_rng_state *rng, unsigned long long n, gptl_stream_t stream);

/* y = resid + dropout(x + bias) over [rows][h]: x (cdt) is the output of a
 * row-split product without its bias; bias [h] (cdt) and resid (fp32 when
 * resid_f32, else cdt) may be NULL; y is fp32 when y_f32, else cdt.  The sum is
 * fp32, rounded once.  y may be x or resid itself where their types agree, and
 * overlaps no input otherwise.  h % 8 == 0, rows*h < 2^35 (GPTL_E_SHAPE);
 * 0 <= p and D < 65536 (GPTL_E_ARG); with D = 0 (p < 2^-17) nothing is dropped,
 * and rng is not read and may be NULL. */
int gptl_dropout_add_fwd(int rows, int h, gptl_dtype dtype, const void *x, const void *bias,
                         const void *resid, int resid_f32, float p, const gptl_rng_state *rng,
                         unsigned site, void *y, int y_f32, gptl_stream_t stream);

/* Scratch bytes gptl_dropout_add_bwd needs for dbias (0 for bad sizes). */
size_t gptl_dropout_scratch_bytes(int rows, int h);

/* dx (cdt) = dy where kept, times the forward's factor, else 0; dbias (fp32
 * [h], may be NULL, else scratch is needed) = the column sums of that product
 * before it is rounded to dx, in a fixed order; calls that share scratch (those of
 * two captured graphs among them) must be ordered on the device.  dy is fp32 when
 * dy_f32, else cdt; dx may be dy itself where the types agree.  The gradient of
 * resid is dy.
 * Other arguments and errors as the forward's. */
int gptl_dropout_add_bwd(int rows, int h, gptl_dtype dtype, const void *dy, int dy_f32, float p,
                         const gptl_rng_state *rng, unsigned site, void *dx, float *dbias,
                         void *scratch, gptl_stream_t stream);

/* ------------------------------------------------------------------------
 * Log probabilities of given tokens under softmax(logits), with the entropy
 * and the top alternatives, in one pass over the logits.
 *   logits: [rows] of vocab elements, ld elements apart (ld >= vocab, any
 *           value below 2^40, rows*ld below 2^56), fp32 when logits_f32, else cdt
 *   m = max_v x_v,  Z = sum_v exp(x_v - m)
 *   logp    = x_target - m - ln Z
 *   entropy = ln Z - sum_v p_v (x_v - m),   p_v = exp(x_v - m) / Z
 *   stats   = (m, ln Z), what the backward needs
 *   top     : the top_k largest x_v in falling order, equal ones by rising
 *             index: top_logp = x_v - m - ln Z and top_id = v, [rows][top_k]
 * All outputs are fp32 (top_id int32).  target: int32 [rows]; a negative one
 * means none (logp = 0); one >= vocab sets bit 2 of the device error word and
 * gives logp = NaN.  target and logp come together or not at all; entropy,
 * stats and the top pair (with top_k = 0) are optional, but one output is
 * given.  0 <= top_k <= 32 and <= vocab (GPTL_E_ARG); 1 <= vocab < 2^30, with
 * alternatives <= 2^20, rows >= 1 (GPTL_E_SHAPE).
 * x_v = -inf has probability 0.  A row of nothing else gives m = ln Z = -inf,
 * entropy 0, logp and top_logp -inf, top_id 0, 1, ...  A row with +inf or NaN
 * gives NaN in every output (m: the largest element that is not NaN; logp of a
 * negative target stays 0) and top_id -1 in every place. */
int gptl_token_logprob_fwd(int rows, int vocab, long long ld, gptl_dtype dtype, int logits_f32,
                           const void *logits, const int *target, float *logp, float *entropy,
                           float *stats, int top_k, float *top_logp, int *top_id,
                           gptl_stream_t stream);

/* dlogits (type and ld of logits; logits itself, or no row of it overlaps one of
 * logits: the columns from vocab to ld of one may hold the other), for
 * the upstream gradients dlogp and dentropy ([rows] fp32, either may be NULL,
 * not both):
 *   dx_v = dlogp (1[v = target] - p_v) - dentropy p_v (ln p_v + entropy)
 * stats, and entropy when dentropy is given, are the forward's.  dlogp needs
 * target; a row whose target is negative (or >= vocab, which also sets bit 2
 * of the device error word) takes dlogp = 0.  A row whose two gradients are
 * both 0 gets exact zeros whatever its logits; a row of -inf alone gets zeros; a
 * row with +inf or NaN gets NaN.  Columns from vocab to ld are not
 * touched: a product that runs over the padded width needs zeros there, and in
 * place they still hold the padded logits. */
int gptl_token_logprob_bwd(int rows, int vocab, long long ld, gptl_dtype dtype, int logits_f32,
                           const void *logits, const int *target, const float *stats,
                           const float *entropy, const float *dlogp, const float *dentropy,
                           void *dlogits, gptl_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GPTLAYER_PARTS_H */
