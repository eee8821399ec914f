/*
 * dg_attn.h — C ABI of the attention half that runs beside the routed-MoE
 * block of dg_moe.h: rotary positions, a paged key/value cache and its page
 * operations, and attention of a chunk of new tokens over that cache.
 *
 * Conventions are those of dg_moe.h: device pointers unless a function says
 * "host", status codes for what the host can see (nothing is launched then),
 * a device status word for what only the device can see (a page id or a
 * length out of range; the kernel skips or clamps it and goes on), calls
 * asynchronous on their stream, no device memory allocated, capturable into a
 * CUDA graph.  Handles own host memory only and may be used from several
 * streams as long as calls that share a workspace do not overlap.
 *
 * Element types: bf16 and fp16 (fp32 too for dg_rope_apply).  All arithmetic
 * is fp32, rounded once on output; attention weights enter the product with V
 * in the element type (fp16: those below 2^-32 of their row's largest as zero),
 * their sums stay fp32.
 */
#ifndef DG_ATTN_H
#define DG_ATTN_H

#include "dg_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { DG_T_BF16 = 0, DG_T_FP16 = 1, DG_T_FP32 = 2 } dg_dtype_t;

/* A [tokens, heads, head_dim] tensor: strides in elements, head_dim
 * contiguous. */
typedef struct {
  void* p;
  int64_t token_stride;
  int64_t head_stride;
} dg_heads_t;

/* ------------------------------------------------------------------------
 * Rotary positions.
 *
 *   f_i  = theta^(-2 i / rot_dim),  i < rot_dim / 2
 *   y    = amplitude * R(p f) x  on the first rot_dim elements of a head,
 *          the others copied
 *
 * R turns the pair (x_i, x_{i + rot_dim/2}) (DG_ROPE_HALF) or
 * (x_2i, x_{2i+1}) (DG_ROPE_INTERLEAVED) by the angle p f_i.  Scaled for
 * contexts longer than the trained orig_len by `factor`:
 *   DG_ROPE_LINEAR  f_i / factor
 *   DG_ROPE_BASE    theta replaced by theta * factor^(rot_dim / (rot_dim - 2))
 *   DG_ROPE_RAMP    g f_i + (1 - g) f_i / factor, where
 *                   g = clamp((r - beta_slow) / (beta_fast - beta_slow), 0, 1)
 *                   and r = orig_len f_i / 2 pi, the turns inside orig_len
 * Angles are exact to 2^-24 of a turn for every 32-bit position.
 * ------------------------------------------------------------------------ */
typedef enum { DG_ROPE_HALF = 0, DG_ROPE_INTERLEAVED = 1 } dg_rope_layout_t;
typedef enum {
  DG_ROPE_PLAIN = 0,
  DG_ROPE_LINEAR = 1,
  DG_ROPE_BASE = 2,
  DG_ROPE_RAMP = 3
} dg_rope_scaling_t;

typedef struct {
  int head_dim; /* 2 .. 512 */
  int rot_dim;  /* even, 2 .. head_dim (DG_ROPE_BASE: at least 4) */
  dg_rope_layout_t layout;
  dg_rope_scaling_t scaling;
  double theta;     /* > 1 */
  double factor;    /* >= 1; unused by DG_ROPE_PLAIN */
  double orig_len;  /* > 0; DG_ROPE_RAMP only */
  double beta_slow; /* 0 <= beta_slow < beta_fast; DG_ROPE_RAMP only */
  double beta_fast;
  double amplitude; /* > 0 */
  unsigned flags;   /* must be 0 */
} dg_rope_config_t;

typedef struct dg_rope dg_rope_t;

/* Frequencies are computed here, in 64 bits on the host. */
dg_status_t dg_rope_create(const dg_rope_config_t* cfg, dg_rope_t** out);
dg_status_t dg_rope_destroy(dg_rope_t* r);

/* out = the rotation of x [n_tokens, n_heads, head_dim] by positions (int32
 * [n_tokens], any value); grad != 0: its transpose, which is the gradient
 * with respect to x of a loss whose gradient with respect to the output is
 * the tensor passed as x.  out may be x (same pointer and strides), else they
 * must not overlap.  Any strides and alignment of the element type; 16-byte
 * aligned pointers and strides take the vectorised path. */
dg_status_t dg_rope_apply(const dg_rope_t* r, dg_dtype_t dtype, const dg_heads_t* x,
                          const dg_heads_t* out, const int32_t* positions, int n_tokens,
                          int n_heads, int grad, dg_stream_t stream);

/* ------------------------------------------------------------------------
 * Paged cache: n_layers pools of n_pages pages, a page holding page_size
 * tokens of n_kv_heads x head_dim keys (and values).  Element (layer, page,
 * token, head, d) of a pool lies at
 *   p + layer*layer_stride + page*page_stride + token*token_stride
 *     + head*head_stride + d                                  (elements).
 * Supported: head_dim 64, 128 or 256; page_size 16, 32, 64, 128 or 256;
 * bf16 or fp16; pointers 16-byte aligned, strides multiples of 8 elements.
 * The two pools do not overlap.  They are borrowed.
 * ------------------------------------------------------------------------ */
typedef struct {
  void* p;
  int64_t layer_stride, page_stride, token_stride, head_stride;
} dg_kv_pool_t;

typedef struct {
  int n_layers, n_pages, page_size, n_kv_heads, head_dim;
  dg_dtype_t dtype;
  dg_kv_pool_t k, v;
  unsigned flags; /* must be 0 */
} dg_kv_config_t;

/* The sequences of one call.  Row s of page_table (row stride table_stride
 * elements) lists the pages of sequence s in order; max_pages is how many of
 * a row may be used.  lens[s]: tokens in the cache, the new ones of this call
 * included.  cu[s] .. cu[s+1]: the new tokens of sequence s among the
 * n_tokens rows of q / k / v; they are its last ones, so row cu[s] + i is at
 * position lens[s] - (cu[s+1] - cu[s]) + i.  All int32 device memory. */
typedef struct {
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* cu; /* [n_seqs + 1], ascending */
  int n_seqs, max_pages;
} dg_kv_batch_t;

typedef struct dg_kv dg_kv_t;

/* status: 256 bytes of device memory, 16-byte aligned, for the device status
 * word; cleared here, through the default stream, before this returns.  No work
 * in flight may still use that memory (the same holds for the workspace of
 * dg_attn_create). */
dg_status_t dg_kv_create(const dg_kv_config_t* cfg, void* status, dg_kv_t** out);
dg_status_t dg_kv_destroy(dg_kv_t* kv);

/* Synchronise `stream`, read the device status word of the cache, clear it. */
dg_status_t dg_kv_last_device_status(dg_kv_t* kv, dg_stream_t stream, unsigned int* where,
                                     unsigned int* info);

/* Write the new tokens' keys and values [n_tokens, n_kv_heads, head_dim] into
 * their pages of `layer`.  With rope, keys are rotated on the way, and q
 * [n_tokens, n_q_heads, head_dim] is rotated into q_out (may be q itself); q
 * NULL: none.  Without rope q, if given, is copied to q_out.
 * positions: int32 [n_tokens] rotary positions, or NULL for the tokens' cache
 * positions.  Tokens outside every sequence are skipped (their q_out rows
 * too); the keys and values of a token at a negative position or with a bad
 * page are not written, which the status word records. */
dg_status_t dg_kv_append(dg_kv_t* kv, int layer, const dg_rope_t* rope, const dg_heads_t* k,
                         const dg_heads_t* v, const dg_heads_t* q, const dg_heads_t* q_out,
                         int n_q_heads, const dg_kv_batch_t* batch, const int32_t* positions,
                         int n_tokens, dg_stream_t stream);

/* Copy pages inside the cache, all layers, keys and values.  copies: int32
 * [n, 3] rows (source page, destination page, tokens); rows with a negative
 * source do nothing.  A page may be the source of several rows and the
 * destination of one, never both. */
dg_status_t dg_kv_copy(dg_kv_t* kv, const int32_t* copies, int n, dg_stream_t stream);

/* Compact: token i of sequence s becomes the token keep[cu[s] + i] that it had
 * (any order, repeats allowed), all layers, keys and values.  src and dst are
 * page tables of n_seqs rows as in dg_kv_batch_t; the pages written must not
 * be among those read.  n_keep: length of keep; cu: int32 [n_seqs + 1].
 * Tokens keep the rotary positions with which they were written. */
dg_status_t dg_kv_gather(dg_kv_t* kv, const int32_t* src_table, int64_t src_stride, int src_pages,
                         const int32_t* dst_table, int64_t dst_stride, int dst_pages,
                         const int32_t* cu, int n_seqs, const int32_t* keep, int n_keep,
                         dg_stream_t stream);

/* ------------------------------------------------------------------------
 * Bookkeeping of pages: which sequence holds which page, shared pages counted.
 *
 * One call takes the sequences from one step to the next.  New sequence j
 * continues old sequence parent[j] (several may continue one: a fork; none:
 * it is freed), or starts empty (parent[j] = -1), and gets room for grow[j]
 * more tokens:
 *   1. ref[page] loses one for every old sequence that holds the page and
 *      gains one for every new one (a sequence holds the first
 *      ceil(len / page_size) pages of its row);
 *   2. a new sequence that grows from a partly filled page which it does not
 *      hold alone gets its own copy of it: (page, fresh page, filled tokens)
 *      in copies[j], else (-1, -1, 0).  Where every holder grows, the first
 *      one keeps the page;
 *   3. pages with ref 0 are taken in ascending order, sequences in order, the
 *      copy's page first.
 * If there are too few free pages, or a sequence would outgrow its row, no
 * sequence grows and none is split: *short_by is the number of pages missing
 * (-1 for a row outgrown) and step 1 stands, which is a valid state.  Else
 * *short_by is 0 and lens_out = len + grow.
 * Run dg_kv_copy with copies before the next append.
 * table_out rows are filled with -1 behind their pages.  ref_out may be
 * ref_in; the other outputs must not overlap the inputs.
 * Inputs out of range (a page id, a length past the row, a parent, a negative
 * growth) are taken as absent or clamped, and recorded in the status word.
 * Supported: page_size as above, up to 4096 old and 4096 new sequences.
 * ------------------------------------------------------------------------ */
typedef struct {
  int n_pages, page_size;
  int row; /* row length of both tables, contiguous rows */
  int n_old, n_new;
  const int32_t* table_in;  /* [n_old, row] */
  const int32_t* lens_in;   /* [n_old] */
  const int32_t* ref_in;    /* [n_pages] */
  const int32_t* parent;    /* [n_new] */
  const int32_t* grow;      /* [n_new] */
  int32_t* table_out;       /* [n_new, row] */
  int32_t* lens_out;        /* [n_new] */
  int32_t* ref_out;         /* [n_pages] */
  int32_t* copies;          /* [n_new, 3] */
  int32_t* short_by;        /* [1] */
} dg_kv_fork_t;

/* Device workspace of a fork (status word first); 16-byte aligned. */
dg_status_t dg_kv_fork_workspace_size(int n_pages, size_t* bytes);
dg_status_t dg_kv_fork(const dg_kv_fork_t* f, void* workspace, size_t workspace_bytes,
                       dg_stream_t stream);
/* Synchronise, read and clear the status word of a fork workspace.  The
 * caller zeroes the first 256 bytes of a new workspace. */
dg_status_t dg_kv_fork_last_device_status(void* workspace, dg_stream_t stream,
                                          unsigned int* where, unsigned int* info);

/* ------------------------------------------------------------------------
 * Attention of new tokens over the paged cache.  Query head h reads key/value
 * head h / (n_q_heads / n_kv_heads).  A query at position p sees key j,
 * 0 <= j < len, if p - left <= j <= p + right; a negative left or right is
 * no limit on that side (right = 0: causal; both negative: a canvas or an
 * encoder memory).
 *
 *   o = sum_j softmax_j(scale q k_j) v_j,   lse = log sum_j exp(scale q k_j)
 *
 * A query that sees nothing gets o = 0 and lse = -inf.  Keys and values at or
 * past len, and whole pages before every window of the call, may hold
 * anything (their table entries too).  Among the other tokens, a non-finite
 * value of v can reach any query of its sequence.
 * ------------------------------------------------------------------------ */
typedef struct {
  int n_q_heads; /* multiple of n_kv_heads, at most 128 of them a group */
  int left, right;
  float scale;    /* > 0 */
  unsigned flags; /* must be 0 */
} dg_attn_config_t;

typedef struct dg_attn dg_attn_t;

/* Device workspace (partial results and the status word); 1024-byte aligned. */
dg_status_t dg_attn_workspace_size(const dg_attn_config_t* cfg, const dg_kv_t* kv, size_t* bytes);

/* kv must outlive the handle. */
dg_status_t dg_attn_create(const dg_attn_config_t* cfg, const dg_kv_t* kv, void* workspace,
                           size_t workspace_bytes, dg_attn_t** out);
dg_status_t dg_attn_destroy(dg_attn_t* a);

/* q, out: [n_tokens, n_q_heads, head_dim], the cache's element type, 16-byte
 * aligned, strides multiples of 8 elements (q's not zero); out must not
 * overlap q.  lse:
 * fp32 [n_tokens, n_q_heads] contiguous, or NULL.  Rows outside every
 * sequence are left alone. */
dg_status_t dg_attn_forward(dg_attn_t* a, int layer, const dg_heads_t* q, const dg_heads_t* out,
                            float* lse, const dg_kv_batch_t* batch, int n_tokens,
                            dg_stream_t stream);

dg_status_t dg_attn_last_device_status(dg_attn_t* a, dg_stream_t stream, unsigned int* where,
                                       unsigned int* info);

#ifdef __cplusplus
}
#endif

#endif /* DG_ATTN_H */
