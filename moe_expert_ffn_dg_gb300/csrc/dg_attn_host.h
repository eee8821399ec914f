// Host-side state and checks shared by the rotary, cache and attention entry
// points of include/dg_attn.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dg_attn.h"
#include "dg_host.h"

struct dg_rope {
  dg_rope_config_t cfg;
  // 2^64 f_i / 2 pi: an angle of position p is the fraction (p * turn[i]) mod
  // 2^64 of a turn, so far positions lose nothing
  uint64_t turn[256];
};

struct dg_kv {
  dg_kv_config_t cfg;
  void* status;
  int sms;  // of the device that it was made on
};

namespace dg {
namespace host {

constexpr int kMaxSeqs = 16384;
// tokens of a sequence and of a call: sums of three stay inside 32 bits
constexpr int kMaxKvTokens = 1 << 28;

inline bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < ((int64_t)1 << 37); }

// Query / key / value rows of the cache's element type for 16-byte accesses.
inline dg_status_t check_heads(const dg_heads_t* t) {
  if (!t || !t->p) return DG_ERR_INVALID_ARG;
  if (t->token_stride < 0 || t->head_stride < 0) return DG_ERR_INVALID_ARG;
  if (!aligned(t->p, 16) || !stride_ok(t->token_stride) || !stride_ok(t->head_stride))
    return DG_ERR_ALIGNMENT;
  return DG_OK;
}

inline dg_status_t check_batch(const dg_kv_batch_t* b, const dg_kv_config_t& c) {
  if (!b || b->n_seqs < 0 || b->max_pages < 0) return DG_ERR_INVALID_ARG;
  if (b->n_seqs == 0) return DG_OK;
  if (!b->lens || !b->cu) return DG_ERR_INVALID_ARG;
  if (b->max_pages > 0 && (!b->page_table || b->table_stride < b->max_pages))
    return DG_ERR_INVALID_ARG;
  if (!aligned(b->page_table, 4) || !aligned(b->lens, 4) || !aligned(b->cu, 4))
    return DG_ERR_ALIGNMENT;
  if (b->n_seqs > kMaxSeqs || (int64_t)b->max_pages * c.page_size > kMaxKvTokens)
    return DG_ERR_UNSUPPORTED;
  return DG_OK;
}

inline int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// Pages of one layer as (64-column block, head, token of the page, page).
inline bool encode_pages(CUtensorMap* map, const dg_kv_config_t& c, const dg_kv_pool_t& pool,
                         int layer, uint32_t box_tokens) {
  const uint16_t* base = static_cast<const uint16_t*>(pool.p) + layer * pool.layer_stride;
  const uint64_t dims[4] = {(uint64_t)c.head_dim, (uint64_t)c.n_kv_heads, (uint64_t)c.page_size,
                            (uint64_t)c.n_pages};
  const uint64_t strides[3] = {(uint64_t)pool.head_stride * 2, (uint64_t)pool.token_stride * 2,
                               (uint64_t)pool.page_stride * 2};
  const uint32_t box[4] = {64, 1, box_tokens, 1};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, base, dims, strides, box);
}

// Query rows as (64-column block, heads of a group, tokens of a box).
// DG_ERR_UNSUPPORTED for a stride of zero, which a descriptor cannot take.
inline dg_status_t encode_queries(CUtensorMap* map, const dg_heads_t& q, int n_q_heads,
                                  int head_dim, int n_tokens, int group, int box_tokens) {
  // a size-1 dimension's stride is never used, but must be a valid one
  const uint64_t hs = n_q_heads > 1 ? q.head_stride : head_dim;
  const uint64_t ts = n_tokens > 1 ? q.token_stride : head_dim;
  if (hs == 0 || ts == 0) return DG_ERR_UNSUPPORTED;
  const uint64_t dims[3] = {(uint64_t)head_dim, (uint64_t)n_q_heads, (uint64_t)n_tokens};
  const uint64_t strides[2] = {hs * 2, ts * 2};
  const uint32_t box[3] = {64, (uint32_t)group, (uint32_t)box_tokens};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, q.p, dims, strides, box)
             ? DG_OK : DG_ERR_CUDA;
}

// ------------------------------------------------------------------ handle

constexpr int kMaxCtas = 160;
constexpr int kRows = 128;  // rows of a query tile
constexpr int kKeys = 128;  // keys of a key tile
constexpr int kWeightKeys = 2 * kKeys;  // keys of a weights item

// An item that several CTAs worked on, written by the CTA that begins it.
struct JoinRec {
  int parts;  // 0: none
  int head, tok0, ntok;
  int shared;  // its sequence shares a prefix, whose part is still to come
};
struct WeightRec {
  int parts;  // 0: none
  int seq, block;
};

// The handle's workspace: status word; partial results of the attention, and
// of the weights of the keys.
struct Layout {
  size_t status, rec, ml, part, wrec, wpart, total;
};
inline Layout layout_of(int head_dim) {
  Layout L;
  const size_t rows = head_dim == 256 ? kRows : 2 * kRows;
  size_t at = 0;
  L.status = at;
  at += 256;
  L.rec = at;
  at = round_up(at + sizeof(JoinRec) * kMaxCtas, 256);
  L.ml = at;
  at = round_up(at + 2 * kMaxCtas * rows * sizeof(float2), 256);
  L.part = at;
  at = round_up(at + 2 * kMaxCtas * rows * head_dim * sizeof(float), 256);
  L.wrec = at;
  at = round_up(at + sizeof(WeightRec) * kMaxCtas, 256);
  L.wpart = at;
  at += 2 * kMaxCtas * kWeightKeys * sizeof(float);
  L.total = at;
  return L;
}

// Kernels whose limits a new handle raises on its device (dg_weights.cu,
// dg_thin.cu).
cudaError_t prepare_weights(int head_dim);
cudaError_t prepare_select();

// Clear the status word of a new handle: through the default stream, done when
// this returns, whatever stream the handle's first call runs on.
bool clear_status(void* word, size_t bytes);

// Synchronise, read and clear a device status word.
dg_status_t read_status(void* word, dg_stream_t stream, unsigned int* where, unsigned int* info);

}  // namespace host
}  // namespace dg

struct dg_attn {
  dg_attn_config_t cfg;
  const dg_kv* kv;
  uint8_t* ws;
  dg::host::Layout L;
  int ctas;
};
