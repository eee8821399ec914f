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

// Clear the status word of a new handle: through the default stream, done when
// this returns, whatever stream the handle's first call runs on.
bool clear_status(void* word, size_t bytes);

// Synchronise, read and clear a device status word.
dg_status_t read_status(void* word, dg_stream_t stream, unsigned int* where, unsigned int* info);

}  // namespace host
}  // namespace dg
