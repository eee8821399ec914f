// The paged cache's handle and its page operations (include/dg_attn.h): the
// bookkeeping of forks, and the moves of cached tokens.
#include <limits.h>

#include <new>

#include "../../include/dg_attn.h"
#include "dg_attn_host.h"
#include "dg_common.cuh"

using namespace dg;
using namespace dg::host;

namespace {

// ------------------------------------------------------------------ moves

enum : unsigned int { kSiteMovePage = 48, kSiteForkPage = 49, kSiteForkLen = 50,
                      kSiteForkParent = 51, kSiteForkRef = 52 };

constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 32;   // tokens of a block
constexpr int kMoveUnroll = 8;    // vectors a thread holds in flight

struct MoveParams {
  const uint16_t* pool[2];  // keys, values
  int64_t layer_stride[2], page_stride[2], token_stride[2], head_stride[2];
  int vec_shift;        // log2 of 16-byte vectors a head
  int row_vecs;         // vectors a token
  uint32_t row_magic;   // ceil(2^32 / row_vecs)
  int page_shift, n_pages;
  // copy: rows (source, destination, tokens)
  const int32_t* copies;
  // gather
  const int32_t* src_table;
  const int32_t* dst_table;
  int64_t src_stride, dst_stride;
  int src_pages, dst_pages;
  const int32_t* cu;
  const int32_t* keep;
  int n_seqs, n_keep;
  DevStatus* status;
};

// Bound by memory: every moved byte is read and written once, 16 bytes a
// thread, kMoveUnroll of them in flight.  A block takes up to kMoveTokens
// tokens of one layer's keys or values (grid y: layer and pool) and first
// finds where each comes from and goes to.  On one GB300: 398 MB in and out in
// 56 us (part of it stays in L2), 800 MB in 120 us (6.7 TB/s).
template <bool GATHER>
__global__ void __launch_bounds__(kMoveThreads) k_kv_move(const __grid_constant__ MoveParams p) {
  __shared__ int s_src[kMoveTokens], s_dst[kMoveTokens];    // page, -1: nothing
  __shared__ int s_from[kMoveTokens], s_to[kMoveTokens];    // token of the page
  const int tid = threadIdx.x, which = blockIdx.y & 1, layer = blockIdx.y >> 1;
  const int mask = (1 << p.page_shift) - 1;
  pdl_trigger();
  pdl_wait();
  int nt;
  if (GATHER) {
    const int t0 = blockIdx.x * kMoveTokens;
    nt = min(kMoveTokens, p.n_keep - t0);
    if (tid < nt) {
      const int t = t0 + tid;
      int lo = 0, hi = p.n_seqs;  // the last s with cu[s] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu + mid) <= t) lo = mid;
        else hi = mid;
      }
      const int a = __ldg(p.cu + lo), b = __ldg(p.cu + lo + 1);
      int src = -1, dst = -1, from = 0, to = 0;
      if (a <= t && t < b) {
        from = __ldg(p.keep + t);
        to = t - a;
        const int sp = from >> p.page_shift, dp = to >> p.page_shift;
        bool ok = from >= 0 && sp < p.src_pages && dp < p.dst_pages;
        if (ok) {
          src = __ldg(p.src_table + lo * p.src_stride + sp);
          dst = __ldg(p.dst_table + lo * p.dst_stride + dp);
          ok = (unsigned)src < (unsigned)p.n_pages && (unsigned)dst < (unsigned)p.n_pages;
        }
        if (!ok) {
          report(p.status, kDevBounds, kSiteMovePage, (unsigned)t, (unsigned)from);
          src = -1;
        }
      }
      s_src[tid] = src;
      s_dst[tid] = dst;
      s_from[tid] = from & mask;
      s_to[tid] = to & mask;
    }
  } else {
    // blocks of a page, page after page
    const int per = ((1 << p.page_shift) + kMoveTokens - 1) / kMoveTokens;
    const int pair = blockIdx.x / per, t0 = (blockIdx.x - pair * per) * kMoveTokens;
    const int32_t* row = p.copies + 3 * (int64_t)pair;
    const int src = __ldg(row), dst = __ldg(row + 1);
    const int n = min(__ldg(row + 2), mask + 1);
    if (src < 0) return;
    nt = min(kMoveTokens, n - t0);
    if (nt <= 0) return;
    if (src >= p.n_pages || (unsigned)dst >= (unsigned)p.n_pages) {
      if (tid == 0) report(p.status, kDevBounds, kSiteMovePage, (unsigned)pair, (unsigned)src);
      return;
    }
    if (tid < nt) {
      s_src[tid] = src;
      s_dst[tid] = dst;
      s_from[tid] = s_to[tid] = t0 + tid;
    }
  }
  __syncthreads();
  const uint16_t* base = p.pool[which] + layer * p.layer_stride[which];
  const int64_t ps = p.page_stride[which], ts = p.token_stride[which], hs = p.head_stride[which];
  const int total = nt * p.row_vecs, vmask = (1 << p.vec_shift) - 1;
  for (int x0 = tid; x0 < total; x0 += kMoveThreads * kMoveUnroll) {
    uint4 v[kMoveUnroll];
    int64_t to[kMoveUnroll];
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i) {
      const int x = x0 + i * kMoveThreads;
      to[i] = -1;
      if (x >= total) continue;
      const int t = (int)__umulhi((uint32_t)x, p.row_magic), r = x - t * p.row_vecs;
      const int src = s_src[t];
      if (src < 0) continue;
      const int64_t in = (int64_t)(r >> p.vec_shift) * hs + (int64_t)(r & vmask) * 8;
      to[i] = s_dst[t] * ps + s_to[t] * ts + in;
      v[i] = *reinterpret_cast<const uint4*>(base + src * ps + s_from[t] * ts + in);
    }
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i)
      if (to[i] >= 0)
        *reinterpret_cast<uint4*>(const_cast<uint16_t*>(base) + to[i]) = v[i];
  }
}

MoveParams move_params(const dg_kv* kv) {
  const dg_kv_config_t& c = kv->cfg;
  MoveParams p = {};
  const dg_kv_pool_t* pools[2] = {&c.k, &c.v};
  for (int i = 0; i < 2; ++i) {
    p.pool[i] = static_cast<const uint16_t*>(pools[i]->p);
    p.layer_stride[i] = pools[i]->layer_stride;
    p.page_stride[i] = pools[i]->page_stride;
    p.token_stride[i] = pools[i]->token_stride;
    p.head_stride[i] = pools[i]->head_stride;
  }
  p.vec_shift = log2_of(c.head_dim / 8);
  p.row_vecs = c.n_kv_heads * (c.head_dim / 8);
  p.row_magic = (uint32_t)((((uint64_t)1 << 32) + p.row_vecs - 1) / p.row_vecs);
  p.page_shift = log2_of(c.page_size);
  p.n_pages = c.n_pages;
  p.status = static_cast<DevStatus*>(kv->status);
  return p;
}

// ------------------------------------------------------------------ fork

// One cluster does the whole step: its phases depend on one another over all
// pages and sequences, and the hardware barrier of a cluster costs far less
// than a launch a phase.  Tables and counts are small (a full server's are a
// few MB), so latency bounds it, not bandwidth: 8.5 us for 8 sequences, 24 us
// for 512 with rows of 512 pages out of 262144.
constexpr int kForkCtas = 8;
constexpr int kForkThreads = 1024;
constexpr int kForkMax = 4096;  // sequences
constexpr int kBatch = 8;       // loads in flight a thread: the loops wait for memory

struct ForkParams {
  dg_kv_fork_t f;
  int page_shift;
  DevStatus* status;
  int32_t* counts;  // [kForkCtas] free pages of each CTA's share
  int32_t* users;   // [n_pages] growing holders of a partly filled page; later the
                    // fresh pages in order
  int32_t* first;   // [n_pages] the lowest of them
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// Held length of old sequence s, clamped.
__device__ __forceinline__ int held_len(const dg_kv_fork_t& f, int s, int shift) {
  return (int)min((int64_t)max(__ldg(f.lens_in + s), 0), (int64_t)f.row << shift);
}

// What a new sequence continues, from the inputs (shared memory, one each).
struct Grow {
  int parent, have, grow;
  int last;  // its partly filled last page, if it grows from one, or -1
};

__global__ void __cluster_dims__(kForkCtas, 1, 1) __launch_bounds__(kForkThreads)
    k_kv_fork(const __grid_constant__ ForkParams p) {
  const dg_kv_fork_t& f = p.f;
  extern __shared__ __align__(16) uint8_t dyn[];
  Grow* grow = reinterpret_cast<Grow*>(dyn);                // [n_new]
  int* child = reinterpret_cast<int*>(grow + f.n_new);      // [n_old] children of an old sequence
  int* start = child;                                       // [n_new + 1] rank of its first fresh
                                                            // page, once child is done with
  __shared__ uint8_t split[kForkMax];
  __shared__ int warp_sum[32], warp_free[32], over;
  __shared__ int s_total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  const int gt = cta * kForkThreads + tid, gw = gt >> 5;
  constexpr int kAll = kForkCtas * kForkThreads, kWarps = kAll / 32;
  const int shift = p.page_shift, ps = 1 << shift;
  pdl_trigger();
  for (int s = tid; s < f.n_old; s += kForkThreads) child[s] = 0;
  if (tid == 0) over = 0;
  pdl_wait();
  __syncthreads();

  // The new sequences (every CTA, all of them); scratch of the pages that may
  // split; children of every old sequence.
  for (int j = tid; j < f.n_new; j += kForkThreads) {
    Grow g;
    g.parent = __ldg(f.parent + j);
    g.grow = __ldg(f.grow + j);
    if (cta == 0) {
      if (g.parent < -1 || g.parent >= f.n_old)
        report(p.status, kDevBounds, kSiteForkParent, (unsigned)j, (unsigned)g.parent);
      if (g.grow < 0) report(p.status, kDevBounds, kSiteForkLen, (unsigned)j, (unsigned)g.grow);
    }
    if (g.parent >= f.n_old || g.parent < 0) g.parent = -1;
    g.grow = max(g.grow, 0);
    g.have = g.parent < 0 ? 0 : held_len(f, g.parent, shift);
    g.last = -1;
    if (g.grow > 0 && (g.have & (ps - 1))) {
      const int id = __ldg(f.table_in + (int64_t)g.parent * f.row + (g.have >> shift));
      if ((unsigned)id < (unsigned)f.n_pages) {
        g.last = id;
        if (cta == 0) {
          p.users[id] = 0;
          p.first[id] = INT_MAX;
        }
      }
    }
    grow[j] = g;
    if (g.parent >= 0) atomicAdd(&child[g.parent], 1);
  }
  if (f.ref_out != f.ref_in) {
#pragma unroll 8
    for (int i = gt; i < f.n_pages; i += kAll) f.ref_out[i] = __ldg(f.ref_in + i);
  }
  cluster_sync();

  // counts of held pages; growing holders of partly filled pages
  for (int s = gw; s < f.n_old; s += kWarps) {
    const int d = child[s] - 1;
    const int raw = __ldg(f.lens_in + s);
    const int pages = (held_len(f, s, shift) + ps - 1) >> shift;
    if (lane == 0 && (raw < 0 || raw > (int64_t)f.row << shift))
      report(p.status, kDevBounds, kSiteForkLen, (unsigned)s, (unsigned)raw);
    if (d == 0) continue;
    const int32_t* held = f.table_in + (int64_t)s * f.row;
    for (int i0 = lane; i0 < pages; i0 += 32 * kBatch) {
      int id[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        id[k] = i0 + 32 * k < pages ? __ldg(held + i0 + 32 * k) : 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (i0 + 32 * k >= pages) break;
        if ((unsigned)id[k] < (unsigned)f.n_pages)
          atomicAdd(f.ref_out + id[k], d);
        else
          report(p.status, kDevBounds, kSiteForkPage, (unsigned)s, (unsigned)id[k]);
      }
    }
  }
  for (int j = gt; j < f.n_new; j += kAll) {
    const int last = grow[j].last;
    if (last >= 0) {
      atomicAdd(p.users + last, 1);
      atomicMin(p.first + last, j);
    }
  }
  cluster_sync();

  // free pages of this CTA's share, one contiguous run a warp
  const int run = (f.n_pages + kWarps - 1) / kWarps;
  const int p0 = min((int64_t)gw * run, (int64_t)f.n_pages), p1 = min(p0 + run, f.n_pages);
  int nfree = 0, least = 0;
  for (int i0 = p0 + lane; i0 < p1; i0 += 32 * kBatch) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = i0 + 32 * k < p1 ? __ldcg(f.ref_out + i0 + 32 * k) : 1;
      nfree += r == 0;
      least = min(least, r);
    }
  }
  if (least < 0) report(p.status, kDevBounds, kSiteForkRef, (unsigned)p0, (unsigned)least);
  nfree = __reduce_add_sync(0xffffffffu, nfree);
  if (lane == 0) warp_free[warp] = nfree;
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    for (int w = 0; w < 32; ++w) n += warp_free[w];
    p.counts[cta] = n;
  }

  // splits and needs of all sequences (every CTA, from the same numbers), and
  // their prefix
  {
    constexpr int kEach = kForkMax / kForkThreads;
    int need[kEach], sum = 0;
    const int each = (f.n_new + kForkThreads - 1) / kForkThreads;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = tid * each + i;
      need[i] = 0;
      if (i < each && j < f.n_new) {
        const Grow g = grow[j];
        bool sp = false;
        if (g.last >= 0)
          sp = __ldcg(f.ref_out + g.last) > __ldcg(p.users + g.last) ||
               __ldcg(p.first + g.last) != j;
        split[j] = sp;
        const int64_t want = (int64_t)g.have + g.grow;
        if (want > (int64_t)f.row << shift) over = 1;
        else
          need[i] =
              (int)((want + ps - 1) >> shift) - ((g.have + ps - 1) >> shift) + (sp ? 1 : 0);
      }
      sum += need[i];
    }
    // at most 4096 sequences of 2^18 pages: the sum fits 32 bits
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    int at = before + incl - sum;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = tid * each + i;
      if (i < each && j < f.n_new) start[j] = at;
      at += need[i];
    }
    if (tid == kForkThreads - 1) {
      start[f.n_new] = at;
      s_total = at;
    }
  }
  cluster_sync();  // the last use of users

  int64_t all_free = 0;
  int rank = 0;
  for (int c = 0; c < kForkCtas; ++c) {
    const int n = __ldcg(p.counts + c);
    all_free += n;
    if (c < cta) rank += n;
  }
  const bool ok = !over && s_total <= all_free;
  const int total = ok ? s_total : 0;
  if (gt == 0) *f.short_by = over ? -1 : (ok ? 0 : (int)(s_total - all_free));

  // the `total` lowest free pages, in order (they may all lie in one warp's
  // run, so it only lists them here)
  int* fresh = p.users;
  for (int w = 0; w < warp; ++w) rank += warp_free[w];
  for (int i0 = p0; i0 < p1 && rank < total; i0 += 32 * kBatch) {
    int r[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + 32 * k + lane;
      r[k] = i < p1 ? __ldcg(f.ref_out + i) : 1;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const unsigned b = __ballot_sync(0xffffffffu, r[k] == 0);
      const int at = rank + __popc(b & ((1u << lane) - 1u));
      if (r[k] == 0 && at < total) fresh[at] = i0 + 32 * k + lane;
      rank += __popc(b);
    }
  }

  // rows of the new sequences, but for their fresh pages
  for (int j = gw; j < f.n_new; j += kWarps) {
    const Grow g = grow[j];
    const bool sp = ok && split[j];
    const int pages = (g.have + ps - 1) >> shift;
    const int stay = pages - (sp ? 1 : 0);
    const int want = ok ? (g.have + g.grow + ps - 1) >> shift : pages;
    const int32_t* held = f.table_in + (int64_t)g.parent * f.row;
    for (int i0 = lane; i0 < f.row; i0 += 32 * kBatch) {
      int id[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) id[k] = i0 + 32 * k < stay ? __ldg(held + i0 + 32 * k) : -1;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + 32 * k;
        if (i >= f.row) break;
        if (i < stay && (unsigned)id[k] >= (unsigned)f.n_pages) {
          report(p.status, kDevBounds, kSiteForkPage, (unsigned)g.parent, (unsigned)id[k]);
          id[k] = -1;
        }
        if (i < stay || i >= want) f.table_out[(int64_t)j * f.row + i] = id[k];
      }
    }
    if (lane == 0) {
      f.lens_out[j] = g.have + (ok ? g.grow : 0);
      if (!sp) {
        f.copies[3 * j] = f.copies[3 * j + 1] = -1;
        f.copies[3 * j + 2] = 0;
      }
    }
  }
  cluster_sync();

  // fresh pages: the one of rank r goes to the sequence whose range holds r
  for (int r = gt; r < total; r += kAll) {
    const int page = __ldcg(fresh + r);
    int lo = 0, hi = f.n_new;  // the last j with start[j] <= r
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= r) lo = mid;
      else hi = mid;
    }
    const Grow g = grow[lo];
    const bool sp = split[lo];
    const int at = ((g.have + ps - 1) >> shift) - (sp ? 1 : 0) + r - start[lo];
    f.table_out[(int64_t)lo * f.row + at] = page;
    f.ref_out[page] = 1;
    if (sp && r == start[lo]) {
      f.copies[3 * lo] = g.last;
      f.copies[3 * lo + 1] = page;
      f.copies[3 * lo + 2] = g.have & (ps - 1);
      atomicSub(f.ref_out + g.last, 1);
    }
  }
}

struct ForkLayout {
  size_t counts, users, first, total;
};
ForkLayout fork_layout(int n_pages) {
  ForkLayout L;
  L.counts = 256;
  L.users = 512;
  L.first = L.users + round_up((size_t)n_pages * 4, 256);
  L.total = L.first + (size_t)n_pages * 4;
  return L;
}

bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }

constexpr int kMaxForkPages = 1 << 28;

}  // namespace

extern "C" {

dg_status_t dg_kv_create(const dg_kv_config_t* cfg, void* status, dg_kv_t** out) {
  if (!out) return DG_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg || cfg->flags != 0) return DG_ERR_INVALID_ARG;
  const dg_kv_config_t& c = *cfg;
  if (c.n_layers <= 0 || c.n_pages <= 0 || c.n_kv_heads <= 0) return DG_ERR_INVALID_ARG;
  if (c.dtype != DG_T_BF16 && c.dtype != DG_T_FP16) return DG_ERR_UNSUPPORTED;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return DG_ERR_UNSUPPORTED;
  if (!page_size_ok(c.page_size) || c.n_kv_heads > 256 || c.n_layers > 32767)
    return DG_ERR_UNSUPPORTED;
  for (const dg_kv_pool_t* q : {&c.k, &c.v}) {
    if (!q->p) return DG_ERR_INVALID_ARG;
    if (!aligned(q->p, 16)) return DG_ERR_ALIGNMENT;
    for (const int64_t s : {q->layer_stride, q->page_stride, q->token_stride, q->head_stride}) {
      if (s < 0) return DG_ERR_INVALID_ARG;
      if (s % 8) return DG_ERR_ALIGNMENT;
    }
    // rows of one pool must not overlap; copies address them with descriptors
    // whose strides are below 2^40 bytes
    if (q->token_stride < c.head_dim || q->page_stride < c.head_dim ||
        (c.n_kv_heads > 1 && q->head_stride < c.head_dim) || !stride_ok(q->page_stride) ||
        !stride_ok(q->token_stride) || !stride_ok(q->head_stride))
      return DG_ERR_INVALID_ARG;
  }
  if (!status) return DG_ERR_WORKSPACE;
  if (!aligned(status, 16)) return DG_ERR_WORKSPACE;
  if (!clear_status(status, 256)) return DG_ERR_CUDA;
  dg_kv* kv = new (std::nothrow) dg_kv();
  if (!kv) return DG_ERR_CUDA;
  kv->cfg = c;
  // a size-1 dimension's stride is never used, but a descriptor wants one
  if (c.n_kv_heads == 1) kv->cfg.k.head_stride = kv->cfg.v.head_stride = c.head_dim;
  kv->status = status;
  *out = kv;
  return DG_OK;
}

dg_status_t dg_kv_destroy(dg_kv_t* kv) {
  delete kv;
  return DG_OK;
}

dg_status_t dg_kv_last_device_status(dg_kv_t* kv, dg_stream_t stream, unsigned int* where,
                                     unsigned int* info) {
  if (!kv) return DG_ERR_INVALID_ARG;
  return read_status(kv->status, stream, where, info);
}

dg_status_t dg_kv_copy(dg_kv_t* kv, const int32_t* copies, int n, dg_stream_t stream) {
  if (!kv || n < 0) return DG_ERR_INVALID_ARG;
  if (n == 0) return DG_OK;
  if (!copies) return DG_ERR_INVALID_ARG;
  if (!aligned(copies, 4)) return DG_ERR_ALIGNMENT;
  if (n > (1 << 24)) return DG_ERR_UNSUPPORTED;
  MoveParams p = move_params(kv);
  p.copies = copies;
  const int per = (kv->cfg.page_size + kMoveTokens - 1) / kMoveTokens;
  const cudaError_t e =
      launch_pdl(k_kv_move<false>, dim3((unsigned)n * per, 2 * kv->cfg.n_layers),
                 dim3(kMoveThreads), 0, reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

dg_status_t dg_kv_gather(dg_kv_t* kv, const int32_t* src_table, int64_t src_stride, int src_pages,
                         const int32_t* dst_table, int64_t dst_stride, int dst_pages,
                         const int32_t* cu, int n_seqs, const int32_t* keep, int n_keep,
                         dg_stream_t stream) {
  if (!kv || n_seqs < 0 || n_keep < 0 || src_pages < 0 || dst_pages < 0) return DG_ERR_INVALID_ARG;
  if (n_seqs == 0 || n_keep == 0) return DG_OK;
  if (!src_table || !dst_table || !cu || !keep) return DG_ERR_INVALID_ARG;
  if (src_stride < src_pages || dst_stride < dst_pages) return DG_ERR_INVALID_ARG;
  for (const void* q : {src_table, dst_table, cu, keep})
    if (!aligned(q, 4)) return DG_ERR_ALIGNMENT;
  if (n_seqs > kMaxSeqs || n_keep > kMaxKvTokens) return DG_ERR_UNSUPPORTED;
  MoveParams p = move_params(kv);
  p.src_table = src_table;
  p.dst_table = dst_table;
  p.src_stride = src_stride;
  p.dst_stride = dst_stride;
  p.src_pages = src_pages;
  p.dst_pages = dst_pages;
  p.cu = cu;
  p.keep = keep;
  p.n_seqs = n_seqs;
  p.n_keep = n_keep;
  const cudaError_t e = launch_pdl(
      k_kv_move<true>, dim3((n_keep + kMoveTokens - 1) / kMoveTokens, 2 * kv->cfg.n_layers),
      dim3(kMoveThreads), 0, reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

dg_status_t dg_kv_fork_workspace_size(int n_pages, size_t* bytes) {
  if (!bytes || n_pages <= 0) return DG_ERR_INVALID_ARG;
  if (n_pages > kMaxForkPages) return DG_ERR_UNSUPPORTED;
  *bytes = fork_layout(n_pages).total;
  return DG_OK;
}

dg_status_t dg_kv_fork(const dg_kv_fork_t* f, void* workspace, size_t workspace_bytes,
                       dg_stream_t stream) {
  if (!f || f->n_pages <= 0 || f->row <= 0 || f->n_old < 0 || f->n_new < 0)
    return DG_ERR_INVALID_ARG;
  if (!page_size_ok(f->page_size) || f->n_pages > kMaxForkPages || f->n_old > kForkMax ||
      f->n_new > kForkMax || (int64_t)f->row * f->page_size > kMaxKvTokens ||
      f->row > (1 << 18))
    return DG_ERR_UNSUPPORTED;
  if (!f->ref_in || !f->ref_out || !f->short_by) return DG_ERR_INVALID_ARG;
  if (f->n_old && (!f->table_in || !f->lens_in)) return DG_ERR_INVALID_ARG;
  if (f->n_new && (!f->parent || !f->grow || !f->table_out || !f->lens_out || !f->copies))
    return DG_ERR_INVALID_ARG;
  for (const void* q : {(const void*)f->table_in, (const void*)f->lens_in, (const void*)f->ref_in,
                        (const void*)f->parent, (const void*)f->grow, (const void*)f->table_out,
                        (const void*)f->lens_out, (const void*)f->ref_out, (const void*)f->copies,
                        (const void*)f->short_by})
    if (!aligned(q, 4)) return DG_ERR_ALIGNMENT;
  if (f->n_old && f->n_new &&
      ((const void*)f->table_in == f->table_out || (const void*)f->lens_in == f->lens_out))
    return DG_ERR_INVALID_ARG;
  const ForkLayout L = fork_layout(f->n_pages);
  if (!workspace || workspace_bytes < L.total || !aligned(workspace, 16)) return DG_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  ForkParams p;
  p.f = *f;
  p.page_shift = log2_of(f->page_size);
  p.status = reinterpret_cast<DevStatus*>(ws);
  p.counts = reinterpret_cast<int32_t*>(ws + L.counts);
  p.users = reinterpret_cast<int32_t*>(ws + L.users);
  p.first = reinterpret_cast<int32_t*>(ws + L.first);
  const int most = f->n_old > f->n_new + 1 ? f->n_old : f->n_new + 1;
  const size_t smem = sizeof(Grow) * f->n_new + sizeof(int) * most;
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024)  // beside 5 KB of static shared memory
    e = cudaFuncSetAttribute(k_kv_fork, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(sizeof(Grow) * kForkMax + sizeof(int) * (kForkMax + 1)));
  if (e == cudaSuccess)
    e = launch_pdl(k_kv_fork, dim3(kForkCtas), dim3(kForkThreads), smem,
                   reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

dg_status_t dg_kv_fork_last_device_status(void* workspace, dg_stream_t stream,
                                          unsigned int* where, unsigned int* info) {
  if (!workspace) return DG_ERR_WORKSPACE;
  return read_status(workspace, stream, where, info);
}

}  // extern "C"
