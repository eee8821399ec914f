// Bookkeeping of forked and thinned sequences (include/dg_attn.h): the pages
// that the sequences of a group have in common, and the choice of the tokens
// that stay when a cache is thinned.
#include <algorithm>

#include "../../include/dg_attn.h"
#include "dg_attn_host.h"
#include "dg_common.cuh"

using namespace dg;
using namespace dg::host;

namespace {

enum : unsigned int { kSiteSharedLen = 56, kSiteSharedGroups = 57, kSiteSelectLen = 58,
                      kSiteSelectWait = 59 };

constexpr int kThinThreads = 1024;
constexpr int kSelectThreads = 1024;
constexpr unsigned kAllLanes = 0xffffffffu;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
// An int of another CTA's shared memory.
__device__ __forceinline__ int peer_int(const int* p, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Add `bytes` of ints to another CTA's, counted on a barrier of that CTA.
__device__ __forceinline__ void peer_add(const int* to, const int* from, int bytes,
                                         const uint64_t* bar, uint32_t rank) {
  uint32_t a, b;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(to)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile(
      "cp.reduce.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes.add.u32"
      " [%0], [%1], %2, [%3];" ::"r"(a),
      "r"(smem_u32(from)), "r"(bytes), "r"(b)
      : "memory");
}

// Sums over the block; `warps` holds one entry a warp.  Ends with a barrier.
__device__ __forceinline__ int block_sum(int v, int* warps) {
  v = __reduce_add_sync(kAllLanes, v);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  v = __reduce_add_sync(
      kAllLanes, (threadIdx.x & 31) < blockDim.x >> 5 ? warps[threadIdx.x & 31] : 0);
  __syncthreads();
  return v;
}
// Sum over the lanes before this one, and over all.
__device__ __forceinline__ int lanes_before(int v, int* total) {
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kAllLanes, incl, o);
    if ((threadIdx.x & 31) >= o) incl += x;
  }
  *total = __shfl_sync(kAllLanes, incl, 31);
  return incl - v;
}
// Sum over the threads before this one, and over all.  Ends with a barrier.
__device__ __forceinline__ int block_before(int v, int* warps, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int all;
  const int lanes = lanes_before(v, &all);
  if (lane == 0) warps[warp] = all;
  __syncthreads();
  const int w = lane < blockDim.x >> 5 ? warps[lane] : 0;
  const int before = __reduce_add_sync(kAllLanes, lane < warp ? w : 0);
  *total = __reduce_add_sync(kAllLanes, w);
  __syncthreads();
  return before + lanes;
}

// ------------------------------------------------------------------ shared

struct SharedParams {
  const int32_t* table;
  int64_t table_stride;
  const int32_t *lens, *cu, *groups;
  int32_t* prefix;
  int n_seqs, n_groups, page_shift, cap;
  DevStatus* status;
};

// prefix = min(page_size * (leading columns in which all rows of the group are
// equal), fewest tokens that a member had before this call).
//
// A block a group: 2.4 us for 8 sequences, 3.6 us for 512 of 40 groups (in a replayed
// graph, 2070 MHz; 11 to 17 for a call from Python), most of it the launch.  What is
// read is little (four bytes a page), so latency bounds it: a warp takes 128 columns
// of a member against the first one, the columns of all members before the next ones,
// and none past the nearest difference found.
__global__ void __launch_bounds__(kThinThreads) k_kv_shared(const __grid_constant__ SharedParams p) {
  __shared__ int least, bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (tid == 0) {
    least = p.cap;
    bad = 0;
  }
  pdl_wait();
  __syncthreads();
  // groups that are not ranges of sequences in ascending order share nothing
  for (int g = tid; g <= p.n_groups; g += kThinThreads) {
    const int a = __ldg(p.groups + g);
    const int b = g < p.n_groups ? __ldg(p.groups + g + 1) : p.n_seqs;
    if (a < 0 || a > b || b > p.n_seqs) bad = 1;
  }
  __syncthreads();
  if (bad) {
    for (int s = blockIdx.x * kThinThreads + tid; s < p.n_seqs; s += gridDim.x * kThinThreads)
      p.prefix[s] = 0;
    if (blockIdx.x == 0 && tid == 0)
      report(p.status, kDevBounds, kSiteSharedGroups, (unsigned)p.n_groups, (unsigned)p.n_seqs);
    return;
  }
  const int a = __ldg(p.groups + blockIdx.x), b = __ldg(p.groups + blockIdx.x + 1);
  if (blockIdx.x == 0)
    for (int s = tid; s < a; s += kThinThreads) p.prefix[s] = 0;
  if ((int)blockIdx.x == p.n_groups - 1)
    for (int s = b + tid; s < p.n_seqs; s += kThinThreads) p.prefix[s] = 0;
  if (b - a < 2) {
    if (b > a && tid == 0) p.prefix[a] = 0;
    return;
  }
  int past = p.cap;
  for (int s = a + tid; s < b; s += kThinThreads) {
    const int kv = __ldg(p.lens + s), n = __ldg(p.cu + s + 1) - __ldg(p.cu + s);
    if (kv < 0 || kv > p.cap || n < 0 || n > kv)
      report(p.status, kDevBounds, kSiteSharedLen, (unsigned)s, (unsigned)kv);
    past = min(past, max(0, min(max(kv, 0), p.cap) - max(n, 0)));
  }
  past = __reduce_min_sync(kAllLanes, past);
  if (lane == 0) atomicMin(&least, past);
  __syncthreads();
  past = least;
  __syncthreads();
  const int pages = (past + (1 << p.page_shift) - 1) >> p.page_shift;
  if (tid == 0) least = pages;  // now the first column that differs
  __syncthreads();
  constexpr int kCols = 128;
  const int32_t* first = p.table + a * p.table_stride;
  const long long tasks = (long long)(b - a - 1) * ((pages + kCols - 1) / kCols);
  for (long long t = warp; t < tasks; t += kThinThreads / 32) {
    const int c0 = (int)(t / (b - a - 1)) * kCols, m = (int)(t % (b - a - 1)) + 1;
    // Later tasks lie no further left.  One lane reads for all: the nearest difference
    // may move meanwhile, and a warp has to leave as one.
    const int end = __shfl_sync(kAllLanes, lane == 0 ? *(volatile int*)&least : 0, 0);
    if (c0 >= end) break;
    const int32_t* row = first + m * p.table_stride;
    int x[kCols / 32], y[kCols / 32], at = pages;
#pragma unroll
    for (int k = 0; k < kCols / 32; ++k) {
      const int c = c0 + lane + 32 * k;
      x[k] = c < pages ? __ldg(first + c) : 0;
      y[k] = c < pages ? __ldg(row + c) : 0;
    }
#pragma unroll
    for (int k = kCols / 32 - 1; k >= 0; --k)
      if (x[k] != y[k]) at = c0 + lane + 32 * k;
    at = __reduce_min_sync(kAllLanes, at);
    if (lane == 0 && at < pages) atomicMin(&least, at);
  }
  __syncthreads();
  const int prefix = min((int)min((long long)least << p.page_shift, (long long)past), past);
  for (int s = a + tid; s < b; s += kThinThreads) p.prefix[s] = prefix;
}

// ------------------------------------------------------------------ select

struct SelectParams {
  dg_kv_select_t s;
  DevStatus* status;
};

// An unsigned order of the weights: NaN above everything, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0xffffffffu;  // kOrderNan
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The weight of an order, but for NaN and the two zeros.
__device__ __forceinline__ float weight_of(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
constexpr uint32_t kOrderNan = 0xffffffffu, kOrderZero = 0x80000000u;

// Digits of the order, from the top: 11, 11 and 10 bits.
constexpr int kDigits = 3;
constexpr int kAllBins = 2048 + 2048 + 1024;
constexpr int kPlaces = 256;  // places of a warp on their way out
constexpr int kListed = 64;  // orders of a run that are listed at most
__device__ __forceinline__ int digit_shift(int d) { return d == 0 ? 21 : d == 1 ? 10 : 0; }
__device__ __forceinline__ int digit_bits(int d) { return d == 2 ? 10 : 11; }

// Kept of a sequence of L tokens, B = budget < L: the first `first`, the last
// `last`, and the m = B - first - last largest weights of those between, equal
// ones in the order of their places.  The m-th largest is found digit by digit
// of its order, a histogram each; what lies above it is kept, and of what
// equals it as much as is missing, from the front.  Then one pass in the order
// of the places, each kept token's rank from a running count.
//
// A cluster a sequence (one CTA where rows are short): each CTA takes a slice
// of the row and keeps its orders in shared memory; each adds its histogram to
// every CTA's, in the fabric between them.  The weights are read once.
//
// Instructions bound it, of the CTAs of the longest row (comparisons and votes go at
// half the rate or less): 48 rows of 8000 to 131072 cut to 16384 in 21 us (in a
// replayed graph, 2070 MHz; 21 to 28 for a call from Python), of which 5 go by with
// loading and the first digit, 4 with listing what has it, 5 with adding up and looking
// through the three histograms, 2 with counting and 4 with writing; 8 rows of up to
// 1500 in 6.5 us (a call 17 to 27, 8 where its outputs are given).  Measured and not
// kept, us for the first: other CTAs' histograms read bin by bin (103, clusters of 8) or
// added up bin by bin in the first CTA's (26; 92 with clusters of 8); two CTAs an SM of
// half the size (22 three to a row, 45 eight); four copies of a histogram against
// colliding additions (37, from 27: the hardware adds equal addresses at once); stores
// straight from the lanes (24); ranks of four rows of places by one scan instead of
// votes (22.5).
template <bool CACHED>
__global__ void __launch_bounds__(kSelectThreads, 1)
    k_kv_select(const __grid_constant__ SelectParams p) {
  // histograms of the slice, a digit each (they are sent from here), and its orders
  extern __shared__ __align__(16) int hists[];
  uint32_t* kept = reinterpret_cast<uint32_t*>(hists + kAllBins);
  __shared__ __align__(16) int sums[kAllBins];  // histograms of the cluster
  __shared__ uint64_t arrived[kDigits];
  __shared__ int warps[32], found[3], counts[2], abort_word;
  // of each run, the orders with the first digit of the m-th largest
  __shared__ uint32_t lists[CACHED ? kSelectThreads / 32 : 1][CACHED ? kListed : 1];
  const dg_kv_select_t& q = p.s;
  const int tid = threadIdx.x;
  const int ctas = (int)cluster_ctas(), rank = (int)cluster_rank();
  const int seq = blockIdx.x / ctas;
  pdl_trigger();
  pdl_wait();
  // kept tokens of the sequences before this one, and of all
  int before = 0, all = 0;
  for (int s = tid; s < q.n_seqs; s += kSelectThreads) {
    const int c = min(min(max(__ldg(q.lens + s), 0), q.width), q.budget);
    all += c;
    if (s < seq) before += c;
  }
  before = block_sum(before, warps);
  all = block_sum(all, warps);
  const int raw = __ldg(q.lens + seq);
  const int L = min(max(raw, 0), q.width), count = min(L, q.budget);
  if (rank == 0 && tid == 0) {
    if (raw < 0 || raw > q.width)
      report(p.status, kDevBounds, kSiteSelectLen, (unsigned)seq, (unsigned)raw);
    q.cu[seq] = before;
    q.lens_out[seq] = count;
    if (seq == q.n_seqs - 1) q.cu[q.n_seqs] = all;
  }
  const int64_t room = (int64_t)q.n_seqs * q.budget;
  for (int64_t i = all + (int64_t)blockIdx.x * kSelectThreads + tid; i < room;
       i += (int64_t)gridDim.x * kSelectThreads)
    q.keep[i] = -1;
  const float* row = q.weights + seq * q.weights_stride;
  int32_t* keep = q.keep + before;
  float* out = q.weights_out + seq * q.out_stride;
  const int wide = ctas * kSelectThreads, at = rank * kSelectThreads + tid;
  for (int i = count + at; i < q.budget; i += wide) out[i] = 0.f;
  if (L <= q.budget) {  // the same for every CTA of the cluster
    for (int i = at; i < L; i += wide) {
      keep[i] = i;
      out[i] = __ldg(row + i);
    }
    return;
  }
  for (int i = at; i < q.first; i += wide) {
    keep[i] = i;
    out[i] = __ldg(row + i);
  }
  for (int i = at; i < q.last; i += wide) {
    keep[count - q.last + i] = L - q.last + i;
    out[count - q.last + i] = __ldg(row + L - q.last + i);
  }
  int m = q.budget - q.first - q.last;
  if (m == 0) return;
  // this CTA's slice of the tokens between
  const int mid = L - q.first - q.last, each = (mid + ctas - 1) / ctas;
  const int lo = min(rank * each, mid), n = min(each, mid - lo);
  const float* src = row + q.first + lo;
  auto order = [&](int i) { return CACHED ? kept[i] : order_of(__ldg(src + i)); };
  for (int i = tid; i < kAllBins; i += kSelectThreads) hists[i] = sums[i] = 0;
  if (ctas > 1) {
    if (tid == 0) {
      abort_word = 0;
      for (int d = 0; d < kDigits; ++d) mbar_init(&arrived[d], 1);
      fence_mbar_init();
      for (int d = 0; d < kDigits; ++d)
        mbar_arrive_expect_tx(&arrived[d], ctas * (int)sizeof(int) << digit_bits(d));
    }
    fence_proxy_async_smem();
    cluster_sync();
  }
  __syncthreads();
  // A warp takes a run of rows of 128 places.
  constexpr int kAtOnce = kSelectThreads * 4;
  const int lane = tid & 31, warp = tid >> 5, run = (n + kAtOnce - 1) / kAtOnce * 128;
  // (zeros behind the last: no weight's order)
  const int full = CACHED ? (n + 127) / 128 * 128 : n;
  const int i0 = min(warp * run, full), i1 = min(i0 + run, full);
  int g_own = 0, e_own = 0;  // of its run: kept for sure, equal to the m-th largest
  bool few = false;          // those with the first digit are listed
  int listed = 0;
  uint32_t* mine = lists[CACHED ? warp : 0];
  uint32_t top = 0;          // the digits found so far
  for (int d = 0; d < kDigits; ++d) {
    const int shift = digit_shift(d), bits = digit_bits(d);
    int* hist = hists + (d << 11);
    if (d == 0) {
      if (CACHED && tid < full - n) kept[n + tid] = 0;
#pragma unroll 8
      for (int i = tid; i < n; i += kSelectThreads) {
        const uint32_t u = order_of(__ldg(src + i));
        if (CACHED) kept[i] = u;
        atomicAdd(&hist[u >> shift], 1);
      }
    } else if (few) {
      for (int i = lane; i < listed; i += 32) {
        const uint32_t u = mine[i];
        if (u >> (shift + bits) == top) atomicAdd(&hist[u >> shift & ((1u << bits) - 1)], 1);
      }
    } else {
#pragma unroll 8
      for (int i = tid; i < n; i += kSelectThreads) {
        const uint32_t u = order(i);
        if (u >> (shift + bits) == top) atomicAdd(&hist[u >> shift & ((1u << bits) - 1)], 1);
      }
    }
    if (ctas > 1) {  // every CTA's to every CTA
      fence_proxy_async_smem();
      __syncthreads();
      if (tid < ctas)
        peer_add(sums + (d << 11), hist, (int)sizeof(int) << bits, &arrived[d],
                 (rank + tid) % ctas);
      const bool ok = mbar_wait(&arrived[d], 0, &abort_word);
      if (__syncthreads_or(!ok)) {  // (the copies on their way still land here)
        if (tid == 0) report(p.status, kDevTimeout, kSiteSelectWait, (unsigned)seq, (unsigned)d);
        abort_word = 0;
        for (int e = d; e < kDigits; ++e) mbar_wait(&arrived[e], 0, &abort_word);
        cluster_sync();
        cluster_sync();
        return;
      }
      hist = sums + (d << 11);
    } else {
      __syncthreads();
    }
    // bins from the largest down, four a thread
    const int b0 = (1 << bits) - 1 - 4 * tid;
    const int4 four =
        b0 >= 0 ? *reinterpret_cast<const int4*>(hist + b0 - 3) : make_int4(0, 0, 0, 0);
    const int bin[4] = {four.w, four.z, four.y, four.x};
    const int here = bin[0] + bin[1] + bin[2] + bin[3];
    int total;
    int over = block_before(here, warps, &total);
    if (over < m && over + here >= m) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (over < m && over + bin[i] >= m) {
          found[0] = b0 - i;
          found[1] = m - over;
          found[2] = bin[i];
        }
        over += bin[i];
      }
    }
    __syncthreads();
    m = found[1];
    top = top << bits | (uint32_t)found[0];
    __syncthreads();
    if (CACHED && d == 0) {  // list those with this digit, if they are few in every run
      const uint32_t least = top << shift, most = least | ((1u << shift) - 1);
      const unsigned before = (1u << lane) - 1;
      for (int i = i0 + lane; i < i1; i += 128) {
        uint32_t u[4], row[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          u[k] = kept[i + 32 * k];
          g_own += u[k] > most;
          row[k] = __ballot_sync(kAllLanes, u[k] >= least && u[k] <= most);
        }
        if (row[0] | row[1] | row[2] | row[3]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at = listed + __popc(row[k] & before);
            if ((row[k] >> lane & 1u) && at < kListed) mine[at] = u[k];
            listed += __popc(row[k]);
          }
        }
      }
      few = !__syncthreads_or(listed > kListed);
      if (!few) g_own = 0;
    }
  }
  // What each run keeps, and what of it equals the m-th largest.
  if (few) {
    for (int i = lane; i < listed; i += 32) {
      g_own += mine[i] > top;
      e_own += mine[i] == top;
    }
  } else {
#pragma unroll 8
    for (int i = i0 + lane; i < i1; i += 32) {
      const uint32_t u = order(i);
      g_own += u > top;
      e_own += u == top;
    }
  }
  int above, equal;  // of the slice
  int gt = block_before(g_own, warps, &above), eq = block_before(e_own, warps, &equal);
  // (the lanes' counts lie between a warp's first lane and its own)
  gt = __shfl_sync(kAllLanes, gt, 0);
  eq = __shfl_sync(kAllLanes, eq, 0);
  if (ctas > 1) {  // and of the slices before
    if (tid == 0) {
      counts[0] = above;
      counts[1] = equal;
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      gt += peer_int(&counts[0], r);
      eq += peer_int(&counts[1], r);
    }
  }
  // Where all that equals the m-th largest is kept, which is where no other weight
  // equals it, one comparison says what stays, and votes give the ranks.  Places go
  // through shared memory (the histograms', which nobody reads any more), so that
  // stores of neighbouring lanes fall together.
  if (CACHED && found[2] == m) {
    uint16_t* places = reinterpret_cast<uint16_t*>(hists) + warp * kPlaces;
    const unsigned lanes = (1u << lane) - 1;
    keep += q.first + gt + eq;
    out += q.first + gt + eq;
    int some = 0;
    for (int i = i0 + lane; i - lane < i1; i += 128) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool stays = kept[i + 32 * k] >= top;
        const unsigned row = __ballot_sync(kAllLanes, stays);
        if (stays) places[some + __popc(row & lanes)] = (uint16_t)(i + 32 * k);
        some += __popc(row);
      }
      if (some > kPlaces - 128 || i - lane + 128 >= i1) {
        __syncwarp();
        for (int t = lane; t < some; t += 32) {
          const int place = places[t];
          const uint32_t u = kept[place];
          keep[t] = q.first + lo + place;
          // (where the order does not say, it is fetched again)
          out[t] = u == kOrderNan || u == kOrderZero ? __ldg(src + place) : weight_of(u);
        }
        __syncwarp();
        keep += some;
        out += some;
        some = 0;
      }
    }
    if (ctas > 1) cluster_sync();  // another CTA may still read this one's counts
    return;
  }
  // Ranks by a scan over the lanes, four places each.
#pragma unroll 2
  for (int i = i0; i < i1; i += 128) {
    uint32_t u[4];
    const int at = i + 4 * lane, in = min(4, i1 - at);  // places of this lane
    if (CACHED) {
      const uint4 x = *reinterpret_cast<const uint4*>(kept + at);  // (there is room behind the last)
      u[0] = x.x, u[1] = x.y, u[2] = x.z, u[3] = x.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = k < in ? order(at + k) : 0u;
    }
    int all, own = 0;  // larger ones; equal ones in the high half
#pragma unroll
    for (int k = 0; k < 4; ++k) own += k < in ? (u[k] > top ? 1 : u[k] == top ? 1 << 16 : 0) : 0;
    const int lanes = lanes_before(own, &all);
    int g = gt + (lanes & 0xffff), e = eq + (lanes >> 16);
    bool open = false;  // where the order does not say what the weight was
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool larger = k < in && u[k] > top, same = k < in && u[k] == top;
      if (larger || (same && e < m)) {
        const int to = q.first + g + min(e, m);
        keep[to] = q.first + lo + at + k;
        out[to] = weight_of(u[k]);
        open |= u[k] == kOrderNan || u[k] == kOrderZero;
      }
      g += larger;
      e += same;
    }
    if (__any_sync(kAllLanes, open)) {  // fetched again
      g = gt + (lanes & 0xffff), e = eq + (lanes >> 16);
#pragma unroll 1
      for (int k = 0; k < in; ++k) {
        const bool larger = order(at + k) > top, same = order(at + k) == top;
        if (larger || (same && e < m)) out[q.first + g + min(e, m)] = __ldg(src + at + k);
        g += larger;
        e += same;
      }
    }
    gt += all & 0xffff;
    eq += all >> 16;
  }
  // another CTA may still read this one's counts
  if (ctas > 1) cluster_sync();
}

// Weights that a CTA holds in shared memory at most (beside 49 KB).
constexpr int kSliceMost = 44 * 1024;

// CTAs of a sequence: so many that each can hold its slice, more where SMs would
// be left over, none with fewer than 20480 weights (us at the least of 2048 / 8192 /
// 20480 / 32768: 8 rows of 4096 10.1 / 7.4 / 7.4 / 7.4, of 16384 16.8 / 12.7 / 10.8 /
// 10.7, of 65536 19.0 / 19.2 / 16.1 / 18.3).  Rows that are not held are read again for
// every digit: 160 rows of 65536 in 62 us by two CTAs each, two rounds of them, 101 by one.
int select_ctas(int n_seqs, int width, int sms) {
  const int cached = (width + kSliceMost - 1) / kSliceMost;
  return std::max(1, std::min({8, std::max(sms / n_seqs, cached), (width + 20479) / 20480}));
}

}  // namespace

namespace dg {
namespace host {
cudaError_t prepare_select() {
  return cudaFuncSetAttribute(k_kv_select<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sizeof(int) * (kAllBins + kSliceMost));
}
}  // namespace host
}  // namespace dg

extern "C" {

dg_status_t dg_kv_shared(dg_kv_t* kv, const dg_kv_batch_t* batch, const int32_t* groups,
                         int n_groups, int32_t* prefix, dg_stream_t stream) {
  if (!kv || n_groups < 0) return DG_ERR_INVALID_ARG;
  const dg_status_t st = check_batch(batch, kv->cfg);
  if (st != DG_OK) return st;
  if (n_groups > kMaxSeqs) return DG_ERR_UNSUPPORTED;
  if (batch->n_seqs == 0) return DG_OK;
  if (!prefix || (n_groups && !groups)) return DG_ERR_INVALID_ARG;
  if (!aligned(prefix, 4) || !aligned(groups, 4)) return DG_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n_groups == 0)
    return cudaMemsetAsync(prefix, 0, sizeof(int32_t) * batch->n_seqs, s) == cudaSuccess
               ? DG_OK : DG_ERR_CUDA;
  SharedParams p;
  p.table = batch->page_table;
  p.table_stride = batch->table_stride;
  p.lens = batch->lens;
  p.cu = batch->cu;
  p.groups = groups;
  p.prefix = prefix;
  p.n_seqs = batch->n_seqs;
  p.n_groups = n_groups;
  p.page_shift = log2_of(kv->cfg.page_size);
  p.cap = batch->max_pages * kv->cfg.page_size;
  p.status = static_cast<DevStatus*>(kv->status);
  return launch_pdl(k_kv_shared, dim3(n_groups), dim3(kThinThreads), 0, s, p) == cudaSuccess
             ? DG_OK : DG_ERR_CUDA;
}

dg_status_t dg_kv_select(dg_kv_t* kv, const dg_kv_select_t* q, dg_stream_t stream) {
  if (!kv || !q || q->n_seqs < 0 || q->width < 0 || q->budget < 0 || q->first < 0 || q->last < 0)
    return DG_ERR_INVALID_ARG;
  if (q->n_seqs == 0) return DG_OK;
  if (q->n_seqs > kMaxSeqs || q->width > kMaxKvTokens) return DG_ERR_UNSUPPORTED;
  SelectParams p;
  p.s = *q;
  if (p.s.budget > p.s.width) p.s.budget = p.s.width;
  if ((int64_t)q->first + q->last > q->budget) return DG_ERR_INVALID_ARG;
  if ((int64_t)q->n_seqs * p.s.budget > kMaxKvTokens) return DG_ERR_UNSUPPORTED;
  if (!q->lens || !q->cu || !q->lens_out) return DG_ERR_INVALID_ARG;
  if (p.s.budget > 0 && (!q->weights || !q->keep || !q->weights_out)) return DG_ERR_INVALID_ARG;
  if (q->weights_stride < 0 || q->out_stride < 0 ||
      (q->n_seqs > 1 && (q->weights_stride < q->width || q->out_stride < p.s.budget)))
    return DG_ERR_INVALID_ARG;
  for (const void* x : {(const void*)q->weights, (const void*)q->lens, (const void*)q->keep,
                        (const void*)q->cu, (const void*)q->lens_out, (const void*)q->weights_out})
    if (!aligned(x, 4)) return DG_ERR_ALIGNMENT;
  if (p.s.budget > 0 && q->weights == q->weights_out) return DG_ERR_INVALID_ARG;
  if (q->lens == q->lens_out || q->lens == q->cu) return DG_ERR_INVALID_ARG;
  const int ctas = select_ctas(q->n_seqs, q->width, kv->sms);
  const int slice = (q->width + ctas - 1) / ctas;
  const bool cached = slice <= kSliceMost;
  p.status = static_cast<DevStatus*>(kv->status);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(q->n_seqs * ctas);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = sizeof(int) * (kAllBins + (cached ? round_up(slice, 128) : 0));
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, cached ? k_kv_select<true> : k_kv_select<false>, p);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

}  // extern "C"
