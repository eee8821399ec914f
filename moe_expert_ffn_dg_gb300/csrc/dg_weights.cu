// Attention weight that each cached token receives from new tokens, on sm_103a.
//
//   w'[j] = decay w[j] + sum over heads h and tokens i that see j of
//           exp(scale q_ih k_j - lse_ih)
//
// with the log-sums that the attention has written: no running maximum, no
// values.  Keys stand in the rows of the product, S^T = K Q^T, so that a thread
// owns a key (a lane of tensor memory) and adds its weights up in a register;
// query rows (the G heads of a group packed with their tokens, row = token * G +
// head of the group) are the columns.
//
// A work item is 256 keys of a sequence (two tiles of 128) against all of its rows
// that see them, head after head; its units are single query tiles.  All units of a
// call lie in one line (sequences, blocks of keys, heads, tiles) and every CTA takes
// a contiguous range, so that long and short sequences balance alike.  An item that
// crosses a range boundary leaves fp32 partial sums in the workspace, joined in a
// fixed order by k_weights_join: the result does not depend on which CTA comes
// first.
//
// What bounds it, on one GB300 (us of a call in a replayed graph, in brackets of calls
// from Python whose inputs change): memory for single tokens (64 of them over 471k
// cached ones, 32 query heads on 8 of 128: 172 us [173 to 179], 6.2 TB/s); shared
// memory for many rows, of which an MMA of 128 x 128 with both operands there takes
// all 128 bytes a cycle while query tiles are copied in and log-sums read (4096 tokens
// behind 12288, same heads: 374 us at 1995 MHz [368 to 413, by the clock under the
// power limit], 1.17 to 1.31 PFLOP/s; 8 canvases of 256 over 36k, 16 heads on 8 of
// 256: 89 us [91 to 93], with the wait for a buffer that the two accumulators of that
// size cost).  Heads of a group that do not divide a tile leave columns without a row,
// so that all of its tiles are masked: the same 4096 with 3, 5 and 7 query heads on
// each of 8 in 498, 824 and 1141 us, 0.73 PFLOP/s (2, 4 and 8: 193, 368 and 747).
// Measured and not kept, us for the 4096 when they took 359: the key tiles in tensor
// memory, whose score tiles then are one fewer and wait for one another (391 to 418);
// eight warps that add 128 columns each (374); an MMA issuer a key tile (354, but 73
// for the canvases, then at 69); 512 keys an item (455); log-sums fetched by every warp
// for itself (480); all 64 columns of a warp loaded at once, which spills (566).
//
// How exact it is: an addition of the tensor core truncates, and loses less than 2^-23
// of the partial sum, so that a weight is off by a factor that grows with the scores:
// at most 2^-23 scale times the sizes of all partial sums, and 2^-24 |lse| for the
// scaled log-sum's rounding.  Root mean square for 512 rows of queries three times
// normal over 1500 normal keys, bf16 and fp16: at head sizes 64 and 128 6e-7 to 1.2e-6
// of the weights with log-sums from 64 bits, 3e-7 to 4e-7 with the attention's own,
// whose scores lose the same; at 256, where the attention has one accumulator and this
// kernel two, 1.0e-6 to 1.5e-6 with either.
//
// Warps: eight (few rows) or sixteen for exponentials and sums, then one each for
// copies of keys, for the MMAs (it owns the tensor memory), for copies of
// queries and for log-sums.
#include <math.h>
#include <string.h>

#include "../../include/dg_attn.h"
#include "dg_attn_dev.cuh"
#include "dg_attn_host.h"
#include "dg_common.cuh"
#include "dg_tmem.cuh"

using namespace dg;
using namespace dg::host;

namespace {

// Sites of the device status word.
enum : unsigned int {
  kSiteWeightLoad = 40, kSiteWeightMma = 41, kSiteWeightSum = 42, kSiteWeightDrain = 43,
  kSiteWeightPage = 44, kSiteWeightLen = 45,
};

struct WeightParams {
  CUtensorMap qm, km;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  int64_t table_stride;
  int n_seqs, cap, n_tokens, n_pages, page_shift;
  int kv_heads, group, step;  // step: tokens of a query tile
  int q_box;                  // tokens of a query box
  int left, right;
  float scale2;  // scale log2 e
  const float* lse;
  const float* w_in;
  float* w_out;
  int64_t in_stride, out_stride;
  int width;
  float decay;
  int fresh;
  float* part;     // [2 ctas][256]
  WeightRec* rec;  // [ctas]
  DevStatus* status;
};

template <int D, int QN>
struct Cfg {
  static constexpr int kChunks = D == 64 ? 1 : 2;         // 64-column chunks of a stage
  static constexpr int kParts = D / 64 / kChunks;         // stages of a tile
  static constexpr int kKeyBytes = kKeys * 128 * kChunks;  // a stage of a key tile
  static constexpr int kRowBytes = QN * 128 * kChunks;    // a stage of a query tile
  static constexpr int kKeyStages = QN == 16 ? (D == 64 ? 12 : 6) : (D == 64 ? 6 : 4);
  static constexpr int kRowStages = QN == 16 ? 6 : (D == 64 ? 7 : 3);
  static constexpr size_t kSmem = (size_t)kKeyStages * kKeyBytes + (size_t)kRowStages * kRowBytes;
  // Score buffers of a key tile, and accumulators of each: the tensor core's additions
  // truncate, and of half the products each they lose less than half as much (head size
  // 256, with log-sums from 64 bits: 1.0e-6 to 1.5e-6 of the weights for 2.1e-6 to
  // 2.9e-6; with those of the attention, which has one accumulator, 1.1e-6 to 1.4e-6 for
  // 5e-7 to 6e-7).  It leaves no room for a second buffer: 8 canvases 92 us for 77; one
  // key tile after the other, for both by a part of the query tile at a time: as long.
  static constexpr int kAccs = D == 256 ? 2 : 1;
  static constexpr int kBufs = QN == 16 ? 4 : 2 / kAccs;
  static constexpr uint32_t kTmem = 2 * kBufs * kAccs * QN;
  // Barriers of a buffer: one for both key tiles, or, where a tile has no second
  // buffer, one each, so that one tile's products run while the other's are read.
  static constexpr int kBars = kBufs == 1 ? 2 : 1;
  // Warpgroups that share a key tile's columns.  Two, 64 columns each: with one
  // the latency of the loads and exponentials shows.
  static constexpr int kColGroups = QN == 16 ? 1 : 2;
  static constexpr int kSumWarps = 8 * kColGroups;
  static constexpr int kThreads = 32 * (kSumWarps + 4);
};

struct Seq {
  int n0, n, kv, blocks;
};

__device__ __forceinline__ Seq load_seq(const WeightParams& p, int b) {
  const int a = __ldg(p.cu + b), e = __ldg(p.cu + b + 1), kv = __ldg(p.lens + b);
  Seq s;
  s.n0 = min(max(a, 0), p.n_tokens);
  s.n = max(min(e, p.n_tokens) - s.n0, 0);
  s.kv = min(max(kv, 0), p.cap);
  s.blocks = (min(s.kv, p.width) + kWeightKeys - 1) / kWeightKeys;
  return s;
}

// Query tiles [x, x + y) of which some token sees some key of block kb.
__device__ __forceinline__ int2 tile_range(const WeightParams& p, const Seq& s, int kb) {
  const int k0 = kb * kWeightKeys, k1 = min(k0 + kWeightKeys, s.kv);
  const int at = s.kv - s.n;  // position of the first token
  const int lo = p.right < 0 ? 0 : max(0, k0 - p.right - at);
  const int hi = p.left < 0 ? s.n - 1 : min(s.n - 1, k1 - 1 + p.left - at);
  if (lo > hi) return make_int2(0, 0);
  const int t = (unsigned)lo / (unsigned)p.step;
  return make_int2(t, (unsigned)hi / (unsigned)p.step - t + 1);
}

// Units of an item: its tiles in every head; one where nothing is seen and the
// weights only decay.
__device__ __forceinline__ long long item_units(const WeightParams& p, int tiles) {
  return max((long long)tiles * p.kv_heads, 1ll);
}

// What a CTA does with one head of an item.
struct Seg {
  int b, kb, head;
  int n0, n, kv;
  int t0, tiles;     // query tiles (may be none)
  bool first, last;  // holds the item's first / last unit
  bool begins, ends; // the first / last segment of the item in this CTA
  long long end;     // unit after the item's last one (where first)
};

struct Start {
  int b, kb;
  long long skip, u, end, total;
  int ctas;
};

// Walk over the segments of a range of units; the same in every role.
struct Walk {
  int b, kb, h, q;  // sequence, block, head, tile of the item's range
  int2 t;
  long long u, end;
  Seq s;
  bool fresh;
  __device__ __forceinline__ void begin(const WeightParams& p, const Start& st) {
    b = st.b;
    kb = st.kb;
    u = st.u;
    end = st.end;
    h = q = 0;
    fresh = true;
    if (u >= end) return;
    s = load_seq(p, b);
    t = tile_range(p, s, kb);
    if (t.y) {
      h = (int)(st.skip / t.y);
      q = (int)(st.skip - (long long)h * t.y);
    }
  }
  __device__ __forceinline__ bool next(const WeightParams& p, Seg& g) {
    if (u >= end) return false;
    g.b = b;
    g.kb = kb;
    g.head = h;
    g.n0 = s.n0;
    g.n = s.n;
    g.kv = s.kv;
    g.first = h == 0 && q == 0;
    g.begins = fresh;
    g.end = u + item_units(p, t.y);
    g.t0 = t.x + q;
    g.tiles = (int)min((long long)(t.y - q), end - u);
    u += max(g.tiles, 1);
    q += g.tiles;
    if (q == t.y) {
      q = 0;
      ++h;
    }
    g.last = h == p.kv_heads || t.y == 0;
    fresh = g.last;
    g.ends = g.last || u >= end;
    if (g.last && u < end) {
      h = 0;
      ++kb;
      while (kb >= s.blocks) {  // ends: there are units left
        kb = 0;
        s = load_seq(p, ++b);
      }
      t = tile_range(p, s, kb);
    }
    return true;
  }
};

// Where this CTA's range of units begins.  Sequences' costs go through `cost`
// (shared memory, n_seqs entries).  All threads; ends with a barrier.
__device__ __forceinline__ void find_start(const WeightParams& p, long long* cost, Start* out) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < 256) {
    int lps = 32;  // lanes a sequence
    while (lps > 1 && lps * p.n_seqs > 256) lps >>= 1;
    const int per = 256 / lps, sub = tid % lps;
    for (int s0 = 0; s0 < p.n_seqs; s0 += per) {
      const int b = s0 + tid / lps;
      long long c = 0;
      if (b < p.n_seqs) {
        const Seq s = load_seq(p, b);
        for (int kb = sub; kb < s.blocks; kb += lps) c += item_units(p, tile_range(p, s, kb).y);
        if (blockIdx.x == 0 && sub == 0) {
          const int a = __ldg(p.cu + b), e = __ldg(p.cu + b + 1), kv = __ldg(p.lens + b);
          if (a < 0 || e < a || e > p.n_tokens || kv < 0 || kv > p.cap || kv > p.width)
            report(p.status, kDevBounds, kSiteWeightLen, (unsigned)b, (unsigned)kv);
        }
      }
      for (int o = lps >> 1; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
      if (b < p.n_seqs && sub == 0) cost[b] = c;
    }
  }
  __syncthreads();
  if (tid < 32) {
    const int ch = (p.n_seqs + 31) / 32;
    const int b0 = min(lane * ch, p.n_seqs), b1 = min(b0 + ch, p.n_seqs);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += cost[b];
    long long incl = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const long long total = __shfl_sync(0xffffffffu, incl, 31);
    const int ctas = (int)min((long long)gridDim.x, total);
    const int c = blockIdx.x;
    Start st{0, 0, 0, 0, 0, total, ctas};
    if (c < ctas) {
      st.u = c * total / ctas;
      st.end = (c + 1) * total / ctas;
    }
    if (st.u < st.end) {
      long long r = st.u;
      const bool mine = r >= incl - sum && r < incl;
      const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
      int b = b0;
      if (mine) {
        r -= incl - sum;
        while (r >= cost[b]) r -= cost[b++];
      }
      st.b = __shfl_sync(0xffffffffu, b, src);
      r = __shfl_sync(0xffffffffu, r, src);
      const Seq s = load_seq(p, st.b);
      for (int base = 0; base < s.blocks; base += 32) {
        const int kb = base + lane;
        const long long cc = kb < s.blocks ? item_units(p, tile_range(p, s, kb).y) : 0;
        long long in = cc;
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, in, o);
          if (lane >= o) in += v;
        }
        const long long all = __shfl_sync(0xffffffffu, in, 31);
        if (r < all) {
          const int l = __ffs(__ballot_sync(0xffffffffu, r < in)) - 1;
          st.kb = base + l;
          st.skip = r - __shfl_sync(0xffffffffu, in - cc, l);
          break;
        }
        r -= all;
      }
    }
    if (lane == 0) *out = st;
  }
  fence_proxy_async_smem();  // `cost` lies where copies will land
  __syncthreads();
}

// A position in a ring of N stages.
template <int N>
struct Cursor {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == N) {
      st = 0;
      ph ^= 1u;
    }
  }
};

// The sum of 16 columns each of two accumulators.
__device__ __forceinline__ void tmem_add16(uint32_t a, uint32_t b, float (&v)[16]) {
  uint32_t x[16], y[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]),
        "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]),
        "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]),
        "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]),
        "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3]),
        "=r"(y[4]), "=r"(y[5]), "=r"(y[6]), "=r"(y[7]),
        "=r"(y[8]), "=r"(y[9]), "=r"(y[10]), "=r"(y[11]),
        "=r"(y[12]), "=r"(y[13]), "=r"(y[14]), "=r"(y[15])
      : "r"(a), "r"(b)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(x[i]) + __uint_as_float(y[i]);
}

// A sum that carries what its additions round away.
struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
  }
  // (the difference of an infinite sum is no number)
  __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
};

// The new weight of key j of a sequence.
__device__ __forceinline__ void write_weight(const WeightParams& p, int b, int n, int kv, int j,
                                             float sum) {
  if (j >= kv || j >= p.width) return;
  const bool old = j < kv - n || !p.fresh;
  const float w = old && p.decay != 0.f ? p.w_in[b * p.in_stride + j] : 0.f;
  p.w_out[b * p.out_stride + j] = fmaf(p.decay, w, sum);
}

template <int D, int QN, bool FP16>
__global__ void __launch_bounds__(Cfg<D, QN>::kThreads, 1) k_weights(const __grid_constant__ WeightParams p) {
  using C = Cfg<D, QN>;
  constexpr int NK = C::kKeyStages, NR = C::kRowStages, NB = C::kBufs, PARTS = C::kParts;
  constexpr int NA = C::kAccs, KB = C::kBars;
  constexpr int LS = NB + 1;  // query tiles whose log-sums are held
  constexpr int CG = C::kColGroups, W0 = C::kSumWarps;  // W0: first of the other warps
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t keys = smem_u32(smem), rows = keys + NK * C::kKeyBytes;
  __shared__ uint64_t k_full[NK], k_empty[NK], q_full[NR], q_empty[NR];
  __shared__ uint64_t s_full[NB * KB], s_empty[NB * KB], drain;
  __shared__ uint64_t x_full[2], x_empty[2];    // sums of a key tile's second column group
  __shared__ float xch[CG == 2 ? kWeightKeys : 1];
  __shared__ __align__(16) float lse[LS][QN];  // -lse log2 e of a query tile
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_word;
  __shared__ Start start;
  volatile int* abort_flag = &abort_word;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (keys & 1023u) {  // the swizzle needs it; the declaration asks for it
    if (tid == 0) report(p.status, kDevBounds, kSiteWeightLoad, keys, 0u);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < NB * KB; ++i) {
      mbar_init(&s_full[i], 2);  // the products, and the log-sums
      mbar_init(&s_empty[i], W0 / KB);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&x_full[i], 4);
      mbar_init(&x_empty[i], 4);
    }
    mbar_init(&drain, 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (tid == W0 * 32) {
    tma_prefetch_map(&p.qm);
    tma_prefetch_map(&p.km);
  }
  if (warp == W0 + 1) {
    tmem_alloc(&tmem_holder, C::kTmem);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  find_start(p, reinterpret_cast<long long*>(smem), &start);
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  Walk w;
  w.begin(p, start);
  Seg g;
  // key tiles of a segment's block
  auto tiles_of = [](const Seg& s) { return s.kv - s.kb * kWeightKeys > kKeys ? 2 : 1; };

  if (warp == W0) {
    // ---------------------------------------------------------------- keys
    const bool leader = elect_one();
    const int piece_shift = min(p.page_shift, 7), piece = 1 << piece_shift;
    const int per = kKeys >> piece_shift;  // boxes of a tile and chunk
    Cursor<NK> c;
    int used = 0;
    bool ok = true;
    int ids = p.n_pages, seen_b = -1, seen_kb = -1;
    while (ok && w.next(p, g)) {
      if (g.tiles == 0) continue;
      // Keys that some token of the sequence sees; others' pages may be gone.
      const int at = g.kv - g.n;
      const int lo = p.left < 0 ? 0 : max(0, at - p.left);
      if (g.b != seen_b || g.kb != seen_kb) {  // the same for all heads
        seen_b = g.b;
        seen_kb = g.kb;
        ids = -1;  // nothing to copy
        const int key = g.kb * kWeightKeys + (lane << piece_shift);
        const int pg = key >> p.page_shift;
        if (lane < 2 * per && key < g.kv && ((pg + 1) << p.page_shift) > lo) {
          ids = __ldg(p.table + (int64_t)g.b * p.table_stride + pg);
          if ((unsigned)ids >= (unsigned)p.n_pages) {
            report(p.status, kDevBounds, kSiteWeightPage, (unsigned)g.b, (unsigned)ids);
            ids = p.n_pages;  // the copy reads zeros
          }
        }
      }
      const int nt = tiles_of(g);
      for (int x = 0; x < PARTS && ok; ++x)
        for (int kt = 0; kt < nt; ++kt) {
          const unsigned live =
              __ballot_sync(0xffffffffu, ids >= 0 && lane >= kt * per && lane < (kt + 1) * per);
          const bool here = mbar_wait(&k_empty[c.st], c.ph ^ 1u, abort_flag);
          ok = __all_sync(0xffffffffu, here);
          if (!ok) break;
          if (leader)
            mbar_arrive_expect_tx(&k_full[c.st], __popc(live) * piece * 128 * C::kChunks);
          for (int r = 0; r < per; ++r) {
            const int l = kt * per + r;
            const int id = __shfl_sync(0xffffffffu, ids, l);
            if (leader && (live >> l & 1u)) {
              const int key = g.kb * kWeightKeys + (l << piece_shift);
#pragma unroll
              for (int i = 0; i < C::kChunks; ++i)
                tma_load_4d(&p.km, &k_full[c.st],
                            keys + c.st * C::kKeyBytes + i * (kKeys * 128) + (r << piece_shift) * 128,
                            (x * C::kChunks + i) * 64, g.head, key & ((1 << p.page_shift) - 1), id);
            }
          }
          __syncwarp();
          c.next();
          ++used;
        }
    }
    if (!ok) {
      if (lane == 0) report(p.status, kDevTimeout, kSiteWeightLoad, (unsigned)used, 8u);
      *abort_flag = 1;
    }
    // no copy may still be landing when the CTA exits
    if (leader) {
      bool done = true;
      for (int i = max(0, used - NK); i < used && done; ++i)
        done = wait_drain(&k_full[i % NK], (uint32_t)(i / NK) & 1u);
      if (!done && ok) report(p.status, kDevTimeout, kSiteWeightDrain, 8u, 0u);
    }
  } else if (warp == W0 + 2) {
    // ------------------------------------------------------------- queries
    const bool leader = elect_one();
    Cursor<NR> c;
    int used = 0;
    bool ok = true;
    while (ok && w.next(p, g))
      for (int t = 0; t < g.tiles && ok; ++t)
        for (int x = 0; x < PARTS; ++x) {
          const bool here = mbar_wait(&q_empty[c.st], c.ph ^ 1u, abort_flag);
          ok = __all_sync(0xffffffffu, here);
          if (!ok) break;
          if (leader) {
            mbar_arrive_expect_tx(&q_full[c.st], C::kChunks * 128 * p.group * p.q_box);
#pragma unroll
            for (int i = 0; i < C::kChunks; ++i)
              tma_load_3d(&p.qm, &q_full[c.st], rows + c.st * C::kRowBytes + i * (QN * 128),
                          (x * C::kChunks + i) * 64, g.head * p.group, g.n0 + (g.t0 + t) * p.step);
          }
          __syncwarp();
          c.next();
          ++used;
        }
    if (!ok) {
      if (lane == 0) report(p.status, kDevTimeout, kSiteWeightLoad, (unsigned)used, 10u);
      *abort_flag = 1;
    }
    if (leader) {
      bool done = true;
      for (int i = max(0, used - NR); i < used && done; ++i)
        done = wait_drain(&q_full[i % NR], (uint32_t)(i / NR) & 1u);
      if (!done && ok) report(p.status, kDevTimeout, kSiteWeightDrain, 10u, 0u);
    }
  } else if (warp == W0 + 3) {
    // ------------------------------------------------------------ log-sums
    // Fetched a tile ahead, written when the tile's score buffer is free: all warps
    // have then taken the scores of tile T - NB, and done with those before it; a
    // place is used again after NB + 1 tiles.
    constexpr int NL = (QN + 31) / 32;
    const int heads = p.kv_heads * p.group;
    int tok[NL], off[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int c = lane + 32 * i;
      tok[i] = (unsigned)c / (unsigned)p.group;
      off[i] = tok[i] * heads + c % p.group;
      if (c >= QN || tok[i] >= p.step) tok[i] = 1 << 30;  // no row
    }
    float ahead[NL];
    int t = 0;
    bool ok = true;
    auto fetch = [&] {  // the next tile's, if there is one
      ++t;
      while (t >= g.tiles) {
        if (!w.next(p, g)) return false;
        t = 0;
      }
      const int i0 = (g.t0 + t) * p.step;
      const float* src = p.lse + (int64_t)(g.n0 + i0) * heads + g.head * p.group;
#pragma unroll
      for (int i = 0; i < NL; ++i)
        ahead[i] = tok[i] < g.n - i0 ? __ldg(src + off[i]) : 0.f;  // no row: any finite number
      return true;
    };
    g.tiles = 0;
    bool more = fetch();
    Cursor<NB> sc;
    Cursor<LS> lc;
    while (more) {
      float now[NL];
#pragma unroll
      for (int i = 0; i < NL; ++i) now[i] = ahead[i];
      more = fetch();
      bool here = mbar_wait(&s_empty[sc.st * KB], sc.ph ^ 1u, abort_flag);
      if (KB == 2) here = here && mbar_wait(&s_empty[sc.st * KB + KB - 1], sc.ph ^ 1u, abort_flag);
      ok = __all_sync(0xffffffffu, here);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < NL; ++i)
        if (QN % 32 == 0 || lane < QN) lse[lc.st][lane + 32 * i] = -1.4426950408889634f * now[i];
      __syncwarp();
      if (lane < KB) mbar_arrive(&s_full[sc.st * KB + lane]);
      sc.next();
      lc.next();
    }
    if (!ok) {
      if (lane == 0) report(p.status, kDevTimeout, kSiteWeightLoad, 0u, 11u);
      *abort_flag = 1;
    }
  } else if (warp == W0 + 1) {
    // ---------------------------------------------------------- MMA issuer
    if (elect_one()) {
      Cursor<NK> kc;
      Cursor<NR> qc;
      Cursor<NB> sc;
      bool ok = true, issued = false;
      int at = 0;
      auto need = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && mbar_wait(bar, parity, abort_flag);
        return ok;
      };
      const uint32_t key_lo = desc_lo(keys, 16), row_lo = desc_lo(rows, 16);
      while (ok && w.next(p, g)) {
        const int nt = tiles_of(g);
        const Cursor<NK> k0 = kc;  // this segment's first key stage
        for (int t = 0; t < g.tiles && ok; ++t) {
          const int live = min(p.step, g.n - (g.t0 + t) * p.step) * p.group;
          const uint32_t idesc =
              idesc_16<FP16>(kKeys, 0, false) | ((uint32_t)((live + 15) & ~15) >> 3 << 17);
          const bool last = t == g.tiles - 1;
          if (KB == 1 && !need(&s_empty[sc.st], sc.ph ^ 1u)) break;
          Cursor<NK> k = k0;
          for (int x = 0; x < PARTS && ok; ++x) {
            if (!need(&q_full[qc.st], qc.ph)) break;
            const uint32_t b = row_lo + qc.st * (C::kRowBytes / 16);
            for (int kt = 0; kt < nt; ++kt) {
              if (t == 0 && !need(&k_full[k.st], k.ph)) break;
              if (KB == 2 && x == 0 && !need(&s_empty[sc.st * KB + kt], sc.ph ^ 1u)) break;
              tc_fence_after();
              const uint32_t a = key_lo + k.st * (C::kKeyBytes / 16);
              const uint32_t d = tmem + ((kt * NB + sc.st) * NA + x % NA) * QN;
#pragma unroll
              for (int i = 0; i < C::kChunks * 4; ++i)
                umma_ss<false>(d, a + ((i >> 2) * (kKeys * 128) + 32 * (i & 3)) / 16,
                               b + ((i >> 2) * (QN * 128) + 32 * (i & 3)) / 16, idesc,
                               NA == PARTS ? i : x | i);
              issued = true;
              if (KB == 2 && x == PARTS - 1) umma_commit(&s_full[sc.st * KB + kt]);
              if (last) umma_commit(&k_empty[k.st]);
              k.next();
            }
            if (!ok) break;
            umma_commit(&q_empty[qc.st]);
            qc.next();
          }
          if (!ok) break;
          if (KB == 1) umma_commit(&s_full[sc.st]);
          if (KB == 2 && nt == 1) {  // the second tile's warps go through it all the same
            if (!need(&s_empty[sc.st * KB + 1], sc.ph ^ 1u)) break;
            umma_commit(&s_full[sc.st * KB + 1]);
          }
          sc.next();
          if (last) kc = k;
          ++at;
        }
      }
      if (!ok) {
        report(p.status, kDevTimeout, kSiteWeightMma, (unsigned)at, 0u);
        *abort_flag = 1;
      }
      // every MMA issued here must have completed before TMEM is released
      if (issued) {
        umma_commit(&drain);
        if (!wait_drain(&drain, 0u)) report(p.status, kDevTimeout, kSiteWeightDrain, 9u, 0u);
      }
    }
  } else {
    // ---------------------------------------------------- weights and sums
    constexpr int NC = QN / CG;  // columns of a thread
    const int kt = warp / (4 * CG), cg = (warp >> 2) % CG, quarter = warp & 3;
    const uint32_t ts = tmem + ((uint32_t)(quarter * 32) << 16) + kt * NB * NA * QN + cg * NC;
    const uint64_t sc2 = f2(p.scale2, p.scale2);
    const int mine = kt * kKeys + quarter * 32 + lane;  // key of the block
    Cursor<NB> sc;
    Cursor<LS> lc;
    bool ok = true;
    int at = 0, items = 0;
    Sum sum;
    WeightRec rec{0, 0, 0};
    bool begun = false;  // the item's first unit is this CTA's
    long long item_end = 0;
    while (ok && w.next(p, g)) {
      if (g.begins) {
        sum = Sum();
        begun = g.first;
        item_end = g.end;
      }
      const int key = g.kb * kWeightKeys + mine;
      const int pos = g.kv - g.n;
      // Tiles [full0, full1) of the segment whose tokens all see all keys of this
      // warp need no mask.
      const int w1 = key - lane + 31;  // its last key
      const int f0 = (p.right < 0 ? 0 : max(0, w1 - p.right - pos)) - g.t0 * p.step;
      const int f1 = w1 >= g.kv || p.step * p.group != QN
                         ? 0
                         : (p.left < 0 ? g.n : min(g.n, w1 - 31 + p.left - pos + 1)) - g.t0 * p.step;
      const int full0 = f0 <= 0 ? 0 : (unsigned)(f0 + p.step - 1) / (unsigned)p.step;
      const int full1 = f1 <= 0 ? 0 : (unsigned)f1 / (unsigned)p.step;
      const bool none = key - lane >= g.kv;  // no keys of this warp
      for (int t = 0; t < g.tiles; ++t) {
        const int bar = sc.st * KB + (KB == 2 ? kt : 0);
        const bool here = mbar_wait(&s_full[bar], sc.ph, abort_flag);
        ok = __all_sync(0xffffffffu, here);
        if (!ok) break;
        tc_fence_after();
        // columns at a time: 64 would spill
        constexpr int W = NC < 32 || NA == 2 ? 16 : 32;
        const float* ls = lse[lc.st] + cg * NC;
        uint64_t acc[4] = {0, 0, 0, 0};
        auto taken = [&] {  // the scores have been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[bar]);
        };
        auto load = [&](int c, float (&s)[W]) {
          const uint32_t at = ts + sc.st * NA * QN + c;
          if constexpr (NA == 2) tmem_add16(at, at + QN, s);
          else if constexpr (W == 16) tmem_ld16(at, s);
          else tmem_load32(at, s);
          if (c + W == NC) taken();
        };
        auto weigh = [&](float (&s)[W], int c) {
#pragma unroll
          for (int e = 0; e < W; e += 4) {
            const float4 l = *reinterpret_cast<const float4*>(ls + c + e);
            const float2 x = unf2(fma2(f2(s[e], s[e + 1]), sc2, f2(l.x, l.y)));
            const float2 y = unf2(fma2(f2(s[e + 2], s[e + 3]), sc2, f2(l.z, l.w)));
            s[e] = exp2_fast(x.x);
            s[e + 1] = exp2_fast(x.y);
            s[e + 2] = exp2_fast(y.x);
            s[e + 3] = exp2_fast(y.y);
          }
        };
        auto gather = [&](const float (&s)[W]) {
#pragma unroll
          for (int e = 0; e < W; e += 2)
            acc[e / 2 & 3] = add2(acc[e / 2 & 3], f2(s[e], s[e + 1]));
        };
        // two loops: the mask must not cost where every row sees every key (and every
        // column is a row: step * group == QN above)
        if (none) {
          taken();
        } else if (t >= full0 && t < full1) {
#pragma unroll
          for (int c = 0; c < NC; c += W) {
            float s[W];
            load(c, s);
            weigh(s, c);
            gather(s);
          }
        } else {
          // tokens [see0, see1) of the sequence see this key, of this thread's
          // columns those from rl to rh
          const int i0 = (g.t0 + t) * p.step;
          const int see0 = p.right < 0 ? 0 : key - p.right - pos;
          const int see1 = key >= g.kv ? 0 : (p.left < 0 ? g.n : key + p.left - pos + 1);
          // (tokens counted inside the tile first: the products stay small)
          const int rl = min(max(0, see0 - i0), p.step) * p.group - cg * NC;
          const int rh = max(0, min(min(p.step, g.n - i0), see1 - i0)) * p.group - cg * NC;
#pragma unroll
          for (int c = 0; c < NC; c += W) {
            float s[W];
            load(c, s);
            if (!__any_sync(0xffffffffu, rl < rh && rh > c && rl < c + W)) continue;
            weigh(s, c);
#pragma unroll
            for (int e = 0; e < W; ++e)
              if (c + e < rl || c + e >= rh) s[e] = 0.f;
            gather(s);
          }
        }
        const float2 x = unf2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])));
        sum.add(x.x + x.y);
        sc.next();
        lc.next();
        ++at;
      }
      if (!ok) break;
      if (!g.ends) continue;
      if (CG == 2) {  // the second group's sums go to the first
        const uint32_t ph = (uint32_t)items++ & 1u;
        const bool here = cg == 1 ? mbar_wait(&x_empty[kt], ph ^ 1u, abort_flag)
                                  : mbar_wait(&x_full[kt], ph, abort_flag);
        ok = __all_sync(0xffffffffu, here);
        if (!ok) break;
        if (cg == 1) xch[CG == 2 ? mine : 0] = sum.value();
        else sum.add(xch[CG == 2 ? mine : 0]);
        __syncwarp();
        if (lane == 0) mbar_arrive(cg == 1 ? &x_full[kt] : &x_empty[kt]);
        if (cg == 1) continue;
      }
      if (begun && g.last) {
        write_weight(p, g.b, g.n, g.kv, key, sum.value());
      } else {
        p.part[(2 * blockIdx.x + (begun ? 1 : 0)) * kWeightKeys + mine] = sum.value();
        if (begun) {  // unit range of CTA c: [c total / ctas, (c + 1) total / ctas)
          rec.parts = (int)((item_end * start.ctas - 1) / start.total) - (int)blockIdx.x + 1;
          rec.seq = g.b;
          rec.block = g.kb;
        }
      }
    }
    if (!ok) {
      if (lane == 0) report(p.status, kDevTimeout, kSiteWeightSum, (unsigned)at, (unsigned)warp);
      *abort_flag = 1;
    }
    if (tid == 0) p.rec[blockIdx.x] = ok ? rec : WeightRec{0, 0, 0};
  }

  tc_fence_before();
  __syncthreads();
  if (warp == W0 + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// The sums of an item that several CTAs worked on, in their order.
__global__ void __launch_bounds__(kWeightKeys) k_weights_join(const __grid_constant__ WeightParams p) {
  pdl_trigger();
  pdl_wait();
  const WeightRec rec = p.rec[blockIdx.x];
  if (rec.parts == 0) return;
  const Seq s = load_seq(p, rec.seq);
  constexpr int kBatch = 8;
  Sum sum;
  for (int k0 = 0; k0 < rec.parts; k0 += kBatch) {
    float v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (k0 + k < rec.parts)
        v[k] = p.part[(2 * (blockIdx.x + k0 + k) + (k0 + k == 0 ? 1 : 0)) * kWeightKeys +
                      threadIdx.x];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (k0 + k < rec.parts) sum.add(v[k]);
  }
  write_weight(p, rec.seq, s.n, s.kv, rec.block * kWeightKeys + threadIdx.x, sum.value());
}

// ------------------------------------------------------------------ host

template <int D, int QN, bool FP16>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(k_weights<D, QN, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)Cfg<D, QN>::kSmem);
}
template <int D>
cudaError_t prepare_dim() {
  cudaError_t e = prepare_one<D, 16, false>();
  if (e == cudaSuccess) e = prepare_one<D, 16, true>();
  if (e == cudaSuccess) e = prepare_one<D, 128, false>();
  if (e == cudaSuccess) e = prepare_one<D, 128, true>();
  return e;
}

template <int D, int QN>
cudaError_t run(const WeightParams& p, bool fp16, int ctas, cudaStream_t s) {
  const cudaError_t e = launch_pdl(fp16 ? k_weights<D, QN, true> : k_weights<D, QN, false>,
                                   dim3(ctas), dim3(Cfg<D, QN>::kThreads),
                                   Cfg<D, QN>::kSmem, s, p);
  return e != cudaSuccess ? e : launch_pdl(k_weights_join, dim3(ctas), dim3(kWeightKeys), 0, s, p);
}
template <int QN>
cudaError_t run_dim(int d, const WeightParams& p, bool fp16, int ctas, cudaStream_t s) {
  return d == 256   ? run<256, QN>(p, fp16, ctas, s)
         : d == 128 ? run<128, QN>(p, fp16, ctas, s)
                    : run<64, QN>(p, fp16, ctas, s);
}

}  // namespace

namespace dg {
namespace host {
cudaError_t prepare_weights(int d) {
  return d == 256 ? prepare_dim<256>() : d == 128 ? prepare_dim<128>() : prepare_dim<64>();
}
}  // namespace host
}  // namespace dg

extern "C" dg_status_t dg_attn_weights(dg_attn_t* a, int layer, const dg_heads_t* q,
                                       const float* lse, const dg_attn_weights_t* w,
                                       const dg_kv_batch_t* batch, int n_tokens,
                                       dg_stream_t stream) {
  if (!a || !w) return DG_ERR_INVALID_ARG;
  const dg_kv_config_t& c = a->kv->cfg;
  if (layer < 0 || layer >= c.n_layers || n_tokens < 0 || w->width < 0) return DG_ERR_INVALID_ARG;
  dg_status_t st = check_batch(batch, c);
  if (st != DG_OK) return st;
  if (n_tokens > kMaxKvTokens || w->width > kMaxKvTokens) return DG_ERR_UNSUPPORTED;
  if (!(w->decay >= 0.f) || !isfinite(w->decay)) return DG_ERR_INVALID_ARG;
  if (batch->n_seqs == 0 || w->width == 0) return DG_OK;
  if (!w->in || !w->out) return DG_ERR_INVALID_ARG;
  if (!aligned(w->in, 4) || !aligned(w->out, 4)) return DG_ERR_ALIGNMENT;
  if (w->in_stride < 0 || w->out_stride < 0 ||
      (batch->n_seqs > 1 && (w->in_stride < w->width || w->out_stride < w->width)) ||
      (w->in == w->out && batch->n_seqs > 1 && w->in_stride != w->out_stride))
    return DG_ERR_INVALID_ARG;
  if (n_tokens > 0) {
    if ((st = check_heads(q)) != DG_OK) return st;
    if (!lse) return DG_ERR_INVALID_ARG;
    if (!aligned(lse, 4)) return DG_ERR_ALIGNMENT;
  }
  const int group = a->cfg.n_q_heads / c.n_kv_heads;
  WeightParams p;
  // Few rows or many, by the average: a long chunk among single tokens is taken by the
  // narrow tiles too (256 single tokens 108 us, 512 behind 4096 26, both in one call 202).
  const int64_t rows = (int64_t)n_tokens * group / batch->n_seqs;
  const bool few = group <= 16 && rows <= 16;
  p.step = (few ? 16 : kRows) / group;
  p.q_box = p.step < n_tokens ? p.step : n_tokens;
  if (n_tokens > 0) {
    st = encode_queries(&p.qm, *q, a->cfg.n_q_heads, c.head_dim, n_tokens, group, p.q_box);
    if (st != DG_OK) return st;
  } else {
    memset(&p.qm, 0, sizeof(p.qm));  // no copy uses it
  }
  const int ps = c.page_size;
  if (!encode_pages(&p.km, c, c.k, layer, ps < kKeys ? ps : kKeys)) return DG_ERR_CUDA;
  p.table = batch->page_table;
  p.table_stride = batch->table_stride;
  p.lens = batch->lens;
  p.cu = batch->cu;
  p.n_seqs = batch->n_seqs;
  p.cap = batch->max_pages * ps;
  p.n_tokens = n_tokens;
  p.n_pages = c.n_pages;
  p.page_shift = log2_of(ps);
  p.kv_heads = c.n_kv_heads;
  p.group = group;
  // a limit past every distance is none
  p.left = a->cfg.left >= p.cap + n_tokens ? -1 : a->cfg.left;
  p.right = a->cfg.right >= p.cap + n_tokens ? -1 : a->cfg.right;
  p.scale2 = a->cfg.scale * 1.4426950408889634f;
  p.lse = lse;
  p.w_in = w->in;
  p.w_out = w->out;
  p.in_stride = w->in_stride;
  p.out_stride = w->out_stride;
  p.width = w->width;
  p.decay = w->decay;
  p.fresh = w->fresh;
  p.part = reinterpret_cast<float*>(a->ws + a->L.wpart);
  p.rec = reinterpret_cast<WeightRec*>(a->ws + a->L.wrec);
  p.status = reinterpret_cast<DevStatus*>(a->ws + a->L.status);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fp16 = c.dtype == DG_T_FP16;
  const cudaError_t e = few ? run_dim<16>(c.head_dim, p, fp16, a->ctas, s)
                            : run_dim<128>(c.head_dim, p, fp16, a->ctas, s);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}
