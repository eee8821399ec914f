// Attention of new tokens over a paged key/value cache on sm_103a.
//
// A work item is one key/value head and a tile of query rows of one sequence:
// the G = n_q_heads / n_kv_heads query heads that share the key/value head
// are packed with their tokens (row = token * G + head of the group), so that
// a single token still fills G rows of the 128-row MMA and every key is read
// once for all of them.  Per 128-key tile j of the item
//   S = Q K_j^T                    tcgen05.mma, operands in shared memory
//   m' = max(m, rowmax(S)),  P = 2^(S scale log2 e - m')
//   O += P V_j,  l += rowsum(P)    tcgen05.mma, P from tensor memory
// with O, l and the statistics in fp32 (running softmax: one pass over the
// keys).  P enters the product rounded to the element type, as the operand of
// a 16-bit MMA must; l sums it before the rounding.
//
// The reference m of a row is only moved when the true maximum has grown past
// it by more than 2^8 (P then stays below 2^8, harmless in fp32 sums and in
// bf16 or fp16): O, which lives in tensor memory, is rescaled a few times a
// row instead of once a tile.  For fp16 the reference lies 2^7 lower (P below
// 2^15, of fp16's 2^16): fp16 ends at 2^-25, and a weight that is lost from
// O but kept in l biases the row (131072 keys of 2^-26 each came out as
// nothing); so the smallest weight kept is 2^-32 of the largest.
//
// The items of a call are cut into units of one key tile (and a few more where
// an item begins, for what its ends cost: 8 canvases take 120 us without those,
// 111 with), and the units dealt evenly to one CTA an SM: a CTA takes a
// contiguous range, so long and short sequences, many and few tokens balance
// alike.  An item that crosses a range boundary leaves fp32 partial results in
// the workspace, joined in a fixed order by k_attn_join.  (Joined by the last
// CTA to come instead: 6 us more, for the code and registers in the main loop.)
//
// Query tiles of one sequence read the same keys.  `team` CTAs take as many
// neighbouring tiles through the same key tiles at the same time, so that the
// keys come from memory once and from the L2 after that; each CTA copies its
// own stages.  At head size 256, where a ring of whole tiles would be too
// shallow, two CTAs are a pair with one tcgen05.mma of 256 rows: each holds its
// own rows and half of every key and value tile, and the first one issues for
// both (a team is made of whole pairs).
//
// Warps 0-3 and 4-7: softmax; 8 and 10: TMA producers of keys and values; 9: MMA
// issuer and TMEM owner.
// NQ = 2 (many rows, head size up to 128): two 128-row tiles an item, one a
// warpgroup, which take turns on the tensor core.  NQ = 1 (few rows, or head
// size 256, whose accumulator takes half of the TMEM): one tile, its key
// tiles double-buffered, its columns halved between the warpgroups.
//
// What bounds it, and what it takes on one GB300 (page size 64, 32 and 16 query
// heads on 8 key/value heads):
//   64 single tokens over 471k cached ones, head size 128: memory, 279 us
//     (6.9 TB/s; 317 us at page size 16, whose copies are 2 KB);
//   8 canvases of 256 over 20k, head size 256: the tensor core at the power
//     limit and the ends of items, 111-122 us (1.28-1.4 PFLOP/s);
//   4096 tokens behind 12288, head size 128: the same and the exponentials
//     between two products, 610-629 us (1.53-1.58 PFLOP/s);
//   one token over 777, head size 64: latency, 9.6 us with the join.
#include <math.h>

#include <new>
#include <type_traits>

#include <cuda_fp16.h>

#include "../../include/dg_attn.h"
#include "dg_attn_dev.cuh"
#include "dg_attn_host.h"
#include "dg_common.cuh"
#include "dg_tmem.cuh"

using namespace dg;
using namespace dg::host;

namespace {

constexpr int kThreads = 384;  // 12 warps: registers are dealt by warpgroup
// Registers a thread: 384 x 168 at launch; the producer and MMA warpgroup
// gives up what the two softmax warpgroups take (2 x 200 + 104 = 3 x 168).
// The compiler reports spills all the same: 200 bytes a thread with two tiles
// at head size 64, 188 at 128, 32 for the pair, 12 for few rows.
constexpr int kRegsSoftmax = 200, kRegsOther = 104;

constexpr int kMinShared = 128;  // tokens of a prefix that are taken together
constexpr int kMaxSharedRows = 128;  // rows of a sequence whose prefix is

// Sites of the device status word.
enum : unsigned int {
  kSiteAttnLoad = 32, kSiteAttnMma = 33, kSiteAttnSoftmax = 34, kSiteAttnDrain = 35,
  kSiteAttnPage = 36, kSiteAttnLen = 37,
};

struct AttnParams {
  CUtensorMap qm, km, vm;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  int64_t table_stride;
  int n_seqs, cap, n_tokens, n_pages, page_shift;
  int kv_heads, group, step;  // step: tokens of a 128-row tile
  int q_box;                  // tokens of a query box
  int team;                   // CTAs that take neighbouring tiles of a sequence
  int over;                   // what beginning an item costs, in key tiles
  int left, right;
  float scale2;  // scale log2 e
  uint16_t* out;
  int64_t o_tok, o_head;
  float* lse;
  float4* part;  // [2 ctas][D / 4][NQ * 128]: four columns of a row
  float2* ml;    // [2 ctas][NQ * 128] (m, l)
  JoinRec* rec;  // [ctas]
  DevStatus* status;
};

template <int D, int NQ, bool PAIR>
struct Cfg {
  // ring stage: 128 keys x D up to 128; at 256 a half of a key tile (128 keys
  // x 128) or of a value tile (64 keys x 256)
  static constexpr int kParts = D == 256 ? 2 : 1;
  // of a key tile a pair's CTA holds half the keys, of a value tile half the
  // columns
  static constexpr int kShare = PAIR ? 2 : 1;
  static constexpr int kStageBytes = kKeys * D * 2 / kParts / kShare;
  static constexpr int kStages = 160 * 1024 / kStageBytes;
  static constexpr int kChunks = D / 64;  // 128-byte columns of a row
  static constexpr int kQTile = kRows * D * 2;
  static constexpr int kQBufs = (NQ == 1 && D <= 128) ? 2 : 1;
  static constexpr size_t kSmem =
      (size_t)kStages * kStageBytes + (size_t)kQBufs * NQ * kQTile;
  // tensor memory columns
  static constexpr uint32_t kO = 256;
};

struct Seq {
  int n0, n, kv;
  int lo;  // its tokens look at keys from here on
};

__device__ __forceinline__ Seq load_seq(const AttnParams& p, int b) {
  const int a = __ldg(p.cu + b), e = __ldg(p.cu + b + 1), kv = __ldg(p.lens + b);
  Seq s;
  s.n0 = min(max(a, 0), p.n_tokens);
  s.n = max(min(e, p.n_tokens) - s.n0, 0);
  s.kv = min(max(kv, 0), p.cap);
  s.lo = 0;
  return s;
}

// Keys [x, y) that the tokens [first, first + n) of a sequence see together.
__device__ __forceinline__ int2 key_range(const AttnParams& p, const Seq& s, int first, int n) {
  const int pos = s.kv - s.n + first;
  const int lo = p.left < 0 ? s.lo : max(s.lo, pos - p.left);
  const int hi = p.right < 0 ? s.kv : min(s.kv, pos + n + p.right);
  return make_int2(lo, max(hi, 0));
}

// Tokens of a team's item.
template <int NQ>
__device__ __forceinline__ int item_tokens(const AttnParams& p) {
  return p.team * NQ * p.step;
}

// Key tiles [x, x + y) of item t of a team.
template <int NQ>
__device__ __forceinline__ int2 tile_range(const AttnParams& p, const Seq& s, int t) {
  const int first = t * item_tokens<NQ>(p);
  const int2 k = key_range(p, s, first, min(item_tokens<NQ>(p), s.n - first));
  if (k.x >= k.y) return make_int2(0, 0);
  const int a = k.x / kKeys;
  return make_int2(a, (k.y + kKeys - 1) / kKeys - a);
}

// The part of an item that a CTA works on.
struct Seg {
  int head, tok0, ntok;  // key/value head; first row of q / out, tokens of this CTA (may be none)
  int pos;               // position of the first token
  int b, kv, klo, khi;   // sequence, its length, keys that the item sees
  int kt0, n;            // key tiles
  bool first, last;      // holds the item's first / last tile
  long long end;         // unit after the item's last one
};

// Walk over the segments of a range of units; the same in every role.
template <int NQ, class P = AttnParams>
struct Walk {
  int h, b, t, skip, over;
  long long u, end;
  Seq s, ahead;  // this sequence and the one after it
  __device__ __forceinline__ void begin(const P& p) {
    if (u >= end) return;
    s = load_seq(p, b);
    ahead = load_seq(p, b + 1 < p.n_seqs ? b + 1 : 0);
  }
  __device__ __forceinline__ bool next(const P& p, Seg& g) {
    if (u >= end) return false;
    const int item = item_tokens<NQ>(p);
    const int2 tr = tile_range<NQ>(p, s, t);
    const int mine = t * item + (int)(blockIdx.x % p.team) * NQ * p.step;
    const int cost = over + max(tr.y, 1);
    const int take = (int)min((long long)(cost - skip), end - u);
    // only the units of its beginning: the next team takes the item whole
    if (skip + take <= over) return false;
    g.head = h;
    g.b = b;
    g.tok0 = s.n0 + mine;
    g.ntok = max(0, min(NQ * p.step, s.n - mine));
    g.pos = s.kv - s.n + mine;
    const int2 k = key_range(p, s, t * item, min(item, s.n - t * item));
    g.kv = s.kv;
    g.klo = k.x;
    g.khi = k.y;
    const int tile = max(skip - over, 0);
    g.kt0 = tr.x + tile;
    g.n = tr.y ? skip + take - over - tile : 0;
    g.first = skip == 0;
    g.last = skip + take == cost;
    g.end = u - skip + cost;
    u += take;
    skip = 0;
    if (u < end) {
      ++t;
      if (t * item >= s.n) {
        t = 0;
        do {
          if (++b == p.n_seqs) {
            b = 0;
            ++h;
          }
          // requested an item ago; the next one now
          s = ahead;
          ahead = load_seq(p, b + 1 < p.n_seqs ? b + 1 : 0);
        } while (s.n == 0);
      }
    }
    return true;
  }
};

struct Start {
  int h, b, t, skip, over;
  long long u, end, total;
  int teams;
};

// Row of the page table of sequence b (of the batch: what a report names), and what
// is wrong with it.
__device__ __forceinline__ int table_row(const AttnParams&, int b) { return b; }
__device__ __forceinline__ void check_seq(const AttnParams& p, int b) {
  const int a = __ldg(p.cu + b), e = __ldg(p.cu + b + 1), kv = __ldg(p.lens + b);
  if (a < 0 || e < a || e > p.n_tokens || kv < 0 || kv > p.cap)
    report(p.status, kDevBounds, kSiteAttnLen, (unsigned)b, (unsigned)kv);
}

// Attention that reads a prefix once for all sequences that share it, in two
// launches.  In the first every sequence attends to what lies behind its prefix;
// where there is one, its results stay as they are, fp32 and with their (m, l), in
// `pre`.  In the second a "sequence" is a group: its rows are the new tokens of all
// of its members, its keys the prefix, all of which every row sees; the first
// one's results are taken in as one more part.  (The other way round each of the
// many short items of the sequences would end in that, and take 13 us more in 40
// for 64 samples of one prompt.)  Rows of one key/value head lie together in `pre`,
// in the order in which tiles hold them, four columns of all rows at a time, so
// that a warp's accesses are contiguous.
struct PreParams : AttnParams {
  float4* pre;    // [D / 4][kv_heads * n_tokens * group]
  float2* pre_ml;
  const int32_t* prefix;  // [n_real]
  const int32_t* groups;  // [n_groups + 1]
  int n_real;             // sequences of the batch
  __device__ __forceinline__ size_t pre_rows() const {
    return (size_t)kv_heads * n_tokens * group;
  }
  __device__ __forceinline__ size_t pre_row(int head, int token, int gh) const {
    return ((size_t)head * n_tokens + token) * group + gh;
  }
  // Tokens that are taken together; a shorter prefix costs more than it saves.
  __device__ __forceinline__ int shared(int b) const {
    const int n = __ldg(prefix + b);
    return n >= kMinShared ? min(n, cap) : 0;
  }
};
struct PrefixParams : PreParams {};  // n_seqs: groups
struct SuffixParams : PreParams {};

__device__ __forceinline__ int table_row(const PrefixParams& p, int g) {
  return min(max(__ldg(p.groups + g), 0), p.n_real - 1);
}
__device__ __forceinline__ Seq load_seq(const PrefixParams& p, int g) {
  const int a = min(max(__ldg(p.groups + g), 0), p.n_real);
  const int b = min(max(__ldg(p.groups + g + 1), a), p.n_real);
  Seq s{0, 0, 0, 0};
  if (b - a < 2) return s;
  const int x = __ldg(p.cu + a), e = __ldg(p.cu + b);
  s.kv = p.shared(a);
  s.n0 = min(max(x, 0), p.n_tokens);
  s.n = s.kv > 0 ? max(min(e, p.n_tokens) - s.n0, 0) : 0;
  return s;
}
__device__ __forceinline__ void check_seq(const PrefixParams&, int) {}  // the first launch did

__device__ __forceinline__ Seq load_seq(const SuffixParams& p, int b) {
  Seq s = load_seq(static_cast<const AttnParams&>(p), b);
  s.lo = p.shared(b);
  return s;
}
__device__ __forceinline__ void check_seq(const SuffixParams& p, int b) {
  check_seq(static_cast<const AttnParams&>(p), b);
  // a prefix that some of the new tokens lie in
  const int past = __ldg(p.lens + b) - (__ldg(p.cu + b + 1) - __ldg(p.cu + b));
  if (p.shared(b) > max(past, 0))
    report(p.status, kDevBounds, kSiteAttnLen, (unsigned)b, (unsigned)past);
}

// Pair of CTAs: a box into this CTA, counted on the first CTA's barrier (`bar`
// is its address in the cluster).
__device__ __forceinline__ void tma_load_4d_pair(const CUtensorMap* map, uint32_t bar,
                                                 uint32_t dst, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(const CUtensorMap* map, uint32_t bar,
                                                 uint32_t dst, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Address of a barrier of the cluster's first CTA, and an arrival there.
__device__ __forceinline__ uint32_t first_cta(uint64_t* bar) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
  return r;
}
// What a softmax warp says so to the issuer is that tensor memory has been read
// or written.  The tcgen05 fences before the arrival and after the wait order
// that, whatever the semantics of the two, as long as their scope holds both
// threads: relaxed at cluster scope.  `wrote`: shared memory was written too
// (cleared values, at the ragged end of an item), which no tcgen05 fence
// orders: a release at cluster scope, after the writer's proxy fence.
template <bool PAIR>
__device__ __forceinline__ void arrive_first(uint64_t* bar, bool wrote = false) {
  if constexpr (PAIR) {
    const uint32_t a = first_cta(bar);
    if (wrote)
      asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(a)
                   : "memory");
    else
      asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(a)
                   : "memory");
  } else {
    mbar_arrive(bar);
  }
}

// try_wait that also acquires what the other CTA of a pair released.
template <bool PAIR>
__device__ __forceinline__ bool try_wait_scope(uint64_t* bar, uint32_t parity) {
  if constexpr (!PAIR) return mbar_try_wait(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait on a barrier that a pair's products, copies or other CTA signal.
// (The phase cannot pass before the second look: the waiter's own next arrival
// or copy is part of every later one.)
template <bool PAIR>
__device__ __forceinline__ bool wait_scope(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (try_wait_scope<PAIR>(bar, parity)) return true;
  return mbar_wait(bar, parity, abort) && (!PAIR || try_wait_scope<PAIR>(bar, parity));
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void set_max_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// log2 of the most tokens of a box.
__host__ __device__ constexpr int key_shift_max(int d, bool pair) {
  return pair || d == 64 ? 6 : 7;
}
__host__ __device__ constexpr int value_shift_max(int d) { return d == 128 ? 7 : 6; }

// umma_ss with A in tensor memory.
template <bool PAIR>
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                        uint32_t idesc, int accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
        : "memory");
}

// Arrive, when this thread's MMAs so far are done, on `bar` of this CTA, or of
// both CTAs of a pair.
template <bool PAIR>
__device__ __forceinline__ void commit_own(uint64_t* bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    umma_commit(bar);
}

// log2 of the largest weight of a row whose reference has just moved.
template <bool FP16>
constexpr float kLift = FP16 ? 7.f : 0.f;

// Barrier of the two warps that share 32 rows (NQ = 1), with an OR of `stop`.
__device__ __forceinline__ bool pair_barrier(int id, bool stop) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, 64, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)stop), "r"(id)
      : "memory");
  return r != 0;
}

// Ring position, inside its segment of n tiles, of the first stage of key
// tile j and of value tile j (order K0, K1, V0, K2, V1, ..., V(n-1)).
template <int PARTS>
__device__ __forceinline__ int k_stage(int j) {
  return j == 0 ? 0 : PARTS * (2 * j - 1);
}
template <int PARTS>
__device__ __forceinline__ int v_stage(int j, int n) {
  return j + 1 < n ? PARTS * (2 * j + 2) : PARTS * (2 * n - 1);
}

// Where this CTA's range of units begins.  Sequence costs go through `cost`
// (shared memory, n_seqs entries).  All threads; ends with a barrier.
template <int NQ, class P>
__device__ __forceinline__ void find_start(const P& p, long long* cost, Start* out) {
  const int tid = threadIdx.x, lane = tid & 31;
  // key tiles in the low bits, items from here on: both add up
  constexpr int kItemBit = 36;
  if (tid < 256) {
    int lps = 32;  // lanes a sequence
    while (lps > 1 && lps * p.n_seqs > 256) lps >>= 1;
    const int per = 256 / lps, sub = tid % lps;
    for (int s0 = 0; s0 < p.n_seqs; s0 += per) {
      const int b = s0 + tid / lps;
      long long c = 0;
      if (b < p.n_seqs) {
        const Seq s = load_seq(p, b);
        for (int t = sub; t * item_tokens<NQ>(p) < s.n; t += lps)
          c += ((long long)1 << kItemBit) + max(tile_range<NQ>(p, s, t).y, 1);
        if (blockIdx.x == 0 && sub == 0) check_seq(p, b);
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
    long long one = __shfl_sync(0xffffffffu, incl, 31);
    const int most = (int)(gridDim.x / p.team);
    // Beginnings count where every team has several times their cost to do:
    // then no two ranges begin inside one beginning.
    const long long tiles = (one & (((long long)1 << kItemBit) - 1)) * p.kv_heads;
    const int over = tiles >= (long long)most * max(8, 3 * p.over) ? p.over : 0;
    auto units = [&](long long x) {
      return (x & (((long long)1 << kItemBit) - 1)) + over * (x >> kItemBit);
    };
    one = units(one);
    incl = units(incl);
    sum = units(sum);
    const long long total = one * p.kv_heads;
    const int teams = (int)min((long long)most, total);
    const int c = blockIdx.x / p.team;
    long long u0 = 0, u1 = 0;
    if (c < teams) {
      if (total < (1 << 22)) {  // at most 160 teams: 32-bit divisions will do
        u0 = (unsigned)c * (unsigned)total / (unsigned)teams;
        u1 = (unsigned)(c + 1) * (unsigned)total / (unsigned)teams;
      } else {
        u0 = (long long)c * total / teams;
        u1 = (long long)(c + 1) * total / teams;
      }
    }
    int h = 0, b = 0, t = 0, skip = 0;
    if (u0 < u1) {
      h = total < (1 << 22) ? (int)((unsigned)u0 / (unsigned)one) : (int)(u0 / one);
      long long r = u0 - h * one;
      const bool mine = r >= incl - sum && r < incl;
      const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
      b = b0;
      if (mine) {
        r -= incl - sum;
        while (r >= units(cost[b])) r -= units(cost[b++]);
      }
      b = __shfl_sync(0xffffffffu, b, src);
      r = __shfl_sync(0xffffffffu, r, src);
      const Seq s = load_seq(p, b);
      for (int base = 0;; base += 32) {
        const int tt = base + lane;
        int cc = 0;
        if (tt * item_tokens<NQ>(p) < s.n) cc = over + max(tile_range<NQ>(p, s, tt).y, 1);
        long long in = cc;
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, in, o);
          if (lane >= o) in += v;
        }
        const long long all = __shfl_sync(0xffffffffu, in, 31);
        if (r < all) {
          const unsigned hit = __ballot_sync(0xffffffffu, r < in);
          const int l = __ffs(hit) - 1;
          t = base + l;
          skip = (int)(r - __shfl_sync(0xffffffffu, in - cc, l));
          break;
        }
        r -= all;
        if (base * item_tokens<NQ>(p) >= s.n) {  // cannot happen: r lies in this sequence
          u1 = u0;
          break;
        }
      }
    }
    if (skip <= over) {  // inside an item's beginning: all of it is this team's
      u0 -= skip;
      skip = 0;
    }
    if (lane == 0) *out = Start{h, b, t, skip, over, u0, u1, total, teams};
  }
  fence_proxy_async_smem();  // `cost` lies where copies will land
  __syncthreads();
}

template <int D, int NQ, bool PAIR, bool FP16, class P = AttnParams>
__global__ void __launch_bounds__(kThreads, 1) k_paged_attn(const __grid_constant__ P p) {
  using C = Cfg<D, NQ, PAIR>;
  constexpr bool PREFIX = std::is_same<P, PrefixParams>::value;
  constexpr bool SUFFIX = std::is_same<P, SuffixParams>::value;
  constexpr int NS = C::kStages, PARTS = C::kParts, SH = C::kShare;
  constexpr int KROWS = kKeys / SH;             // keys of a tile in this CTA
  constexpr int NC = NQ == 2 ? 128 : 64;        // score columns a softmax thread
  constexpr int OC = NQ == 2 ? D : D / 2;       // output columns a softmax thread
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t ring = smem_u32(smem);
  const uint32_t qbase = ring + NS * C::kStageBytes;
  __shared__ uint64_t full[NS], empty[NS];
  __shared__ uint64_t q_full[C::kQBufs], q_empty[C::kQBufs];
  __shared__ uint64_t s_full[2], p_half[2], p_full[2], pv_done[2], o_full[2], drain;
  // Pair, second CTA: the values that it clears.  One a stage: several may be on
  // their way, and a barrier must not be armed again before its phase is over.
  __shared__ uint64_t tail_full[PAIR ? NS : 1];
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_word;
  __shared__ Start start;
  __shared__ float xch[2][NQ == 1 ? 256 : 1];
  volatile int* abort_flag = &abort_word;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if constexpr (!SUFFIX) pdl_trigger();
  if (ring & 1023u) {  // the swizzle needs it; the declaration asks for it
    if constexpr (PREFIX) pdl_wait();
    if (tid == 0) report(p.status, kDevBounds, kSiteAttnLoad, ring, 0u);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kQBufs; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_half[i], 4 * SH);
      mbar_init(&p_full[i], (NQ == 2 ? 4 : 8) * SH);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(&drain, 1);
    for (int i = 0; i < (PAIR ? NS : 0); ++i) mbar_init(&tail_full[i], 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (tid == 8 * 32) {
    tma_prefetch_map(&p.qm);
    tma_prefetch_map(&p.km);
    tma_prefetch_map(&p.vm);
  }
  if (PAIR) {  // the pair allocates together: both CTAs have to be there
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 9) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                       smem_u32(&tmem_holder))
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(&tmem_holder, 512);
      tmem_relinquish();
    }
  }
  // The launch over the prefixes runs beside the one before it (the sequences' own
  // parts) and its join, and waits for them where it takes their results in.  What
  // came before those is done: the first lets others begin only once it is.
  if constexpr (!PREFIX) pdl_wait();
  if constexpr (SUFFIX) pdl_trigger();
  tc_fence_before();
  find_start<NQ>(p, reinterpret_cast<long long*>(smem), &start);
  tc_fence_after();
  if (PAIR) {  // the other CTA's copies and arrivals need the ring to be free
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  const uint32_t tmem = tmem_holder;
  const int rank = PAIR ? blockIdx.x % 2 : 0;
  Walk<NQ, P> w;
  w.h = start.h;
  w.b = start.b;
  w.t = start.t;
  w.skip = start.skip;
  w.over = start.over;
  w.u = start.u;
  w.end = start.end;
  w.begin(p);
  Seg g;

  // nested, so that the registers of each side are its own
  if (warp >= 8) {
    set_max_regs_down<kRegsOther>();
    if (warp == 8 || warp == 10) {
      // ------------------------------------------------------------ producers
      // Warp 8 fills the key stages (and the query tiles), warp 10 the value
      // stages.  Uniform loops, one elected lane issues; of a pair's CTAs each
      // takes its own half of the tile.
      const bool leader = elect_one(), keys = warp == 8;
      // whether stage h of a value tile holds the last keys seen, in a part of
      // their 16-key step
      auto clears_stage = [](int vis, int h) {
        return vis < kKeys && (vis & 15) && vis / (kKeys / PARTS) == h;
      };
      const int ps = 1 << p.page_shift;
      const int piece_shift =
          min(p.page_shift, keys ? key_shift_max(D, PAIR) : value_shift_max(D));
      const int piece = 1 << piece_shift;                    // tokens of a box
      const int tokens = keys ? KROWS : kKeys / PARTS;       // of a stage
      const int chunks = keys ? C::kChunks / PARTS : C::kChunks / SH;
      const CUtensorMap* map = keys ? &p.km : &p.vm;
      int pos = 0, qn = 0;
      bool ok = true;
      auto acquire = [&](uint64_t* bar, uint32_t parity) {
        const bool here = wait_scope<PAIR>(bar, parity, abort_flag);
        ok = __all_sync(0xffffffffu, here);
        return ok;
      };
      while (ok && w.next(p, g)) {
        if (g.n == 0) continue;
        if (keys) {
          const int qb = qn % C::kQBufs;
          if (!acquire(&q_empty[qb], ((uint32_t)(qn / C::kQBufs) & 1u) ^ 1u)) break;
          ++qn;
          if (leader) {
            if (!PAIR || rank == 0)
              mbar_arrive_expect_tx(&q_full[qb],
                                    SH * NQ * C::kChunks * 128 * p.group * p.q_box);
#pragma unroll 1
            for (int x = 0; x < NQ * C::kChunks; ++x) {
              const uint32_t dst = qbase + qb * NQ * C::kQTile + x * (kRows * 128);
              const int c = 64 * (x % C::kChunks), row = g.tok0 + x / C::kChunks * p.step;
              if (PAIR)
                tma_load_3d_pair(&p.qm, first_cta(&q_full[qb]), dst, c, g.head * p.group, row);
              else
                tma_load_3d(&p.qm, &q_full[qb], dst, c, g.head * p.group, row);
            }
          }
          __syncwarp();
        }
        // Page ids of 32 consecutive boxes, one a lane, and of the next 32.  An
        // id out of range (or of a box that no query sees, whose page may be
        // gone) becomes n_pages: the copy then reads zeros.
        auto ids_at = [&](int base) {
          int id = p.n_pages;
          const int key = (base + lane) << piece_shift, pg = key >> p.page_shift;
          if (key < g.khi && ((pg + 1) << p.page_shift) > g.klo) {
            id = __ldg(p.table + (int64_t)table_row(p, g.b) * p.table_stride + pg);
            if ((unsigned)id >= (unsigned)p.n_pages) {
              report(p.status, kDevBounds, kSiteAttnPage, (unsigned)table_row(p, g.b),
                     (unsigned)id);
              id = p.n_pages;
            }
          }
          return id;
        };
        int base = ((g.kt0 * kKeys) >> piece_shift) & ~31;
        int ids = ids_at(base), ids_next = ids_at(base + 32);
#pragma unroll 1
        for (int j = 0; j < g.n && ok; ++j) {
          const int rp = pos + (keys ? k_stage<PARTS>(j) : v_stage<PARTS>(j, g.n));
          const int key_t = (g.kt0 + j) * kKeys;
#pragma unroll 1
          for (int h = 0; h < PARTS; ++h) {
            const int st = (rp + h) % NS;
            if (!acquire(&empty[st], ((uint32_t)((rp + h) / NS) & 1u) ^ 1u)) break;
            const int key0 = key_t + (keys ? rank * (SH - 1) * KROWS : h * tokens);
            // Tokens of a stage from `key` on that are fetched.  Of a pair both CTAs copy
            // something of every stage (zeros, where no key is seen): one that could be
            // filled, used and given back without the second CTA's producer might pass
            // twice the phase that it waits for, which then looks like none.
            auto live_from = [&](int key) {
              return max(PAIR ? piece : 0, min(tokens, (g.khi - key + piece - 1) & -piece));
            };
            const int live = live_from(key0);
            // Pair: counted in the first CTA, both shares together; but values
            // that the second CTA clears in part, it has to wait for itself.
            uint64_t* bar = &full[st];
            bool other = PAIR && rank == 1;
            if (PAIR) {
              const bool clears = !keys && clears_stage(g.khi - key_t, h);
              if (other && clears) bar = &tail_full[PAIR ? st : 0];
              if (leader && (!other || clears))
                mbar_arrive_expect_tx(bar, (live + (keys ? live_from(key_t + KROWS)
                                                         : (clears ? 0 : live))) *
                                               128 * chunks);
              other = other && !clears;
            } else if (leader) {
              mbar_arrive_expect_tx(bar, live * 128 * chunks);
            }
            const uint32_t bar_addr = other ? first_cta(bar) : smem_u32(bar);
#pragma unroll 1
            for (int r = 0; r < live; r += piece) {
              const int x = (key0 + r) >> piece_shift;
              if (x - base >= 32) {
                base += 32;
                ids = ids_next;
                ids_next = ids_at(base + 32);
              }
              const int id = __shfl_sync(0xffffffffu, ids, x & 31);
              if (leader)
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                  const uint32_t dst = ring + st * C::kStageBytes + (c * tokens + r) * 128;
                  const int col = ((keys ? h : rank * (SH - 1)) * chunks + c) * 64;
                  if (PAIR)
                    tma_load_4d_pair(map, bar_addr, dst, col, g.head, (key0 + r) & (ps - 1), id);
                  else
                    tma_load_4d(map, bar, dst, col, g.head, (key0 + r) & (ps - 1), id);
                }
              __syncwarp();
            }
          }
        }
        pos += 2 * PARTS * g.n;
      }
      if (!ok) {
        if (lane == 0) report(p.status, kDevTimeout, kSiteAttnLoad, (unsigned)pos, (unsigned)warp);
        *abort_flag = 1;
      }
      // No copy may still be landing in shared memory when the CTA exits: the
      // last use of every stage and query tile.  After a timeout some of these
      // never began; the first wait that runs out ends the list.
      if (keys && leader) {
        bool done = true;
        if (!(PAIR && rank == 1)) {
          for (int i = max(0, pos - NS); i < pos && done; ++i)
            done = wait_drain(&full[i % NS], (uint32_t)(i / NS) & 1u);
          for (int i = max(0, qn - C::kQBufs); i < qn && done; ++i)
            done = wait_drain(&q_full[i % C::kQBufs], (uint32_t)(i / C::kQBufs) & 1u);
        }
        // Nor may an arrival of the pair's products still be on its way to this
        // CTA's barriers: it must not meet a CTA that has gone.
        if (PAIR) {
          for (int i = max(0, pos - NS); i < pos && done; ++i)
            done = wait_drain(&empty[i % NS], (uint32_t)(i / NS) & 1u);
          for (int i = max(0, qn - C::kQBufs); i < qn && done; ++i)
            done = wait_drain(&q_empty[i % C::kQBufs], (uint32_t)(i / C::kQBufs) & 1u);
          const int tiles = pos / (2 * PARTS);
          for (int i = 0; i < NQ && tiles > 0 && done; ++i)
            done = wait_drain(&pv_done[i], (uint32_t)(tiles - 1) & 1u);
        }
        if (!done && ok) report(p.status, kDevTimeout, kSiteAttnDrain, 0u, 0u);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------ MMA issuer
      // One elected lane.  Its instructions between a wait and the MMAs that the
      // wait releases are on the critical path of the whole CTA (with a division
      // for the ring position and warp votes around the waits 4096 tokens behind
      // 12288 took 690 us), so ring positions are running counters.
      if ((!PAIR || rank == 0) && elect_one()) {
        struct Cursor {
          int st;
          uint32_t ph;
          __device__ __forceinline__ void add(int n) {
            st += n;
            if (st >= NS) {
              st -= NS;
              ph ^= 1u;
            }
          }
        };
        Cursor base{0, 0u};
        int qb = 0, at = 0;  // query buffer, key tiles
        uint32_t qph = 0;
        bool ok = true, issued = false;
        auto need = [&](uint64_t* bar, uint32_t parity) {
          ok = wait_scope<PAIR>(bar, parity, abort_flag);
          return ok;
        };
        while (ok && w.next(p, g)) {
          if (g.n == 0) continue;
          Cursor kc = base, vc = base;
          vc.add(g.n == 1 ? PARTS : 2 * PARTS);
          if (!need(&q_full[qb], qph)) break;
          const uint32_t q_lo = desc_lo(qbase + qb * NQ * C::kQTile, 16);
          const uint32_t ring_k = desc_lo(ring, 16);
          constexpr int SK = 8 / PARTS;  // 16-key steps of a value stage
          const uint32_t ring_v = desc_lo(ring, SK * 2048);
          int rem = g.khi - g.kt0 * kKeys;  // keys from the tile at hand on that some row sees
          // S_i(j) = Q_i K_j^T for the tile under kc; `keys` of it are seen
          auto scores = [&](int i, int j, int keys) {
            const int buf = NQ == 2 ? i : ((at + j) & 1);
            const uint32_t d = tmem + buf * 128u;
            // only the 16-key steps that are seen; a pair's keys lie in halves
            const uint32_t cols = PAIR ? kKeys : min(kKeys, (keys + 15) & ~15);
            const uint32_t idesc = idesc_16<FP16>(128 * SH, 0, false) | (cols >> 3 << 17);
            Cursor c = kc;
#pragma unroll
            for (int h = 0; h < PARTS; ++h) {
              if (i == 0 && !need(&full[c.st], c.ph)) return;
              tc_fence_after();
              constexpr int CH = C::kChunks / PARTS;
              const uint32_t a = q_lo + (i * C::kQTile + h * CH * (kRows * 128)) / 16;
              const uint32_t b = ring_k + c.st * (C::kStageBytes / 16);
#pragma unroll
              for (int x = 0; x < CH * 4; ++x)
                umma_ss<PAIR>(d, a + ((x >> 2) * (kRows * 128) + 32 * (x & 3)) / 16,
                        b + ((x >> 2) * (KROWS * 128) + 32 * (x & 3)) / 16, idesc, h | x);
              if (i == NQ - 1) commit_own<PAIR>(&empty[c.st]);
              c.add(1);
            }
            commit_own<PAIR>(&s_full[buf]);
            issued = true;
            if (i == NQ - 1) {
              if (j == g.n - 1) commit_own<PAIR>(&q_empty[qb]);
              kc.add(j == 0 ? PARTS : 2 * PARTS);
            }
          };
          // O_i += P_i(j) V_j for the tile under vc
          auto values = [&](int i, int j) {
            const int buf = NQ == 2 ? i : ((at + j) & 1);
            const uint32_t use = NQ == 2 ? (uint32_t)(at + j) : (uint32_t)(at + j) >> 1;
            const uint32_t d = tmem + C::kO + i * D;
            const uint32_t a = tmem + buf * 128u;
            constexpr uint32_t idesc = idesc_16<FP16>(128 * SH, D, true);
            Cursor c = vc;
            // NQ = 2: the first 64 keys' weights come ahead of the others'.  A
            // segment's first weights also say that O has been read: a warp
            // writes out the last segment's before it makes them.
            if (!need(NQ == 2 ? &p_half[buf] : &p_full[buf], use & 1u)) return;
            if (i == 0 && !need(&full[c.st], c.ph)) return;
            tc_fence_after();
            if (rem >= kKeys) {
#pragma unroll
              for (int h = 0; h < PARTS; ++h) {
                if (h > 0 && i == 0) {
                  if (!need(&full[c.st], c.ph)) return;
                  tc_fence_after();
                }
                const uint32_t b = ring_v + c.st * (C::kStageBytes / 16);
#pragma unroll
                for (int k = 0; k < SK; ++k) {
                  if (NQ == 2 && h * SK + k == 4) {
                    if (!need(&p_full[buf], use & 1u)) return;
                    tc_fence_after();
                  }
                  umma_ts<PAIR>(d, a + 8 * (h * SK + k), b + k * 2048 / 16, idesc,
                          h + k == 0 ? j != 0 : 1);
                }
                if (i == NQ - 1) commit_own<PAIR>(&empty[c.st]);
                c.add(1);
              }
            } else {  // the item's last keys: only their 16-key steps
              if (NQ == 2) {
                if (!need(&p_full[buf], use & 1u)) return;
                tc_fence_after();
              }
              const int ks = (rem + 15) >> 4;
#pragma unroll 1
              for (int h = 0; h < PARTS; ++h) {
                if (h > 0 && i == 0) {
                  if (!need(&full[c.st], c.ph)) return;
                  tc_fence_after();
                }
                const uint32_t b = ring_v + c.st * (C::kStageBytes / 16);
#pragma unroll 1
                for (int k = 0; k < SK && h * SK + k < ks; ++k)
                  umma_ts<PAIR>(d, a + 8 * (h * SK + k), b + k * 2048 / 16, idesc, j | h | k);
                if (i == NQ - 1) commit_own<PAIR>(&empty[c.st]);
                c.add(1);
              }
            }
            commit_own<PAIR>(&pv_done[i]);
            if (j == g.n - 1) commit_own<PAIR>(&o_full[i]);
            if (i == NQ - 1) {
              if (j == g.n - 1) {
                base = vc;
                base.add(PARTS);
              }
              vc.add(j + 1 < g.n - 1 ? 2 * PARTS : PARTS);
              rem -= kKeys;
            }
          };
          if (NQ == 2) {
            scores(0, 0, rem);
            if (ok) scores(1, 0, rem);
            for (int j = 0; j < g.n && ok; ++j) {
              const int next = rem - kKeys;
              values(0, j);
              if (ok && j + 1 < g.n) scores(0, j + 1, next);
              if (ok) values(1, j);
              if (ok && j + 1 < g.n) scores(1, j + 1, next);
            }
          } else {
            scores(0, 0, rem);
            if (ok && g.n > 1) scores(0, 1, rem - kKeys);
            for (int j = 0; j < g.n && ok; ++j) {
              values(0, j);
              if (ok && j + 2 < g.n) scores(0, j + 2, rem - kKeys);
            }
          }
          at += g.n;
          if (++qb == C::kQBufs) {
            qb = 0;
            qph ^= 1u;
          }
        }
        if (!ok) {
          report(p.status, kDevTimeout, kSiteAttnMma, (unsigned)at, 0u);
          *abort_flag = 1;
        }
        // every MMA issued here must have completed before TMEM is released
        if (issued) {
          if constexpr (PAIR)
            asm volatile(
                "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                    smem_u32(&drain))
                : "memory");
          else
            umma_commit(&drain);
          if (!wait_drain(&drain, 0u)) report(p.status, kDevTimeout, kSiteAttnDrain, 99u, 0u);
        }
      }
    }
  } else {
    set_max_regs_up<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax
    const int wg = warp >> 2, quarter = warp & 3;
    const int i = NQ == 2 ? wg : 0;        // tile of the item
    const int c0 = NQ == 2 ? 0 : wg * NC;  // first score column
    const int o0 = NQ == 2 ? 0 : wg * OC;  // first output column
    const int row = quarter * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    const int tok = row / p.group, gh = row - tok * p.group;
    int pos = 0, at = 0, segs = 0;  // ring position, key tiles, segments
    int xn = 0;           // exchanges (NQ = 1)
    uint32_t tails = 0;   // phase of each stage's tail_full
    bool ok = true;
    JoinRec rec{0, 0, 0, 0, 0};
    while (ok && w.next(p, g)) {
      const bool row_live = tok < p.step && tok + i * p.step < g.ntok;
      const bool live = __any_sync(0xffffffffu, row_live);
      // rows that are not there see all of the item, so that they need no mask
      // (a warp with one takes the masked path at every tile otherwise: 1100
      // cycles more a tile for single tokens); nothing of theirs is kept
      int lo = 0, hi = g.khi;
      if (row_live) {
        const int qp = g.pos + i * p.step + tok;
        lo = p.left < 0 ? 0 : max(0, qp - p.left);
        if constexpr (SUFFIX) lo = max(lo, g.klo);
        hi = max(lo, p.right < 0 ? g.kv : min(g.kv, qp + p.right + 1));
      }
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < g.n; ++j) {
        const int buf = NQ == 2 ? i : ((at + j) & 1);
        const uint32_t use = NQ == 2 ? (uint32_t)(at + j) : (uint32_t)(at + j) >> 1;
        const int key0 = (g.kt0 + j) * kKeys;
        if (!wait_scope<PAIR>(&s_full[buf], use & 1u, abort_flag)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && (NQ == 2 || !live)) break;  // a live pair leaves at its barrier
        tc_fence_after();
        // The last tile of an item may hold keys that no row sees, and rows
        // that were never written: their V is zeroed up to the 16-key step,
        // so that 0 * V cannot bring in a NaN.
        const int vis = g.khi - key0;
        const bool clears = vis < kKeys && (vis & 15) && i == 0;
        if (clears) {
          const int rp = pos + v_stage<PARTS>(j, g.n);
          constexpr int VK = kKeys / PARTS;
          const int h = vis / VK;  // the stage that holds the step
          const int st = (rp + h) % NS;
          bool here;
          if (PAIR && rank == 1) {
            here = mbar_wait(&tail_full[PAIR ? st : 0], (tails >> st) & 1u, abort_flag);
            tails ^= 1u << st;
          } else {
            here = wait_scope<PAIR>(&full[st], (uint32_t)((rp + h) / NS) & 1u, abort_flag);
          }
          ok = __all_sync(0xffffffffu, here) && ok;
          const int r0 = vis - h * VK, r1 = (r0 + 15) & ~15;
          constexpr int NT = NQ == 2 ? 128 : 256;
          constexpr int VCH = C::kChunks / SH;
          for (int x = (tid & (NT - 1)); x < (r1 - r0) * VCH * 8; x += NT) {
            const int u = x & 7, r = r0 + (x >> 3) / VCH, c = (x >> 3) % VCH;
            *reinterpret_cast<uint4*>(smem + st * C::kStageBytes + c * (VK * 128) + r * 128 +
                                      u * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (live) {
          const uint32_t ts = tl + buf * 128u;
          float s[NC];
          if constexpr (NC == 128) tmem_load128(ts, s);
          else tmem_load64(ts + c0, s);
          const int rl = lo - key0 - c0, rh = hi - key0 - c0;
          // blocks of columns that every row sees need no mask
          if (!__all_sync(0xffffffffu, rl <= 0 && rh >= NC)) {
#pragma unroll
            for (int b = 0; b < NC; b += 32)
              if (!__all_sync(0xffffffffu, rl <= b && rh >= b + 32)) {
#pragma unroll
                for (int c = b; c < b + 32; ++c)
                  if ((unsigned)(c - rl) >= (unsigned)(rh - rl)) s[c] = -INFINITY;
              }
          }
          float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c + 7 < NC; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx4[e] = fmaxf(fmaxf(mx4[e], s[c + e]), s[c + 4 + e]);
#pragma unroll
          for (int e = 0; e < 4; ++e) mx4[e] = fmaxf(mx4[e], s[NC - 4 + e]);
          float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          if (NQ == 1) {
            float* x = xch[xn & 1];
            x[wg * 128 + row] = mx;
            // also orders the partner's loads of S before this warp's P
            tc_fence_before();
            if (pair_barrier(1 + quarter, !ok)) {
              ok = false;
              break;
            }
            tc_fence_after();
            mx = fmaxf(mx, x[(wg ^ 1) * 128 + row]);
            ++xn;
          }
          // what the reference would be
          const float mt = fmaf(mx, p.scale2, -kLift<FP16>);
          // also true of the first key that a row sees (m is -inf before it)
          const bool grown = row_live && mt > m + 8.f;
          if (__any_sync(0xffffffffu, grown)) {
            const float fac = grown && m != -INFINITY ? exp2_fast(m - mt) : 1.f;
            if (grown) m = mt;
            l *= fac;
            if (j > 0 && __any_sync(0xffffffffu, fac != 1.f)) {
              // O holds the tiles before this one once their product is done.
              // The products before that one are: S of this tile was issued
              // after them, so the barrier is at most one phase behind.
              bool here = wait_scope<PAIR>(&pv_done[i], (uint32_t)(at + j - 1) & 1u, abort_flag);
              here = __all_sync(0xffffffffu, here);
              if (!here) {
                ok = false;
                if (NQ == 2) break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < OC; c += 16) {
                float o[16];
                uint32_t r[16];
                tmem_ld16(tl + C::kO + i * D + o0 + c, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(o[e] * fac);
                tmem_store16(tl + C::kO + i * D + o0 + c, r);
              }
            }
          }
          const float mr = m == -INFINITY ? 0.f : m;
          const uint64_t sc2 = f2(p.scale2, p.scale2), mr2 = f2(-mr, -mr);
          uint64_t l2[2] = {0, 0};
#pragma unroll
          for (int b = 0; b < NC; b += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float2 x = unf2(fma2(f2(s[b + c], s[b + c + 1]), sc2, mr2));
              const float e0 = exp2_fast(x.x), e1 = exp2_fast(x.y);
              l2[(c >> 1) & 1] = add2(l2[(c >> 1) & 1], f2(e0, e1));
              pk[c / 2] = pack16<FP16>(e0, e1);
            }
            tmem_store16(ts + c0 / 2 + b / 2, pk);
            if (NQ == 2 && b == 32) {
              tmem_store_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_first<PAIR>(&p_half[buf]);
            }
          }
          {
            const float2 x = unf2(add2(l2[0], l2[1]));
            l += x.x + x.y;
          }
          tmem_store_wait();
        } else if (NQ == 2) {
          __syncwarp();
          if (lane == 0) arrive_first<PAIR>(&p_half[buf]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first<PAIR>(&p_full[buf], clears);
      }
      // ------------------------------------------------- end of the segment
      if (g.n) {
        if (ok && !wait_scope<PAIR>(&o_full[i], (uint32_t)segs & 1u, abort_flag)) ok = false;
        ++segs;
        ok = __all_sync(0xffffffffu, ok);
        if (NQ == 2 && !ok) break;
        tc_fence_after();
      }
      if (live) {
        if (NQ == 1 && g.n) {
          float* x = xch[xn & 1];
          x[wg * 128 + row] = l;
          if (pair_barrier(1 + quarter, !ok)) {
            ok = false;
            break;
          }
          l += x[(wg ^ 1) * 128 + row];
          ++xn;
        }
        const bool whole = g.first && g.last;
        // the part of a shared prefix, and what this one counts beside it
        bool pre = false;
        size_t pre_at = 0;
        float own = 1.f, pre_f = 0.f;
        if constexpr (PREFIX || SUFFIX) {
          pre_at = p.pre_row(g.head, g.tok0 + i * p.step + tok, gh);
          if (PREFIX && whole) pdl_wait();
          if (PREFIX && whole && row_live) {
            const float2 q = p.pre_ml[pre_at];
            pre = !(q.y == 0.f);  // one that saw nothing holds nothing
            if (pre) {
              const float top = fmaxf(m, q.x);
              own = l == 0.f ? 0.f : exp2f(m - top);
              pre_f = exp2f(q.x - top);
              l = (l == 0.f ? 0.f : own * l) + pre_f * q.y;
              m = top;
            }
          }
        }
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        const int trow = g.tok0 + i * p.step + tok;
        const int head = g.head * p.group + gh;
        const int slot = 2 * blockIdx.x + (g.first ? 1 : 0);
        const size_t prow = (size_t)slot * (NQ * kRows) + i * kRows + row;
        // (few rows: the code is fetched again for every item, so it stays short)
#pragma unroll(NQ == 1 && !PAIR ? 1 : OC / 32)
        for (int c = 0; c < OC; c += 32) {
          float o[32];
          if (g.n) {
            __syncwarp();
            tmem_load32(tl + C::kO + i * D + o0 + c, o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
          }
          if (!row_live) continue;
          if constexpr (PREFIX) {
            if (pre) {
              const float4* src = p.pre + (size_t)((o0 + c) / 4) * p.pre_rows() + pre_at;
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 x = src[e / 4 * p.pre_rows()];
                const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)  // (O may hold anything where nothing was seen)
                  o[e + k] = (own == 0.f ? 0.f : own * o[e + k]) + pre_f * y[k];
              }
            }
          }
          if (SUFFIX && whole && g.klo > 0) {
            if constexpr (SUFFIX) {
              float4* dst = p.pre + (size_t)((o0 + c) / 4) * p.pre_rows() + pre_at;
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                dst[e / 4 * p.pre_rows()] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          } else if (whole) {
            uint16_t* dst = p.out + trow * p.o_tok + head * p.o_head + o0 + c;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 v;
              // nothing seen: O may hold what was there before
              const bool z = l == 0.f;
              v.x = z ? 0u : pack16<FP16>(o[e] * inv, o[e + 1] * inv);
              v.y = z ? 0u : pack16<FP16>(o[e + 2] * inv, o[e + 3] * inv);
              v.z = z ? 0u : pack16<FP16>(o[e + 4] * inv, o[e + 5] * inv);
              v.w = z ? 0u : pack16<FP16>(o[e + 6] * inv, o[e + 7] * inv);
              *reinterpret_cast<uint4*>(dst + e) = v;
            }
          } else {
            // four columns of all rows together, so that a warp's rows are
            // contiguous
            float4* dst = p.part + ((size_t)slot * (D / 4) + (o0 + c) / 4) * (NQ * kRows) +
                          i * kRows + row;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              dst[e / 4 * (NQ * kRows)] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        if (row_live && (NQ == 2 || wg == 0)) {
          if (!whole)
            p.ml[prow] = make_float2(m, l);
          else if (SUFFIX && g.klo > 0) {
            if constexpr (SUFFIX) p.pre_ml[pre_at] = make_float2(m, l);
          } else if (p.lse)
            p.lse[(size_t)trow * (p.kv_heads * p.group) + head] =
                l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
        }
      }
      if (g.first && !g.last) {
        // unit range of team c: [c total / teams, (c + 1) total / teams)
        const long long x = g.end * start.teams - 1;
        const int lastc = start.total < (1 << 22) ? (int)((unsigned)x / (unsigned)start.total)
                                                  : (int)(x / start.total);
        rec.parts = lastc - (int)(blockIdx.x / p.team) + 1;
        rec.head = g.head;
        rec.tok0 = g.tok0;
        rec.ntok = g.ntok;
        if constexpr (SUFFIX) rec.shared = g.klo > 0;
      }
      if (g.n) {
        pos += 2 * PARTS * g.n;
        at += g.n;
      }
    }
    if (!ok) {
      if (lane == 0) report(p.status, kDevTimeout, kSiteAttnSoftmax, (unsigned)at, (unsigned)warp);
      *abort_flag = 1;
    }
    if (tid == 0) p.rec[blockIdx.x] = ok ? rec : JoinRec{0, 0, 0, 0, 0};
  }

  if constexpr (PREFIX) pdl_wait();  // completion stays transitive
  tc_fence_before();
  __syncthreads();
  if (PAIR) {  // the first CTA has waited for the pair's products
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    else
      tmem_dealloc(tmem, 512);
  }
  if (PAIR) {  // the other CTA's arrivals may still come here
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
}

// Join the parts of the item that CTA blockIdx.x began: with m the largest
// reference, o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i, parts in order,
// BATCH of them in flight.  A thread takes eight columns of a row,
// neighbouring threads neighbouring rows.
template <int D, int NQ, int BATCH, bool FP16, class P = AttnParams>
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ P p) {
  constexpr bool PREFIX = std::is_same<P, PrefixParams>::value;
  constexpr bool SUFFIX = std::is_same<P, SuffixParams>::value;
  pdl_trigger();
  pdl_wait();
  const JoinRec rec = p.rec[blockIdx.x];
  if (rec.parts == 0) return;
  constexpr int ROWS = NQ * kRows;
  const int live = rec.ntok * p.group;
  for (int u = threadIdx.x + 256 * (int)blockIdx.y; u < live * (D / 8);
       u += 256 * (int)gridDim.y) {
    const int c = u / live, vr = u - c * live;  // eight columns, row
    const int tok = vr / p.group, gh = vr - tok * p.group;
    const int i = tok / p.step;
    const int row = i * kRows + (tok - i * p.step) * p.group + gh;
    const int trow = rec.tok0 + tok, head = rec.head * p.group + gh;
    float2 pre_ml;  // the first launch's part
    float4 pre_lo, pre_hi;
    if constexpr (PREFIX) {
      const size_t at = p.pre_row(rec.head, trow, gh);
      pre_ml = p.pre_ml[at];
      pre_lo = p.pre[2 * c * p.pre_rows() + at];
      pre_hi = p.pre[(2 * c + 1) * p.pre_rows() + at];
    }
    float m = -INFINITY, l = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < rec.parts; k0 += BATCH) {
      float4 v[BATCH][2];
      float2 ml[BATCH];
      float top = m;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        if (k0 + k < rec.parts) {
          const size_t slot = 2 * ((int)blockIdx.x + (k0 + k) * p.team) + (k0 + k == 0 ? 1 : 0);
          ml[k] = p.ml[slot * ROWS + row];
          const float4* src = p.part + (slot * (D / 4) + 2 * c) * ROWS + row;
          v[k][0] = src[0];
          v[k][1] = src[ROWS];
        }
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) top = fmaxf(top, ml[k].x);
      if (m != -INFINITY) {
        const float f = exp2f(m - top);
        l *= f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= f;
      }
      m = top;
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        // A part that saw nothing holds nothing.  One whose scores are all NaN has
        // no reference either, but its sum is NaN and makes the row's NaN.
        if (!(ml[k].y == 0.f)) {
          const float f = exp2f(ml[k].x - m);
          l += f * ml[k].y;
          acc[0] += f * v[k][0].x;
          acc[1] += f * v[k][0].y;
          acc[2] += f * v[k][0].z;
          acc[3] += f * v[k][0].w;
          acc[4] += f * v[k][1].x;
          acc[5] += f * v[k][1].y;
          acc[6] += f * v[k][1].z;
          acc[7] += f * v[k][1].w;
        }
    }
    if constexpr (SUFFIX) {
      if (rec.shared) {
        const size_t at = p.pre_row(rec.head, trow, gh);
        p.pre[2 * c * p.pre_rows() + at] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        p.pre[(2 * c + 1) * p.pre_rows() + at] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (c == 0) p.pre_ml[at] = make_float2(m, l);
        continue;
      }
    }
    if constexpr (PREFIX) {
      if (!(pre_ml.y == 0.f)) {
        const float top = fmaxf(m, pre_ml.x), f = exp2f(pre_ml.x - top);
        const float own = l == 0.f ? 0.f : exp2f(m - top);  // (acc is 0 with l)
        const float z[8] = {pre_lo.x, pre_lo.y, pre_lo.z, pre_lo.w,
                            pre_hi.x, pre_hi.y, pre_hi.z, pre_hi.w};
        l = own * l + f * pre_ml.y;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = own * acc[e] + f * z[e];
        m = top;
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (l != 0.f)
      r = make_uint4(
          pack16<FP16>(acc[0] * inv, acc[1] * inv), pack16<FP16>(acc[2] * inv, acc[3] * inv),
          pack16<FP16>(acc[4] * inv, acc[5] * inv), pack16<FP16>(acc[6] * inv, acc[7] * inv));
    *reinterpret_cast<uint4*>(p.out + trow * p.o_tok + head * p.o_head + 8 * c) = r;
    if (p.lse && c == 0)
      p.lse[(size_t)trow * (p.kv_heads * p.group) + head] =
          l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
  }
}

// ------------------------------------------------------------------ host

// Head sizes whose many-row variant is a pair of CTAs with shared products.
constexpr bool pair_of(int d) { return d == 256; }

// The variants of a head size: few rows (one tile) and many rows (as wide an
// item as fits; dg_attn_forward chooses).
template <int D, bool FP16>
struct Variant {
  static constexpr int kManyNq = D == 256 ? 1 : 2;
  static constexpr bool kPair = pair_of(D);
  static constexpr auto few = k_paged_attn<D, 1, false, FP16>;
  static constexpr auto many = k_paged_attn<D, kManyNq, kPair, FP16>;
  template <class P>
  static constexpr auto few_of = k_paged_attn<D, 1, false, FP16, P>;
  template <class P>
  static constexpr auto many_of = k_paged_attn<D, kManyNq, kPair, FP16, P>;
  // P: plain, PrefixParams, or SuffixParams (few rows alone)
  template <class P>
  static cudaError_t run(bool m, const P& p, int ctas, cudaStream_t s) {
    constexpr bool kSuffix = std::is_same<P, SuffixParams>::value;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = m ? Cfg<D, kManyNq, kPair>::kSmem : Cfg<D, 1, false>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = m && kPair ? 2 : 1;
    cudaError_t e;
    if constexpr (kSuffix)
      e = cudaLaunchKernelEx(&cfg, few_of<P>, p);
    else
      e = cudaLaunchKernelEx(&cfg, m ? many_of<P> : few_of<P>, p);
    if (e != cudaSuccess) return e;
    // few rows are split into many parts, many rows into two or three, but a
    // prefix's into many again
    if constexpr (std::is_same<P, PrefixParams>::value) {
      if (m && kManyNq == 2)
        return launch_pdl(k_attn_join<D, kManyNq, 8, FP16, P>, dim3(ctas, 16), dim3(256), 0, s, p);
      return launch_pdl(k_attn_join<D, 1, 8, FP16, P>, dim3(ctas, 16), dim3(256), 0, s, p);
    } else if constexpr (!kSuffix) {
      if (m && kManyNq == 2)
        return launch_pdl(k_attn_join<D, kManyNq, 2, FP16, P>, dim3(ctas, 8), dim3(256), 0, s, p);
      if (m) return launch_pdl(k_attn_join<D, 1, 2, FP16, P>, dim3(ctas, 8), dim3(256), 0, s, p);
    }
    if constexpr (!std::is_same<P, PrefixParams>::value)
      return launch_pdl(k_attn_join<D, 1, 8, FP16, P>, dim3(ctas), dim3(256), 0, s, p);
  }
  template <class K>
  static cudaError_t limit(K kernel, size_t smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  }
  static cudaError_t prepare() {
    cudaError_t e = limit(few, Cfg<D, 1, false>::kSmem);
    if (e == cudaSuccess) e = limit(many, Cfg<D, kManyNq, kPair>::kSmem);
    if (e == cudaSuccess) e = limit(few_of<PrefixParams>, Cfg<D, 1, false>::kSmem);
    if (e == cudaSuccess) e = limit(many_of<PrefixParams>, Cfg<D, kManyNq, kPair>::kSmem);
    if (e == cudaSuccess) e = limit(few_of<SuffixParams>, Cfg<D, 1, false>::kSmem);
    return e;
  }
};

template <bool FP16>
cudaError_t prepare_dim(int d) {
  return d == 256   ? Variant<256, FP16>::prepare()
         : d == 128 ? Variant<128, FP16>::prepare()
                    : Variant<64, FP16>::prepare();
}
template <bool FP16, class P>
cudaError_t run_dim(int d, bool many, const P& p, int ctas, cudaStream_t s) {
  return d == 256   ? Variant<256, FP16>::run(many, p, ctas, s)
         : d == 128 ? Variant<128, FP16>::run(many, p, ctas, s)
                    : Variant<64, FP16>::run(many, p, ctas, s);
}
template <class P>
dg_status_t run_call(const dg_attn* a, bool many, const P& p, dg_stream_t stream) {
  const dg_kv_config_t& c = a->kv->cfg;
  const int ctas = a->ctas / p.team * p.team;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c.dtype == DG_T_FP16 ? run_dim<true>(c.head_dim, many, p, ctas, s)
                                             : run_dim<false>(c.head_dim, many, p, ctas, s);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

// Workspace of a call with shared prefixes: results of the sequences' own parts
// (fp32 rows, and their (m, l)), and a place for that launch's partial results, which
// runs beside the one over the prefixes.
struct PreLayout {
  size_t o, ml, rec, part_ml, part, total;
};
PreLayout pre_layout(const dg_attn_config_t& a, const dg_kv_config_t& c, int n_tokens) {
  const size_t rows = (size_t)n_tokens * a.n_q_heads;
  PreLayout L;
  size_t at = 0;
  L.o = at;
  at = round_up(at + rows * c.head_dim * sizeof(float), 256);
  L.ml = at;
  at = round_up(at + rows * sizeof(float2), 256);
  L.rec = at;
  at = round_up(at + sizeof(JoinRec) * kMaxCtas, 256);
  L.part_ml = at;
  at = round_up(at + 2 * kMaxCtas * kRows * sizeof(float2), 256);
  L.part = at;
  at += 2 * kMaxCtas * kRows * c.head_dim * sizeof(float);
  L.total = at;
  return L;
}

dg_status_t check_config(const dg_attn_config_t* c, const dg_kv* kv) {
  if (!c || !kv) return DG_ERR_INVALID_ARG;
  if (c->n_q_heads <= 0 || c->flags != 0 || !(c->scale > 0.f) || !isfinite(c->scale))
    return DG_ERR_INVALID_ARG;
  if (c->n_q_heads % kv->cfg.n_kv_heads) return DG_ERR_INVALID_ARG;
  if (c->n_q_heads / kv->cfg.n_kv_heads > kRows) return DG_ERR_UNSUPPORTED;
  return DG_OK;
}

// Checks of a call's arguments; *done: nothing to do.
dg_status_t check_call(const dg_attn* a, int layer, const dg_heads_t* q, const dg_heads_t* out,
                       const float* lse, const dg_kv_batch_t* batch, int n_tokens, bool* done) {
  *done = false;
  if (!a) return DG_ERR_INVALID_ARG;
  const dg_kv_config_t& c = a->kv->cfg;
  if (layer < 0 || layer >= c.n_layers || n_tokens < 0) return DG_ERR_INVALID_ARG;
  dg_status_t st = check_batch(batch, c);
  if (st != DG_OK) return st;
  if (n_tokens > kMaxKvTokens) return DG_ERR_UNSUPPORTED;
  *done = n_tokens == 0 || batch->n_seqs == 0;
  if (*done) return DG_OK;
  if ((st = check_heads(q)) != DG_OK || (st = check_heads(out)) != DG_OK) return st;
  if (lse && !aligned(lse, 4)) return DG_ERR_ALIGNMENT;
  if (q->p == out->p) return DG_ERR_INVALID_ARG;
  return DG_OK;
}

// The parameters of a launch over sequences of `rows` rows on average, and
// whether it takes the variant for many.
dg_status_t set_up(const dg_attn* a, int layer, const dg_heads_t* q, const dg_heads_t* out,
                   float* lse, const dg_kv_batch_t* batch, int n_tokens, int64_t rows,
                   AttnParams& p, bool* takes_many) {
  const dg_kv_config_t& c = a->kv->cfg;
  const int group = a->cfg.n_q_heads / c.n_kv_heads;
  p.step = kRows / group;
  p.q_box = p.step < n_tokens ? p.step : n_tokens;
  const dg_status_t st = encode_queries(&p.qm, *q, a->cfg.n_q_heads, c.head_dim, n_tokens, group, p.q_box);
  if (st != DG_OK) return st;
  // Few rows (one tile a CTA) or many, by the average rows of a sequence.  16
  // sequences behind 4000 cached tokens, 4 query heads a key/value head, us few
  // / many: head size 64: 41 / 48 at 128 rows, 65 / 53 at 192, 112 / 94 at 512;
  // 128: 65 / 63 at 128, 104 / 69 at 192, 180 / 123 at 512; 256: 93 / 95 at 32,
  // 102 / 99 at 64, 199 / 113 at 256.
  const bool many = rows > (c.head_dim == 256 ? 32 : 128);
  const int ps = c.page_size;
  const int kmax = 1 << key_shift_max(c.head_dim, many && pair_of(c.head_dim));
  const int vmax = 1 << value_shift_max(c.head_dim);
  const uint32_t kbox = ps < kmax ? ps : kmax, vbox = ps < vmax ? ps : vmax;
  if (!encode_pages(&p.km, c, c.k, layer, kbox) || !encode_pages(&p.vm, c, c.v, layer, vbox))
    return DG_ERR_CUDA;
  p.table = batch->page_table;
  p.table_stride = batch->table_stride;
  p.lens = batch->lens;
  p.cu = batch->cu;
  p.n_seqs = batch->n_seqs;
  p.cap = batch->max_pages * c.page_size;
  p.n_tokens = n_tokens;
  p.n_pages = c.n_pages;
  p.page_shift = log2_of(c.page_size);
  p.kv_heads = c.n_kv_heads;
  p.group = group;
  // a limit past every distance is none
  p.left = a->cfg.left >= p.cap + n_tokens ? -1 : a->cfg.left;
  p.right = a->cfg.right >= p.cap + n_tokens ? -1 : a->cfg.right;
  p.scale2 = a->cfg.scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(out->p);
  p.o_tok = out->token_stride;
  p.o_head = out->head_stride;
  p.lse = lse;
  p.part = reinterpret_cast<float4*>(a->ws + a->L.part);
  p.ml = reinterpret_cast<float2*>(a->ws + a->L.ml);
  p.rec = reinterpret_cast<JoinRec*>(a->ws + a->L.rec);
  p.status = reinterpret_cast<DevStatus*>(a->ws + a->L.status);
  // Many, head size 256: a pair, and teams of two pairs when there are that
  // many tiles (us teams of two CTAs / four: 113 / 174 at 256 rows, 202 / 181 at
  // 512).  Up to 128: every CTA by itself, unless a sequence's keys and values
  // can be past the L2 (129 MB) and its tiles are many: then teams of four read
  // them from memory once (heads of 128, 4 query heads on each of 8, us by
  // itself / four: 4096 tokens behind 131072 6350 / 5712, behind 12288 572 / 615;
  // 12 sequences of 20 to 600 283 / 357).
  const int wide = c.head_dim == 256 ? kRows : 2 * kRows;
  const int64_t seq_bytes = (int64_t)batch->max_pages * ps * c.n_kv_heads * c.head_dim * 4;
  const bool past_l2 = seq_bytes > ((int64_t)256 << 20);
  if (!many) p.team = 1;
  else if (c.head_dim == 256) p.team = rows > 2 * wide ? 4 : 2;
  else p.team = rows > 4 * wide && past_l2 ? 4 : 1;
  // Ending one item and beginning the next, in key tiles: results to write, and
  // a pipeline to fill again (8 canvases at 0, 2, 4, 6, 8: 120, 117, 114, 111,
  // 110 us; the other two barely move).
  p.over = !many ? 1 : (c.head_dim == 256 ? 6 : 2);
  *takes_many = many;
  return DG_OK;
}

}  // namespace

namespace dg {
namespace host {
bool clear_status(void* word, size_t bytes) {
  return cudaMemset(word, 0, bytes) == cudaSuccess && cudaStreamSynchronize(nullptr) == cudaSuccess;
}

dg_status_t read_status(void* word, dg_stream_t stream, unsigned int* where, unsigned int* info) {
  // all on the caller's stream: it need not be ordered with the default one
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DevStatus st;
  if (cudaMemcpyAsync(&st, word, sizeof(st), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemsetAsync(word, 0, sizeof(st), s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return DG_ERR_CUDA;
  if (where) *where = st.where;
  if (info) *info = st.info0;
  if (st.code == kDevTimeout) return DG_ERR_TIMEOUT;
  if (st.code == kDevBounds) return DG_ERR_DEVICE_CHECK;
  return DG_OK;
}
}  // namespace host
}  // namespace dg

extern "C" {

dg_status_t dg_attn_workspace_size(const dg_attn_config_t* cfg, const dg_kv_t* kv, size_t* bytes) {
  if (!bytes) return DG_ERR_INVALID_ARG;
  const dg_status_t s = check_config(cfg, kv);
  if (s != DG_OK) return s;
  *bytes = layout_of(kv->cfg.head_dim).total;
  return DG_OK;
}

dg_status_t dg_attn_create(const dg_attn_config_t* cfg, const dg_kv_t* kv, void* workspace,
                           size_t workspace_bytes, dg_attn_t** out) {
  if (!out) return DG_ERR_INVALID_ARG;
  *out = nullptr;
  const dg_status_t s = check_config(cfg, kv);
  if (s != DG_OK) return s;
  const Layout L = layout_of(kv->cfg.head_dim);
  if (!workspace || workspace_bytes < L.total || !aligned(workspace, 1024)) return DG_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return DG_ERR_CUDA;
  const cudaError_t e = kv->cfg.dtype == DG_T_FP16 ? prepare_dim<true>(kv->cfg.head_dim)
                                                   : prepare_dim<false>(kv->cfg.head_dim);
  if (e != cudaSuccess || prepare_weights(kv->cfg.head_dim) != cudaSuccess) return DG_ERR_CUDA;
  if (!clear_status(static_cast<uint8_t*>(workspace) + L.status, sizeof(DevStatus)))
    return DG_ERR_CUDA;
  dg_attn* a = new (std::nothrow) dg_attn();
  if (!a) return DG_ERR_CUDA;
  a->cfg = *cfg;
  a->kv = kv;
  a->ws = static_cast<uint8_t*>(workspace);
  a->L = L;
  a->ctas = sms < kMaxCtas ? sms : kMaxCtas;
  *out = a;
  return DG_OK;
}

dg_status_t dg_attn_destroy(dg_attn_t* a) {
  delete a;
  return DG_OK;
}

dg_status_t dg_attn_forward(dg_attn_t* a, int layer, const dg_heads_t* q, const dg_heads_t* out,
                            float* lse, const dg_kv_batch_t* batch, int n_tokens,
                            dg_stream_t stream) {
  bool done, many;
  dg_status_t st = check_call(a, layer, q, out, lse, batch, n_tokens, &done);
  if (st != DG_OK || done) return st;
  const int group = a->cfg.n_q_heads / a->kv->cfg.n_kv_heads;
  const int64_t rows = (int64_t)n_tokens * group / batch->n_seqs;
  AttnParams p;
  st = set_up(a, layer, q, out, lse, batch, n_tokens, rows, p, &many);
  return st != DG_OK ? st : run_call(a, many, p, stream);
}

dg_status_t dg_attn_shared_workspace_size(const dg_attn_config_t* cfg, const dg_kv_t* kv,
                                          int n_tokens, size_t* bytes) {
  if (!bytes) return DG_ERR_INVALID_ARG;
  const dg_status_t s = check_config(cfg, kv);
  if (s != DG_OK) return s;
  if (n_tokens < 0) return DG_ERR_INVALID_ARG;
  if (n_tokens > kMaxKvTokens) return DG_ERR_UNSUPPORTED;
  *bytes = pre_layout(*cfg, kv->cfg, n_tokens).total;
  return DG_OK;
}

dg_status_t dg_attn_forward_shared(dg_attn_t* a, int layer, const dg_heads_t* q,
                                   const dg_heads_t* out, float* lse, const dg_kv_batch_t* batch,
                                   const dg_attn_shared_t* shared, int n_tokens,
                                   dg_stream_t stream) {
  bool done, many;
  dg_status_t st = check_call(a, layer, q, out, lse, batch, n_tokens, &done);
  if (st != DG_OK || done) return st;
  if (!shared || shared->n_groups < 0) return DG_ERR_INVALID_ARG;
  if (shared->n_groups > kMaxSeqs) return DG_ERR_UNSUPPORTED;
  if (!shared->prefix || (shared->n_groups && !shared->groups)) return DG_ERR_INVALID_ARG;
  if (!aligned(shared->prefix, 4) || !aligned(shared->groups, 4)) return DG_ERR_ALIGNMENT;
  const dg_kv_config_t& c = a->kv->cfg;
  const PreLayout L = pre_layout(a->cfg, c, n_tokens);
  if (!shared->workspace || shared->workspace_bytes < L.total ||
      !aligned(shared->workspace, 1024))
    return DG_ERR_WORKSPACE;
  const int group = a->cfg.n_q_heads / c.n_kv_heads;
  const int64_t rows = (int64_t)n_tokens * group / batch->n_seqs;
  // One by one: with many rows a sequence the keys are read once for all of them
  // anyway; and where all that the sequences can hold is little, a second launch
  // costs more than reading a prefix again, mostly from the L2 (2 to 32 sequences,
  // one token each, us one by one / together: at 140 to 170 MB 24 / 29, 24 / 34, 44 /
  // 47; at 270 to 300 MB 65 / 47, 34 / 31, 30 / 32; at 550 to 600 MB 60 / 55, 48 / 35).
  // It is the table's room that the host knows, not the lengths: short sequences in a
  // wide table go together all the same (4 behind 2000 tokens, room for 131072 each: 23
  // together, 13 one by one).
  const int64_t held = (int64_t)batch->n_seqs * batch->max_pages * c.page_size * c.n_kv_heads *
                       c.head_dim * 4;
  if (shared->n_groups == 0 || a->cfg.left >= 0 || rows > kMaxSharedRows ||
      held <= ((int64_t)256 << 20))
    return dg_attn_forward(a, layer, q, out, lse, batch, n_tokens, stream);
  uint8_t* ws = static_cast<uint8_t*>(shared->workspace);
  auto with = [&](PreParams& p) {
    p.pre = reinterpret_cast<float4*>(ws + L.o);
    p.pre_ml = reinterpret_cast<float2*>(ws + L.ml);
    p.prefix = shared->prefix;
    p.groups = shared->groups;
    p.n_real = batch->n_seqs;
  };
  SuffixParams own;
  bool unused;
  st = set_up(a, layer, q, out, lse, batch, n_tokens, 1, own, &unused);
  if (st != DG_OK) return st;
  with(own);
  own.part = reinterpret_cast<float4*>(ws + L.part);
  own.ml = reinterpret_cast<float2*>(ws + L.part_ml);
  own.rec = reinterpret_cast<JoinRec*>(ws + L.rec);
  // A prefix's items are split into many parts, and parts of few rows cost less to
  // write and join (behind 16384 tokens, us few / many: head size 64 39.6 / 40.4 at
  // 256 rows, 58.6 / 56.3 at 512; 128: 45.7 / 51.8, 69.7 / 75.4, at 2048 rows behind
  // 65536 643 / 392; 256: 58.8 / 66.8 at 128, 78.2 / 73.6 at 192).  By the average of
  // the groups, those without a fork counted too.
  PrefixParams prefix;
  const int64_t prefix_rows = (int64_t)n_tokens * group / shared->n_groups;
  st = set_up(a, layer, q, out, lse, batch, n_tokens,
              prefix_rows > (c.head_dim == 256 ? 160 : 512) ? prefix_rows : 1, prefix, &many);
  if (st != DG_OK) return st;
  with(prefix);
  prefix.n_seqs = shared->n_groups;
  prefix.left = prefix.right = -1;
  st = run_call(a, false, own, stream);
  return st != DG_OK ? st : run_call(a, many, prefix, stream);
}

dg_status_t dg_attn_last_device_status(dg_attn_t* a, dg_stream_t stream, unsigned int* where,
                                       unsigned int* info) {
  if (!a) return DG_ERR_INVALID_ARG;
  return read_status(a->ws + a->L.status, stream, where, info);
}

}  // extern "C"
