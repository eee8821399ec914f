// Rotary positions, and the append of new tokens to the paged cache with the
// rotation fused (include/dg_attn.h).
//
// The angle of position p and pair i is p f_i modulo one turn.  With
// F_i = round(2^64 f_i / 2 pi) the product p F_i mod 2^64 is that fraction of
// a turn in 64-bit fixed point: exact but for |p| 2^-65 turns, whatever the
// position, with one integer product and no 64-bit floating point.  Its top 32
// bits go through sincospi.
//
// Bound by memory: every element is read once and written once.  A block
// takes a few tokens: each thread requests its elements, the block computes
// the cosines of its tokens (shared by all heads) while they arrive, then
// rotates and stores.  On one GB300: 16384 tokens of 24 heads of 256, half of
// each rotated, 63.5 us (6.35 TB/s); the append of 64 canvases of 256 tokens,
// 16 query and 8 key/value heads of 256, 89.5 us (6.0 TB/s: the tokens' pages
// have to be looked up first); one step of 64 sequences 3.5 us.
#include <math.h>

#include <new>

#include <cuda_fp16.h>

#include "../../include/dg_attn.h"
#include "dg_attn_host.h"
#include "dg_common.cuh"

using namespace dg;
using namespace dg::host;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;  // tokens of a block
constexpr int kUnits = 2;       // units a thread holds in flight

enum : unsigned int { kSiteAppendPos = 40, kSiteAppendPage = 41 };

// One of up to three tensors of a call.
struct Part {
  const void* src;
  void* dst;
  int64_t s_tok, s_head, d_tok, d_head, d_page;
  int rotated;  // else copied
  int paged;    // rows of dst are (page, token of the page)
};

struct RopeParams {
  Part part[3];
  int first[2];  // first head of parts 1 and 2 among the heads of a token
  int heads;     // of a token, all parts
  // Units of a head: vector path: two 16-byte vectors; else one pair or
  // element.  unit_magic, head_magic: ceil(2^32 / x) for quotients of small
  // numbers.
  int units;
  uint32_t unit_magic, head_magic;
  int n_tokens, per_block;
  int dim, half, interleaved, grad;
  float amplitude;
  const int32_t* positions;
  const int32_t* table;  // null: no cache
  const int32_t* lens;
  const int32_t* cu;
  int64_t table_stride;
  int n_seqs, max_pages, page_shift, n_pages;
  DevStatus* status;
  uint64_t turn[256];
};

template <typename T>
struct Vec {  // 16 bytes
  static constexpr int N = 16 / (int)sizeof(T);
};
__device__ __forceinline__ float to_f(uint16_t v, __nv_bfloat16*) { return bf16_to_f32(v); }
__device__ __forceinline__ float to_f(uint16_t v, __half*) {
  return __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ uint16_t from_f(float v, __nv_bfloat16*) { return f32_to_bf16_rne(v); }
__device__ __forceinline__ uint16_t from_f(float v, __half*) {
  return __half_as_ushort(__float2half_rn(v));
}
template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[Vec<T>::N]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = to_f((uint16_t)(w[i] & 0xffffu), (T*)nullptr);
      f[2 * i + 1] = to_f((uint16_t)(w[i] >> 16), (T*)nullptr);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[Vec<T>::N]) {
  uint32_t w[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (uint32_t)from_f(f[2 * i], (T*)nullptr) |
             ((uint32_t)from_f(f[2 * i + 1], (T*)nullptr) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ float get(const T* p) {
  if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float*>(p);
  else return to_f(*reinterpret_cast<const uint16_t*>(p), (T*)nullptr);
}
template <typename T>
__device__ __forceinline__ void put(T* p, float v) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float*>(p) = v;
  else *reinterpret_cast<uint16_t*>(p) = from_f(v, (T*)nullptr);
}

// The sequence that holds row `tok`: the last s with cu[s] <= tok, or -1.  A
// warp probes 32 places a round.
__device__ __forceinline__ int find_seq(const int32_t* cu, int n, int tok, int lane) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;
    const bool below = at < hi && __ldg(cu + at) <= tok;
    const int k = __popc(__ballot_sync(0xffffffffu, below));
    const int nlo = lo + k * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  return (__ldg(cu + lo) <= tok && tok < __ldg(cu + lo + 1)) ? lo : -1;
}

// Quotient by d with its magic number m: exact while x (m d - 2^32) < 2^32, and
// m d - 2^32 < d.
__device__ __forceinline__ int quot(int x, uint32_t magic) {
  return magic ? (int)__umulhi((uint32_t)x, magic) : x;  // 0: divisor 1
}

// VEC: a unit is two 16-byte vectors of a head: in the half layout the two
// halves of eight (four) pairs, else, and where nothing rotates, neighbours.
// Otherwise a unit is one pair or one copied element.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, VEC ? 6 : 4)
    k_rope(const __grid_constant__ RopeParams p) {
  constexpr int N = Vec<T>::N;
  // Cosines and sines of the block's tokens.  Pair i of a token lies at column
  // i / PAIRS of row i % PAIRS: the threads of neighbouring units read
  // neighbouring places (in the order of the pairs they met in the same banks:
  // an append of 64 canvases took 119 us).
  constexpr int PAIRS = VEC ? N : 1;  // of a unit
  extern __shared__ float2 cs[];
  __shared__ int s_pos[kMaxTokens], s_page[kMaxTokens], s_rot[kMaxTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  const int t0 = blockIdx.x * p.per_block;
  const int nt = min(p.per_block, p.n_tokens - t0);
  const int total = nt * p.heads * p.units;

  struct Unit {
    int tok, head, u;  // head among those of the token
  };
  auto locate = [&](int x) {
    Unit a;
    const int row = quot(x, p.unit_magic);
    a.u = x - row * p.units;
    a.tok = quot(row, p.head_magic);
    a.head = row - a.tok * p.heads;
    return a;
  };
  auto part_of = [&](Unit& a) -> const Part& {
    const int i = (a.head >= p.first[0]) + (a.head >= p.first[1]);
    a.head -= i == 0 ? 0 : p.first[i - 1];
    return p.part[i];
  };
  // first elements of a unit's two vectors (scalars; e1 < 0: only one), and
  // whether they rotate
  auto place = [&](const Part& q, int u, int& e0, int& e1) {
    const int half = q.rotated ? p.half : 0;
    if (VEC) {
      if (!p.interleaved && u * N < half) {
        e0 = u * N;
        e1 = e0 + half;
        return true;
      }
      e0 = 2 * u * N;
      e1 = e0 + N;
      return p.interleaved && e0 < 2 * half;
    }
    if (u < half) {
      e0 = p.interleaved ? 2 * u : u;
      e1 = p.interleaved ? e0 + 1 : half + u;
      return true;
    }
    e0 = half + u;
    e1 = -1;
    // heads of more units than a copied one has
    if (e0 >= p.dim) e0 = -1;
    return false;
  };

  uint4 va[kUnits], vb[kUnits];
  auto load = [&](int i, Unit a) {
    const Part& q = part_of(a);
    const T* src = static_cast<const T*>(q.src) + (int64_t)(t0 + a.tok) * q.s_tok +
                   (int64_t)a.head * q.s_head;
    int e0, e1;
    place(q, a.u, e0, e1);
    if (VEC) {
      va[i] = __ldcs(reinterpret_cast<const uint4*>(src + e0));
      vb[i] = __ldcs(reinterpret_cast<const uint4*>(src + e1));
    } else {
      if (e0 >= 0) va[i].x = __float_as_uint(get(src + e0));
      if (e1 >= 0) vb[i].x = __float_as_uint(get(src + e1));
    }
  };
  auto finish = [&](int i, Unit a) {
    const Part& q = part_of(a);
    T* dst = static_cast<T*>(q.dst) + (int64_t)a.head * q.d_head;
    if (q.paged) {
      const int page = s_page[a.tok];
      if (page < 0) return;
      dst += (int64_t)page * q.d_page +
             (int64_t)(s_pos[a.tok] & ((1 << p.page_shift) - 1)) * q.d_tok;
    } else {
      if (p.table && s_page[a.tok] == -2) return;  // outside every sequence
      dst += (int64_t)(t0 + a.tok) * q.d_tok;
    }
    int e0, e1;
    const bool rot = place(q, a.u, e0, e1);
    const float2* c = cs + a.tok * p.half + a.u;
    const int cols = p.half / PAIRS;
    if (VEC) {
      if (rot) {
        float x[N], y[N];
        unpack<T>(va[i], x);
        unpack<T>(vb[i], y);
        if (p.interleaved) {
#pragma unroll
          for (int k = 0; k < N; k += 2) {
            const float2 w = c[(k >> 1) * cols], z = c[((N + k) >> 1) * cols];
            const float x0 = fmaf(x[k], w.x, -x[k + 1] * w.y);
            const float y0 = fmaf(y[k], z.x, -y[k + 1] * z.y);
            x[k + 1] = fmaf(x[k + 1], w.x, x[k] * w.y);
            y[k + 1] = fmaf(y[k + 1], z.x, y[k] * z.y);
            x[k] = x0;
            y[k] = y0;
          }
        } else {
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const float2 w = c[k * cols];
            const float x0 = fmaf(x[k], w.x, -y[k] * w.y);
            y[k] = fmaf(y[k], w.x, x[k] * w.y);
            x[k] = x0;
          }
        }
        va[i] = pack<T>(x);
        vb[i] = pack<T>(y);
      }
      *reinterpret_cast<uint4*>(dst + e0) = va[i];
      *reinterpret_cast<uint4*>(dst + e1) = vb[i];
    } else if (rot) {
      const float2 w = *c;
      const float x = __uint_as_float(va[i].x), y = __uint_as_float(vb[i].x);
      put(dst + e0, fmaf(x, w.x, -y * w.y));
      put(dst + e1, fmaf(y, w.x, x * w.y));
    } else if (e0 >= 0) {
      put(dst + e0, __uint_as_float(va[i].x));
    }
  };

#pragma unroll
  for (int i = 0; i < kUnits; ++i)
    if (tid + i * kThreads < total) load(i, locate(tid + i * kThreads));
  if (p.table) {
    for (int t = warp; t < nt; t += kThreads / 32) {
      const int s = find_seq(p.cu, p.n_seqs, t0 + t, lane);
      if (lane == 0) {
        int page = -2, pos = 0;
        if (s >= 0) {
          page = -1;
          pos = __ldg(p.lens + s) - (__ldg(p.cu + s + 1) - (t0 + t));
          const int pg = pos >> p.page_shift;
          if (pos < 0 || pg >= p.max_pages) {
            report(p.status, kDevBounds, kSiteAppendPos, (unsigned)(t0 + t), (unsigned)pos);
          } else {
            page = __ldg(p.table + (int64_t)s * p.table_stride + pg);
            if ((unsigned)page >= (unsigned)p.n_pages) {
              report(p.status, kDevBounds, kSiteAppendPage, (unsigned)(t0 + t), (unsigned)page);
              page = -1;
            }
          }
        }
        s_page[t] = page;
        s_pos[t] = pos;
        s_rot[t] = p.positions ? __ldg(p.positions + t0 + t) : pos;
      }
    }
    __syncthreads();
  }
  for (int x = tid; x < nt * p.half; x += kThreads) {
    const int t = x / p.half, y = x - t * p.half, cols = p.half / PAIRS;
    const int i = y % cols * PAIRS + y / cols;
    const int pos = p.table ? s_rot[t] : __ldg(p.positions + t0 + t);
    const uint64_t a = p.turn[i] * (uint64_t)(int64_t)pos;
    float s, c;
    sincospif((float)(int32_t)(a >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    cs[x] = make_float2(c * p.amplitude, (p.grad ? -s : s) * p.amplitude);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
    if (tid + i * kThreads < total) finish(i, locate(tid + i * kThreads));
  for (int x0 = tid + kUnits * kThreads; x0 < total; x0 += kUnits * kThreads) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (x0 + i * kThreads < total) load(i, locate(x0 + i * kThreads));
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (x0 + i * kThreads < total) finish(i, locate(x0 + i * kThreads));
  }
}

// Whether every part can be moved in pairs of 16-byte vectors.
template <typename T>
bool vector_ok(const RopeParams& p, int n_parts, int dim, int rot) {
  const int n = Vec<T>::N;
  if (dim % (2 * n) || rot % (2 * n)) return false;
  for (int i = 0; i < n_parts; ++i) {
    const Part& q = p.part[i];
    if (!aligned(q.src, 16) || !aligned(q.dst, 16)) return false;
    for (const int64_t s : {q.s_tok, q.s_head, q.d_tok, q.d_head, q.d_page})
      if (s % n) return false;
  }
  return true;
}

// The quotients by magic numbers are exact for this many.
bool heads_ok(int heads, int dim) { return heads <= 16384 && (int64_t)heads * dim <= 1 << 22; }

uint32_t magic_of(int d) { return d <= 1 ? 0 : (uint32_t)((((uint64_t)1 << 32) + d - 1) / d); }

template <typename T>
cudaError_t launch(RopeParams& p, int n_parts, const int* heads, int dim, int rot,
                   cudaStream_t s) {
  const bool vec = vector_ok<T>(p, n_parts, dim, rot);
  bool copies = false;
  for (int i = 0; i < n_parts; ++i) copies = copies || !p.part[i].rotated;
  p.dim = dim;
  p.half = rot / 2;
  p.units = vec ? dim / (2 * Vec<T>::N) : (copies ? dim : dim - p.half);
  p.heads = 0;
  for (int i = 0; i < n_parts; ++i) {
    if (i) p.first[i - 1] = p.heads;
    p.heads += heads[i];
  }
  for (int i = n_parts; i < 3; ++i) p.first[i - 1] = p.heads;  // nothing from here on
  p.unit_magic = magic_of(p.units);
  p.head_magic = magic_of(p.heads);
  // Several blocks an SM (of 152) before a block takes more than one token, at
  // most 32 KB of cosines, and about kUnits units a thread, twice that where no
  // token is looked up (16384 x 24 x 256: 63.3 us so, 67.5 with kUnits; an
  // append of 64 canvases 90.9 and 89.4 us).
  const int64_t token_units = (int64_t)p.heads * p.units;
  int per = (int)((p.table ? 1 : 2) * kUnits * kThreads / token_units);
  const int spread = p.n_tokens / (152 * 4);
  if (per > spread) per = spread;
  if (per > kMaxTokens) per = kMaxTokens;
  if (p.half > 0 && per > 4096 / p.half) per = 4096 / p.half;
  if (per < 1) per = 1;
  p.per_block = per;
  const dim3 grid((p.n_tokens + per - 1) / per);
  const size_t smem = (size_t)per * p.half * sizeof(float2);
  return vec ? launch_pdl(k_rope<T, true>, grid, dim3(kThreads), smem, s, p)
             : launch_pdl(k_rope<T, false>, grid, dim3(kThreads), smem, s, p);
}

void set_rope(RopeParams& p, const dg_rope* r) {
  p.interleaved = r->cfg.layout == DG_ROPE_INTERLEAVED;
  p.amplitude = (float)r->cfg.amplitude;
  for (int i = 0; i < r->cfg.rot_dim / 2; ++i) p.turn[i] = r->turn[i];
}

dg_status_t check_rope_heads(const dg_heads_t* t, size_t elem) {
  if (!t || !t->p) return DG_ERR_INVALID_ARG;
  if (t->token_stride < 0 || t->head_stride < 0) return DG_ERR_INVALID_ARG;
  if (!aligned(t->p, elem)) return DG_ERR_ALIGNMENT;
  return DG_OK;
}

}  // namespace

extern "C" {

dg_status_t dg_rope_create(const dg_rope_config_t* cfg, dg_rope_t** out) {
  if (!out) return DG_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg || cfg->flags != 0) return DG_ERR_INVALID_ARG;
  const dg_rope_config_t& c = *cfg;
  if (c.head_dim < 2 || c.rot_dim < 2 || c.rot_dim > c.head_dim || c.rot_dim % 2)
    return DG_ERR_INVALID_ARG;
  if (c.head_dim > 512) return DG_ERR_UNSUPPORTED;
  if (c.layout != DG_ROPE_HALF && c.layout != DG_ROPE_INTERLEAVED) return DG_ERR_INVALID_ARG;
  if (!(c.theta > 1.0) || !isfinite(c.theta)) return DG_ERR_INVALID_ARG;
  if (!(c.amplitude > 0.0) || !isfinite(c.amplitude)) return DG_ERR_INVALID_ARG;
  if (c.scaling < DG_ROPE_PLAIN || c.scaling > DG_ROPE_RAMP) return DG_ERR_INVALID_ARG;
  if (c.scaling != DG_ROPE_PLAIN && (!(c.factor >= 1.0) || !isfinite(c.factor)))
    return DG_ERR_INVALID_ARG;
  if (c.scaling == DG_ROPE_BASE && c.rot_dim < 4) return DG_ERR_INVALID_ARG;
  if (c.scaling == DG_ROPE_RAMP &&
      (!(c.orig_len > 0.0) || !isfinite(c.orig_len) || !(c.beta_slow >= 0.0) ||
       !(c.beta_fast > c.beta_slow) || !isfinite(c.beta_fast)))
    return DG_ERR_INVALID_ARG;
  dg_rope* r = new (std::nothrow) dg_rope();
  if (!r) return DG_ERR_CUDA;
  r->cfg = c;
  const double two_pi = 6.283185307179586476925286766559;
  double theta = c.theta;
  if (c.scaling == DG_ROPE_BASE) theta *= pow(c.factor, c.rot_dim / (c.rot_dim - 2.0));
  for (int i = 0; i < c.rot_dim / 2; ++i) {
    double f = pow(theta, -2.0 * i / c.rot_dim);
    if (c.scaling == DG_ROPE_LINEAR) f /= c.factor;
    if (c.scaling == DG_ROPE_RAMP) {
      double g = (c.orig_len * f / two_pi - c.beta_slow) / (c.beta_fast - c.beta_slow);
      g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
      f = g * f + (1.0 - g) * f / c.factor;
    }
    // f <= 1, so the product is below 2^62
    r->turn[i] = (uint64_t)llrint(ldexp(f / two_pi, 64));
  }
  *out = r;
  return DG_OK;
}

dg_status_t dg_rope_destroy(dg_rope_t* r) {
  delete r;
  return DG_OK;
}

dg_status_t dg_rope_apply(const dg_rope_t* r, dg_dtype_t dtype, const dg_heads_t* x,
                          const dg_heads_t* out, const int32_t* positions, int n_tokens,
                          int n_heads, int grad, dg_stream_t stream) {
  if (!r || n_tokens < 0 || n_heads < 0) return DG_ERR_INVALID_ARG;
  if (dtype != DG_T_BF16 && dtype != DG_T_FP16 && dtype != DG_T_FP32) return DG_ERR_INVALID_ARG;
  if (n_tokens == 0 || n_heads == 0) return DG_OK;
  const size_t elem = dtype == DG_T_FP32 ? 4 : 2;
  dg_status_t st;
  if ((st = check_rope_heads(x, elem)) != DG_OK || (st = check_rope_heads(out, elem)) != DG_OK)
    return st;
  if (!positions) return DG_ERR_INVALID_ARG;
  if (!aligned(positions, 4)) return DG_ERR_ALIGNMENT;
  if (!heads_ok(n_heads, r->cfg.head_dim)) return DG_ERR_UNSUPPORTED;
  RopeParams p = {};
  set_rope(p, r);
  p.part[0] = Part{x->p, out->p, x->token_stride, x->head_stride, out->token_stride,
                   out->head_stride, 0, 1, 0};
  p.n_tokens = n_tokens;
  p.grad = grad != 0;
  p.positions = positions;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int d = r->cfg.head_dim, rd = r->cfg.rot_dim;
  const cudaError_t e = dtype == DG_T_BF16   ? launch<__nv_bfloat16>(p, 1, &n_heads, d, rd, s)
                        : dtype == DG_T_FP16 ? launch<__half>(p, 1, &n_heads, d, rd, s)
                                             : launch<float>(p, 1, &n_heads, d, rd, s);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

dg_status_t dg_kv_append(dg_kv_t* kv, int layer, const dg_rope_t* rope, const dg_heads_t* k,
                         const dg_heads_t* v, const dg_heads_t* q, const dg_heads_t* q_out,
                         int n_q_heads, const dg_kv_batch_t* batch, const int32_t* positions,
                         int n_tokens, dg_stream_t stream) {
  if (!kv) return DG_ERR_INVALID_ARG;
  const dg_kv_config_t& c = kv->cfg;
  if (layer < 0 || layer >= c.n_layers || n_tokens < 0) return DG_ERR_INVALID_ARG;
  if (rope && rope->cfg.head_dim != c.head_dim) return DG_ERR_INVALID_ARG;
  dg_status_t st = check_batch(batch, c);
  if (st != DG_OK) return st;
  if (n_tokens > kMaxKvTokens) return DG_ERR_UNSUPPORTED;
  if (n_tokens == 0 || batch->n_seqs == 0) return DG_OK;
  if ((st = check_heads(k)) != DG_OK || (st = check_heads(v)) != DG_OK) return st;
  if (q) {
    if (n_q_heads <= 0) return DG_ERR_INVALID_ARG;
    if (!heads_ok(n_q_heads, c.head_dim)) return DG_ERR_UNSUPPORTED;
    if ((st = check_heads(q)) != DG_OK || (st = check_heads(q_out)) != DG_OK) return st;
  }
  if (!batch->page_table) return DG_ERR_INVALID_ARG;
  if (positions && !aligned(positions, 4)) return DG_ERR_ALIGNMENT;
  RopeParams p = {};
  p.amplitude = 1.f;
  if (rope) set_rope(p, rope);
  int heads[3], parts = 0;
  auto add = [&](const dg_heads_t* src, int n, bool rot, const dg_kv_pool_t* pool,
                 const dg_heads_t* dst) {
    heads[parts] = n;
    if (pool)
      p.part[parts] = Part{src->p, static_cast<uint16_t*>(pool->p) + layer * pool->layer_stride,
                           src->token_stride, src->head_stride, pool->token_stride,
                           pool->head_stride, pool->page_stride, rot, 1};
    else
      p.part[parts] = Part{src->p, dst->p, src->token_stride, src->head_stride,
                           dst->token_stride, dst->head_stride, 0, rot, 0};
    ++parts;
  };
  add(k, c.n_kv_heads, rope != nullptr, &c.k, nullptr);
  add(v, c.n_kv_heads, false, &c.v, nullptr);
  if (q) add(q, n_q_heads, rope != nullptr, nullptr, q_out);
  p.n_tokens = n_tokens;
  p.positions = positions;
  p.table = batch->page_table;
  p.lens = batch->lens;
  p.cu = batch->cu;
  p.table_stride = batch->table_stride;
  p.n_seqs = batch->n_seqs;
  p.max_pages = batch->max_pages;
  p.page_shift = log2_of(c.page_size);
  p.n_pages = c.n_pages;
  p.status = static_cast<DevStatus*>(kv->status);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rd = rope ? rope->cfg.rot_dim : 0;
  const cudaError_t e = c.dtype == DG_T_BF16
                            ? launch<__nv_bfloat16>(p, parts, heads, c.head_dim, rd, s)
                            : launch<__half>(p, parts, heads, c.head_dim, rd, s);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

}  // extern "C"
