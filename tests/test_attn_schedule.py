"""How k_paged_attn deals its work (moe_expert_ffn_dg_gb300/csrc/dg_attn.cu).

The items of a call (key/value head, sequence, team's tile of query rows) are
cut into units, a team of CTAs takes a contiguous range of them, and beginning
an item costs units of its own once every team has several times that to do.
The kernel's own code of key ranges and of the walk over a range is compiled
for the host here; where a range begins is worked out again from its
definition.  Checked for every call: each item's key tiles are taken exactly
once, in order, by neighbouring teams; the first of them knows how many there
are; no CTA uses a place of the workspace twice; a team's CTAs split its rows."""

import ctypes
import os
import random
import subprocess

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(__file__)), "moe_expert_ffn_dg_gb300", "csrc",
                   "dg_attn.cu")

HEAD = r"""
#include <stdint.h>
#include <algorithm>
#include <map>
#include <tuple>
#include <vector>
using std::max; using std::min;
#define __device__
#define __forceinline__ inline
template <typename T> T __ldg(const T* p) { return *p; }
struct int2 { int x, y; };
static int2 make_int2(int x, int y) { return int2{x, y}; }
static struct { unsigned x; } blockIdx;
constexpr int kKeys = 128;
struct AttnParams {
  const int32_t *lens, *cu;
  int n_seqs, cap, n_tokens, kv_heads, step, team, over, left, right;
};
"""

TAIL = r"""
struct Begin { int h, b, t, skip; long long u, end; };

// The range of team c: units [c total / teams, (c + 1) total / teams) of all
// items in order, an item being `over` units and one a key tile (at least one).
template <int NQ>
static Begin begin_of(const AttnParams& p, int c, int over, long long total, int teams) {
  Begin r{0, 0, 0, 0, 0, 0};
  if (c >= teams) return r;
  r.u = c * total / teams;
  r.end = (c + 1) * total / teams;
  if (r.u >= r.end) return r;
  long long at = 0;
  for (int h = 0; h < p.kv_heads; ++h)
    for (int b = 0; b < p.n_seqs; ++b) {
      const Seq s = load_seq(p, b);
      for (int t = 0; t * item_tokens<NQ>(p) < s.n; ++t) {
        const int cost = over + max(tile_range<NQ>(p, s, t).y, 1);
        if (r.u < at + cost) {
          r.h = h, r.b = b, r.t = t, r.skip = (int)(r.u - at);
          if (r.skip <= over) r.u -= r.skip, r.skip = 0;
          return r;
        }
        at += cost;
      }
    }
  return r;
}

struct Item { int taken, next, teams, last_team, parts, firsts, lasts; std::vector<char> rows; };

// 0, or the number of the check that failed; *used: what a beginning cost.
template <int NQ>
static int simulate(const AttnParams& p, int ctas, int* used) {
  long long tiles = 0, items = 0;
  std::map<std::tuple<int, int, int>, Item> all;
  for (int b = 0; b < p.n_seqs; ++b) {
    const Seq s = load_seq(p, b);
    for (int t = 0; t * item_tokens<NQ>(p) < s.n; ++t) {
      tiles += max(tile_range<NQ>(p, s, t).y, 1);
      ++items;
      for (int h = 0; h < p.kv_heads; ++h)
        all[{h, b, t}] = Item{0, -1, 0, -1, 0, 0, 0,
                              std::vector<char>(min(item_tokens<NQ>(p), s.n - t * item_tokens<NQ>(p)))};
    }
  }
  const int most = ctas / p.team;
  const int over = tiles * p.kv_heads >= (long long)most * max(8, 3 * p.over) ? p.over : 0;
  *used = over;
  const long long total = (tiles + over * items) * p.kv_heads;
  const int teams = (int)min((long long)most, total);
  for (unsigned cta = 0; cta < (unsigned)(most * p.team); ++cta) {
    blockIdx.x = cta;
    const int team = cta / p.team, rank = cta % p.team;
    const Begin g0 = begin_of<NQ>(p, team, over, total, teams);
    Walk<NQ> w;
    w.h = g0.h, w.b = g0.b, w.t = g0.t, w.skip = g0.skip, w.over = over;
    w.u = g0.u, w.end = g0.end;
    w.begin(p);
    Seg g;
    int early = 0, late = 0, segs = 0;
    while (w.next(p, g)) {
      ++segs;
      const Seq s = load_seq(p, g.b);
      const int t = (g.tok0 - s.n0 - rank * NQ * p.step) / item_tokens<NQ>(p);
      auto it = all.find({g.head, g.b, t});
      if (it == all.end()) return 1;
      Item& x = it->second;
      const int2 tr = tile_range<NQ>(p, s, t);
      if (!g.first && (++early > 1 || segs > 1)) return 2;    // one part at the start
      if (late) return 3;                                     // nothing behind an open item
      if (g.first && !g.last) ++late;
      if (g.pos != s.kv - s.n + (g.tok0 - s.n0) || g.kv != s.kv) return 4;
      if (g.n < 0 || (tr.y > 0 && g.n == 0)) return 5;
      if (g.first)
        for (int i = 0; i < g.ntok; ++i) {
          const int at = g.tok0 - s.n0 - t * item_tokens<NQ>(p) + i;
          if (at < 0 || at >= (int)x.rows.size() || x.rows[at]++) return 6;
        }
      if (rank) continue;
      if (g.first) x.firsts++, x.next = tr.x;
      if (g.last) x.lasts++;
      if (g.n && g.kt0 != x.next) return 7;
      x.next = g.kt0 + g.n;
      x.taken += g.n;
      if (x.last_team >= 0 && team != x.last_team + 1) return 8;
      x.last_team = team;
      ++x.teams;
      if (g.first)
        x.parts = g.last ? 1 : (int)((g.end * teams - 1) / total) - team + 1;
    }
  }
  for (auto& e : all) {
    const Item& x = e.second;
    const Seq s = load_seq(p, std::get<1>(e.first));
    if (x.firsts != 1 || x.lasts != 1) return 9;
    if (x.taken != tile_range<NQ>(p, s, std::get<2>(e.first)).y) return 10;
    if (x.parts != x.teams) return 11;
    for (char r : x.rows)
      if (r != 1) return 12;
  }
  return 0;
}

extern "C" int run(int nq, const int32_t* lens, const int32_t* cu, int n_seqs, int cap, int n_tokens,
                   int kv_heads, int step, int team, int over, int left, int right, int ctas,
                   int* used) {
  AttnParams p{lens, cu, n_seqs, cap, n_tokens, kv_heads, step, team, over, left, right};
  return nq == 1 ? simulate<1>(p, ctas, used) : simulate<2>(p, ctas, used);
}
"""


def kernel_code(plant=None):
    """Sequences, key ranges, segments and the walk, as the kernel has them."""
    src = open(SRC).read()
    body = src[src.index("struct Seq {"):src.index("struct Start {")]
    assert "struct Walk" in body and "tile_range" in body
    # what the definitions above take over from find_start and the host
    for line in ("if (skip <= over) {", "max(8, 3 * p.over) ? p.over : 0",
                 "u1 = (long long)(c + 1) * total / teams;",
                 "const long long x = g.end * start.teams - 1;"):
        assert line in src, line
    if plant:
        assert plant[0] in body
        body = body.replace(*plant)
    return body


def library(path, plant=None):
    cpp, so = str(path / "schedule.cpp"), str(path / "schedule.so")
    with open(cpp, "w") as f:
        f.write(HEAD + kernel_code(plant) + TAIL)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wno-unknown-pragmas", "-shared", "-fPIC", "-o", so,
                    cpp], check=True)
    return ctypes.CDLL(so)


def rule(d, many, rows, seq_bytes=0):
    """Tiles of an item's CTA, CTAs of a team and the cost of a beginning, as
    dg_attn_forward chooses them."""
    src = open(SRC).read()
    for line in ("const bool many = rows > (c.head_dim == 256 ? 32 : 128);",
                 "else if (c.head_dim == 256) p.team = rows > 2 * wide ? 4 : 2;",
                 "else p.team = rows > 4 * wide && past_l2 ? 4 : 1;",
                 "p.over = !many ? 1 : (c.head_dim == 256 ? 6 : 2);",
                 "static constexpr int kManyNq = D == 256 ? 1 : 2;"):
        assert line in src, line
    if not many:
        return 1, 1, 1
    if d == 256:
        return 1, 4 if rows > 256 else 2, 6
    return 2, 4 if rows > 1024 and seq_bytes > 256 << 20 else 1, 2


def go(lib, nq, team, over, lens, n, kv_heads, group, left, right, ctas=152, cap=None):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    used = ctypes.c_int(-1)
    arr = [(ctypes.c_int32 * len(a))(*a) for a in (lens, cu)]
    bad = lib.run(nq, *arr, len(lens), cap or max(lens + [1]), cu[-1], kv_heads, 128 // group, team,
                  over, left, right, ctas, ctypes.byref(used))
    return bad, used.value


def case(rng):
    nq, team, over = rng.choice([(1, 1, 1), (2, 1, 2), (2, 4, 2), (1, 2, 6), (1, 4, 6)])
    seqs = rng.choice([1, 2, 7, 40])
    longest, most = rng.choice([50, 900, 9000]), rng.choice([1, 9, 300, 900])
    lens = [rng.choice([0, rng.randint(0, longest), longest]) for _ in range(seqs)]
    n = [rng.choice([0, 1, rng.randint(0, most)]) for _ in range(seqs)]
    n[rng.randrange(seqs)] = rng.randint(1, most)
    group = rng.choice([1, 2, 3, 8, 128])
    if group == 128:
        n = [min(x, 60) for x in n]
    return dict(nq=nq, team=team, over=over, lens=lens, n=n, kv_heads=rng.choice([1, 3, 8]),
                group=group, left=rng.choice([-1, -1, 0, 5, 127, 700]),
                right=rng.choice([0, 0, -1, 3, 200]), ctas=rng.choice([152, 152, 148, 12, 4]))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return library(tmp_path_factory.mktemp("schedule"))


def test_every_tile_is_taken_once(lib):
    costly = 0
    for seed in range(3000):
        c = case(random.Random(seed))
        bad, used = go(lib, **c)
        assert bad == 0, (bad, seed, c)
        costly += used > 0
    assert costly > 500  # of them with beginnings that count


@pytest.mark.parametrize("plant", [
    # a range's last units inside a beginning are worked on here as well
    ("if (skip + take <= over) return false;", ""),
    # a range that begins in an item forgets the beginning's units
    ("const int tile = max(skip - over, 0);", "const int tile = skip;"),
    # the row of a new sequence is one behind
    ("} while (s.n == 0);", "} while (false);")])
def test_planted_mistakes_are_caught(plant, tmp_path):
    bad = library(tmp_path, plant)
    assert any(go(bad, **case(random.Random(seed)))[0] for seed in range(300))
