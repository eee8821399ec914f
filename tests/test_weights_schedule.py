"""How k_weights deals its work (moe_expert_ffn_dg_gb300/csrc/dg_weights.cu).

The kernel's own code of sequences, tile ranges and the walk over a range of
units is compiled for the host; where a range begins is worked out again from its
definition.  Checked for every call: each (256 keys, head, query tile) in which
a token sees a key is taken exactly once and no other is; every block of keys is
written once, by one CTA or as parts of neighbouring ones that the first of them
counts right; no CTA uses a place of the workspace twice."""

import ctypes
import os
import random
import subprocess

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(__file__)), "moe_expert_ffn_dg_gb300", "csrc",
                   "dg_weights.cu")

HEAD = r"""
#include <stdint.h>
#include <algorithm>
#include <map>
#include <set>
#include <tuple>
#include <vector>
using std::max; using std::min;
#define __device__
#define __forceinline__ inline
template <typename T> T __ldg(const T* p) { return *p; }
struct int2 { int x, y; };
static int2 make_int2(int x, int y) { return int2{x, y}; }
constexpr int kWeightKeys = 256;
struct WeightParams {
  const int32_t *lens, *cu;
  int n_seqs, cap, n_tokens, kv_heads, step, left, right, width;
};
"""

TAIL = r"""
// The range of CTA c: units [c total / ctas, (c + 1) total / ctas) of all items
// in order.
static Start begin_of(const WeightParams& p, int c, long long total, int ctas) {
  Start st{0, 0, 0, 0, 0, total, ctas};
  if (c >= ctas) return st;
  st.u = c * total / ctas, st.end = (c + 1) * total / ctas;
  long long at = 0;
  for (int b = 0; b < p.n_seqs; ++b) {
    const Seq s = load_seq(p, b);
    for (int kb = 0; kb < s.blocks; ++kb) {
      const long long n = item_units(p, tile_range(p, s, kb).y);
      if (st.u < at + n) {
        st.b = b, st.kb = kb, st.skip = st.u - at;
        return st;
      }
      at += n;
    }
  }
  return st;
}

struct Item { int whole, begun, ended, next_cta, parts; std::map<std::pair<int, int>, int> tiles; };

static int simulate(const WeightParams& p, int grid) {
  long long total = 0;
  std::map<std::pair<int, int>, Item> all;
  for (int b = 0; b < p.n_seqs; ++b) {
    const Seq s = load_seq(p, b);
    for (int kb = 0; kb < s.blocks; ++kb) {
      total += item_units(p, tile_range(p, s, kb).y);
      all[{b, kb}] = Item{0, 0, 0, -1, 0, {}};
    }
  }
  const int ctas = (int)min((long long)grid, total);
  for (int c = 0; c < grid; ++c) {
    Walk w;
    w.begin(p, begin_of(p, c, total, ctas));
    Seg g;
    std::set<int> slots;
    bool begun = false, open = false;
    long long item_end = 0;
    while (w.next(p, g)) {
      auto it = all.find({g.b, g.kb});
      if (it == all.end()) return 1;
      Item& x = it->second;
      if (g.begins == open) return 2;  // an item's segments are one run
      open = !g.ends;
      if (g.begins) begun = g.first, item_end = g.end;
      else if (g.first) return 3;
      for (int t = 0; t < g.tiles; ++t)
        if (x.tiles[{g.head, g.t0 + t}]++) return 4;
      if (!g.ends) continue;
      if (begun && g.last) { ++x.whole; continue; }
      if (!slots.insert(begun ? 1 : 0).second) return 5;
      if (begun) {
        ++x.begun;
        x.next_cta = c;
        x.parts = (int)((item_end * ctas - 1) / total) - c + 1;
      }
      if (x.next_cta != c) return 6;  // parts of neighbours
      ++x.next_cta;
      if (--x.parts < 0) return 7;
      if (g.last) {
        ++x.ended;
        if (x.parts != 0) return 8;
      }
    }
    if (open) return 9;
  }
  for (auto& e : all) {
    const Item& x = e.second;
    if (x.whole + x.begun != 1 || x.begun != x.ended) return 10;
    const int b = e.first.first, kb = e.first.second;
    const Seq s = load_seq(p, b);
    // token by token and key by key
    std::set<int> want;
    for (int i = 0; i < s.n; ++i) {
      const int pos = s.kv - s.n + i;
      const int lo = p.left < 0 ? 0 : max(0, pos - p.left);
      const int hi = p.right < 0 ? s.kv : min(s.kv, pos + p.right + 1);
      const int k0 = kb * 256, k1 = min(k0 + 256, s.kv);
      if (max(lo, k0) < min(hi, k1)) want.insert(i / p.step);
    }
    // tiles between two that see something count as well
    if (!want.empty())
      for (int t = *want.begin(); t < *want.rbegin(); ++t) want.insert(t);
    if (x.tiles.size() != want.size() * p.kv_heads) return 11;
    for (auto& t : x.tiles)
      if (t.second != 1 || !want.count(t.first.second)) return 12;
  }
  return 0;
}

extern "C" int run(const int32_t* lens, const int32_t* cu, int n_seqs, int cap, int n_tokens,
                   int kv_heads, int step, int left, int right, int width, int grid) {
  WeightParams p{lens, cu, n_seqs, cap, n_tokens, kv_heads, step, left, right, width};
  return simulate(p, grid);
}
"""


def library(path, plant=None):
    src = open(SRC).read()
    body = src[src.index("struct Seq {"):src.index("// Where this CTA's range of units begins.")]
    assert "struct Walk" in body
    for line in ("st.u = c * total / ctas;", "st.end = (c + 1) * total / ctas;",
                 "rec.parts = (int)((item_end * start.ctas - 1) / start.total) - "
                 "(int)blockIdx.x + 1;",
                 "p.part[(2 * blockIdx.x + (begun ? 1 : 0)) * kWeightKeys + mine]"):
        assert line in src, line
    if plant:
        assert plant[0] in body
        body = body.replace(*plant)
    cpp, so = str(path / "weights.cpp"), str(path / "weights.so")
    with open(cpp, "w") as f:
        f.write(HEAD + body + TAIL)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wno-unknown-pragmas", "-shared", "-fPIC", "-o", so,
                    cpp], check=True)
    return ctypes.CDLL(so)


def go(lib, lens, n, kv_heads, group, left, right, cols, grid, width):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    arr = [(ctypes.c_int32 * len(a))(*a) for a in (lens, cu)]
    return lib.run(*arr, len(lens), max(lens + [1]), cu[-1], kv_heads, cols // group, left, right,
                   width, grid)


def case(rng):
    seqs = rng.choice([1, 2, 7, 40])
    longest, most = rng.choice([50, 900, 9000]), rng.choice([1, 9, 300, 900])
    lens = [rng.choice([0, rng.randint(0, longest), longest]) for _ in range(seqs)]
    n = [rng.choice([0, 1, rng.randint(0, most)]) for _ in range(seqs)]
    group = rng.choice([1, 2, 3, 8, 16])
    return dict(lens=lens, n=n, kv_heads=rng.choice([1, 3, 8]), group=group,
                left=rng.choice([-1, -1, 0, 5, 127, 700]), right=rng.choice([0, 0, -1, 3, 200]),
                cols=rng.choice([16, 128]), grid=rng.choice([152, 152, 148, 12, 4]),
                width=rng.choice([max(lens) + 3, max(lens), max(1, max(lens) // 2)]))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return library(tmp_path_factory.mktemp("weights"))


def test_every_tile_is_taken_once(lib):
    for seed in range(1500):
        c = case(random.Random(seed))
        bad = go(lib, **c)
        assert bad == 0, (bad, seed, c)


@pytest.mark.parametrize("plant", [
    ("while (kb >= s.blocks) {", "if (kb >= s.blocks) {"),
    ("g.last = h == p.kv_heads || t.y == 0;", "g.last = h == p.kv_heads;"),
    ("g.ends = g.last || u >= end;", "g.ends = g.last;")])
def test_planted_mistakes_are_caught(plant, tmp_path):
    bad = library(tmp_path, plant)
    found = False
    for seed in range(300):
        c = case(random.Random(seed))
        c["lens"] = [max(1, x) if plant[0].startswith("g.") else x for x in c["lens"]]
        if plant[0].startswith("g.last"):
            c["n"], c["grid"] = [max(1, x) for x in c["n"]], 1  # a single CTA cannot run away
            c["left"] = 0
            c["lens"] = [min(x, 600) for x in c["lens"]]
        if plant[0].startswith("while") and 0 in c["lens"][-1:]:
            continue  # the walk would leave the list
        found = found or go(bad, **c) != 0
        if found:
            break
    assert found
