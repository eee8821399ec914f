"""k_kv_shared (moe_expert_ffn_dg_gb300/csrc/dg_thin.cu) with lanes that run one by
one.

The kernel's own code is compiled for the host, each thread a context of its own
that runs until it waits for others: for its warp, or for the block.  A warp's
lanes need not run together between two waits, so every order has to do: that of
their numbers, the reverse, and random ones.  Checked: nobody waits for a lane that
waits elsewhere or has left, and the prefixes are those of the definition."""

import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from test_attn_sources import CSRC

HEAD = r"""
#include <stdint.h>
#include <string.h>
#include <ucontext.h>
#include <algorithm>
#include <random>
#include <vector>
using std::max; using std::min;
#define __device__
#define __global__
#define __forceinline__ inline
#define __grid_constant__
#define __launch_bounds__(...)
#define __shared__ static
struct Dim { int x; };
static Dim blockIdx, gridDim;
struct DevStatus { int reports; };
enum : unsigned { kDevBounds = 2, kSiteSharedLen = 56, kSiteSharedGroups = 57 };
constexpr int kThinThreads = 128;  // of a block, here
constexpr unsigned kAllLanes = 0xffffffffu;

enum Wait { kRuns, kWarp, kBlock, kGone };
struct Thread { ucontext_t at; Wait wait; int value, from; std::vector<char> stack; };
static Thread threads[kThinThreads];
static ucontext_t scheduler;
static int current;
struct Me { struct { operator int() const { return current; } } x; };
static Me threadIdx;
static void wait_for(Wait w) {
  threads[current].wait = w;
  swapcontext(&threads[current].at, &scheduler);
}
static void __syncthreads() { wait_for(kBlock); }
// What all lanes of a warp bring to a meeting: kept until its last lane has left, as
// none can come to the next one before.
static int brought[2][kThinThreads], turn[kThinThreads];
static const int* meet(int v) {
  int* all = brought[turn[current]++ & 1];
  all[current] = v;
  wait_for(kWarp);
  return all + current / 32 * 32;
}
static int __reduce_min_sync(unsigned, int v) {
  const int* a = meet(v);
  return *std::min_element(a, a + 32);
}
static int __shfl_sync(unsigned, int v, int from) { return meet(v)[from]; }
template <typename T> T __ldg(const T* p) { return *p; }
static int atomicMin(int* p, int v) { int old = *p; *p = min(old, v); return old; }
static void pdl_trigger() {}
static void pdl_wait() {}
static void report(DevStatus* s, unsigned, unsigned, unsigned, unsigned) { ++s->reports; }
"""

TAIL = r"""
static const SharedParams* params;
static void thread_main() {
  k_kv_shared(*params);
  threads[current].wait = kGone;
  swapcontext(&threads[current].at, &scheduler);
}

// 0, or 1: somebody waits for a lane that will not come.
static int block(int order, std::mt19937& rng) {
  std::vector<int> who;
  for (int t = 0; t < kThinThreads; ++t) {
    Thread& x = threads[t];
    if (x.stack.empty()) x.stack.resize(64 << 10);
    getcontext(&x.at);
    x.at.uc_stack.ss_sp = x.stack.data();
    x.at.uc_stack.ss_size = x.stack.size();
    x.at.uc_link = &scheduler;
    makecontext(&x.at, thread_main, 0);
    x.wait = kRuns;
    turn[t] = 0;
    who.push_back(t);
  }
  if (order == 1) std::reverse(who.begin(), who.end());
  while (true) {
    if (order == 2) std::shuffle(who.begin(), who.end(), rng);
    bool ran = false;
    for (int t : who)
      if (threads[t].wait == kRuns) {
        current = t;
        swapcontext(&scheduler, &threads[t].at);
        ran = true;
      }
    int at_block = 0, gone = 0;
    for (int w = 0; w < kThinThreads; w += 32) {
      int n = 0;
      for (int l = 0; l < 32; ++l) n += threads[w + l].wait == kWarp;
      if (n == 32) {
        ran = true;
        for (int l = 0; l < 32; ++l) threads[w + l].wait = kRuns;
      }
      for (int l = 0; l < 32; ++l) {
        at_block += threads[w + l].wait == kBlock;
        gone += threads[w + l].wait == kGone;
      }
    }
    if (gone == kThinThreads) return 0;
    if (at_block && at_block + gone == kThinThreads) {
      for (int t = 0; t < kThinThreads; ++t)
        if (threads[t].wait == kBlock) threads[t].wait = kRuns;
      ran = true;
    }
    if (!ran) return 1;
  }
}

extern "C" int run(const int32_t* table, int64_t stride, const int32_t* lens, const int32_t* cu,
                   const int32_t* groups, int32_t* prefix, int n_seqs, int n_groups, int page_shift,
                   int max_pages, int order, int seed, int* reports) {
  DevStatus st{0};
  SharedParams p;
  p.table = table, p.table_stride = stride, p.lens = lens, p.cu = cu, p.groups = groups;
  p.prefix = prefix, p.n_seqs = n_seqs, p.n_groups = n_groups, p.page_shift = page_shift;
  p.cap = max_pages << page_shift, p.status = &st;
  params = &p;
  std::mt19937 rng(seed);
  gridDim.x = n_groups;
  for (blockIdx.x = 0; blockIdx.x < n_groups; ++blockIdx.x)
    if (const int bad = block(order, rng)) return bad;
  *reports = st.reports;
  return 0;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    src = open(os.path.join(CSRC, "dg_thin.cu")).read()
    body = src[src.index("struct SharedParams {"):src.index("struct SelectParams {")]
    assert "k_kv_shared(" in body and body.count("__shared__") == 1
    path = tmp_path_factory.mktemp("shared")
    cpp, so = str(path / "shared.cpp"), str(path / "shared.so")
    with open(cpp, "w") as f:
        f.write(HEAD + body + TAIL)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wno-unknown-pragmas", "-shared", "-fPIC", "-o", so,
                    cpp], check=True)
    return ctypes.CDLL(so)


def common(table, lens, cu, bounds, page):
    """The definition."""
    out = [0] * len(lens)
    for a, b in zip(bounds[:-1], bounds[1:]):
        if b - a < 2:
            continue
        differ = np.nonzero((table[a:b] != table[a]).any(0))[0]
        pages = int(differ[0]) if len(differ) else table.shape[1]
        least = min([pages * page] + [lens[s] - (cu[s + 1] - cu[s]) for s in range(a, b)])
        out[a:b] = [least] * (b - a)
    return out


def check(lib, table, lens, n, bounds, shift, order, seed):
    def ints(a):
        return np.ascontiguousarray(a, np.int32)

    def ptr(a):
        return a.ctypes.data_as(ctypes.c_void_p)
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    table = ints(table)
    arr = [ints(lens), ints(cu), ints(bounds)]
    prefix, reports = np.full(len(lens), -9, np.int32), ctypes.c_int(0)
    bad = lib.run(ptr(table), ctypes.c_int64(table.shape[1]), *map(ptr, arr), ptr(prefix), len(lens),
                  len(bounds) - 1, shift, table.shape[1], order, seed, ctypes.byref(reports))
    assert bad == 0, "a lane waits for one that does not come"
    assert reports.value == 0
    assert prefix.tolist() == common(table, lens, cu, bounds, 1 << shift)


ORDERS = pytest.mark.parametrize("order", [0, 1, 2], ids=["ascending", "descending", "random"])


@ORDERS
@pytest.mark.parametrize("members", [2, 3, 9, 40])
@pytest.mark.parametrize("differ", [0, 5, 127, 128, 300, 899, None])
def test_one_difference(lib, order, members, differ):
    """Rows of 900 columns: several tasks a warp behind the one that finds it."""
    table = np.tile(np.random.default_rng(1).integers(0, 1 << 20, 900), (members, 1))
    if differ is not None:
        table[members - 1, differ] += 1
    check(lib, table, [900 * 16] * members, [1] * members, [0, members], 4, order, 2)


@ORDERS
def test_forks(lib, order):
    for seed in range(60):
        rng = random.Random(seed)
        width, shift = rng.choice([3, 130, 700]), rng.choice([4, 6])
        rows, lens, n, bounds = [], [], [], [0]
        for _ in range(rng.randint(1, 4)):
            top = [rng.randint(0, 99) for _ in range(width)]
            for _ in range(rng.choice([0, 1, 2, 7, 33])):
                row = list(top)
                for _ in range(rng.choice([0, 0, 1, 3])):
                    row[rng.randrange(width)] += 100
                rows.append(row)
                lens.append(rng.choice([width << shift, rng.randint(0, width << shift)]))
                n.append(rng.randint(0, min(5, lens[-1])))
            bounds.append(len(rows))
        if rows:
            check(lib, rows, lens, n, bounds, shift, order, seed)
