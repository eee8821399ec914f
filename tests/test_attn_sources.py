"""Rules of the compiled sources that can be read off them, and the constants
of k_paged_attn that its host-side models stand on."""

import glob
import os
import random
import re

import test_attn_protocol as protocol

ROOT = os.path.dirname(os.path.dirname(__file__))
CSRC = os.path.join(ROOT, "moe_expert_ffn_dg_gb300", "csrc")


def asm_statements():
    """(file, text) of every inline PTX statement, its literals joined."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*")) + glob.glob(os.path.join(CSRC, "*.h"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\b[^;]*?\(((?:\s*\"(?:[^\"\\]|\\.)*\")+)", src):
            yield os.path.basename(path), "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1)))


def test_statements_are_found():
    text = [t for _, t in asm_statements()]
    assert sum("cp.async.bulk.tensor" in t for t in text) >= 5
    assert sum("tcgen05.commit" in t for t in text) >= 3


def test_no_copy_is_multicast():
    """The library also runs as one replica a GPU, where a multicast copy is
    ruled out: no copy names more than one destination.  (A commit that
    arrives in both CTAs of a pair moves no data.)"""
    bad = [(f, t) for f, t in asm_statements() if "cp.async" in t and "multicast" in t]
    assert not bad, bad


def test_every_stage_is_the_ctas_own():
    """One CTA with two query tiles (many rows, head sizes 64 and 128): the
    protocol's model, each stage filled and freed by one CTA."""
    for stages in (10, 5):
        for seed in range(40):
            rng = random.Random(f"own {stages} {seed}")
            protocol.Model("single", 2, 1, stages, 1, protocol.segments(rng), rng).run()


def test_signals_between_ctas_have_their_scope():
    """An arrival at another CTA's barrier without a scope is a release of the
    CTA's scope, which does not hold the thread that waits for it."""
    far = [(f, t) for f, t in asm_statements()
           if re.match(r"\s*mbarrier\.arrive", t) and "shared::cluster" in t]
    assert far
    bad = [x for x in far
           if not re.search(r"mbarrier\.arrive\.(release|relaxed)\.cluster\.shared::cluster", x[1])]
    assert not bad, bad


def test_waits_for_the_other_cta_have_their_scope():
    """In k_paged_attn the barriers that a pair's products or other CTA signal
    are waited for at cluster scope; a CTA's own `tail_full` is not among them."""
    src = open(os.path.join(CSRC, "dg_attn.cu")).read()
    body = src[src.index("k_paged_attn(const"):src.index("k_attn_join(const")]
    plain = re.findall(r"\bmbar_(?:try_)?wait\(([^,]*),", body)
    assert set(plain) == {"&tail_full[PAIR ? st : 0]"}, plain
    assert len(re.findall(r"\bwait_scope<PAIR>\(", body)) >= 5
