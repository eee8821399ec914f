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


def variants():
    """Name in the protocol's model -> (D, NQ, pair) of the kernel's variants."""
    src = open(os.path.join(CSRC, "dg_attn.cu")).read()
    pair_of = re.search(r"constexpr bool pair_of\(int d\) \{ return (.*?); \}", src).group(1)
    many_nq = {d: eval(py(re.search(r"kManyNq = (.*?);", src).group(1)), {"D": d})
               for d in (64, 128, 256)}
    assert "few = k_paged_attn<D, 1, false, FP16>;" in src
    assert "many = k_paged_attn<D, kManyNq, kPair, FP16>;" in src
    out = {}
    for d in (64, 128, 256):
        out[f"one token, {d}"] = (d, 1, False)
        out[f"many rows, {d}"] = (d, many_nq[d], eval(pair_of, {"d": d}))
    return src, out


def py(expr):
    """A C expression of conditionals, comparisons and integers as Python."""
    expr = expr.strip().replace("&&", " and ").replace("||", " or ").replace("/", "//")
    while expr.startswith("(") and expr.endswith(")") and expr[1:-1].count("(") == 0:
        expr = expr[1:-1]
    m = re.match(r"(.*?)\?(.*?):(.*)$", expr, re.S)
    if m and m.group(1).count("(") > m.group(1).count(")"):  # a conditional inside a product
        m2 = re.match(r"\((.*?)\?(.*?):(.*?)\)(.*)$", expr, re.S)
        a, b, c, rest = m2.groups()
        return f"(({b}) if ({a}) else ({c})){rest}"
    return f"(({m.group(2)}) if ({m.group(1)}) else ({m.group(3)}))" if m else expr


def test_the_models_constants_are_the_kernels():
    """Ring stages, parts of a tile, query buffers, arrival counts and ring
    positions of tests/test_attn_protocol.py, worked out from the kernel."""
    src, kinds = variants()
    cfg = src[src.index("struct Cfg {"):src.index("struct Seq {")]

    def const(name, env):
        text = re.search(rf"static constexpr \w+ {name} =\s*(.*?);", cfg, re.S).group(1)
        return eval(py(text), {}, env)
    for name, (d, nq, pair) in kinds.items():
        env = {"D": d, "NQ": nq, "PAIR": pair, "kKeys": 128, "kRows": 128}
        for k in ("kParts", "kShare", "kStageBytes", "kStages", "kQBufs"):
            env[k] = const(k, env)
        mode, m_nq, parts, stages, q_bufs = protocol.MODES[name]
        assert (m_nq, parts, stages, q_bufs) == (nq, env["kParts"], env["kStages"], env["kQBufs"])
        # head sizes up to 128 take many rows by single CTAs now
        assert (mode == "pair") == pair
        # arrivals of a phase
        init = dict(re.findall(r"mbar_init\(&(\w+)(?:\[i\])?, (.*?)\);", src))
        env["SH"] = env["kShare"]
        got = {k: eval(py(v), {}, env) for k, v in init.items()}
        model = protocol.Model("pair" if pair else "single", nq, parts, stages, q_bufs, [],
                               random.Random(0))
        first = model.cta[0]
        for bar, ours in (("full", "full"), ("empty", "empty"), ("q_full", "q_full"),
                          ("q_empty", "q_empty"), ("s_full", "s"), ("p_half", "half"),
                          ("p_full", "p"), ("pv_done", "pv"), ("o_full", "o"),
                          ("tail_full", "tail")):
            assert first[ours][0].count == got[bar], (name, bar)
    # ring positions
    for fn, args in (("k_stage", "j"), ("v_stage", "j n")):
        text = re.search(rf"int {fn}\([^)]*\) \{{\s*return (.*?);\s*\}}", src, re.S).group(1)
        for parts in (1, 2):
            for n in (1, 2, 3, 9):
                for j in range(n):
                    want = getattr(protocol, fn)(parts, *([j] if args == "j" else [j, n]))
                    assert eval(py(text), {}, {"PARTS": parts, "j": j, "n": n}) == want


def test_registers_are_dealt_within_the_launch():
    """setmaxnreg draws on what the block was launched with: the three
    warpgroups' shares add up to it, as the comment beside them says."""
    src = open(os.path.join(CSRC, "dg_attn.cu")).read()
    soft, other = map(int, re.search(r"kRegsSoftmax = (\d+), kRegsOther = (\d+)", src).groups())
    launch = 65536 // 384 // 8 * 8
    assert 2 * soft + other <= 3 * launch and soft % 8 == other % 8 == 0
    assert f"2 x {soft} + {other} = 3 x {launch}" in src
