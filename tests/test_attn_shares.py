"""What a pair's second CTA copies of each stage (k_paged_attn, head size 256), in
the model of tests/test_attn_protocol.py.

A wait compares parities, so nobody may be two phases behind the barrier that it
waits for.  A producer is not as long as its own next copy is part of the phase to
come.  A stage of which the second CTA copies nothing (the second half of a tile
whose seen keys all lie in the first one) is filled, used and given back without it:
then it may come to its wait for the use before when both are over, wait for the
next one, and the pair with it.  So it copies at least one piece of every stage,
zeros if need be.

The shares are the kernel's: its own lines, compiled for the host."""

import ctypes
import os
import random
import re
import subprocess

import pytest

import test_attn_protocol as protocol
from test_attn_sources import CSRC

NAME = "many rows, 256"


@pytest.fixture(scope="module")
def live_from(tmp_path_factory):
    """Tokens that a CTA fetches of a stage: (khi, key, tokens, piece)."""
    src = open(os.path.join(CSRC, "dg_attn.cu")).read()
    body = re.search(r"auto live_from = \[&\]\(int key\) \{.*?\n\s*\};", src, re.S).group(0)
    # both CTAs' shares of a stage are counted where the first one awaits them
    assert "(live + (keys ? live_from(key_t + KROWS)" in src
    assert "const int key0 = key_t + (keys ? rank * (SH - 1) * KROWS : h * tokens);" in src
    path = tmp_path_factory.mktemp("shares")
    cpp, so = str(path / "shares.cpp"), str(path / "shares.so")
    with open(cpp, "w") as f:
        f.write("#include <algorithm>\nusing std::max; using std::min;\n"
                'extern "C" int share(int khi, int key_, int tokens, int piece) {\n'
                "constexpr bool PAIR = true; (void)PAIR;\nstruct { int khi; } g{khi};\n"
                + body + "\nreturn live_from(key_); }\n")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-o", so, cpp], check=True)
    return ctypes.CDLL(so).share


class Bar(protocol.Bar):
    def landed(self, tokens=1):
        self.tx -= tokens
        self._advance()


class Model(protocol.Model):
    """With each copy's tokens, and producers that dawdle."""

    def __init__(self, segs, rng, share, piece):
        self.share, self.piece = share, piece
        self.nothing = set()  # (CTA, tile, part) of which nothing is copied
        super().__init__(*protocol.MODES[NAME], segs, rng)
        for me in self.cta:
            for bars in me.values():
                if isinstance(bars[0], protocol.Bar):
                    for b in bars:
                        b.__class__ = Bar

    def dawdle(self):
        if self.rng.random() < 0.1:
            for _ in range(self.rng.randint(0, 40)):
                yield

    def producer(self, c, keys):
        me, first, ns = self.cta[c], self.cta[0], self.ns
        pos = 0
        for si, seg in enumerate(self.segs):
            n, vis, last = seg
            khi = 128 * n - (128 - vis if last else 0)
            if keys:
                yield from me["q_empty"][0].wait(si - 1)
                if c == 0:
                    me["q_full"][0].arrive(2)
                self.copies.append(first["q_full"][0].landed)
            for j in range(n):
                rp = pos + (protocol.k_stage(2, j) if keys else protocol.v_stage(2, j, n))
                for h in range(2):
                    st = (rp + h) % ns
                    yield from self.dawdle()
                    yield from me["empty"][st].wait((rp + h) // ns - 1)
                    tag = ("K" if keys else "V", si, j, h)
                    at = [128 * j + 64 * (x if keys else h) for x in range(2)]
                    live = [self.share(khi, x, 64, self.piece) for x in at]
                    clears = not keys and self.cleared_stage(seg, j) == h
                    bar = first["full"][st]
                    if c == 0:
                        bar.arrive(live[0] + (0 if clears else live[1]))
                    elif clears:
                        bar = me["tail"][st]
                        bar.arrive(live[1])
                    if not live[c]:
                        self.nothing.add((c, tag))
                        me["slot"][st] = tag
                        continue

                    def land(bar=bar, st=st, tag=tag, tokens=live[c]):
                        me["slot"][st] = tag
                        bar.landed(tokens)
                    self.copies.append(land)
                    yield
            pos += 4 * n
        if keys:
            for i in range(max(0, pos - ns), pos):
                yield from me["empty"][i % ns].wait(i // ns)
            if pos:
                yield from me["q_empty"][0].wait(len(self.segs) - 1)
                yield from me["pv"][0].wait(pos // 4 - 1)

    def finish_product(self, c):
        op = self.mma_queue[c][0]
        if op[0] != "commit":  # an operand of which nothing is copied is not read
            for x, t in enumerate(op[1]):
                tag = op[3]
                _, si, j, h = tag
                n, vis, last = self.segs[si]
                khi = 128 * n - (128 - vis if last else 0)
                at = 128 * j + 64 * (x if tag[0] == "K" else h)
                if not self.share(khi, at, 64, self.piece):
                    t["slot"][op[2]] = tag
        super().finish_product(c)


def segments(rng):
    """Many short items, as sequences of few tokens make them."""
    out = []
    for _ in range(rng.randint(1, 12)):
        out.append((rng.choice([1, 1, 2, 5]), rng.choice([rng.randint(1, 64), rng.randint(1, 128)]),
                    rng.random() < 0.9))
    return out


@pytest.mark.parametrize("piece", [16, 32, 64])
def test_no_producer_is_left_behind(piece, live_from):
    for seed in range(150):
        rng = random.Random(f"shares {piece} {seed}")
        segs = segments(rng)
        Model(segs, rng, live_from, piece).run()


@pytest.mark.parametrize("piece", [16, 32, 64])
def test_shares_hold_what_is_seen(piece, live_from):
    """Whole pieces from the stage's first token on, one at least, up to the last
    key that is seen; never more than the stage."""
    for khi in range(0, 400):
        for key in range(0, 512, 64):
            live = live_from(khi, key, 64, piece)
            assert piece <= live <= 64 and live % piece == 0
            seen = max(0, min(64, khi - key))
            assert live == max(piece, -(-seen // piece) * piece)


def test_the_model_sees_a_producer_left_behind():
    """Shares of nothing, as they were."""
    def none(khi, key, tokens, piece):
        return max(0, min(tokens, -(-(khi - key) // piece) * piece))
    caught = 0
    for seed in range(150):
        rng = random.Random(f"shares 16 {seed}")
        segs = segments(rng)
        try:
            Model(segs, rng, none, 16).run()
        except protocol.ProtocolError:
            caught += 1
    assert caught > 0
