"""Host-side model of the barrier protocol of k_paged_attn
(moe_expert_ffn_dg_gb300/csrc/dg_attn.cu), run on random segments.

Two key / value producers, the MMA issuer and the softmax warps of one CTA, of
a cluster that shares copies by multicast, or of a pair with shared products
run as coroutines with the kernel's ring positions, arrival counts and wait
parities, interleaved at random with the copies (landing in any order) and the
products (completing in issue order, their arrivals delivered in order).  It
checks that

* every wait returns on the phase it means (an mbarrier compares parities),
* no barrier receives an arrival beyond its count (the hardware faults),
* every product reads the operands it means, scores are read before they are
  overwritten, cleared values are in place, and an accumulator is read whole,
* every run ends, and in a cluster nothing is still to arrive then.

Planted mistakes must be caught."""

import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(__file__)), "moe_expert_ffn_dg_gb300", "csrc",
                   "dg_attn.cu")


class ProtocolError(AssertionError):
    pass


def need(ok, *what):
    if not ok:
        raise ProtocolError(what)


class Bar:
    def __init__(self, count, name):
        self.count, self.pending, self.tx, self.phase, self.name = count, count, 0, 0, name

    def _advance(self):
        if self.pending == 0 and self.tx == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def arrive(self, tx=0):
        need(self.pending > 0, "over-arrival", self.name, self.phase)
        self.tx, self.pending = self.tx + tx, self.pending - 1
        self._advance()

    def landed(self):
        self.tx -= 1
        self._advance()

    def wait(self, k):
        """Wait for phase k by its parity, as the kernel does."""
        while (self.phase & 1) == (k & 1):
            yield
        need(self.phase > k, "parity alias", self.name, self.phase, k)


def k_stage(parts, j):
    return 0 if j == 0 else parts * (2 * j - 1)


def v_stage(parts, j, n):
    return parts * (2 * j + 2) if j + 1 < n else parts * (2 * n - 1)


class Model:
    """segs: (key tiles, keys of the last tile that are seen, whether the item
    ends there).  plant: a mistake."""

    def __init__(self, mode, nq, parts, stages, q_bufs, segs, rng, plant=None):
        self.mode, self.nq, self.parts, self.ns, self.qb = mode, nq, parts, stages, q_bufs
        self.segs, self.rng, self.plant = segs, rng, plant
        self.swift = rng.choice([0.6, 0.1])  # of arrivals
        self.n_cta = 1 if mode == "single" else 2
        self.pair = mode == "pair"
        share = 2 if self.pair else 1
        warps = 4 if nq == 2 else 8
        free = self.n_cta if mode == "cluster" and plant != "free_alone" else 1
        self.cta = []
        for c in range(self.n_cta):
            def bars(name, n, count):
                return [Bar(count, f"{name}{i} of {c}") for i in range(n)]
            self.cta.append({
                "full": bars("full", stages, 1), "empty": bars("empty", stages, free),
                "q_full": bars("q_full", q_bufs, 1), "q_empty": bars("q_empty", q_bufs, 1),
                "s": bars("s_full", 2, 1), "half": bars("p_half", 2, 4 * share),
                "p": bars("p_full", 2, warps * share), "pv": bars("pv_done", 2, 1),
                "o": bars("o_full", 2, 1),
                "tail": bars("tail_full", 1 if plant == "one_tail" else stages, 1),
                "slot": [None] * stages, "S": [None, None], "P": [None, None], "Pw": [0, 0],
                "O": [[], []]})
        self.copies = []                                   # landing in any order
        self.mma_queue = [[] for _ in self.cta]            # in order
        self.arrivals = [[] for _ in self.cta]             # of finished products, in order
        self.roles = {}
        for c in range(self.n_cta):
            self.roles[f"keys {c}"] = self.producer(c, True)
            self.roles[f"values {c}"] = self.producer(c, False)
            if not self.pair or c == 0:
                self.roles[f"mma {c}"] = self.mma(c)
            for w in range(8):
                self.roles[f"softmax {c}.{w}"] = self.softmax(c, w)

    def cleared_stage(self, seg, j):
        n, vis, last = seg
        if last and j == n - 1 and vis < 128 and vis & 15:
            return vis // (128 // self.parts)
        return None

    def producer(self, c, keys):
        me, first, ns = self.cta[c], self.cta[0], self.ns
        pos = qn = 0
        for si, seg in enumerate(self.segs):
            n = seg[0]
            if keys:
                i = qn % self.qb
                yield from me["q_empty"][i].wait(qn // self.qb - 1)
                qn += 1
                if not self.pair or c == 0:
                    me["q_full"][i].arrive(2 if self.pair else 1)
                self.copies.append((first if self.pair else me)["q_full"][i].landed)
            for j in range(n):
                rp = pos + (k_stage(self.parts, j) if keys else v_stage(self.parts, j, n))
                for h in range(self.parts):
                    st = (rp + h) % ns
                    yield from me["empty"][st].wait((rp + h) // ns - 1)
                    tag = ("K" if keys else "V", si, j, h)
                    if self.mode == "cluster":
                        me["full"][st].arrive(2)
                        for to in self.cta:
                            def land(to=to, st=st, tag=tag):
                                half = to["slot"][st] == ("half", tag)
                                to["slot"][st] = tag if half else ("half", tag)
                                to["full"][st].landed()
                            self.copies.append(land)
                    else:
                        bar = me["full"][st]
                        if self.pair:
                            clears = not keys and self.cleared_stage(seg, j) == h
                            if c == 0:
                                bar.arrive(1 if clears else 2)
                            elif clears:
                                bar = me["tail"][st % len(me["tail"])]
                                bar.arrive(1)
                            else:
                                bar = first["full"][st]
                        else:
                            bar.arrive(1)

                        def land(bar=bar, st=st, tag=tag):
                            me["slot"][st] = tag
                            bar.landed()
                        self.copies.append(land)
                    yield
            pos += 2 * self.parts * n
        if keys and self.n_cta > 1:
            for i in range(max(0, pos - ns), pos):
                yield from me["empty"][i % ns].wait(i // ns)
            for i in range(max(0, qn - self.qb), qn):
                yield from me["q_empty"][i % self.qb].wait(i // self.qb)
            tiles = pos // (2 * self.parts)
            for i in range(self.nq if tiles else 0):
                yield from me["pv"][i].wait(tiles - 1)

    def mma(self, c):
        me, queue = self.cta[c], self.mma_queue[c]
        both = self.cta if self.pair else [me]
        everyone = self.cta if self.n_cta > 1 else [me]
        pos = at = 0
        for si, (n, _, _) in enumerate(self.segs):
            qi = si % self.qb
            yield from me["q_full"][qi].wait(si // self.qb)

            def commit(bars):
                queue.append(("commit", bars))

            def stage(rp, i):
                if i == 0:
                    yield from me["full"][rp % self.ns].wait(rp // self.ns)

            def scores(i, j):
                buf = i if self.nq == 2 else (at + j) & 1
                for h in range(self.parts):
                    rp = pos + k_stage(self.parts, j) + h
                    yield from stage(rp, i)
                    queue.append(("S", both, rp % self.ns, ("K", si, j, h), buf, (si, j, i)))
                    if i == self.nq - 1:
                        commit([t["empty"][rp % self.ns] for t in everyone])
                commit([t["s"][buf] for t in both])
                if i == self.nq - 1 and j == n - 1:
                    commit([t["q_empty"][qi] for t in both])

            def values(i, j):
                buf = i if self.nq == 2 else (at + j) & 1
                use = at + j if self.nq == 2 else (at + j) >> 1
                if self.nq == 2:
                    yield from me["half"][buf].wait(use)
                yield from me["p"][buf].wait(use)
                for h in range(self.parts):
                    rp = pos + v_stage(self.parts, j, n) + h
                    yield from stage(rp, i)
                    queue.append(("PV", both, rp % self.ns, ("V", si, j, h), buf, (si, j, i), i,
                                  j + h == 0))
                    if i == self.nq - 1:
                        commit([t["empty"][rp % self.ns] for t in everyone])
                commit([t["pv"][i] for t in both])
                if j == n - 1:
                    commit([t["o"][i] for t in both])
            if self.nq == 2:
                yield from scores(0, 0)
                yield from scores(1, 0)
                for j in range(n):
                    for i in (0, 1):
                        yield from values(i, j)
                        if j + 1 < n:
                            yield from scores(i, j + 1)
            else:
                for j in range(min(2, n)):
                    yield from scores(0, j)
                for j in range(n):
                    yield from values(0, j)
                    if j + 2 < n:
                        yield from scores(0, j + 2)
            pos += 2 * self.parts * n
            at += n
        while queue:
            yield

    def softmax(self, c, w):
        me = self.cta[c]
        first = self.cta[0] if self.pair else me
        wg = w >> 2
        i = wg if self.nq == 2 else 0
        warps = 4 if self.nq == 2 else 8
        pos = at = tails = 0
        tail_of = [0] * self.ns
        for si, seg in enumerate(self.segs):
            n = seg[0]
            for j in range(n):
                buf = i if self.nq == 2 else (at + j) & 1
                use = at + j if self.nq == 2 else (at + j) >> 1
                yield from me["s"][buf].wait(use)
                need(me["S"][buf] == (si, j, i), "scores", c, w, me["S"][buf])
                h = self.cleared_stage(seg, j)
                if h is not None and i == 0:
                    rp = pos + v_stage(self.parts, j, n) + h
                    st = rp % self.ns
                    if not self.pair or c == 0:
                        yield from me["full"][st].wait(rp // self.ns)
                    elif self.plant == "one_tail":
                        yield from me["tail"][0].wait(tails)
                        tails += 1
                    else:
                        yield from me["tail"][st].wait(tail_of[st])
                        tail_of[st] += 1
                    need(me["slot"][st] == ("V", si, j, h), "cleared", c, me["slot"][st])
                if j > 0 and self.rng.random() < 0.2:  # the reference moved
                    yield from me["pv"][i].wait(at + j - 1)
                    need(me["O"][i][-1][:2] == (si, j - 1), "rescaled", c, me["O"][i][-1:])
                yield
                me["Pw"][buf] += 1
                if me["Pw"][buf] == warps:
                    me["Pw"][buf], me["P"][buf] = 0, (si, j, i)
                if self.nq == 2:
                    first["half"][buf].arrive()
                first["p"][buf].arrive()
                yield
            if self.plant == "end_by_tile":
                yield from me["pv"][i].wait(at + n - 1)
            else:
                yield from me["o"][i].wait(si)
            for _ in range(3):  # the accumulator is read
                need(me["O"][i] == [(si, j, h) for j in range(n) for h in range(self.parts)],
                     "accumulator", c, w, si)
                yield
            pos += 2 * self.parts * n
            at += n

    def finish_product(self, c):
        op = self.mma_queue[c].pop(0)
        if op[0] == "commit":
            self.arrivals[c].append(op[1])
            return
        kind, ctas, st, tag, buf, val = op[:6]
        for t in ctas:
            need(t["slot"][st] == tag, "operand", kind, t["slot"][st], tag)
            if kind == "S":
                t["S"][buf] = val
            else:
                need(t["P"][buf] == val, "weights", t["P"][buf], val)
                i, fresh = op[6:]
                if fresh:
                    t["O"][i] = []
                t["O"][i].append(tag[1:])

    def run(self):
        idle = 0
        while self.roles:
            moved = False
            if self.copies and self.rng.random() < 0.3:
                self.copies.pop(self.rng.randrange(len(self.copies)))()
                moved = True
            for c in range(self.n_cta):
                if self.mma_queue[c] and self.rng.random() < 0.5:
                    self.finish_product(c)
                    moved = True
                if self.arrivals[c] and self.rng.random() < self.swift:
                    for bar in self.arrivals[c].pop(0):
                        bar.arrive()
                    moved = True
            for name in self.rng.sample(list(self.roles), k=min(len(self.roles), 6)):
                try:
                    next(self.roles[name])
                except StopIteration:
                    del self.roles[name]
                    moved = True
            busy = moved or self.copies or any(self.mma_queue) or any(self.arrivals)
            idle = 0 if busy else idle + 1
            need(idle < 400, "deadlock", sorted(self.roles))
        if self.n_cta > 1:
            need(not self.copies and not any(self.arrivals), "still to arrive")


def segments(rng):
    longest = rng.choice([1, 2, 9])
    out = []
    for _ in range(rng.randint(1, 12)):
        last = rng.random() < 0.8
        out.append((rng.randint(1, longest), rng.choice([rng.randint(1, 127), 128, 64]), last))
    return out


def ring(d):
    """Stages and their bytes from the kernel's constants."""
    src = open(SRC).read()
    total = int(re.search(r"kStages = (\d+) \* 1024 / kStageBytes", src).group(1)) * 1024
    assert "kParts = D == 256 ? 2 : 1;" in src and "kDescHi" in src
    pair = d == 256
    parts = 2 if d == 256 else 1
    return parts, [total // (128 * d * 2 // parts // s) for s in ((2,) if pair else (1,))][0], pair


# mode, query tiles, parts of a tile, ring stages, query buffers
MODES = {
    "one token, 64": ("single", 1, 1, 10, 2), "one token, 128": ("single", 1, 1, 5, 2),
    "one token, 256": ("single", 1, 2, 5, 1), "many rows, 64": ("cluster", 2, 1, 10, 1),
    "many rows, 128": ("cluster", 2, 1, 5, 1), "many rows, 256": ("pair", 1, 2, 10, 1),
}


def test_modes_are_the_kernels():
    assert ring(64) == (1, MODES["many rows, 64"][3], False)
    assert ring(128) == (1, MODES["many rows, 128"][3], False)
    assert ring(256) == (2, MODES["many rows, 256"][3], True)


@pytest.mark.parametrize("name", MODES)
def test_protocol(name):
    for seed in range(40):
        rng = random.Random(f"{name} {seed}")
        Model(*MODES[name], segments(rng), rng).run()


@pytest.mark.parametrize("name,plant", [
    ("many rows, 256", "one_tail"),      # one barrier for all cleared values
    ("one token, 256", "end_by_tile"),   # a segment's end taken from the per-tile barrier
    ("many rows, 128", "free_alone"),    # a shared stage freed by one CTA
])
def test_planted_mistakes_are_caught(name, plant):
    caught = 0
    for seed in range(60):
        rng = random.Random(f"{name} {seed}")
        try:
            Model(*MODES[name], segments(rng), rng, plant).run()
        except ProtocolError:
            caught += 1
    assert caught > 0
