"""A model on the CPU of who waits for whom in the wide paged-attention kernel (csrc/paged_attn.cu,
paged_attn): the walk, the MMA issuer, two softmax groups and the loaders of K and V, with their
mbarriers, over one CTA's stops.  Each role is a generator that yields (barrier, phase) where the
kernel waits; a warp or a group counts as one arrival.  No data, no time: a stall is a state in which
every unfinished role waits for a phase that nobody left can complete.

The bf16 loaders bring a tile of pages by asynchronous copies or by TMA, and block tokens by TMA.  TMA
announces a tile by itself, copies are announced by the loader once they have landed, which it sees to
one tile later.  `announce` says what happens to a stop's last tile:
  "late"    it is announced with the next stop's first tile, or when the walk is over
  "poll"    it is announced at the end of the stop unless the next stop is there already
  "always"  it is announced at the end of the stop
  "at once" every tile is announced when it is issued (the 4-bit cache's loaders)
"""
from __future__ import annotations

import random

COPY, TMA = "copy", "tma"


class Stall(Exception):
    pass


class Aliased(Exception):
    """A wait by parity met a phase two away from its own."""


class Bar:
    def __init__(self, name, count=1):
        self.name, self.count, self.here, self.done = name, count, 0, 0

    def arrive(self):
        self.here += 1
        if self.here == self.count:
            self.here, self.done = 0, self.done + 1

    def passed(self, phase):
        if not phase <= self.done <= phase + 1:
            raise Aliased(f"{self.name}: phase {phase} of {self.done}")
        return self.done > phase


class Cta:
    """stops: a list of stops, each a list of (kind, masked) per tile; masked: the softmax group zeroes
    value rows, so it waits for V before it decides the tile."""

    def __init__(self, stops, stages, announce, rng, pv_first=None):
        self.stops, self.st, self.announce, self.rng = stops, stages, announce, rng
        # a softmax group that waits for V(k) waits for PV(k - stages) first
        self.pv_first = stages < 3 if pv_first is None else pv_first
        bars = lambda name, n, count=1: [Bar(f"{name}[{i}]", count) for i in range(n)]  # noqa: E731
        self.k_full, self.k_empty = bars("k_full", stages), bars("k_empty", stages)
        self.v_full, self.v_empty = bars("v_full", stages), bars("v_empty", stages)
        self.tab_full = bars("tab_full", 8)
        self.s_full, self.p_full = bars("s_full", 3), bars("p_full", 3)
        self.pv_done, self.decided = bars("pv_done", 2), bars("decided", 2)
        self.q_full, self.q_empty, self.o_full = Bar("q_full"), Bar("q_empty"), Bar("o_full")
        self.o_free, self.meet = Bar("o_free", 2), Bar("meet", 2)
        self.stop_full, self.stop_empty = bars("stop_full", 3), bars("stop_empty", 3, 5)
        self.pv = 0  # MMAs of P V that were issued

    def nt(self, it):
        return len(self.stops[it]) if it < len(self.stops) else 0

    def walk(self):
        for it in range(len(self.stops) + 1):
            if it >= 3:
                yield self.stop_empty[it % 3], it // 3 - 1
            self.stop_full[it % 3].arrive()
            if self.nt(it) == 0:
                return
            if it > 0:
                yield self.q_empty, it - 1
            self.q_full.arrive()

    def issuer(self):
        s = dict(it=0, left=0, ks=0, more=True)

        def issue_s():
            if s["left"] == 0:
                if not s["more"]:
                    return
                yield self.stop_full[s["it"] % 3], s["it"] // 3
                s["left"] = self.nt(s["it"])
                self.stop_empty[s["it"] % 3].arrive()
                s["more"] = s["left"] > 0
                if not s["more"]:
                    return
                yield self.q_full, s["it"]
                s["it"] += 1
            ks = s["ks"]
            yield self.k_full[ks % self.st], ks // self.st
            if ks >= 3:
                yield self.pv_done[(ks - 3) % 2], (ks - 3) // 2
            self.s_full[ks % 3].arrive()
            self.k_empty[ks % self.st].arrive()
            s["ks"] += 1
            s["left"] -= 1
            if s["left"] == 0:
                self.q_empty.arrive()

        yield from issue_s()
        yield from issue_s()
        k = 0
        for it in range(len(self.stops)):
            for j in range(self.nt(it)):
                yield from issue_s()
                yield self.p_full[k % 3], k // 3
                yield self.v_full[k % self.st], k // self.st
                if j == 0 and it > 0:
                    yield self.o_free, it - 1
                self.pv += 1
                self.pv_done[k % 2].arrive()
                self.v_empty[k % self.st].arrive()
                k += 1
            self.o_full.arrive()

    def softmax(self, g):
        k0 = met = 0
        for it in range(len(self.stops) + 1):
            yield self.stop_full[it % 3], it // 3
            if self.nt(it) == 0:
                return
            k1 = k0 + self.nt(it)
            for k in range(k0 + ((k0 ^ g) & 1), k1, 2):
                yield self.tab_full[k % 8], k // 8
                yield self.s_full[k % 3], k // 3
                if self.stops[it][k - k0][1]:
                    if self.pv_first and k >= self.st:
                        yield self.pv_done[(k - self.st) % 2], (k - self.st) // 2
                    yield self.v_full[k % self.st], k // self.st
                if k > k0:
                    yield self.decided[(k - 1) % 2], (k - 1) // 2
                    if self.rng.random() < 0.5:  # O is rescaled
                        yield self.pv_done[(k - 1) % 2], (k - 1) // 2
                self.decided[k % 2].arrive()
                self.p_full[k % 3].arrive()
            yield self.o_full, it
            yield self.decided[(k1 - 1) % 2], (k1 - 1) // 2
            for _ in range(2):
                self.meet.arrive()
                yield self.meet, met
                met += 1
            self.o_free.arrive()
            k0 = k1
            self.stop_empty[it % 3].arrive()

    def loader(self, isv):
        full, empty = (self.v_full, self.v_empty) if isv else (self.k_full, self.k_empty)
        k = told = 0

        def tell(upto):
            nonlocal told
            while told < upto:
                full[told % self.st].arrive()
                told += 1

        for it in range(len(self.stops) + 1):
            yield self.stop_full[it % 3], it // 3
            if self.nt(it) == 0:
                break
            for kind, _ in self.stops[it]:
                if k >= self.st:
                    yield empty[k % self.st], k // self.st - 1
                if not isv:
                    self.tab_full[k % 8].arrive()
                tell(k)
                if kind == TMA or self.announce == "at once":
                    tell(k + 1)
                k += 1
            if self.announce == "always" or (self.announce == "poll" and not self.stop_full[(it + 1) % 3].passed((it + 1) // 3)):
                tell(k)
            self.stop_empty[it % 3].arrive()
        tell(k)

    def run(self):
        """Runs the roles in random order to their ends; raises Stall."""
        roles = [self.walk(), self.issuer(), self.softmax(0), self.softmax(1), self.loader(False), self.loader(True)]
        names = ["walk", "issuer", "softmax 0", "softmax 1", "K", "V"]
        live = [[n, r, None] for n, r in zip(names, roles)]
        # some roles are slower than others by up to three powers of ten, so that each gets far ahead
        speed = {n: 10.0 ** -self.rng.choice((0, 0, 1, 3)) for n in names}
        while live:
            ready = [r for r in live if r[2] is None or r[2][0].passed(r[2][1])]
            if not ready:
                tiles = sum(map(len, self.stops))
                raise Stall(f"{self.pv} of {tiles} PVs; " + ", ".join(f"{n} at {w[0].name}" for n, _, w in live))
            role = self.rng.choices(ready, [speed[r[0]] for r in ready])[0]
            try:
                role[2] = next(role[1])
            except StopIteration:
                live.remove(role)
        return self


def stalls(stops, stages, announce, seed=0):
    try:
        Cta(stops, stages, announce, random.Random(seed)).run()
    except Stall:
        return True
    return False


# ------------------------------------------------------ the tiles of a call, its shares ----
def unit_tiles(n, b0, rows, new, page, window, sinks, causal, block, run):
    """Tiles (kind, masked) of the unit of tokens [b0, b0 + rows) in dsa_window_attn: pages in which
    some row sees a token, then block tokens.  run: a tile's pages lie one after the other."""
    if min(new, b0 + rows) <= b0:
        return []
    last = min(new, b0 + rows) - 1
    low = n + b0 - window + 1
    pages = [p for p in range(-(-n // page))
             if any(t < sinks or t >= low for t in range(p * page, min(n, (p + 1) * page)))]
    per = 128 // page
    tiles = [(TMA if run and len(pages[i:i + per]) == per else COPY, True) for i in range(0, len(pages), per)]
    if block:
        top = last if causal else min(new - 1, last + window - 1)
        near = max(0, min(sinks, n + top + 1) - n) if sinks > n else 0
        first = max(near, low - n)
        tiles += [(TMA, True)] * (-(-near // 128) + -(-max(0, top + 1 - first) // 128))
    return tiles or [(COPY, True)]


def shares(units, ctas, whole):
    """The stops of every CTA: equal shares of all tiles in a row, or whole units dealt out in turn."""
    if whole:
        return [[u for u in units[c::ctas] if u] for c in range(ctas)]
    total = sum(map(len, units))
    n = max(1, min(ctas, total))
    out = []
    for c in range(n):
        lo, hi, at, stops = total * c // n, total * (c + 1) // n, 0, []
        for u in units:
            a, b = max(lo, at), min(hi, at + len(u))
            if a < b:
                stops.append(u[a - at:b - at])
            at += len(u)
        out.append(stops)
    return out


def call(n, new, B, G, Hkv, page, window, sinks, causal, block=True, run=False, ctas=148):
    """Every CTA's stops of a call with prefix lengths n and block lengths new on `ctas` CTAs."""
    bpt = min(128 // G, B)
    units = []
    for s in range(len(n)):
        for _ in range(Hkv):
            for b0 in range(0, B, bpt):
                units.append(unit_tiles(n[s], b0, min(bpt, B - b0), new[s], page, window, sinks, causal, block, run))
    return shares(units, ctas, len(units) > min(8 * ctas, 1536))


# Calls with many stops per CTA: mixed batches with fresh sequences, the prefix alone, prompts in
# parts.  held_back: some CTA of 148 stalls if a stop's last tile is announced with the next stop.
def _mixed(S, every, n, fresh=0):
    return [fresh if s % every == 0 else n for s in range(S)]


WALKS = {
    "fresh_every_4th": dict(n=_mixed(24, 4, 100), B=32, G=4, Hkv=8, d=128, page=16, window=1024, sinks=0, causal=False, held_back=True),
    "fresh_every_2nd": dict(n=_mixed(32, 2, 100), B=32, G=4, Hkv=8, d=64, page=32, window=1024, sinks=0, causal=True, held_back=True),
    "prefix_alone": dict(n=[90 + 7 * (s % 60) for s in range(64)], B=20, G=1, Hkv=8, d=128, page=16, window=60, sinks=0, causal=False,
                         block=False, held_back=True),
    "prefix_alone_p32": dict(n=[90 + 7 * (s % 60) for s in range(64)], B=20, G=1, Hkv=8, d=64, page=32, window=60, sinks=3, causal=True,
                             block=False, held_back=True),
    "prefix_alone_many": dict(n=[s % 100 for s in range(160)], B=17, G=1, Hkv=8, d=64, page=16, window=100, sinks=0, causal=True,
                              block=False, held_back=True),
    "prefix_alone_empty": dict(n=[0] * 160, B=17, G=1, Hkv=4, d=128, page=16, window=100, sinks=0, causal=True, block=False,
                               held_back=True),
    "prefix_of_a_prompt": dict(n=[100], B=4000, G=4, Hkv=16, d=64, page=16, window=1024, sinks=4, causal=True, block=False,
                               held_back=True),
    "mostly_fresh_few_long": dict(n=[3000 if s in (9, 30, 31) else 0 for s in range(64)], B=24, G=2, Hkv=4, d=128, page=16,
                                  window=2000, sinks=5, causal=True, held_back=False),
    "fresh_identity_table": dict(n=_mixed(24, 4, 300), B=32, G=4, Hkv=8, d=128, page=16, window=1024, sinks=0, causal=False,
                                 table=False, held_back=False),
    "padded_mixed": dict(n=_mixed(48, 3, 70), new=[(5 * s) % 21 for s in range(48)], B=20, G=2, Hkv=8, d=128, page=16, window=50,
                         sinks=9, causal=False, held_back=True),
}


def walk_call(c, ctas=148):
    B = c["B"]
    return call(c["n"], c.get("new") or [B] * len(c["n"]), B, c["G"], c["Hkv"], c["page"], c["window"], c["sinks"], c["causal"],
                c.get("block", True), run=not c.get("table", True), ctas=ctas)
