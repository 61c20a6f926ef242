"""The waits of the wide paged-attention kernel, in a model of its roles (walk_model.py): every walk
comes to its end, whatever the stops' lengths and however their tiles are brought."""
import itertools
import random

import pytest

import walk_model as wm
from walk_model import COPY, TMA

# d = 128 and d = 64 in bf16: three and five stages; the 4-bit cache: two, and nothing is announced late
KINDS = [(3, "poll"), (5, "poll"), (3, "always"), (2, "at once")]


def every_stop(longest):
    return [list(t) for n in range(1, longest + 1) for t in itertools.product((COPY, TMA), repeat=n)]


@pytest.mark.parametrize("stages,announce", KINDS)
def test_every_short_walk_ends(stages, announce):
    """All walks of up to three stops of one to three tiles, random schedules and masks."""
    rng = random.Random(stages)
    for n in range(4):
        for stops in itertools.product(every_stop(3), repeat=n):
            wm.Cta([[(k, rng.random() < 0.5) for k in s] for s in stops], stages, announce, rng).run()


@pytest.mark.parametrize("stages,announce", KINDS)
def test_longer_walks_end(stages, announce):
    """Four and five stops of one tile in every order, and random walks."""
    rng = random.Random(10 + stages)
    for n in (4, 5):
        for kinds in itertools.product((COPY, TMA), repeat=n):
            wm.Cta([[(k, True)] for k in kinds], stages, announce, rng).run()
    for _ in range(3000):
        stops = [[(rng.choice((COPY, TMA)), rng.random() < 0.5) for _ in range(rng.choice((1, 1, 1, 2, 3, 4, 9)))]
                 for _ in range(rng.randint(4, 9))]
        wm.Cta(stops, stages, announce, rng).run()


def test_the_model_shows_a_tile_held_back():
    """A last tile that is announced with the next stop's first only: three stops of one tile, the
    last one copied, stall, and so does a longer first stop; none does that ends by TMA."""
    for stages in (3, 5):
        assert wm.stalls([[(COPY, True)]] * 3, stages, "late")
        assert wm.stalls([[(COPY, True)] * 5, [(COPY, True)], [(COPY, True)]], stages, "late")
        assert not wm.stalls([[(COPY, True)]] * 2, stages, "late")
        assert not wm.stalls([[(COPY, True)], [(COPY, True)], [(TMA, True)]], stages, "late")


def random_stops(rng):
    return [[(rng.choice((COPY, TMA)), rng.random() < 0.4) for _ in range(rng.choice((1, 1, 2, 3, 4, 9)))]
            for _ in range(rng.randint(1, 7))]


def test_every_wait_names_its_own_phase():
    """Roles of very different speeds: a wait by parity never meets a phase two away from its own
    (Aliased).  With two stages a softmax group may reach tile k before V(k - 2) has come, so that
    waiting for V(k) alone passes at once, and the rows it zeroes are V(k - 2)'s; three stages
    need no more, since S(k) follows PV(k - 3)."""
    for stages, announce in KINDS:
        for seed in range(2000):
            rng = random.Random(seed)
            wm.Cta(random_stops(rng), stages, announce, rng).run()
    met = 0
    for seed in range(2000):
        rng = random.Random(seed)
        try:
            wm.Cta(random_stops(rng), 2, "at once", rng, pv_first=False).run()
        except wm.Aliased as e:
            assert "v_full" in str(e)
            met += 1
    assert met > 20


# the GPU tests' shapes (test_walks.py)
@pytest.mark.parametrize("name", sorted(wm.WALKS))
def test_calls_end(name):
    """The stops of every CTA of these calls, as 148 SMs share them: each of the two kinds of
    loader brings every CTA to its end, and the order that holds a tile back does not."""
    c = wm.WALKS[name]
    for ctas in (148, 40):
        stops = wm.walk_call(c, ctas)
        for i, s in enumerate(stops):
            assert not wm.stalls(s, 3 if c["d"] == 128 else 5, "poll", seed=i), (name, i)
    late = sum(wm.stalls(s, 3 if c["d"] == 128 else 5, "late", seed=i) for i, s in enumerate(wm.walk_call(c)))
    assert (late > 0) == c["held_back"], (name, late)
