"""The ring of hs_mla_decode_int4's kernel, as the kernel's own header (csrc/hs_ring.hpp) orders it: every stage gets its arrivals
and no more, the MMAs read as many stages as are filled, and the stages of a loader are close enough for its waits.

A loader waits for a place by its barrier's parity, which tells a phase only from its neighbours. Stage x is overwritten once the
one NSTAGE before it has been read; the phase before that one is over for sure if the loader has waited for a place among the
NSTAGE stages before x, that is if its stages are at most NSTAGE - 1 apart and it takes them in rising order.
"""
import os
import subprocess
from collections import Counter

import pytest

from hierarchical_sparse_attention_hs_gb300 import build as hs_build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("ring") / "ring_walk")
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(os.path.dirname(hs_build.__file__), "csrc"),
                           os.path.join(HERE, "ring_walk.cpp"), "-o", exe])
    lines = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    places, full = map(int, lines[0].split())
    cases = {}
    for line in lines[1:]:
        head, tail = line.split(":")
        *key, who = head.split()
        cases.setdefault(tuple(map(int, key)), {})[who] = tail.split()
    return places, full, cases


def stages(items):
    return [tuple(map(int, x.split("@")[0].split("x"))) for x in items]


def test_every_stage_is_filled_once(walk):
    places, full, cases = walk
    assert len(cases) == 2 * 6 * 4
    for key, who in cases.items():
        arrivals, loaders = Counter(), Counter()
        for name, items in who.items():
            if name != "issuer":
                for at, count in stages(items):
                    arrivals[at] += count
                    loaders[at] += 1
        read = [tuple(map(int, x.split("+"))) for x in who["issuer"]]
        assert sorted(arrivals) == list(range(sum(k + v for k, v in read))), key
        assert all(2 * n == full for n in arrivals.values()), key  # the pair's two CTAs alike
        keys = {at for at, _ in stages(who["keys"])}
        # the stages in the order in which the MMAs read them: K(0), then K(g) and V(g - 1), at last V(n - 1)
        kinds = []
        for g in range(len(read) + 1):
            kinds += ["K"] * (read[g][0] if g < len(read) else 0) + ["V"] * (read[g - 1][1] if g else 0)
        for at, kind in enumerate(kinds):
            assert loaders[at] == (1 if at in keys else 4 if kind == "K" else 2), (key, at)
        assert all(kinds[at] == "K" for at in keys) and len(keys) == len(read), key


def test_a_stage_is_made_of_the_rows_and_columns_that_the_mmas_take_it_for(walk):
    """K stage i of a tile is 64 columns of 128 rows, block i (the keys in between); V stage c 128 columns of the 64 rows of a
    segment, or with two stages a segment its columns' first or second 128."""
    places, full, cases = walk
    for (lv, n, last), who in cases.items():
        read = [tuple(map(int, x.split("+"))) for x in who["issuer"]]
        want, at = {}, 0
        for g in range(n + 1):
            for i in range(read[g][0] if g < n else 0):
                blk = i if i < 4 else i - 1
                want[at] = None if i == 4 else [(32 * r, 64 * blk) for r in range(4)]
                at += 1
            for c in range(read[g - 1][1] if g else 0):
                segment, half = (c, 0) if lv else (c >> 1, c & 1)
                want[at] = [(64 * segment + 32 * r, 128 * half) for r in range(2)]
                at += 1
        got = {x: [] for x in want}
        for name, items in who.items():
            if name not in ("issuer", "keys"):
                for item in items:
                    stage, place = item.split("@")
                    got[int(stage.split("x")[0])].append(tuple(map(int, place.split("/"))))
        assert all(sorted(got[x]) == sorted(want[x] or []) for x in want), (lv, n, last)


def test_stages_of_a_loader_are_less_than_the_ring_apart(walk):
    places, _, cases = walk
    for key, who in cases.items():
        for name, items in who.items():
            if name in ("issuer", "keys"):
                continue
            at = [x for x, _ in stages(items)]
            assert at[0] < places and all(0 < b - a < places for a, b in zip(at, at[1:])), (key, name, at)


def test_the_keys_place_is_free_when_they_are_told_so(walk):
    """The keys of tile 1 wait for all scores of tile 0, those of tile t for all of V(t - 2): what their place held is among it."""
    places, _, cases = walk
    for (lv, n, last), who in cases.items():
        read = [tuple(map(int, x.split("+"))) for x in who["issuer"]]
        at = [x for x, _ in stages(who["keys"])]
        assert at[0] < places
        done = 0  # stages read once K(0), then K(g) and V(g - 1), are
        for t in range(1, n):
            done += read[t - 1][0] + (read[t - 2][1] if t > 1 else 0)
            assert at[t] - places < done, (lv, n, last, t)
