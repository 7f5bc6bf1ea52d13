"""Model check of the shared memory of a block of the beam step, between its barriers.

A block of eight warps goes through its part of a row: the threshold of the first tile (``tops``,
``sh_top``), the tiles' hits, the warps' maxima, where needed a second pass with its own threshold
and list, the sums, and the word that says which block is the last.  This file restates the warps'
reads and writes in order and runs them under random interleavings with the checker of
protocol_model: a read has to find the value that the algorithm means, whichever warp is ahead.

The maxima once lay in ``tops``, which the second pass's threshold writes without a barrier after the
warps have read them: a warp that was late then missed other warps' maxima, and summed against
another power of two than its neighbours.  That form must be caught for every path that takes the
second threshold, and for more than one beam (with one the value is the same).  Host logic only.
"""

import random

import pytest

from protocol_model import Barrier, Violation, run_roles

WARPS = 8


def warp(w, K, path, own_place):
    """One warp of a block.  path: "listed" (hits fit their places), "many" (more reach the
    threshold), "equal" (more than the list holds), "slow" (NaN, infinities, far logits)."""
    phase = [0]

    def sync():
        yield ("arrive", "cta", 1)
        yield ("wait", "cta", phase[0])
        phase[0] += 1

    def everyones(name, tag):
        for i in range(WARPS):
            yield ("read", f"{name}{i}", tag(i) if callable(tag) else tag)

    def kth_largest(tag):
        # (a warp's largest value stands first: with one beam that is its maximum)
        for i in range(K):
            yield ("write", f"tops{w * K + i}", f"max{w}" if i == 0 else f"{tag}{w}.{i}")
        yield from sync()
        if w * 32 < WARPS * K:
            for i in range(WARPS * K):
                v, at = divmod(i, K)
                yield ("read", f"tops{i}", f"max{v}" if at == 0 else f"{tag}{v}.{at}")
        yield ("write", f"sh_top{w}", tag)
        yield from sync()
        yield from everyones("sh_top", tag)

    if w == 0:
        yield ("write", "n_list", 0)
    yield from kth_largest("first")
    maxima = "warp_top" if own_place else "tops"
    own = lambda i: f"max{i}"
    yield ("write", f"{maxima}{w}", own(w))
    yield from sync()                                   # (whether any thread met NaN)
    if path == "slow":
        yield ("write", f"{maxima}{w}", own(w))
        yield from sync()
    yield from everyones(maxima, own)
    yield ("write", f"sums{w}", "sum")
    if path != "listed":
        yield from kth_largest("second")
        yield from sync()
    yield ("write", f"list{w}", "found")
    yield from sync()
    yield ("read", "n_list", 0)
    if path == "equal":
        for n in range(K):
            yield from sync()
            yield ("write", f"list{w}", f"best{n}")
            yield from sync()
            yield from everyones("list", f"best{n}")
    else:
        yield from everyones("list", "found")
    yield from sync()
    if w == 0:
        yield from everyones("sums", "sum")
    # the counters of the row and of the group; the last block's keys take the list's place
    for which in ("row", "group"):
        yield from sync()
        if w == 0:
            yield ("write", "last_of", which)
        yield from sync()
        yield ("read", "last_of", which)
        yield ("write", f"list{w}", f"keys of the {which}")
        yield from sync()
        yield from everyones("list", f"keys of the {which}")


def run(K, path, own_place, seed):
    bars = {"cta": Barrier("cta", WARPS)}
    roles = {f"warp{w}": warp(w, K, path, own_place) for w in range(WARPS)}
    run_roles(roles, bars, (), random.Random(seed))


@pytest.mark.parametrize("path", ["listed", "many", "equal", "slow"])
@pytest.mark.parametrize("K", [1, 2, 5, 32])
def test_every_read_finds_what_is_meant(K, path):
    for seed in range(30 if K < 32 else 5):
        run(K, path, True, seed)


@pytest.mark.parametrize("path", ["many", "equal", "slow"])
@pytest.mark.parametrize("K", [2, 5, 32])
def test_maxima_in_the_thresholds_list_are_caught(K, path):
    caught = 0
    for seed in range(30):
        try:
            run(K, path, False, seed)
        except Violation as e:
            caught += "tops" in str(e)
    assert caught > 0
