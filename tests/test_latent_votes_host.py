"""The rescale votes of the latent attention's softmax warps, without a GPU: the order of events that its barriers
give, as a graph, over every way in which a few tiles fall into items.  A buffer of votes may be written again only
after every warp's look at what it held."""

import itertools
import os
import re

import pytest

from paged_kv_cache_111_gb300 import _build

WARPS = 4


def constant(name):
    src = open(os.path.join(os.path.dirname(_build.__file__), "csrc", "latent_attn.cu")).read()
    return int(re.search(rf"constexpr int {name} = (\d+);", src).group(1))


def ancestors(first):
    """{event: events before it}, tile g the first of its item where first[g].  No warp votes: a vote only adds waits
    (the second products' for the rescaling warps)."""
    stages = constant("kLaStages")
    before, last = {}, {}

    def event(process, name, *after):
        """`name` happens in `process`, after what the process did and after the events waited for."""
        seen = set()
        for e in (last.get(process), *after):
            if e is not None:
                seen |= {e} | before[e]
        before[name] = seen
        last[process] = name

    for g in range(len(first)):
        # a stage is loaded again once its second products are done; its S once the S buffer has been read
        event("load", ("load", g), ("products", g - stages) if g >= stages else None)
        event("scores", ("scores", g), ("load", g), *([("read S", g - 2, w) for w in range(WARPS)] if g >= 2 else []))
        for w in range(WARPS):
            event(w, ("read S", g, w), ("scores", g))
            event(w, ("write", g, w))
            event(w, ("arrive", g, w))                      # kLaPFull
        arrived = [("arrive", g, w) for w in range(WARPS)]
        for w in range(WARPS):
            if not first[g]:
                event(w, ("look", g, w), *arrived)
        event("products", ("products", g), *arrived)
    return before


def unordered(first, buffers):
    before = ancestors(first)
    return [(g, x, y) for g in range(len(first) - buffers) if not first[g]
            for x in range(WARPS) for y in range(WARPS)
            if ("look", g, x) not in before[("write", g + buffers, y)]]


RUNS = [(True,) + rest for rest in itertools.product([True, False], repeat=9)]


def test_votes_are_written_again_only_after_every_look():
    buffers = constant("kLaVotes")
    assert all(not unordered(first, buffers) for first in RUNS)


@pytest.mark.parametrize("buffers,holds", [(2, False), (3, True)])
def test_how_many_buffers_hold(buffers, holds):
    """Two hold within an item, but not where a tile without a look lies between."""
    assert all(not unordered(first, buffers) for first in RUNS) == holds
    assert not unordered((True,) + (False,) * 9, buffers)
