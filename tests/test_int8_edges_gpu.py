"""Attention over an int8 cache on the GPU: queries that are no numbers, keys that take nearly all of the weight, many
query heads a kv head, few work items of very many keys, and the same call again and again."""

import math

import pytest
import torch

import int8_ref as ref
import paged_kv_cache_111_gb300 as pkv
from test_int8_attn_gpu import BLOCK, batch, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def built():
    from paged_kv_cache_111_gb300 import _build
    _build.build()


@pytest.mark.parametrize("value", [-math.inf, math.inf, math.nan])
@pytest.mark.parametrize("reqs", [[(1, 100), (1, 16)], [(3, 40), (2, 2)], [(70, 70), (1, 30)], [(200, 333)], [(40, 6000)]])
@pytest.mark.parametrize("scale", [0.1, -0.1])
def test_queries_that_are_no_numbers(value, reqs, scale):
    """Such a row is NaN, wherever the mask cuts it; the others are as if it were not there."""
    s = batch(reqs, 8, 2, 64, seed=21)
    s["scale"] = scale
    want, bound = ref.attention(s["query"], s["cache"], s["scales"], s["tables"], s["lens"], s["qsl"], scale)
    T = s["query"].shape[0]
    spoiled = torch.zeros(T, 8, dtype=torch.bool, device="cuda")
    spoiled[::3, 1] = spoiled[::7, 6] = spoiled[T - 1, 3] = True
    query = s["query"].clone()
    query[..., 5][spoiled] = value
    out = run(s, query=query)
    assert torch.isnan(out[spoiled].float()).all()
    ref.check(out[~spoiled], want[~spoiled], bound[~spoiled])


@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("reqs", [[(4, 34)], [(200, 300)], [(40, 5990)]])
def test_rows_that_do_not_see_a_block_of_an_infinite_scale(side, reqs):
    s = batch(reqs, 4, 2, 64, seed=25)
    q, n = reqs[0]
    page = (n - 1) // BLOCK
    want, bound = ref.attention(s["query"], s["cache"], s["scales"], s["tables"], s["lens"], s["qsl"], s["scale"])
    s["scales"][s["tables"][0, page].long(), 1, side] = float("inf")
    out = run(s)
    blind = (torch.arange(n - q, n) < page * BLOCK).cuda()
    assert blind.any()
    ref.check(out[:, :2], want[:, :2], bound[:, :2])
    ref.check(out[blind], want[blind], bound[blind])


@pytest.mark.parametrize("reqs,hq,hkv", [([(1, 2000)] * 300 + [(300, 9000)] * 5, 32, 1),
                                         ([(1, 30)] * 1100 + [(33, 9000)] * 40, 8, 1),
                                         ([(64, 40000), (64, 40000), (64, 36000)] * 3, 8, 2)])
def test_the_same_again_and_again(reqs, hq, hkv):
    """Work items of one size, cut along their keys: which of them are cut, and where, must not vary between calls."""
    s = batch(reqs, hq, hkv, 64, seed=23)
    one = run(s)
    check(s, one)
    for k in range(100):
        assert torch.equal(run(s), one), k
