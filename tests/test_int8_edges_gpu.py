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
