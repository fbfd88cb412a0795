"""The binding's size query against the calls' own, without a GPU."""

import ctypes

import pytest

import paged_kv_cache_111_gb300 as pkv
from paged_kv_cache_111_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def needed(fn, before, S, T, max_q, max_n, hq, hkv, d, floats):
    need = ctypes.c_size_t(0)
    width = -(-max_n // 16)
    assert fn(*before, None, width, None, None, S, T, max_q, max_n, hq, hkv, d, 16, *floats, 0, None, 0,
              ctypes.byref(need), None) in (0, 1, 5)
    return need.value


@pytest.mark.parametrize("sizes", [
    (4, 4, 1, 300, 32, 8, 128), (4, 64, 16, 300, 32, 8, 128), (4, 68, 17, 300, 32, 8, 128),
    (3, 2050, 2046, 8190, 32, 8, 128), (2, 100, 99, 400, 8, 8, 64), (1, 1, 1, 17, 65, 1, 64), (0, 0, 0, 0, 4, 2, 64)])
def test_each_cache_pays_for_what_its_call_needs(lib, sizes):
    hq, hkv, d = sizes[4:]
    step = hq * d
    plain = needed(lib.pkv_paged_attn, (None, None, step, None, 1), *sizes, (1.0,))
    e4m3 = needed(lib.pkv_paged_attn_fp8, (None, None, step, None, 1), *sizes, (1.0, 1.0, 1.0))
    int8 = needed(lib.pkv_paged_attn_int8, (None, None, step, None, None, 1), *sizes, (1.0,))
    assert pkv.paged_attn_workspace_size(*sizes, int8=False) == plain == e4m3
    assert pkv.paged_attn_workspace_size(*sizes) == pkv.paged_attn_workspace_size(*sizes, int8=True) == int8
    # pieces of cut work items: two places for each of 152 CTAs, 256 rows of sums, and a record and states
    more = 152 * 32 + 2 * 152 * 256 * 4 * (2 + d)
    assert int8 - plain == (more if sizes[2] * (hq // hkv) > 64 else 0)


def test_sizes_that_no_call_takes(lib):
    for int8 in (False, True):
        with pytest.raises(pkv.PagedKVError):
            pkv.paged_attn_workspace_size(1, 1, 1, 16, 3, 2, 64, int8=int8)
