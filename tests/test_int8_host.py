"""Argument checks of the int8 cache's calls, without a GPU: each refusal returns its code before anything is enqueued,
and the binding refuses what it cannot pass on."""

import ctypes

import numpy as np
import pytest
import torch

import int8_ref as ref
import paged_kv_cache_111_gb300 as pkv
from paged_kv_cache_111_gb300 import _build

OK, NULL, SHAPE, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4, 5
A, B = 0x10000, 0x20000          # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def caller(fn, defaults):
    def call(**kw):
        assert not set(kw) - set(defaults), kw
        return fn(*dict(defaults, **kw).values())
    return call


CACHE = (("cache", A), ("scales", A), ("nb", 4), ("hkv", 2), ("d", 128), ("bs", 16))
BAD_CACHE = ((dict(nb=0), SHAPE), (dict(hkv=0), SHAPE), (dict(d=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED),
             (dict(nb=1 << 31), SHAPE), (dict(hkv=1 << 21), SHAPE))


def test_write_refusals(lib):
    call = caller(lib.pkv_kv_write_int8, dict(CACHE, key=A, k_stride=256, value=A, v_stride=256, slots=B, T=0,
                                              status=None, stream=None))
    assert call() == OK                                     # no tokens: nothing enqueued
    for kw, code in BAD_CACHE + ((dict(T=-1), SHAPE),):
        assert call(**kw) == code, kw
    for name in ("cache", "scales", "key", "value", "slots"):
        assert call(T=3, **{name: None}) == NULL, name
    for name, off in (("cache", 8), ("key", 8), ("value", 8), ("scales", 4), ("slots", 4)):
        assert call(T=3, **{name: A + off}) == ALIGNMENT, name
    for name in ("k_stride", "v_stride"):
        assert call(T=3, **{name: 248}) == SHAPE and call(T=3, **{name: 260}) == ALIGNMENT
    assert call(T=(1 << 31) - 1, hkv=40, k_stride=1 << 20, v_stride=1 << 20) == SHAPE       # more warps than a launch has


def test_norm_rope_write_refusals(lib):
    call = caller(lib.pkv_qk_norm_rope_kv_write_int8,
                  dict(query_out=A, out_stride=1024, cache=A, scales=A, nb=4, hq=8, hkv=2, d=128, bs=16, query=A,
                       q_stride=1024, key=A, k_stride=256, value=A, v_stride=256, wq=A, wk=A, eps=1e-6, cos_sin=A,
                       max_pos=100, rot=128, inter=0, positions=B, slots=B, T=0, status=None, stream=None))
    assert call() == OK
    for kw, code in BAD_CACHE + ((dict(T=-1), SHAPE), (dict(hq=0), SHAPE), (dict(max_pos=0), SHAPE),
                                 (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(rot=0), UNSUPPORTED),
                                 (dict(rot=24), UNSUPPORTED), (dict(rot=144), UNSUPPORTED)):
        assert call(**kw) == code, kw
    for name in ("query_out", "cache", "scales", "query", "key", "value", "cos_sin", "positions", "slots"):
        assert call(T=3, **{name: None}) == NULL, name
    for name in ("query_out", "cache", "query", "key", "value", "wq", "wk", "cos_sin"):
        assert call(T=3, **{name: A + 8}) == ALIGNMENT, name
    for name in ("scales", "positions", "slots"):
        assert call(T=3, **{name: B + 4}) == ALIGNMENT, name
    for name, least in (("out_stride", 1024), ("q_stride", 1024), ("k_stride", 256), ("v_stride", 256)):
        assert call(T=3, **{name: least - 8}) == SHAPE and call(T=3, **{name: least + 4}) == ALIGNMENT, name


def test_gather_refusals(lib):
    call = caller(lib.pkv_kv_gather_int8, dict(key_out=A, value_out=A, rows=100, **dict(CACHE), bt=B, width=4, lens=B,
                                               starts=B, S=0, max_len=64, status=None, stream=None))
    assert call() == OK
    for kw, code in BAD_CACHE + ((dict(S=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(S=65536), SHAPE),
                                 (dict(S=2, max_len=65), SHAPE), (dict(S=2, max_len=-1), SHAPE)):
        assert call(**kw) == code, kw
    for name in ("key_out", "value_out", "cache", "scales", "bt", "lens", "starts"):
        assert call(S=2, **{name: None}) == NULL, name
    for name, off in (("key_out", 8), ("value_out", 2), ("cache", 8), ("scales", 4), ("bt", 2), ("lens", 2), ("starts", 1)):
        assert call(S=2, **{name: A + off}) == ALIGNMENT, name


def test_copy_refusals(lib):
    call = caller(lib.pkv_copy_blocks_int8, dict(CACHE, mapping=B, pairs=0, status=None, stream=None))
    assert call() == OK
    for kw, code in BAD_CACHE + ((dict(pairs=-1), SHAPE),):
        assert call(**kw) == code, kw
    for name in ("cache", "scales", "mapping"):
        assert call(pairs=2, **{name: None}) == NULL, name
    for name, off in (("cache", 8), ("scales", 4), ("mapping", 4)):
        assert call(pairs=2, **{name: A + off}) == ALIGNMENT, name
    assert call(pairs=(1 << 31) - 1, hkv=40) == SHAPE


def test_attention_refusals_and_size_query(lib):
    need = ctypes.c_size_t(0)
    call = caller(lib.pkv_paged_attn_int8,
                  dict(out=A, query=A, q_stride=512, cache=A, scales=A, nb=16, bt=B, width=4, lens=B, qsl=B, S=2, T=2,
                       max_q=1, max_n=64, H=4, hkv=2, d=128, bs=16, scale=0.1, splits=0, ws=None, ws_bytes=0,
                       need=ctypes.byref(need), stream=None))
    assert call() == WORKSPACE
    size = need.value
    assert size == pkv.paged_attn_workspace_size(2, 2, 1, 64, 4, 2, 128) > 256
    ok = dict(ws=0x40000, ws_bytes=size)
    for kw, code in ((dict(d=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(H=3), SHAPE), (dict(width=3), SHAPE),
                     (dict(S=0), SHAPE), (dict(max_q=65), SHAPE), (dict(scale=float("nan")), SHAPE),
                     (dict(nb=1 << 30), SHAPE), (dict(ws_bytes=size - 1), WORKSPACE), (dict(ws=0x40010), ALIGNMENT),
                     (dict(q_stride=500), SHAPE), (dict(q_stride=516), ALIGNMENT), (dict(scales=A + 4), ALIGNMENT),
                     (dict(cache=A + 8), ALIGNMENT), (dict(splits=-1), SHAPE)):
        assert call(**dict(ok, **kw)) == code, kw
    for name in ("out", "query", "cache", "scales", "bt", "lens", "qsl"):
        assert call(**ok, **{name: None}) == NULL, name
    assert call(S=0, T=0) == OK


def test_binding_refusals():
    cache, scales = ref.new_cache(4, 2, 64)
    x, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    i32 = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: pkv.kv_write_int8(cache, scales, x, x, slots),
                 lambda: pkv.copy_blocks_int8(cache, scales, torch.zeros(1, 2, dtype=torch.int64)),
                 lambda: pkv.kv_gather_int8(x, x, cache, scales, i32.view(1, 4), i32[:1], i32[:1], 3),
                 lambda: pkv.paged_attn_int8(x, x, cache, scales, i32.view(1, 4), i32[:1], i32[:2], 3, 3, 1.0, i32),
                 lambda: pkv.qk_norm_rope_kv_write_int8(x, cache, scales, x, x, x, None, None, 0.0, torch.zeros(4, 64),
                                                        slots, slots)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()


def test_the_model_of_the_write():
    """The tests' model against the definition, by hand: a fresh block, one that grows, one that does not."""
    cache, scales = np.full((2, 1, 2, 16, 64), 100, np.int8), np.full((2, 1, 2), 0.5, np.float32)
    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, 0], x[1, 0, 0] = 254.0, -127.0
    ref.write(cache, scales, x, x / 254, np.array([16, 3]))
    assert scales[1, 0, 0] == 2.0 and cache[1, 0, 0, 0, 0] == 127 and cache[1, 0, 0, 1, 0] == 100
    assert scales[0, 0, 0] == 1.0 and cache[0, 0, 0, 3, 0] == -127 and (cache[0, 0, 0, :3] == 50).all()
    assert scales[0, 0, 1] == 0.5 and cache[0, 0, 1, 3, 0] == -1 and (cache[0, 0, 1, 4:] == 100).all()
