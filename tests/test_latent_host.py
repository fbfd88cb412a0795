"""Argument checks of the norm, rotation and latent-attention calls, without a GPU: each refusal returns its code
before anything is enqueued, and the binding refuses what it cannot pass on."""

import ctypes

import pytest
import torch

import paged_kv_cache_111_gb300 as pkv
from paged_kv_cache_111_gb300 import _build

OK, NULL, SHAPE, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4, 5
A, B = 0x10000, 0x20000          # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def caller(fn, names, defaults):
    def call(**kw):
        unknown = set(kw) - set(names)
        assert not unknown, unknown
        a = dict(defaults, **kw)
        return fn(*[a[n] for n in names])
    return call


QK = ("query_out", "out_stride", "cache", "nb", "hq", "hkv", "d", "bs", "query", "q_stride", "key", "k_stride", "value",
      "v_stride", "wq", "wk", "eps", "cos_sin", "max_pos", "rot", "inter", "positions", "slots", "T")
QK_OK = dict(query_out=A, out_stride=1024, cache=A, nb=4, hq=8, hkv=2, d=128, bs=16, query=A, q_stride=1024, key=A,
             k_stride=256, value=A, v_stride=256, wq=A, wk=A, eps=1e-6, cos_sin=A, max_pos=100, rot=128, inter=0,
             positions=B, slots=B, T=0, status=None, stream=None, ks=1.0, vs=1.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_qk_norm_rope_refusals(lib, fp8):
    names = QK + (("ks", "vs") if fp8 else ()) + ("status", "stream")
    call = caller(lib.pkv_qk_norm_rope_kv_write_fp8 if fp8 else lib.pkv_qk_norm_rope_kv_write, names, QK_OK)
    assert call() == OK                                    # no tokens: nothing enqueued
    for kw, code in ((dict(T=-1), SHAPE), (dict(nb=0), SHAPE), (dict(hq=0), SHAPE), (dict(hkv=0), SHAPE),
                     (dict(max_pos=0), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
                     (dict(d=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(rot=0), UNSUPPORTED),
                     (dict(rot=24), UNSUPPORTED), (dict(rot=144), UNSUPPORTED), (dict(nb=1 << 62), SHAPE)):
        assert call(**kw) == code, kw
    if fp8:
        for s in (0.0, -1.0, float("nan"), float("inf")):
            assert call(ks=s) == SHAPE and call(vs=s) == SHAPE
    for name in ("query_out", "cache", "query", "key", "value", "cos_sin", "positions", "slots"):
        assert call(T=3, **{name: None}) == NULL, name
    for name in ("query_out", "cache", "query", "key", "value", "wq", "wk", "cos_sin"):
        assert call(T=3, **{name: A + 8}) == ALIGNMENT, name
    for name in ("positions", "slots"):
        assert call(T=3, **{name: B + 4}) == ALIGNMENT, name
    for name, least in (("out_stride", 1024), ("q_stride", 1024), ("k_stride", 256), ("v_stride", 256)):
        assert call(T=3, **{name: least - 8}) == SHAPE, name
        assert call(T=3, **{name: least + 4}) == ALIGNMENT, name


def test_latent_write_refusals(lib):
    names = ("cache", "nb", "bs", "latent", "l_stride", "key_rope", "k_stride", "weight", "eps", "cos_sin", "max_pos",
             "inter", "positions", "slots", "T", "q_out", "qo_tok", "qo_head", "q", "q_tok", "q_head", "H", "status",
             "stream")
    call = caller(lib.pkv_latent_kv_write, names,
                  dict(cache=A, nb=4, bs=16, latent=A, l_stride=576, key_rope=A, k_stride=576, weight=A, eps=1e-6,
                       cos_sin=A, max_pos=10, inter=0, positions=B, slots=B, T=0, q_out=A, qo_tok=4 * 576, qo_head=576,
                       q=A, q_tok=4 * 192, q_head=192, H=4, status=None, stream=None))
    assert call() == OK
    for kw, code in ((dict(T=-1), SHAPE), (dict(nb=0), SHAPE), (dict(bs=8), UNSUPPORTED), (dict(eps=-0.5), SHAPE),
                     (dict(max_pos=0), SHAPE), (dict(H=-1), SHAPE),
                     (dict(T=2, l_stride=504), SHAPE), (dict(T=2, l_stride=580), ALIGNMENT),
                     (dict(T=2, k_stride=56), SHAPE), (dict(T=2, qo_head=56), SHAPE),
                     (dict(T=2, q_tok=3 * 192 + 56), SHAPE), (dict(T=2, q_head=240), SHAPE),
                     (dict(T=2, q_head=196, q_tok=1000), ALIGNMENT), (dict(T=2, q=None), NULL),
                     (dict(T=2, q_out=None), NULL), (dict(T=2, q_out=A + 2), ALIGNMENT),
                     (dict(T=2, weight=A + 4), ALIGNMENT), (dict(T=2, slots=B + 4), ALIGNMENT)):
        assert call(**kw) == code, kw
    for name in ("cache", "latent", "key_rope", "cos_sin", "positions", "slots"):
        assert call(T=2, **{name: None}) == NULL, name


def test_gather_refusals(lib):
    names = ("out", "rows", "cache", "nb", "bs", "bt", "width", "lens", "starts", "S", "max_len", "status", "stream")
    call = caller(lib.pkv_latent_gather, names, dict(out=A, rows=100, cache=A, nb=4, bs=16, bt=B, width=4, lens=B,
                                                     starts=B, S=0, max_len=64, status=None, stream=None))
    assert call() == OK and call(S=3, max_len=0) == OK
    for kw, code in ((dict(S=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(nb=0), SHAPE), (dict(bs=32), UNSUPPORTED),
                     (dict(S=65536), SHAPE), (dict(S=2, max_len=65), SHAPE), (dict(S=2, out=A + 8), ALIGNMENT),
                     (dict(S=2, lens=B + 2), ALIGNMENT)):
        assert call(**kw) == code, kw
    for name in ("out", "cache", "bt", "lens", "starts"):
        assert call(S=2, **{name: None}) == NULL, name


def latent_attn(lib, **kw):
    need = ctypes.c_size_t(0)
    names = ("out", "query", "q_stride", "cache", "nb", "bt", "width", "lens", "qsl", "S", "T", "max_q", "max_n", "H",
             "bs", "scale", "ws", "ws_bytes", "need", "stream")
    d = dict(out=A, query=A, q_stride=16 * 576, cache=A, nb=8, bt=B, width=4, lens=B, qsl=B, S=2, T=2, max_q=1, max_n=64,
             H=16, bs=16, scale=0.07, ws=None, ws_bytes=0, need=ctypes.byref(need), stream=None)
    return caller(lib.pkv_latent_paged_attn, names, d)(**kw), need.value


def test_latent_attn_refusals_and_size_query(lib):
    rc, need = latent_attn(lib)
    assert rc == WORKSPACE and need == pkv.latent_paged_attn_workspace_size(2, 2, 1, 64, 16) > 1 << 20
    # the size is the same whatever the batch
    assert pkv.latent_paged_attn_workspace_size(500, 9000, 4096, 100000, 128) == need
    ok = dict(ws=0x40000, ws_bytes=need)
    assert latent_attn(lib, S=0, T=0)[0] == OK
    for kw, code in ((dict(S=0), SHAPE), (dict(S=-1), SHAPE), (dict(H=0), SHAPE), (dict(nb=0), SHAPE),
                     (dict(H=1025), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(max_n=65), SHAPE),
                     (dict(max_q=65), SHAPE), (dict(nb=1 << 31), SHAPE), (dict(T=1 << 28), SHAPE),
                     (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE)):
        assert latent_attn(lib, **ok, **kw)[0] == code, kw
    assert latent_attn(lib, ws=0x40000, ws_bytes=need - 1)[0] == WORKSPACE
    assert latent_attn(lib, ws=0x40010, ws_bytes=need)[0] == ALIGNMENT
    for name in ("out", "query", "cache", "bt", "lens", "qsl"):
        assert latent_attn(lib, **ok, **{name: None})[0] == NULL, name
    for kw, code in ((dict(q_stride=15 * 576), SHAPE), (dict(q_stride=16 * 576 + 4), ALIGNMENT),
                     (dict(out=A + 8), ALIGNMENT), (dict(cache=A + 2), ALIGNMENT), (dict(lens=B + 1), ALIGNMENT)):
        assert latent_attn(lib, **ok, **kw)[0] == code, kw


def test_expanded_refusals(lib):
    names = ("out", "query", "q_tok", "key", "k_tok", "k_head", "rope", "r_tok", "value", "v_tok", "v_head", "qsl",
             "ksl", "S", "T", "K", "max_q", "max_k", "H", "scale", "status", "stream")
    call = caller(lib.pkv_latent_attn_expanded, names,
                  dict(out=A, query=A, q_tok=4 * 192, key=A, k_tok=4 * 256, k_head=256, rope=A, r_tok=576, value=A,
                       v_tok=4 * 256, v_head=256, qsl=B, ksl=B, S=2, T=5, K=9, max_q=4, max_k=6, H=4, scale=0.07,
                       status=None, stream=None))
    assert call(S=0, T=0) == OK and call(T=0) == OK and call(max_q=0) == OK
    for kw, code in ((dict(S=0), SHAPE), (dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(max_q=7), SHAPE),
                     (dict(scale=float("nan")), SHAPE), (dict(k_head=120), SHAPE), (dict(v_head=120), SHAPE),
                     (dict(q_tok=4 * 192 - 8), SHAPE), (dict(k_tok=120), SHAPE), (dict(r_tok=56), SHAPE),
                     (dict(v_tok=120), SHAPE), (dict(q_tok=4 * 192 + 4), ALIGNMENT), (dict(k_head=260), ALIGNMENT),
                     (dict(r_tok=580), ALIGNMENT), (dict(value=A + 8), ALIGNMENT), (dict(ksl=B + 2), ALIGNMENT)):
        assert call(**kw) == code, kw
    for name in ("out", "query", "key", "rope", "value", "qsl", "ksl"):
        assert call(**{name: None}) == NULL, name


def test_binding_refuses_cpu_tensors_and_wrong_forms():
    bf = torch.bfloat16
    cache = torch.zeros(1, 16, 576, dtype=bf)
    i32, i64 = torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    t64 = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        pkv.latent_kv_write(cache, torch.zeros(1, 512, dtype=bf), torch.zeros(1, 64, dtype=bf), None, 0.0, t64, i64, i64)
    with pytest.raises(ValueError):
        pkv.latent_gather(torch.zeros(1, 576, dtype=bf), cache, i32[None], i32, i32, 1)
    with pytest.raises(ValueError):
        pkv.latent_paged_attn(torch.zeros(1, 1, 512, dtype=bf), torch.zeros(1, 1, 576, dtype=bf), cache, i32[None], i32,
                              torch.zeros(2, dtype=torch.int32), 1, 1, 1.0, torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        x = torch.zeros(1, 1, 128, dtype=bf)
        pkv.latent_attn_expanded(x, torch.zeros(1, 1, 192, dtype=bf), x, torch.zeros(1, 64, dtype=bf), x, i32, i32, 1, 1,
                                 1.0)
    with pytest.raises(ValueError):
        x = torch.zeros(1, 1, 64, dtype=bf)
        pkv.qk_norm_rope_kv_write(x, torch.zeros(1, 1, 2, 16, 64, dtype=bf), x, x, x, None, None, 0.0, t64, i64, i64)
