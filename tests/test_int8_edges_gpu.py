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
@pytest.mark.parametrize("reqs", [[(1, 100), (1, 16)], [(3, 40), (2, 2)], [(70, 70), (1, 30)], [(200, 333)],
                                  [(40, 6000)]])
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


# The kernels' references: a row's largest weight (times its V scale) is 2^7 (decode) or 2^3 (chunks) or more of the
# unit that a weight's f16 has, so a subnormal weight is off by 2^-25 / 2^7, 2^-25 / 2^3 of the largest at most.
SUBNORMAL_DECODE, SUBNORMAL_CHUNK = 2.0 ** -32, 2.0 ** -28


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("reqs,num_splits", [([(1, 579)], 1), ([(1, 579), (3, 2000)], 0), ([(200, 779)], 0),
                                             ([(40, 6000)], 0)])
def test_a_key_that_takes_nearly_all_of_the_weight(reqs, num_splits, d):
    """The first key has a value of zero and the others a weight of 5.45 * 2^-24 of its own each, with values of one
    sign: an f16 against that weight would be off by 9%, and all of them the same way."""
    s = batch(reqs, 8, 2, d, seed=22)
    lift = -math.log(5.45 * 2.0 ** -24)
    s["scales"].fill_(1 / 36)
    s["scale"] = lift * 36 / (127 * d)
    s["query"].fill_(1.0)
    g = torch.Generator().manual_seed(3)
    shape = s["cache"][:, :, 1].shape
    s["cache"][:, :, 0] = 0
    s["cache"][:, :, 1] = torch.randint(64, 128, shape, generator=g, dtype=torch.int8).cuda()
    first = s["tables"][:, 0].long()
    s["cache"][first, :, 0, 0] = 127
    s["cache"][first, :, 1, 0] = 0
    out = run(s, num_splits=num_splits)
    want, _ = ref.attention(s["query"], s["cache"], s["scales"], s["tables"], s["lens"], s["qsl"], s["scale"])
    # per row, all of `want` positive: f16 of the weights, subnormal weights, the scores' errors (int8_ref.attention's
    # bound of them: the largest term of S is 1152 sum q, 1152 / 127 times the largest score), the output's bf16
    rows = torch.tensor([q for q, _ in reqs], device="cuda")
    keys = torch.tensor([n for _, n in reqs], device="cuda").repeat_interleave(rows)
    slip = 2 * 16 * 2 * ref.FP32_STEP * (1152 / 127 * lift) + 2.0 ** -18
    least = SUBNORMAL_DECODE if s["max_q"] * 4 <= 64 else SUBNORMAL_CHUNK
    top = (127 * least * keys.double() / 36)[:, None, None]                   # (the largest weight is below one)
    e = (ref.F16_HALF_STEP + slip) * want + top
    ref.check(out, want, ref.BF16_HALF_STEP * want + (1 + ref.BF16_HALF_STEP) * e)


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


@pytest.mark.parametrize("hq,hkv", [(32, 1), (24, 1), (64, 1), (65, 1), (128, 1), (300, 1), (256, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_query_heads_a_kv_head(hq, hkv, d):
    """One token is two or more tiles of 16 rows up to 64 heads a kv head, and a chunk's work item beyond."""
    for reqs in ([(1, 1)], [(1, 17), (1, 300), (1, 128)], [(1, 9000)], [(2, 40), (1, 500)], [(3, 9000), (1, 5)]):
        s = batch(reqs, hq, hkv, d, seed=hq)
        check(s, run(s), str(reqs))


@pytest.mark.parametrize("q,n", [(1, 131072), (16, 131072), (40, 100003)])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (128, 1, 64)])
def test_few_work_items_of_very_many_keys(q, n, hq, hkv, d):
    s = batch([(q, n)], hq, hkv, d, seed=24)
    check(s, run(s))


@pytest.mark.parametrize("reqs", [[(1, 900)] * 20, [(200, 6000), (1, 40)], [(2046, 2100)]])
def test_two_calls_at_once(reqs):
    """On two streams, each with a workspace of its own and the cache in common."""
    s = batch(reqs, 8, 2, 128, seed=26)
    one = run(s)
    T, hq, d = s["query"].shape
    lens, qsl = (torch.tensor(s[k], dtype=torch.int32, device="cuda") for k in ("lens", "qsl"))
    n = pkv.paged_attn_workspace_size(len(reqs), T, s["max_q"], s["max_n"], hq, 2, d)
    sides = [(torch.cuda.Stream(), torch.empty(n, dtype=torch.uint8, device="cuda"), torch.zeros_like(one))
             for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for stream, ws, out in sides:
            pkv.paged_attn_int8(out, s["query"], s["cache"], s["scales"], s["tables"], lens, qsl, s["max_q"],
                                s["max_n"], s["scale"], ws, stream=stream)
            pkv.paged_attn_combine(out, ws, stream=stream)
    torch.cuda.synchronize()
    for _, ws, out in sides:
        assert pkv.workspace_status(ws) == 0
        assert torch.equal(out, one)


def test_the_combine_without_the_module(monkeypatch, tmp_path):
    """As built without Python's headers: attention over the other caches still has its combine."""
    from paged_kv_cache_111_gb300 import _build
    s = batch([(1, 900), (3, 400), (70, 90)], 8, 2, 64, seed=27)
    one = run(s)
    combine = pkv.paged_attn_combine

    def without(*args, **kw):
        with monkeypatch.context() as m:
            m.setattr(pkv, "_module", None)
            m.setattr(_build, "CALLS", str(tmp_path / "none.so"))
            combine(*args, **kw)

    monkeypatch.setattr(pkv, "paged_attn_combine", without)
    assert torch.equal(run(s), one)
