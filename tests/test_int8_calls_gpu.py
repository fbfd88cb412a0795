"""The int8 calls' marshalling: what each refuses, by its argument, and the streams and views that it takes."""

import pytest
import torch

import int8_ref as ref
import paged_kv_cache_111_gb300 as pkv

pytestmark = pytest.mark.gpu
NB, HKV, HQ, D, T = 6, 2, 4, 64, 3


@pytest.fixture(autouse=True, scope="module")
def built():
    from paged_kv_cache_111_gb300 import _build
    _build.build()


def arguments():
    cache, scales = (x.cuda() for x in ref.new_cache(NB, HKV, D))
    g = torch.Generator().manual_seed(0)
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    i64 = lambda v: torch.tensor(v, dtype=torch.int64, device="cuda")
    size = pkv.paged_attn_workspace_size(2, T, 2, 32, HQ, HKV, D)
    status = i32([0])
    return {
        "kv_write_int8": dict(kv_cache=cache, kv_scales=scales, key=bf(T, HKV, D), value=bf(T, HKV, D),
                              slot_mapping=i64([16, 17, 40]), device_status=status),
        "qk_norm_rope_kv_write_int8": dict(
            query_out=bf(T, HQ, D), kv_cache=cache, kv_scales=scales, query=bf(T, HQ, D), key=bf(T, HKV, D),
            value=bf(T, HKV, D), q_weight=bf(D), k_weight=bf(D), eps=1e-6, cos_sin=torch.ones(8, D, device="cuda"),
            positions=i64([0, 1, 2]), slot_mapping=i64([16, 17, 40]), device_status=status),
        "paged_attn_int8": dict(
            out=bf(T, HQ, D), query=bf(T, HQ, D), kv_cache=cache, kv_scales=scales, block_tables=i32([[1, 2], [3, 4]]),
            seq_lens=i32([20, 9]), query_start_loc=i32([0, 1, 3]), max_query_len=2, max_seq_len=32, scale=0.1,
            workspace=torch.zeros(size, dtype=torch.uint8, device="cuda")),
        "kv_gather_int8": dict(
            key_out=bf(29, HKV, D), value_out=bf(29, HKV, D), kv_cache=cache, kv_scales=scales,
            block_tables=i32([[1, 2], [3, 4]]), seq_lens=i32([20, 9]), key_start_loc=i32([0, 20]), max_seq_len=32,
            device_status=status),
        "copy_blocks_int8": dict(kv_cache=cache, kv_scales=scales, block_mapping=i64([[1, 5]]), device_status=status),
    }


NAMES = ["kv_write_int8", "qk_norm_rope_kv_write_int8", "paged_attn_int8", "kv_gather_int8", "copy_blocks_int8"]
OPTIONAL = ("q_weight", "k_weight", "device_status")


def wrong_forms(name, x):
    """(what is wrong, the tensor) for a tensor argument."""
    yield "on the CPU", x.cpu()
    if name != "workspace":
        yield "of another type", x.to(torch.float16 if x.is_floating_point() else torch.int16)
        yield "of one dim more", x[None]
        if name != "device_status" and name != "key_start_loc" and x.numel():
            yield "with a last entry less", x[..., :-1].contiguous()
    if x.dim() == 1:
        yield "not contiguous", x.repeat_interleave(2)[::2]
    else:
        yield "not contiguous", x.transpose(-1, -2).contiguous().transpose(-1, -2)


@pytest.mark.parametrize("name", NAMES)
def test_every_argument_of_another_form_is_refused(name):
    call = getattr(pkv, name)
    args = arguments()[name]
    call(**args)
    torch.cuda.synchronize()
    before = {k: v.clone() for k, v in args.items() if torch.is_tensor(v) and k != "workspace"}
    for what, x in args.items():
        if not torch.is_tensor(x):
            continue
        for wrong, y in wrong_forms(what, x):
            if wrong == "not contiguous" and y.is_contiguous():
                continue                                       # (a vector of one entry)
            if wrong == "with a last entry less":              # (which contradicts other sizes, or is no head size)
                with pytest.raises((ValueError, pkv.PagedKVError)):
                    call(**dict(args, **{what: y}))
                continue
            with pytest.raises(ValueError):
                call(**dict(args, **{what: y}))
        for wrong in [3, "x"] + ([] if what in OPTIONAL else [None]):
            with pytest.raises((AttributeError, TypeError)):
                call(**dict(args, **{what: wrong}))
    torch.cuda.synchronize()
    for k, v in before.items():
        assert torch.equal(args[k].view(torch.uint8), v.view(torch.uint8)), k
    for what in OPTIONAL:
        if what in args:
            call(**dict(args, **{what: None}))


def test_numbers_that_are_none_or_too_large():
    args = arguments()["paged_attn_int8"]
    for what in ("max_query_len", "max_seq_len"):
        with pytest.raises(OverflowError):
            pkv.paged_attn_int8(**dict(args, **{what: (1 << 32) + 2}))
        with pytest.raises(TypeError):
            pkv.paged_attn_int8(**dict(args, **{what: "2"}))
    with pytest.raises(TypeError):
        pkv.paged_attn_int8(**dict(args, scale="1"))
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attn_int8(**dict(args, workspace=args["workspace"][:64]))
    with pytest.raises(OverflowError):
        pkv.kv_gather_int8(**dict(arguments()["kv_gather_int8"], max_seq_len=1 << 40))


@pytest.mark.parametrize("form", ["object", "handle", "current"])
def test_streams(form):
    args = arguments()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = arguments()
    for name in NAMES:
        getattr(pkv, name)(**want[name])
    pkv.paged_attn_combine(want[NAMES[2]]["out"], want[NAMES[2]]["workspace"])
    torch.cuda.synchronize()
    given = {"object": stream, "handle": stream.cuda_stream, "current": None}[form]
    with torch.cuda.stream(stream if form == "current" else torch.cuda.current_stream()):
        for name in NAMES:
            getattr(pkv, name)(**args[name], stream=given)
        pkv.paged_attn_combine(args[NAMES[2]]["out"], args[NAMES[2]]["workspace"], stream=given)
    stream.synchronize()
    for name in NAMES:
        for k, v in args[name].items():
            if torch.is_tensor(v) and k != "workspace":
                assert torch.equal(v.view(torch.uint8), want[name][k].view(torch.uint8)), (name, k)


def test_a_row_or_a_head_of_any_stride():
    # the stride of a dim of one entry means nothing
    args = arguments()["kv_write_int8"]
    one = torch.randn(1, HKV, D, device="cuda").bfloat16()
    slots = args["slot_mapping"][:1]
    got = []
    for k in (one, one.as_strided((1, HKV, D), (3, D, 1))):
        cache, scales = args["kv_cache"].clone(), args["kv_scales"].clone()
        pkv.kv_write_int8(cache, scales, k, k, slots)
        got.append((cache, scales))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    cache, scales = (x.cuda() for x in ref.new_cache(NB, 1, D))
    x = torch.randn(T, 1, D, device="cuda").bfloat16()
    other, oscales = cache.clone(), scales.clone()
    pkv.kv_write_int8(cache, scales, x, x, args["slot_mapping"])
    y = x.as_strided((T, 1, D), (D, 7, 1))
    pkv.kv_write_int8(other, oscales, y, y, args["slot_mapping"])
    assert torch.equal(cache, other) and torch.equal(scales, oscales)
