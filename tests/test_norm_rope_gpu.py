"""Norm, rotation and cache write in one pass, the latent cache's write and gather, against plain 64-bit forms.

The bound of a comparison is half a bf16 step of the value plus the fp32 steps of the arithmetic (latent_ref)."""

import pytest
import torch

import paged_kv_cache_111_gb300 as pkv
from latent_ref import angles, check_rounded, norm_rotate

pytestmark = pytest.mark.gpu


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).cuda()


def poisoned(*shape, dtype=torch.bfloat16):
    if dtype == torch.uint8:
        return torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def qk_case(seed, T, hq, hkv, d, rot, fused=True, max_pos=5000, blocks=None):
    g = torch.Generator().manual_seed(seed)
    blocks = blocks or 2 * (T // 16) + 3
    if fused:
        qkv = randn(g, T, hq + 2 * hkv, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = randn(g, T, hq, d, scale=30.0), randn(g, T, hkv, d, scale=0.01), randn(g, T, hkv, d)
    return dict(q=q, k=k, v=v, wq=randn(g, d), wk=randn(g, d), table=angles(rot, max_pos).cuda(),
                pos=torch.randint(0, max_pos, (T,), generator=g).cuda(),
                slots=torch.randperm(blocks * 16, generator=g)[:T].cuda(), blocks=blocks)


@pytest.mark.parametrize("T,hq,hkv,d,rot,inter,fused", [
    (1, 1, 1, 64, 16, False, True), (1, 8, 8, 64, 64, True, True), (3, 5, 1, 128, 128, False, False),
    (17, 32, 8, 128, 128, True, True), (64, 32, 4, 64, 48, False, True), (33, 40, 40, 128, 64, True, False),
    (257, 7, 7, 128, 112, False, True), (1000, 3, 1, 64, 32, True, True), (2046, 32, 8, 128, 128, False, True)])
def test_qk_against_64_bits(T, hq, hkv, d, rot, inter, fused):
    c = qk_case(T + hq, T, hq, hkv, d, rot, fused)
    c["slots"][::7] = -1 if T > 8 else c["slots"][::7]           # padding among them
    cache = poisoned(c["blocks"], hkv, 2, 16, d)
    before = cache.clone()
    out = poisoned(T, hq, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.qk_norm_rope_kv_write(out, cache, c["q"], c["k"], c["v"], c["wq"], c["wk"], 1e-6, c["table"], c["pos"],
                              c["slots"], interleaved=inter, device_status=status)
    check_rounded(out, *norm_rotate(c["q"], c["wq"], 1e-6, c["table"], c["pos"], inter), "query")
    kept = c["slots"] >= 0
    s = c["slots"][kept]
    k, m = norm_rotate(c["k"], c["wk"], 1e-6, c["table"], c["pos"], inter)
    check_rounded(cache[s // 16, :, 0, s % 16], k[kept], m[kept], "key")
    assert torch.equal(cache[s // 16, :, 1, s % 16].view(torch.int16), c["v"][kept].contiguous().view(torch.int16))
    # every other slot as it was, bit for bit
    before[s // 16, :, :, s % 16] = cache[s // 16, :, :, s % 16]
    assert torch.equal(before.view(torch.int16), cache.view(torch.int16))
    assert int(status.item()) == 0


@pytest.mark.parametrize("inter", [False, True])
def test_qk_without_weights_and_in_place(inter):
    c = qk_case(5, 50, 6, 2, 128, 96)
    ref, mag = norm_rotate(c["q"], None, 0.0, c["table"], c["pos"], inter)
    cache = poisoned(c["blocks"], 2, 2, 16, 128)
    pkv.qk_norm_rope_kv_write(c["q"], cache, c["q"], c["k"], c["v"], None, c["wk"], 0.0, c["table"], c["pos"],
                              c["slots"], interleaved=inter)
    check_rounded(c["q"], ref, mag, "query in place")


def test_qk_only_rotates_where_asked():
    """An all-zero row has no direction: the norm leaves zeros (eps), never NaN; cosine 1 and sine 0 leave values."""
    T, d = 4, 64
    q = torch.zeros(T, 2, d, dtype=torch.bfloat16, device="cuda")
    k = torch.randn(T, 1, d, device="cuda").bfloat16()
    table = torch.zeros(8, 32, device="cuda")
    table[:, :16] = 1
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    cache = poisoned(1, 1, 2, 16, d)
    pos, slots = torch.arange(T, device="cuda"), torch.arange(T, device="cuda")
    out = poisoned(T, 2, d)
    pkv.qk_norm_rope_kv_write(out, cache, q, k, k, w, None, 1e-6, table, pos, slots)
    assert torch.equal(out, q)
    assert torch.equal(cache[0, 0, 0, :T].view(torch.int16), k[:, 0].contiguous().view(torch.int16))


@pytest.mark.parametrize("T,hq,hkv,d,rot,inter", [(5, 8, 2, 64, 64, True), (130, 16, 8, 128, 64, False),
                                                  (40, 4, 4, 128, 128, True)])
def test_qk_fp8(T, hq, hkv, d, rot, inter):
    c = qk_case(T, T, hq, hkv, d, rot)
    ks, vs = 0.0173, 0.003                                       # the second saturates some values
    cache = poisoned(c["blocks"], hkv, 2, 16, d, dtype=torch.uint8)
    other = cache.clone()
    out = poisoned(T, hq, d)
    pkv.qk_norm_rope_kv_write_fp8(out, cache, c["q"], c["k"], c["v"], c["wq"], c["wk"], 1e-6, c["table"], c["pos"],
                                  c["slots"], ks, vs, interleaved=inter)
    check_rounded(out, *norm_rotate(c["q"], c["wq"], 1e-6, c["table"], c["pos"], inter), "query")
    # V exactly as the plain write stores it, and nothing but the tokens' slots touched
    pkv.kv_write_fp8(other, c["k"], c["v"], c["slots"], ks, vs)
    assert torch.equal(cache[:, :, 1], other[:, :, 1])
    touched = torch.zeros(c["blocks"] * 16, dtype=torch.bool, device="cuda")
    touched[c["slots"]] = True
    rows = cache[:, :, 0].transpose(1, 2).reshape(c["blocks"] * 16, hkv, d)
    assert (rows[~touched] == 0x7F).all()
    # K within half an E4M3 step (2^-4 of the value, 2^-10 below the normal range) of the quotient, which the
    # fp32 scale enters as its fp32 value
    k, m = norm_rotate(c["k"], c["wk"], 1e-6, c["table"], c["pos"], inter)
    want = (k / torch.tensor(ks, dtype=torch.float32).double().item()).clamp(-448, 448)
    got = rows[c["slots"]].view(torch.float8_e4m3fn).double()
    bound = torch.maximum(want.abs() * 2.0 ** -4, torch.full_like(want, 2.0 ** -10)) + 1e-4 * m / ks
    assert ((got - want).abs() <= bound).all()
    # and with nothing to norm or turn, K as the plain write stores it
    still = torch.zeros(1, rot, device="cuda")
    still[:, :rot // 2] = 1
    pkv.qk_norm_rope_kv_write_fp8(out, cache, c["q"], c["k"], c["v"], None, None, 0.0, still,
                                  torch.zeros_like(c["pos"]), c["slots"], ks, vs, interleaved=inter)
    assert torch.equal(cache, other)
    assert torch.equal(out.view(torch.int16), c["q"].contiguous().view(torch.int16))


def test_qk_reports_bad_positions_and_slots():
    c = qk_case(9, 6, 4, 2, 64, 64, max_pos=100, blocks=2)
    c["pos"][:] = torch.tensor([0, 100, 5, -1, 7, 8])
    c["slots"][:] = torch.tensor([0, 1, 32, 2, -1, 3])
    cache = poisoned(2, 2, 2, 16, 64)
    out = poisoned(6, 4, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (c["q"], c["k"], c["v"], c["wq"], c["wk"], 1e-6, c["table"])
    pkv.qk_norm_rope_kv_write(out, cache, *args, c["pos"], c["slots"], device_status=status)
    assert int(status.item()) == 7
    done = torch.isfinite(out.float()).all(-1).all(-1)
    assert done.tolist() == [True, False, True, False, True, True]
    stored = torch.isfinite(cache.float()).all(-1).all(1).all(1)    # [block, slot]
    assert stored.nonzero().tolist() == [[0, 0], [0, 3]]
    # padding with a position from nowhere is no error
    status.zero_()
    c["pos"][:] = 1 << 40
    c["slots"][:] = -5
    pkv.qk_norm_rope_kv_write(out, cache, *args, c["pos"], c["slots"], device_status=status)
    assert int(status.item()) == 0


def test_qk_then_attention_is_the_step_by_hand():
    """A layer-step through the fused write gives the bits of the same rows written by kv_write."""
    g = torch.Generator().manual_seed(3)
    S, hq, hkv, d, L = 5, 8, 2, 128, 70
    table_rows = angles(d, 256).cuda()
    w = randn(g, d)
    width = -(-L // 16)
    bt = torch.randperm(S * width, generator=g).view(S, width).to(torch.int32).cuda()
    pool = poisoned(S * width, hkv, 2, 16, d)
    lens = torch.tensor([L, 1, 16, 17, 33])
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    seq = torch.repeat_interleave(torch.arange(S), lens).cuda()
    slots = bt[seq, pos // 16].long() * 16 + pos % 16
    T = int(lens.sum())
    q, k, v = randn(g, T, hq, d), randn(g, T, hkv, d), randn(g, T, hkv, d)
    qo = torch.empty_like(q)
    pkv.qk_norm_rope_kv_write(qo, pool, q, k, v, w, w, 1e-5, table_rows, pos, slots)
    lens_d = lens.to(torch.int32).cuda()
    qsl = torch.tensor([0] + lens.tolist()).cumsum(0).to(torch.int32).cuda()
    ws = torch.zeros(pkv.paged_attn_workspace_size(S, T, L, L, hq, hkv, d), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    pkv.paged_attn(out, qo, pool, bt, lens_d, qsl, L, L, d ** -0.5, ws)
    pkv.paged_attn_combine(out, ws)
    again = poisoned(S * width, hkv, 2, 16, d)
    pkv.kv_write(again, pool[slots // 16, :, 0, slots % 16].contiguous(), v, slots)
    out2 = torch.empty_like(q)
    pkv.paged_attn(out2, qo, again, bt, lens_d, qsl, L, L, d ** -0.5, ws)
    pkv.paged_attn_combine(out2, ws)
    assert torch.equal(pool.view(torch.int16), again.view(torch.int16))
    assert torch.equal(out, out2) and torch.isfinite(out.float()).all()


# ---- latent cache -------------------------------------------------------------------------------------------------

def latent_case(seed, T, H, blocks=None, max_pos=3000):
    g = torch.Generator().manual_seed(seed)
    blocks = blocks or 2 * (T // 16) + 3
    down = randn(g, T, 576)
    return dict(c=down[:, :512], kr=down[:, 512:], w=randn(g, 512), table=angles(64, max_pos).cuda(),
                pos=torch.randint(0, max_pos, (T,), generator=g).cuda(), blocks=blocks,
                slots=torch.randperm(blocks * 16, generator=g)[:T].cuda(),
                q=randn(g, T, max(H, 1), 192), rows=randn(g, T, max(H, 1), 576))


@pytest.mark.parametrize("T,H,inter", [(1, 1, False), (1, 128, True), (7, 5, True), (64, 16, False), (300, 17, True),
                                       (1025, 33, False)])
def test_latent_write_against_64_bits(T, H, inter):
    c = latent_case(T, T, H)
    if T > 8:
        c["slots"][3::5] = -1
    cache = poisoned(c["blocks"], 16, 576)
    rows = c["rows"].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.latent_kv_write(cache, c["c"], c["kr"], c["w"], 1e-6, c["table"], c["pos"], c["slots"],
                        query_rope_out=rows[:, :, 512:], query_rope=c["q"][:, :, 128:], interleaved=inter,
                        device_status=status)
    assert int(status.item()) == 0
    check_rounded(rows[:, :, 512:], *norm_rotate(c["q"][:, :, 128:], None, 0, c["table"], c["pos"], inter), "query")
    assert torch.equal(rows[:, :, :512], c["rows"][:, :, :512])
    kept = c["slots"] >= 0
    flat = cache.view(-1, 576)
    got = flat[c["slots"][kept]]
    lat = c["c"].double()[kept]
    ref = lat / (lat.square().mean(-1, keepdim=True) + 1e-6).sqrt() * c["w"].double()
    check_rounded(got[:, :512], ref, ref.abs(), "latent")
    kr, m = norm_rotate(c["kr"][:, None], None, 0, c["table"], c["pos"], inter)
    check_rounded(got[:, 512:], kr[kept][:, 0], m[kept][:, 0], "rotated key")
    untouched = torch.ones(flat.shape[0], dtype=torch.bool, device="cuda")
    untouched[c["slots"][kept]] = False
    assert torch.isnan(flat[untouched].float()).all()


def test_latent_write_without_norm_or_query_and_its_reports():
    c = latent_case(2, 6, 0, blocks=1, max_pos=50)
    c["pos"][:] = torch.tensor([0, 1, 50, 3, -1, 49])
    c["slots"][:] = torch.tensor([0, 16, 2, -1, -1, 15])
    cache = poisoned(1, 16, 576)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.latent_kv_write(cache, c["c"], c["kr"], None, 0.0, c["table"], c["pos"], c["slots"], device_status=status)
    assert int(status.item()) == 7
    assert torch.equal(cache[0, [0, 15], :512].view(torch.int16), c["c"][[0, 5]].contiguous().view(torch.int16))
    assert torch.isnan(cache[0, 1:15].float()).all()
    # in place: the query's own memory
    q = c["q"][:, :, 128:]
    c["pos"].clamp_(0, 49)
    c["slots"][1] = 5
    ref = norm_rotate(q, None, 0, c["table"], c["pos"], True)
    status.zero_()
    pkv.latent_kv_write(cache, c["c"], c["kr"], None, 0.0, c["table"], c["pos"], c["slots"], query_rope_out=q,
                        query_rope=q, interleaved=True, device_status=status)
    check_rounded(q, *ref, "query in place")
    assert int(status.item()) == 0


@pytest.mark.parametrize("lens", [[1], [16], [0, 17, 32, 1], [33, 0, 48, 31, 5000]])
def test_gather_is_the_pages(lens):
    g = torch.Generator().manual_seed(sum(lens))
    S, width = len(lens), max(1, max(-(-n // 16) for n in lens))
    nb = S * width + 4
    cache = randn(g, nb, 16, 576)
    bt = torch.randperm(nb, generator=g)[:S * width].view(S, width).to(torch.int32)
    for r, n in enumerate(lens):
        bt[r, -(-n // 16):] = -1
    starts = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    total = sum(lens)
    out = poisoned(total + 3, 576)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.latent_gather(out, cache, bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), starts, max(lens),
                      device_status=status)
    want = [cache[bt[r, :-(-n // 16)].long().cuda()].reshape(-1, 576)[:n] for r, n in enumerate(lens) if n]
    assert torch.equal(out[:total], torch.cat(want)) and int(status.item()) == 0
    assert torch.isnan(out[total:].float()).all()


def test_gather_reports():
    cache = torch.zeros(4, 16, 576, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    bt = torch.tensor([[0, 4], [1, -3]], **i32)
    out = poisoned(40, 576)
    status = torch.zeros(1, **i32)
    pkv.latent_gather(out, cache, bt, torch.tensor([20, 10], **i32), torch.tensor([0, 20], **i32), 32,
                      device_status=status)
    assert int(status.item()) == 7
    done = torch.isfinite(out.float()).all(-1).nonzero()[:, 0].tolist()
    assert done == list(range(16)) + list(range(20, 30))
    for lens, starts in (([33, 1], [0, 1]), ([20, 21], [0, 20]), ([1, -1], [0, 1]), ([1, 1], [0, -1])):
        status.zero_()
        pkv.latent_gather(out, cache, torch.zeros_like(bt), torch.tensor(lens, **i32), torch.tensor(starts, **i32),
                          32, device_status=status)
        assert int(status.item()) == 8, (lens, starts)


def test_writes_captured_and_replayed_on_another_stream():
    c = qk_case(1, 20, 4, 4, 64, 64)
    n = latent_case(1, 20, 4)
    cache, lat = poisoned(c["blocks"], 4, 2, 16, 64), poisoned(n["blocks"], 16, 576)
    out = poisoned(20, 4, 64)

    def step():
        pkv.qk_norm_rope_kv_write(out, cache, c["q"], c["k"], c["v"], c["wq"], c["wk"], 1e-6, c["table"], c["pos"],
                                  c["slots"])
        pkv.latent_kv_write(lat, n["c"], n["kr"], n["w"], 1e-6, n["table"], n["pos"], n["slots"],
                            query_rope_out=n["rows"][:, :, 512:], query_rope=n["q"][:, :, 128:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (out, cache, lat, n["rows"])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in (out, cache, lat):
        x.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip((out, cache, lat, n["rows"]), want):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_slots_past_four_gigabytes():
    blocks = 140_000                                              # 4.6 GB of K/V, 2.6 GB of latent rows
    c = qk_case(4, 9, 4, 4, 128, 128)
    n = latent_case(4, 9, 0)
    slots = torch.arange(blocks * 16 - 9, blocks * 16, device="cuda")
    cache = torch.empty(blocks, 4, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    out = poisoned(9, 4, 128)
    pkv.qk_norm_rope_kv_write(out, cache, c["q"], c["k"], c["v"], c["wq"], c["wk"], 1e-6, c["table"], c["pos"], slots)
    check_rounded(cache[-1, :, 0, 7:].transpose(0, 1), *norm_rotate(c["k"], c["wk"], 1e-6, c["table"], c["pos"], False),
                  "key")
    assert torch.equal(cache[-1, :, 1, 7:].transpose(0, 1).contiguous().view(torch.int16),
                       c["v"].contiguous().view(torch.int16))
    del cache
    lat = torch.empty(240_000, 16, 576, dtype=torch.bfloat16, device="cuda")           # 4.4 GB
    slots = torch.arange(240_000 * 16 - 9, 240_000 * 16, device="cuda")
    pkv.latent_kv_write(lat, n["c"], n["kr"], None, 0.0, n["table"], n["pos"], slots)
    assert torch.equal(lat[-1, 7:, :512].view(torch.int16), n["c"].contiguous().view(torch.int16))


def test_no_tokens():
    c = qk_case(4, 3, 4, 4, 64, 64)
    cache = poisoned(c["blocks"], 4, 2, 16, 64)
    e = slice(0, 0)
    pkv.qk_norm_rope_kv_write(c["q"][e], cache, c["q"][e], c["k"][e], c["v"][e], c["wq"], c["wk"], 1e-6, c["table"],
                              c["pos"][e], c["slots"][e])
    n = latent_case(4, 3, 2)
    lat = poisoned(n["blocks"], 16, 576)
    pkv.latent_kv_write(lat, n["c"][e], n["kr"][e], None, 0.0, n["table"], n["pos"][e], n["slots"][e])
    assert torch.isnan(cache.float()).all() and torch.isnan(lat.float()).all()


def test_refused_forms_on_the_gpu():
    c = qk_case(4, 3, 4, 4, 64, 64)
    cache = poisoned(c["blocks"], 4, 2, 16, 64)
    good = [c["q"].clone(), cache, c["q"], c["k"], c["v"], c["wq"], c["wk"], 1e-6, c["table"], c["pos"], c["slots"]]
    pkv.qk_norm_rope_kv_write(*good)
    for i, bad in ((0, good[0].float()), (1, cache.float()), (2, c["q"][:, :, ::2]), (3, c["k"][:2]), (5, c["wq"][:32]),
                   (8, c["table"].double()), (9, c["pos"].int()), (10, c["slots"].cpu()), (10, c["slots"][:2])):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            pkv.qk_norm_rope_kv_write(*args)
    with pytest.raises(pkv.PagedKVError):                          # the C call's own refusal: rotary_dim 24
        args = list(good)
        args[8] = torch.zeros(8, 24, device="cuda")
        pkv.qk_norm_rope_kv_write(*args)
    n = latent_case(4, 3, 2)
    lat = poisoned(n["blocks"], 16, 576)
    ok = dict(latent_cache=lat, latent=n["c"], key_rope=n["kr"], weight=n["w"], eps=1e-6, cos_sin=n["table"],
              positions=n["pos"], slot_mapping=n["slots"])
    pkv.latent_kv_write(**ok)
    for k, bad in (("latent", n["c"][:, :500]), ("latent_cache", lat[:, :, :512]), ("weight", n["w"].float()),
                   ("query_rope", n["q"][:, :, 128:]), ("cos_sin", n["table"][:, :32]), ("key_rope", n["kr"].t())):
        with pytest.raises(ValueError):
            pkv.latent_kv_write(**dict(ok, **{k: bad}))


def test_fp8_codes_beside_the_midpoints():
    """Codes whose quotients lie on a midpoint between two codes, or an ulp or two beside it, powers of two and ends
    of the range among the scales: bit for bit those of the rounded fp32 quotient."""
    g = torch.Generator().manual_seed(31)
    mid = [(2 * m + 1) * 2.0 ** e for e in range(-10, 5) for m in (0, 1, 4, 7, 8, 11, 13, 15)]
    scales = [1.0, 0.5, 2.0 ** -40, 2.0 ** 30, 3e-38, 1e-42, 2.9e38, 448.0, 1e-31, 2.0 ** -101, 1.5 * 2.0 ** 99]
    x0 = (torch.rand(40, generator=g) + 1).to(torch.bfloat16).float()
    for i, m in enumerate(mid):
        s = x0[i % 40] / m
        for _ in range(i % 4):
            s = torch.nextafter(s, torch.tensor(0.0 if i % 8 < 4 else 1e9))
        scales.append(s.item())
    T, h, d = 16, 4, 128
    dims = torch.arange(T * h * d)
    table = torch.zeros(1, 16, device="cuda")
    table[:, :8] = 1
    at, slots = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.arange(T, device="cuda")
    for s in scales:
        s32 = torch.tensor(s, dtype=torch.float32)
        s = s32.item()
        x = x0[dims % 40] * 2.0 ** (dims // 40 % 23 - 11)
        x = torch.where(dims % 3 == 0, (torch.randn(dims.numel(), generator=g) * s32 * 100), x)
        x[:8] = torch.tensor([0.0, -0.0, float("inf"), float("-inf"), float("nan"), 3e38, -3e38, 1e-38])
        x = torch.where(dims % 2 == 0, x, -x).to(torch.bfloat16).reshape(T, h, d).cuda()
        cache = torch.zeros(1, h, 2, 16, d, dtype=torch.uint8, device="cuda")
        q = torch.zeros(T, h, d, dtype=torch.bfloat16, device="cuda")
        pkv.qk_norm_rope_kv_write_fp8(q, cache, q, x, x, None, None, 0.0, table, at, slots, s, s)
        quotient = (x.cpu().float() / s32).clamp(-448, 448)          # fp32, then the nearest code
        want = quotient.to(torch.float8_e4m3fn).view(torch.uint8).transpose(0, 1)
        nan = torch.isnan(quotient).transpose(0, 1)
        # (a turn by no angle: x * 1 - y * 0 is NaN beside an infinity or a NaN, and +0 for -0)
        plain = torch.isfinite(x.float()).cpu() & (x.float().cpu() != 0)
        finite = (plain & plain.roll(-8, -1) & plain.roll(8, -1)).transpose(0, 1)
        got_k, got_v = cache[0, :, 0].cpu(), cache[0, :, 1].cpu()
        assert torch.equal(torch.where(nan, 0x7F, got_v & torch.where(nan, 0x7F, 0xFF)), torch.where(nan, 0x7F, want)), s
        assert torch.equal(got_k[finite], want[finite]), s
