"""The int8 cache's writes, reading back and block copies on the GPU, to the bit where they are defined to it."""

import numpy as np
import pytest
import torch

import int8_ref as ref
import latent_ref
import paged_kv_cache_111_gb300 as pkv

pytestmark = pytest.mark.gpu
BLOCK = 16


@pytest.fixture(autouse=True, scope="module")
def built():
    from paged_kv_cache_111_gb300 import _build
    _build.build()


def heads(T, hkv, d, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hkv, d, generator=g) * std
    x = x * torch.exp(torch.randn(1, hkv, 1, generator=g))            # heads of several magnitudes
    return x.bfloat16()


def slots_of(requests, blocks, seed):
    """Slots of [(first position, tokens)], each request's blocks in random places."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(blocks, generator=g).tolist()
    out = []
    for first, n in requests:
        own = [order.pop() for _ in range(-(-(first + n) // BLOCK))]
        out += [own[p // BLOCK] * BLOCK + p % BLOCK for p in range(first, first + n)]
    return out


def run_write(cache, scales, key, value, slots, status=0):
    dc, ds = cache.cuda(), scales.cuda()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.tensor(slots, dtype=torch.int64)
    pkv.kv_write_int8(dc, ds, key.cuda() if not key.is_cuda else key, value.cuda() if not value.is_cuda else value,
                      s.cuda(), device_status=word)
    c, sc = cache.numpy().copy(), scales.numpy().copy()
    ref.write(c, sc, key.float().cpu().numpy(), value.float().cpu().numpy(), np.array(slots, dtype=np.int64).reshape(-1))
    torch.cuda.synchronize()
    assert word.item() == status
    ref.same(dc, ds, c, sc)
    return dc, ds


PLACES = {
    "one": [(0, 1)],
    "one in a block": [(5, 1)],
    "last of a block": [(15, 1)],
    "decodes": [(p, 1) for p in (0, 1, 7, 15, 16, 31, 40, 3, 2, 9)],
    "a block": [(0, 16)],
    "across two": [(9, 12)],
    "pairs": [(14, 2), (15, 2), (16, 2), (3, 2)],
    "chunk": [(0, 200)],
    "chunk in a block": [(37, 131)],
    "mixed": [(20, 1), (33, 1), (7, 77), (0, 3)],
    "odd": [(1, 15), (2, 31), (11, 5), (4, 9)],
    # so many that a warp takes more heads than in the others
    "many": [(p % 40, 1) for p in range(1500)] + [(5, 700), (0, 333), (47, 1), (30, 3)],
}


@pytest.mark.parametrize("hkv,d", [(1, 64), (8, 128), (3, 128), (5, 64), (40, 128), (17, 64)])
@pytest.mark.parametrize("place", list(PLACES))
def test_write_to_the_bit(place, hkv, d):
    requests = PLACES[place]
    blocks = sum(-(-(a + n) // BLOCK) for a, n in requests) + 3
    slots = slots_of(requests, blocks, 7)
    T = len(slots)
    cache, scales = ref.new_cache(blocks, hkv, d, seed=hkv)
    run_write(cache, scales, heads(T, hkv, d, 1), heads(T, hkv, d, 2), slots)


@pytest.mark.parametrize("d", [64, 128])
def test_views_of_a_projection_and_padding(d):
    hq, hkv, blocks = 4, 2, 9
    slots = slots_of([(0, 20), (30, 1), (5, 1)], blocks, 3) + [-1, -5]
    g = torch.Generator().manual_seed(0)
    fused = torch.randn(len(slots), hq + 2 * hkv, d, generator=g).bfloat16().cuda()
    cache, scales = ref.new_cache(blocks, hkv, d)
    run_write(cache, scales, fused[:, hq:hq + hkv], fused[:, hq + hkv:], slots)
    # padding in the middle of a batch (each request padded to three tokens), one token of each alone
    slots = [16 * 3 + 2, -1, -1, 16 * 5 + 9, 16 * 5 + 10, -1, 7, 8, 9]
    run_write(cache, scales, fused[:9, hq:hq + hkv], fused[:9, hq + hkv:], slots)


def test_order_and_repeats_within_a_block():
    hkv, d, blocks = 2, 128, 4
    cache, scales = ref.new_cache(blocks, hkv, d)
    for slots in ([35, 33, 47, 32], [40, 39, 38], [20, 20], [16, 17, 16, 18, 17], [5] * 16, list(range(47, 31, -1))):
        run_write(cache, scales, heads(len(slots), hkv, d, 4), heads(len(slots), hkv, d, 5), slots)


def test_more_than_sixteen_of_one_block():
    hkv, d = 2, 64
    cache, scales = ref.new_cache(4, hkv, d)
    slots = list(range(16, 32)) + [18, 19] + [40]
    run_write(cache, scales, heads(19, hkv, d, 4), heads(19, hkv, d, 5), slots, status=7)


def test_slots_past_the_cache():
    hkv, d = 3, 128
    cache, scales = ref.new_cache(4, hkv, d)
    slots = [64, 65, 17, 18, 1 << 40, 63, 35]
    run_write(cache, scales, heads(7, hkv, d, 4), heads(7, hkv, d, 5), slots, status=7)


@pytest.mark.parametrize("what", ["zeros", "tiny", "subnormal", "huge", "one large", "nan", "inf"])
@pytest.mark.parametrize("start", [0, 6])
def test_values(what, start):
    hkv, d, T = 3, 64, 21
    cache, scales = ref.new_cache(6, hkv, d)
    key, value = heads(T, hkv, d, 1), heads(T, hkv, d, 2)
    for x in (key, value):
        if what == "zeros":
            x.zero_()
        elif what == "tiny":
            x.mul_(2.0 ** -64)
        elif what == "subnormal":
            x.mul_(2.0 ** -130)
        elif what == "huge":
            x.copy_(x.sign() * 3.3e38)
        elif what == "one large":
            x[4, 1, 3] = 3e30
        else:
            x[4, 1, 3] = float(what)
            x[9, 2, 0] = -float(what)
    slots = slots_of([(start, T)], 6, 1)
    dc, ds = run_write(cache, scales, key, value, slots)
    if what in ("nan", "inf"):
        # the block stays without a scale while it is filled, and has one when it starts anew
        assert torch.isnan(ds).any()
        again = slots[:1]
        k2, v2 = heads(1, hkv, d, 3), heads(1, hkv, d, 4)
        run_write(dc.cpu(), ds.cpu(), k2, v2, [again[0] // 16 * 16 + 15])
        dc, ds = run_write(dc.cpu(), ds.cpu(), k2, v2, [again[0] // 16 * 16])
        assert torch.isfinite(ds[again[0] // 16]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_block_filled_one_token_at_a_time(d):
    """Codes to the bit at every step, and the growths' error: half a step of the final scale for each and one more."""
    hkv, T = 4, 32
    key, value = heads(T, hkv, d, 11), heads(T, hkv, d, 12)
    key *= torch.linspace(0.1, 3.0, T)[:, None, None]                  # a scale that grows often
    cache, scales = ref.new_cache(3, hkv, d)
    dc, ds = cache, scales
    growths = torch.zeros(hkv, 2)
    for t in range(T):
        before = ds.cpu()[1 + t // BLOCK]
        dc, ds = run_write(dc.cpu(), ds.cpu(), key[t:t + 1], value[t:t + 1], [BLOCK + t])
        after = ds.cpu()[1 + t // BLOCK]
        growths = torch.zeros(hkv, 2) if t % BLOCK == 0 else growths + (after > before)
        if t % BLOCK == BLOCK - 1:
            x = ref.values(dc.cpu(), ds.cpu())[1 + t // BLOCK]         # [Hkv, 2, 16, d]
            want = torch.stack([key[t - 15:t + 1], value[t - 15:t + 1]], 2).permute(1, 2, 0, 3).double()
            step = after.double()[..., None, None]
            # (a quotient near 127 in fp32: 2^-17 of a step at most, at each of the roundings)
            assert ((x - want).abs() <= step * ((growths[..., None, None] + 1) * (0.5 + 2.0 ** -16))).all()
            assert growths.max() >= 3


def test_far_blocks():
    """Codes past 2^32 bytes."""
    hkv, d, blocks = 40, 128, 30000
    cache = torch.zeros(blocks, hkv, 2, BLOCK, d, dtype=torch.int8, device="cuda")
    scales = torch.ones(blocks, hkv, 2, device="cuda") * 0.001
    assert cache.numel() > 1 << 32
    slots = list(range(29999 * 16, 29999 * 16 + 16)) + [28000 * 16 + 3] + list(range(27000 * 16 + 2, 27000 * 16 + 5))
    key, value = heads(20, hkv, d, 1), heads(20, hkv, d, 2)
    pkv.kv_write_int8(cache, scales, key.cuda(), value.cuda(), torch.tensor(slots, device="cuda"))
    at = [29999, 28000, 27000]
    c, s = np.zeros((3, hkv, 2, BLOCK, d), np.int8), np.full((3, hkv, 2), 0.001, np.float32)
    where = {b: i for i, b in enumerate(at)}
    ref.write(c, s, key.float().numpy(), value.float().numpy(),
              np.array([where[x // 16] * 16 + x % 16 for x in slots], dtype=np.int64))
    ref.same(cache[at], scales[at], c, s)
    assert (cache != 0).any(-1).any(-1).any(-1).any(-1).nonzero().flatten().tolist() == sorted(at)
    mapping = torch.tensor([[29999, 5], [28000, 29998]], device="cuda")
    pkv.copy_blocks_int8(cache, scales, mapping)
    assert torch.equal(cache[[5, 29998]], cache[[29999, 28000]]) and torch.equal(scales[[5, 29998]], scales[[29999, 28000]])
    out = [torch.zeros(20, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.tensor([[29999, 27000]], dtype=torch.int32, device="cuda")
    pkv.kv_gather_int8(*out, cache, scales, table, torch.tensor([20], dtype=torch.int32, device="cuda"),
                       torch.zeros(1, dtype=torch.int32, device="cuda"), 20)
    for got, want in zip(out, ref.rows_of(cache, scales, table[0], 20)):
        assert torch.equal(got, want.float().bfloat16())


# ---- behind norm and rotation -----------------------------------------------------------------------------------

def norm_case(hq, hkv, d, rot, inter, requests, normed, seed=0):
    blocks = sum(-(-(a + n) // BLOCK) for a, n in requests) + 2
    slots = slots_of(requests, blocks, seed + 1)
    T = len(slots)
    g = torch.Generator().manual_seed(seed)
    fused = torch.randn(T, hq + 2 * hkv, d, generator=g).bfloat16()
    weights = [(torch.randn(d, generator=g) * 0.3 + 1).bfloat16() if normed else None for _ in range(2)]
    positions = torch.randint(0, 500, (T,), generator=g)
    return blocks, slots, fused, weights, positions


@pytest.mark.parametrize("hq,hkv,d,rot,inter", [(8, 8, 64, 64, False), (6, 2, 128, 128, False), (5, 5, 128, 64, True),
                                                (32, 4, 64, 16, True), (40, 40, 128, 32, False)])
@pytest.mark.parametrize("place", ["decodes", "chunk in a block", "mixed"])
@pytest.mark.parametrize("normed", [True, False])
def test_norm_rope_write(hq, hkv, d, rot, inter, place, normed):
    blocks, slots, fused, weights, positions = norm_case(hq, hkv, d, rot, inter, PLACES[place], normed)
    T = len(slots)
    cache, scales = ref.new_cache(blocks, hkv, d)
    table = latent_ref.angles(rot, 500)
    dev = fused.cuda()
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    dc, ds = cache.cuda(), scales.cuda()
    out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    wq, wk = (None if w is None else w.cuda() for w in weights)
    pkv.qk_norm_rope_kv_write_int8(out, dc, ds, q, k, v, wq, wk, 1e-6, table.cuda(), positions.cuda(),
                                   torch.tensor(slots).cuda(), interleaved=inter)
    want, mag = latent_ref.norm_rotate(fused[:, :hq], weights[0], 1e-6, table, positions, inter)
    latent_ref.check_rounded(out.cpu(), want, mag, "query")
    key, kmag = latent_ref.norm_rotate(fused[:, hq:hq + hkv], weights[1], 1e-6, table, positions, inter)
    # the values' side to the bit
    c, s = cache.numpy().copy(), scales.numpy().copy()
    ref.write(c, s, key.float().numpy(), fused[:, hq + hkv:].float().numpy(), np.array(slots, dtype=np.int64))
    got_c, got_s = dc.cpu().numpy(), ds.cpu().numpy()
    assert np.array_equal(got_s[:, :, 1], s[:, :, 1]) and np.array_equal(got_c[:, :, 1], c[:, :, 1])
    # the keys': scales within the fp32 slack of the largest key, new rows within half a step and the slack
    largest = float(kmag.max())
    assert np.abs(got_s[:, :, 0] - s[:, :, 0]).max() <= (latent_ref.FP32_SLACK + 2.0 ** -22) * largest / 127
    x = ref.values(dc.cpu(), ds.cpu())
    st = torch.tensor(slots)
    got = x[st // BLOCK, :, 0, st % BLOCK]                             # [T, Hkv, d]
    step = ds.cpu().double()[st // BLOCK, :, 0][..., None]
    assert ((got - key).abs() <= step * (0.5 + 2.0 ** -16) + latent_ref.FP32_SLACK * kmag).all()
    # older rows: as the model requantises them but for a step where a quotient is near a border
    assert np.abs(got_c[:, :, 0].astype(int) - c[:, :, 0].astype(int)).max() <= 1
    assert (got_c[:, :, 0] != c[:, :, 0]).mean() < 1e-3


@pytest.mark.parametrize("hq,hkv,d,rot,inter", [(8, 8, 64, 64, False), (6, 2, 128, 128, False), (17, 17, 128, 64, True),
                                                (20, 4, 64, 16, True)])
def test_norm_rope_write_of_many_tokens(hq, hkv, d, rot, inter):
    test_norm_rope_write(hq, hkv, d, rot, inter, "many", True)


def test_norm_rope_in_place_padding_and_positions():
    hq = hkv = 2
    d = rot = 64
    slots = [16, 17, -1, 50, 51, 35]
    positions = torch.tensor([0, 5, 7, 900, 8, -1])                    # the 4th and 6th are outside the table
    g = torch.Generator().manual_seed(0)
    fused = torch.randn(6, 6, d, generator=g).bfloat16()
    table = latent_ref.angles(rot, 500)
    cache, scales = ref.new_cache(4, hkv, d)
    dc, ds, dev = cache.cuda(), scales.cuda(), fused.cuda()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = dev[:, :2]
    pkv.qk_norm_rope_kv_write_int8(q, dc, ds, q, dev[:, 2:4], dev[:, 4:], None, None, 0.0, table.cuda(),
                                   positions.cuda(), torch.tensor(slots).cuda(), device_status=word)
    assert word.item() == 7
    ok = [0, 1, 2, 4]
    want, mag = latent_ref.norm_rotate(fused[ok][:, :2], None, 0.0, table, positions[ok], False)
    latent_ref.check_rounded(q.cpu()[ok], want, mag, "query")
    assert torch.equal(q.cpu()[[3, 5]], fused[[3, 5]][:, :2])          # skipped
    c, s = cache.numpy().copy(), scales.numpy().copy()
    ref.write(c, s, fused[:, 4:].float().numpy(), fused[:, 4:].float().numpy(), np.array(slots), ignored=(3, 5))
    assert np.array_equal(ds.cpu().numpy()[:, :, 1], s[:, :, 1]) and np.array_equal(dc.cpu().numpy()[:, :, 1], c[:, :, 1])
    assert torch.equal(dc.cpu()[[0, 2]], cache[[0, 2]])                # the token outside the table writes nothing
    c, s = cache.numpy().copy(), scales.numpy().copy()
    # a token outside the table counts for no scale
    dc, ds = cache.cuda(), scales.cuda()
    big = fused.clone()
    big[1, 4:] = 1e6
    pos = torch.tensor([3, 900, 4])
    dev = big[:3].cuda()
    pkv.qk_norm_rope_kv_write_int8(dev[:, :2], dc, ds, dev[:, :2], dev[:, 2:4], dev[:, 4:], None, None, 0.0,
                                   table.cuda(), pos.cuda(), torch.tensor([32, 33, 34]).cuda())
    ref.write(c, s, big[:3, 4:].float().numpy(), big[:3, 4:].float().numpy(), np.array([32, 33, 34]), ignored=(1,))
    assert np.array_equal(ds.cpu().numpy()[:, :, 1], s[:, :, 1]) and np.array_equal(dc.cpu().numpy()[:, :, 1], c[:, :, 1])


# ---- reading back, copies ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("hkv,d", [(1, 64), (8, 128), (3, 64), (40, 128)])
@pytest.mark.parametrize("lens", [[1], [16, 17, 15], [0, 33, 0, 700], [5] * 70])
def test_gather(hkv, d, lens):
    S, width = len(lens), max(-(-n // BLOCK) for n in lens) + 1
    blocks = sum(-(-n // BLOCK) for n in lens) + 2
    cache, scales = (x.cuda() for x in ref.new_cache(blocks, hkv, d))
    scales[-1] = float("nan")
    g = torch.Generator().manual_seed(0)
    order = torch.randperm(blocks - 1, generator=g).tolist()
    tables = torch.full((S, width), -1, dtype=torch.int32)
    for r, n in enumerate(lens):
        for b in range(-(-n // BLOCK)):
            tables[r, b] = order.pop()
    tables = tables.cuda()
    starts = torch.tensor([2] + lens).cumsum(0).to(torch.int32).cuda()             # rows 0, 1 and the last belong to nobody
    rows = sum(lens) + 3
    out = [torch.full((rows, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.kv_gather_int8(*out, cache, scales, tables, torch.tensor(lens, dtype=torch.int32).cuda(), starts,
                       max(lens), device_status=word)
    at = 2
    for r, n in enumerate(lens):
        for got, want in zip(out, ref.rows_of(cache, scales, tables[r], n) if n else ()):
            assert torch.equal(got[at:at + n], want.float().bfloat16())
        at += n
    for got in out:
        assert (got[:2] == 7).all() and (got[at:] == 7).all()
    assert word.item() == 0


def test_gather_of_no_numbers_and_bad_requests():
    hkv, d = 2, 64
    cache, scales = (x.cuda() for x in ref.new_cache(4, hkv, d))
    scales[1, 0, 1] = float("nan")
    scales[2, 1, 0] = 0.0
    tables = torch.tensor([[0, 1], [2, 9], [3, 0], [3, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 20, 33, 4], dtype=torch.int32, device="cuda")          # the second's page, the third's length
    starts = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device="cuda")
    out = [torch.full((64, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.kv_gather_int8(*out, cache, scales, tables, lens, starts, 32, device_status=word)
    assert word.item() in (7, 8)
    k, v = out
    assert torch.isnan(v[16:20, 0]).all() and torch.isfinite(v[:16].float()).all() and torch.isfinite(k[:20].float()).all()
    assert torch.isfinite(v[16:20, 1].float()).all()
    assert (k[20:36, 1] == 0).all() and (k[36:40] == 7).all() and (k[40:60] == 7).all()
    assert torch.equal(k[60:], ref.rows_of(cache, scales, tables[3], 4)[0].float().bfloat16())
    # a request whose rows end behind the output
    word.zero_()
    pkv.kv_gather_int8(k[:10], v[:10], cache, scales, tables[:1], lens[:1], starts, 32, device_status=word)
    assert word.item() == 8


@pytest.mark.parametrize("hkv,d", [(1, 64), (8, 128), (3, 64), (40, 128)])
def test_copy(hkv, d):
    blocks = 30
    cache, scales = (x.cuda() for x in ref.new_cache(blocks, hkv, d))
    want_c, want_s = cache.clone(), scales.clone()
    pairs = [(0, 29), (5, 6), (5, 7), (28, 1), (9, 9)]
    for a, b in pairs:
        want_c[b], want_s[b] = cache[a], scales[a]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.copy_blocks_int8(cache, scales, torch.tensor(pairs, device="cuda"), device_status=word)
    assert torch.equal(cache, want_c) and torch.equal(scales, want_s) and word.item() == 0
    pkv.copy_blocks_int8(cache, scales, torch.tensor([(2, 30), (-1, 3), (4, 10)], device="cuda"), device_status=word)
    want_c[10], want_s[10] = want_c[4].clone(), want_s[4].clone()
    assert torch.equal(cache, want_c) and torch.equal(scales, want_s) and word.item() == 7


# ---- one after the other, with nothing waited for between ---------------------------------------------------------

@pytest.mark.parametrize("hkv,d,tokens", [(8, 128, 1), (3, 64, 1), (8, 128, 5), (40, 128, 1)])
def test_writes_and_read_backs_in_a_row(hkv, d, tokens):
    # each read-back sees the codes and scales of the write before it, while the scales of neighbouring heads (one
    # stretch of memory) grow under other warps
    steps, S = 32, 64
    blocks = S * -(-steps * tokens // BLOCK)
    order = torch.randperm(blocks, generator=torch.Generator().manual_seed(3)).reshape(S, -1)
    cache, scales = ref.new_cache(blocks, hkv, d)
    dc, ds = cache.cuda(), scales.cuda()
    table = order.int().cuda()
    data, slots, lens = [], [], []
    for i in range(steps):
        at = torch.arange(i * tokens, (i + 1) * tokens)
        slots.append((order[:, at // BLOCK] * BLOCK + at % BLOCK).flatten())
        data.append([heads(S * tokens, hkv, d, 2 * i + k, std=1.5 ** i) for k in range(2)])
        lens.append((i + 1) * tokens)
    on = [(k.cuda(), v.cuda(), s.cuda(), torch.full((S,), n, dtype=torch.int32, device="cuda"),
           torch.arange(0, S * n, n, dtype=torch.int32, device="cuda")) for (k, v), s, n in zip(data, slots, lens)]
    outs = [[torch.empty(S * n, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for n in lens]
    torch.cuda.synchronize()
    for (k, v, s, n, start), out in zip(on, outs):
        pkv.kv_write_int8(dc, ds, k, v, s)
        pkv.kv_gather_int8(*out, dc, ds, table, n, start, int(out[0].shape[0] // S))
    torch.cuda.synchronize()
    c, sc = cache.numpy().copy(), scales.numpy().copy()
    for i, ((k, v), s, n) in enumerate(zip(data, slots, lens)):
        ref.write(c, sc, k.float().numpy(), v.float().numpy(), s.numpy())
        if i % 5 and i != steps - 1:
            continue
        for r in range(0, S, 7):
            for got, want in zip(outs[i], ref.rows_of(torch.from_numpy(c), torch.from_numpy(sc), order[r], n)):
                assert torch.equal(got[r * n:(r + 1) * n].cpu(), want.float().bfloat16()), (i, r)
