"""The expanded form of latent attention against a plain 64-bit form, and a prompt through both forms.

The bound of an output: half a bf16 step of it; half a bf16 step of every weight; and the fp32 score's error (2^-20
of the sum of its absolute products) twice, as a relative error of the weights."""

import pytest
import torch

import paged_kv_cache_111_gb300 as pkv
from latent_ref import BF16_HALF_STEP, angles

pytestmark = pytest.mark.gpu


class Ragged:
    """reqs: [(query tokens, keys)]; rows between and behind the requests' are poison."""

    def __init__(self, seed, reqs, H, head_major=False, gap=0, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        self.reqs, self.H = reqs, H
        q, n = [a for a, _ in reqs], [b for _, b in reqs]
        self.T, self.K = sum(q) + 3, sum(n) + gap + 2

        def rows(*shape, used):
            x = (torch.randn(*shape, generator=g) * gain).to(torch.bfloat16)
            x[used:] = float("nan")
            return x.cuda()
        self.query = rows(self.T, H, 192, used=sum(q))
        up = rows(self.K, H, 256, used=sum(n))
        if head_major:
            up = up.transpose(0, 1).contiguous().transpose(0, 1)
        self.key, self.value = up[:, :, :128], up[:, :, 128:]
        self.rope = rows(self.K, 80, used=sum(n))[:, 16:]
        self.qsl = torch.tensor([0] + q).cumsum(0).to(torch.int32).cuda()
        self.ksl = torch.tensor([0] + n).cumsum(0).to(torch.int32).cuda()
        self.scale = 192 ** -0.5
        self.out = torch.full((self.T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.max_q, self.max_n = max(q), max(n)

    def run(self):
        pkv.latent_attn_expanded(self.out, self.query, self.key, self.rope, self.value, self.qsl, self.ksl,
                                 self.max_q, self.max_n, self.scale, device_status=self.status)
        return self.out

    def check(self, what="", skip=()):
        t = k = 0
        for r, (q, n) in enumerate(self.reqs):
            if r in skip:
                assert (self.out[t:t + q] == 7.0).all()
            elif q:
                qd = self.query[t:t + q].double()
                hid = torch.arange(n, device="cuda")[None] > torch.arange(n - q, n, device="cuda")[:, None]
                for h0 in range(0, self.H, 8):
                    sl = slice(h0, h0 + 8)
                    kd = torch.cat([self.key[k:k + n, sl], self.rope[k:k + n, None].expand(-1, self.key[0, sl].shape[0],
                                                                                          -1)], -1).double()
                    vd = self.value[k:k + n, sl].double()
                    s = torch.einsum("qhd,nhd->hqn", qd[:, sl], kd) * self.scale
                    w = torch.softmax(s.masked_fill(hid[None], float("-inf")), -1)
                    ref, mag = torch.einsum("hqn,nhd->qhd", w, vd), torch.einsum("hqn,nhd->qhd", w, vd.abs())
                    score = torch.einsum("qhd,nhd->qhn", qd[:, sl].abs(), kd.abs()).amax(-1) * abs(self.scale)
                    bound = BF16_HALF_STEP * ref.abs() + mag * (BF16_HALF_STEP * (1 + BF16_HALF_STEP)
                                                                + 2 * 2.0 ** -20 * score[..., None])
                    got = self.out[t:t + q, sl].double()
                    assert torch.isfinite(got).all(), f"{what} request {r}: not finite"
                    worst = ((got - ref).abs() - bound).max().item()
                    assert worst <= 0, f"{what} request {r} ({q}, {n}) heads {h0}: {worst:.3e} past the bound"
            t, k = t + q, k + n
        assert (self.out[t:] == 7.0).all(), "rows behind the last request changed"


@pytest.mark.parametrize("H,reqs", [
    (1, [(1, 1)]), (2, [(1, 300)]), (3, [(2, 2), (127, 127), (128, 128), (129, 129)]),
    (5, [(255, 300), (256, 256), (257, 700), (0, 10), (1, 128), (1, 129)]),
    (16, [(300, 300), (500, 1500)]), (1, [(1000, 1000)]), (9, [(513, 513), (64, 4000)]), (128, [(130, 200)])])
@pytest.mark.parametrize("head_major", [False, True])
def test_against_64_bits(H, reqs, head_major):
    b = Ragged(H * 31 + len(reqs), reqs, H, head_major)
    b.run()
    assert int(b.status.item()) == 0
    b.check()


def test_many_short_requests():
    g = torch.Generator().manual_seed(0)
    reqs = [(int(min(a, b)), int(max(a, b))) for a, b in torch.randint(1, 40, (500, 2), generator=g)]
    b = Ragged(5, reqs, 2)
    b.run()
    b.check()


@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_scales(scale):
    b = Ragged(2, [(200, 333)], 3)
    b.scale = scale
    b.run()
    b.check()


@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_grow_along_the_keys(sign):
    b = Ragged(3, [(300, 900)], 4, gain=0.25)
    b.rope[:900] = 0
    b.rope[:900, 5] = (torch.arange(900, dtype=torch.float64) / 16 * sign).to(torch.bfloat16).cuda()
    b.query[:300, :, 128 + 5] = 40.0
    b.run()
    b.check(what=f"sign {sign}")


def test_reports_and_leaves_bad_requests():
    b = Ragged(4, [(20, 40), (30, 60), (50, 50)], 4)
    b.max_n = 59
    b.run()
    assert int(b.status.item()) == 8
    b.check(skip=(1,))


def test_same_bits_again_and_in_a_graph():
    b = Ragged(6, [(400, 900), (3, 5)], 8)
    first = b.run().clone()
    b.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for _ in range(3):
        b.out.fill_(7.0)
        graph.replay()
        assert torch.equal(b.out, first)


def test_a_chunk_through_both_forms():
    """Latent write, then the chunk with its cached context attended in the latent space (absorbed projections) and
    over expanded keys and values: the same attention, each within the roundings of its own bf16 projections."""
    g = torch.Generator().manual_seed(9)
    H, ctx, q = 4, 70, 150
    n = ctx + q

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).cuda()
    pages = -(-n // 16)
    cache = torch.full((pages + 2, 16, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    bt = torch.randperm(pages + 2, generator=g)[:pages].to(torch.int32).cuda()[None].contiguous()
    pos = torch.arange(n).cuda()
    slots = bt[0, pos // 16].long() * 16 + pos % 16
    table = angles(64, n).cuda()
    w = randn(512)
    w_uk, w_uv = randn(H, 512, 128, scale=512 ** -0.5), randn(H, 512, 128, scale=512 ** -0.5)
    query = randn(q, H, 192)
    down = randn(n, 576)
    # earlier steps wrote the context, this one the chunk and its queries' rotated part
    pkv.latent_kv_write(cache, down[:ctx, :512], down[:ctx, 512:], w, 1e-6, table, pos[:ctx], slots[:ctx])
    rows = torch.empty(q, H, 576, dtype=torch.bfloat16, device="cuda")
    pkv.latent_kv_write(cache, down[ctx:, :512], down[ctx:, 512:], w, 1e-6, table, pos[ctx:], slots[ctx:],
                        query_rope_out=query[:, :, 128:], query_rope=query[:, :, 128:])
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, qsl, ksl = torch.tensor([n], **i32), torch.tensor([0, q], **i32), torch.tensor([0, n], **i32)
    scale = 192 ** -0.5
    # absorbed
    rows[:, :, :512] = torch.einsum("qhd,hcd->qhc", query[:, :, :128].float(), w_uk.float()).bfloat16()
    rows[:, :, 512:] = query[:, :, 128:]
    ws = torch.empty(pkv.latent_paged_attn_workspace_size(1, q, q, n, H), dtype=torch.uint8, device="cuda")
    lat = torch.empty(q, H, 512, dtype=torch.bfloat16, device="cuda")
    pkv.latent_paged_attn(lat, rows, cache, bt, lens, qsl, q, n, scale, ws)
    absorbed = torch.einsum("qhc,hcd->qhd", lat.double(), w_uv.double())
    # expanded
    flat = torch.empty(n, 576, dtype=torch.bfloat16, device="cuda")
    pkv.latent_gather(flat, cache, bt, lens, ksl, n)
    assert torch.equal(flat, cache.view(-1, 576)[slots])
    key = torch.einsum("nc,hcd->nhd", flat[:, :512].float(), w_uk.float()).bfloat16()
    value = torch.einsum("nc,hcd->nhd", flat[:, :512].float(), w_uv.float()).bfloat16()
    out = torch.empty(q, H, 128, dtype=torch.bfloat16, device="cuda")
    pkv.latent_attn_expanded(out, query, key, flat[:, 512:], value, qsl, ksl, q, n, scale)
    # exact, in 64 bits from the cached rows
    c = flat.double()
    kd = torch.cat([torch.einsum("nc,hcd->nhd", c[:, :512], w_uk.double()), c[:, None, 512:].expand(-1, H, -1)], -1)
    vd = torch.einsum("nc,hcd->nhd", c[:, :512], w_uv.double())
    s = torch.einsum("qhd,nhd->hqn", query.double(), kd) * scale
    hid = torch.arange(n, device="cuda")[None] > torch.arange(ctx, n, device="cuda")[:, None]
    p = torch.softmax(s.masked_fill(hid[None], float("-inf")), -1)
    ref, mag = torch.einsum("hqn,nhd->qhd", p, vd), torch.einsum("hqn,nhd->qhd", p, vd.abs())
    # A bf16 projection moves a score by at most half a step of each of its terms, so every weight by at most twice
    # that (numerator and sum); the values, the weights and the result round once each (absorbed: the latent result
    # rounds, and is projected after).
    terms = 2 * BF16_HALF_STEP * scale
    up = w_uv.double().abs()
    ds_e = (torch.einsum("qhd,nhd->qhn", query[..., :128].double().abs(), kd[..., :128].abs()).amax(-1) * terms)[..., None]
    bound_e = mag * (ds_e.exp() - 1 + 2 * BF16_HALF_STEP * 1.01) + BF16_HALF_STEP * ref.abs() * 1.02
    assert ((out.double() - ref).abs() <= bound_e).all()
    qa = torch.einsum("qhd,hcd->qhc", query[:, :, :128].double(), w_uk.double()).abs()
    ds_a = (torch.einsum("qhc,nc->qhn", qa, c[:, :512].abs()).amax(-1) * terms)[..., None]
    lat_mag = torch.einsum("hqn,nc->qhc", p, c[:, :512].abs())
    bound_a = torch.einsum("qhc,hcd->qhd", lat_mag * (ds_a.exp() - 1 + 2 * BF16_HALF_STEP * 1.02), up)
    assert ((absorbed - ref).abs() <= bound_a).all()


@pytest.mark.parametrize("seed", range(6))
def test_random_batches_twice(seed):
    g = torch.Generator().manual_seed(50 + seed)

    def draw(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=g))
    reqs = []
    for _ in range(draw(1, 12)):
        q = draw(0, (3, 130, 600)[draw(0, 2)])
        reqs.append((q, q + draw(0, (1, 140, 900)[draw(0, 2)])))
    if not any(q for q, _ in reqs):
        reqs.append((5, 9))
    b = Ragged(seed, reqs, (1, 2, 7, 16)[draw(0, 3)], head_major=bool(draw(0, 1)))
    first = b.run().clone()
    assert int(b.status.item()) == 0
    b.check()
    b.out.fill_(7.0)
    assert torch.equal(b.run(), first)


def test_heads_one_after_another():
    """Keys and values past 64 MB: the token tiles of a head run side by side."""
    b = Ragged(2, [(600, 4200), (300, 5000)], 16)
    assert b.K * b.H * 512 > 64 << 20
    b.run()
    b.check()


@pytest.mark.parametrize("S", [1, 3])
def test_a_call_without_a_query_keeps_the_order_around_it(S):
    """A cache write, then a call in which no request has a query, then attention over what was written: each may
    start before the one in front has ended, so the call in between has to outlast the write."""
    g = torch.Generator().manual_seed(3)
    n, H, Hkv, d = 8192, 8, 8, 128
    blocks = n // 16

    def randn(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()
    q, k, v = randn(n, H, d), randn(n, Hkv, d), randn(n, Hkv, d)
    table = angles(d, n).cuda()
    at = torch.arange(n, device="cuda")
    bt = torch.arange(blocks, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    slots = bt[0].long()[at // 16] * 16 + at % 16
    lens, qsl = torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda()
    ws = torch.empty(pkv.paged_attn_workspace_size(1, 1, 1, n, H, Hkv, d), dtype=torch.uint8, device="cuda")
    c = Ragged(4, [(1, 1)] * S, 2)
    c.qsl.zero_()

    def step(between):
        cache = torch.zeros(blocks, Hkv, 2, 16, d, dtype=torch.bfloat16, device="cuda")
        q_out, out = torch.empty_like(q), torch.empty(1, H, d, dtype=torch.bfloat16, device="cuda")
        last = q_out[n - 1:]
        torch.cuda.synchronize()
        pkv.qk_norm_rope_kv_write(q_out, cache, q, k, v, None, None, 1e-6, table, at, slots)
        if between:
            c.run()
        pkv.paged_attn(out, last, cache, bt, lens, qsl, 1, n, d ** -0.5, ws)
        pkv.paged_attn_combine(out, ws)
        torch.cuda.synchronize()
        return out
    want = step(False)
    for _ in range(20):
        assert torch.equal(step(True), want)
    assert (c.out == 7.0).all() and int(c.status) == 0


@pytest.mark.parametrize("H,reqs,scale", [
    (1, [(1, 5000)], None),                                 # one row, eight shares
    (3, [(300, 2001)], None),
    (2, [(7, 129), (256, 1100), (0, 40), (1, 1), (257, 257)], None),     # shares without a key
    (16, [(129, 640), (40, 41), (513, 513)], None),
    (40, [(2, 900), (128, 128)], None),
    (5, [(33, 1500), (1, 1030)], -0.2),
])
def test_keys_shared_out_over_a_cluster(H, reqs, scale):
    """Few rows and many keys: the shares' sums are joined, and the rows behind and between stay as they were."""
    c = Ragged(21, reqs, H, gain=2.0)
    if scale is not None:
        c.scale = scale
    first = c.run().clone()
    c.check(f"{H} heads {reqs}")
    assert int(c.status) == 0
    assert torch.equal(c.run(), first)


def test_scores_that_grow_from_share_to_share():
    """The shares' references lie hundreds of powers of two apart; a share whose weights vanish adds nothing."""
    for sign in (1.0, -1.0):
        c = Ragged(22, [(5, 2048)], 2)
        c.query[:5] = 1.0
        steps = sign * torch.arange(2048, device="cuda") / 2048 * 40
        c.key[:2048] = steps[:, None, None].to(torch.bfloat16)
        c.rope[:2048] = 0
        c.run()
        c.check(f"sign {sign}")


def test_a_bad_request_beside_a_shared_one():
    c = Ragged(23, [(4, 1600), (9, 700)], 2)
    c.qsl[1] = 2000                                         # past the bound, and the next one starts there
    before = c.out.clone()
    c.run()
    assert int(c.status) != 0
    assert torch.equal(c.out, before)


@pytest.mark.parametrize("H,q,n", [(2, 70, 150), (1, 600, 600), (16, 257, 900), (200, 130, 140), (1, 2, 5000), (3, 256, 256)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["value", "key", "rope"])
def test_infinities_and_nan_in_later_tokens_rows(H, q, n, what, where):
    """The chunk's own keys or values hold infinities or NaN: the tokens before them come out as without, bit for
    bit; those that see one are no numbers where NaN is seen."""
    c = Ragged(31, [(q, n), (1, 40)], H)
    want = c.run().clone()
    c.check()
    first = n - q + max(1, q // 3)                         # the first key with such a value
    if where == "rope":
        c.rope[first:n:7, 63] = what
    else:
        (c.value if where == "value" else c.key)[first:n:7, :, 77] = what
    c.out.fill_(7.0)
    c.run()
    seen = first - (n - q)                                 # query tokens before it
    assert torch.equal(c.out[:seen], want[:seen])
    assert torch.equal(c.out[q:], want[q:])
    if what != what:
        assert torch.isnan(c.out[seen:q, :, 77]).all()
    assert int(c.status) == 0
