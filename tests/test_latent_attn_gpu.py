"""Attention over the latent cache in the latent space, against a plain 64-bit form.

The bound of an output: half a bf16 step of it; half a bf16 step of every weight (2^-8 of the sum of weight times
|value|); and the fp32 score's error (2^-20 of the sum of its absolute products, four steps of a 576-term sum in the
tensor core's fp32) twice, as a relative error of the weights."""

import pytest
import torch

import paged_kv_cache_111_gb300 as pkv
from latent_ref import BF16_HALF_STEP, attention

pytestmark = pytest.mark.gpu

D, W = 576, 512


class Batch:
    """reqs: [(query tokens, keys)]; unwritten slots, and table entries past a request's pages, are poison."""

    def __init__(self, seed, reqs, H, extra_rows=0, gain=1.0, stride_pad=0):
        g = torch.Generator().manual_seed(seed)
        self.reqs, self.H = reqs, H
        q, n = [a for a, _ in reqs], [b for _, b in reqs]
        self.T = sum(q) + extra_rows
        pages = [-(-x // 16) for x in n]
        nb = sum(pages) + 3
        width = max(1, max(pages)) + 1
        order = torch.randperm(nb, generator=g)
        self.bt = torch.full((len(reqs), width), 1 << 29, dtype=torch.int32)
        self.cache = torch.full((nb, 16, D), float("nan"), dtype=torch.bfloat16)
        self.rows, at = [], 0
        for r, x in enumerate(n):
            ids = order[at:at + pages[r]]
            at += pages[r]
            self.bt[r, :pages[r]] = ids.to(torch.int32)
            rows = (torch.randn(x, D, generator=g) * gain).to(torch.bfloat16)
            self.rows.append(rows.double())
            page, off = ids[torch.arange(x) // 16], torch.arange(x) % 16
            self.cache[page, off] = rows
        store = torch.randn(self.T, H * D + stride_pad, generator=g).to(torch.bfloat16).cuda()
        self.query = store[:, :H * D].view(self.T, H, D) if not stride_pad else store.as_strided(
            (self.T, H, D), (H * D + stride_pad, D, 1))
        self.cache, self.bt = self.cache.cuda(), self.bt.cuda()
        self.lens = torch.tensor(n, dtype=torch.int32).cuda()
        self.qsl = torch.tensor([0] + q).cumsum(0).to(torch.int32).cuda()
        self.max_q, self.max_n = max(q), max(n)
        self.scale = 192 ** -0.5
        self.ws = torch.full((pkv.latent_paged_attn_workspace_size(len(reqs), self.T, self.max_q, self.max_n, H),),
                             0xFF, dtype=torch.uint8, device="cuda")
        self.out = torch.full((self.T, H, W), 7.0, dtype=torch.bfloat16, device="cuda")

    def run(self, **kw):
        pkv.latent_paged_attn(self.out, self.query, self.cache, self.bt, self.lens, self.qsl, self.max_q, self.max_n,
                              self.scale, self.ws, **kw)
        return self.out

    def check(self, out=None, what=""):
        out = self.out if out is None else out
        t = 0
        for r, (q, n) in enumerate(self.reqs):
            if q == 0:
                continue
            query, rows = self.query[t:t + q].double(), self.rows[r].cuda()
            lim = torch.arange(n - q + 1, n + 1, device="cuda")
            ref, mag = attention(query, rows, lim, self.scale, W)
            score = (torch.einsum("qhd,nd->qhn", query.abs(), rows.abs()).amax(-1) * abs(self.scale))[..., None]
            bound = BF16_HALF_STEP * ref.abs() + mag * (BF16_HALF_STEP * (1 + BF16_HALF_STEP) + 2 * 2.0 ** -20 * score)
            got = out[t:t + q].double()
            assert torch.isfinite(got).all(), f"{what} request {r}: not finite"
            worst = ((got - ref).abs() - bound).max().item()
            assert worst <= 0, f"{what} request {r} ({q}, {n}): {worst:.3e} past the bound"
            t += q
        assert (out[t:] == 7.0).all(), "rows behind the last request changed"


@pytest.mark.parametrize("H", [1, 2, 5, 16, 33, 64, 65, 80, 128, 200])
def test_decode_lengths(H):
    b = Batch(H, [(1, n) for n in (1, 2, 15, 16, 17, 63, 64, 65, 128, 300, 1000)], H, extra_rows=2)
    b.run()
    assert pkv.workspace_status(b.ws) == 0
    b.check()


@pytest.mark.parametrize("H,reqs", [
    (16, [(2, 2), (3, 70), (4, 4), (5, 64), (1, 1), (0, 40), (7, 129)]),
    (1, [(64, 64), (65, 200), (100, 100)]),
    (3, [(33, 90), (1, 17), (16, 16)]),
    (5, [(9, 9), (130, 131)]),
    (20, [(40, 333), (3, 3)]),
    (40, [(17, 64), (2, 1000)]),
    (128, [(5, 70), (1, 600), (33, 33)]),
])
def test_chunks_and_several_tokens(H, reqs):
    b = Batch(H + len(reqs), reqs, H, extra_rows=1, stride_pad=64)
    b.run()
    assert pkv.workspace_status(b.ws) == 0
    b.check()


@pytest.mark.parametrize("H,n", [(16, 20000), (128, 9001)])
def test_one_long_request_is_split_over_every_sm(H, n):
    b = Batch(n, [(1, n)], H)
    b.run()
    b.check()


def test_many_requests():
    """More requests than the kernel has threads to scan them in one go, empty ones among them."""
    g = torch.Generator().manual_seed(0)
    reqs = [(int(x > 2), int(x)) for x in torch.randint(1, 90, (700,), generator=g)]
    b = Batch(1, reqs, 16)
    b.run()
    assert pkv.workspace_status(b.ws) == 0
    b.check()


def test_long_prompt_chunk():
    b = Batch(4, [(1, 700), (1, 1500), (600, 1100)], 16)
    b.run()
    b.check()


@pytest.mark.parametrize("H", [4, 128])
def test_scores_that_grow_along_the_keys(H):
    """Scores rising by hundreds (in the log2 domain) from one key tile to the next move the running maximum past
    its bound again and again; falling ones underflow."""
    for sign in (1, -1):
        b = Batch(8, [(1, 400), (3, 500)], H)
        for r, (q, n) in enumerate(b.reqs):
            ramp = torch.arange(n, dtype=torch.float64) / 16 * sign
            rows = b.rows[r]
            rows[:, W:] = 0
            rows[:, W] = ramp.to(torch.bfloat16).double()
            rows[:, :W] = (rows[:, :W] * 0.25).to(torch.bfloat16).double()
            ids = b.bt[r, torch.arange(n) // 16].long()
            b.cache[ids, (torch.arange(n) % 16).cuda()] = rows.to(torch.bfloat16).cuda()
        b.query[:, :, W] = 40.0
        b.run()
        assert pkv.workspace_status(b.ws) == 0
        b.check(what=f"sign {sign}")


@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_scales(scale):
    b = Batch(3, [(1, 100), (6, 66)], 16)
    b.scale = scale
    b.run()
    b.check()


def test_values_far_apart():
    b = Batch(6, [(1, 200), (2, 130)], 8, gain=1.0)
    for r in range(2):
        b.rows[r][::3, :W] *= 2.0 ** 20
        n = b.reqs[r][1]
        ids = b.bt[r, torch.arange(n) // 16].long()
        b.cache[ids, (torch.arange(n) % 16).cuda()] = b.rows[r].to(torch.bfloat16).cuda()
    b.query[:, :, :W] *= 2.0 ** -20
    b.run()
    b.check()


def test_reports_and_leaves_bad_requests():
    b = Batch(2, [(1, 40), (1, 50), (1, 20)], 16)
    b.bt[0, 1] = -1
    b.run()
    assert pkv.workspace_status(b.ws) == 7
    b = Batch(2, [(1, 40), (1, 50), (2, 20)], 16)
    lens = b.lens.clone()
    b.lens[1], b.lens[2] = 51, 1                                # past the bound; fewer keys than queries
    b.run()
    assert pkv.workspace_status(b.ws) == 8
    assert (b.out[1:] == 7.0).all() and not (b.out[0] == 7.0).any()
    b.lens.copy_(lens)
    b.run()                                                     # the status starts afresh
    assert pkv.workspace_status(b.ws) == 0
    b.check()


def test_nothing_to_do():
    b = Batch(1, [(0, 30), (0, 1)], 4, extra_rows=2)
    b.run()
    assert pkv.workspace_status(b.ws) == 0
    assert (b.out == 7.0).all()


def test_repeated_calls_give_the_same_bits():
    b = Batch(12, [(1, n) for n in (900, 33, 1, 4000, 128, 77)] + [(70, 300)], 32)
    first = b.run().clone()
    b.check()
    for _ in range(5):
        b.out.fill_(7.0)
        assert torch.equal(b.run(), first)


def test_write_then_attend_captured_in_a_graph():
    """A decode step through the latent write and the attention, eager and replayed with new inputs."""
    b = Batch(20, [(1, 100), (1, 17), (1, 65)], 16)
    g = torch.Generator().manual_seed(1)
    new = torch.randn(3, D, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(W, generator=g).to(torch.bfloat16).cuda()
    from latent_ref import angles
    table = angles(64, 128).cuda()
    pos = (b.lens - 1).long()
    slots = b.bt[torch.arange(3), pos // 16].long() * 16 + pos % 16
    qr = torch.randn(3, 16, 64, generator=g).to(torch.bfloat16).cuda()

    def step():
        pkv.latent_kv_write(b.cache, new[:, :W], new[:, W:], w, 1e-6, table, pos, slots,
                            query_rope_out=b.query[:, :, W:], query_rope=qr)
        b.run()

    def refresh():
        for r in range(3):
            b.rows[r][-1] = b.cache.view(-1, D)[slots[r]].double().cpu()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    refresh()
    b.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    new.copy_(torch.randn(3, D, generator=g).to(torch.bfloat16))
    b.query[:, :, :W] = torch.randn(3, 16, W, generator=g).to(torch.bfloat16).cuda()
    for _ in range(2):
        b.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        refresh()
        b.check()


@pytest.mark.parametrize("seed", range(8))
def test_random_batches_twice(seed):
    """Batches drawn over the range of heads, lengths and chunks: within the bound, and the same bits again from a
    workspace full of something else."""
    g = torch.Generator().manual_seed(100 + seed)

    def draw(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=g))
    H = (1, 3, 8, 16, 24, 32, 64, 72, 128)[draw(0, 8)]
    reqs = []
    for _ in range(draw(1, 40)):
        n = draw(1, (80, 700, 2500)[draw(0, 2)])
        q = min(n, (1, 1, 1, draw(1, 5), draw(1, 90))[draw(0, 4)]) if H <= 32 else min(n, (1, 1, draw(1, 3))[draw(0, 2)])
        reqs.append((q, n))
    b = Batch(seed, reqs, H, extra_rows=draw(0, 3))
    first = b.run().clone()
    assert pkv.workspace_status(b.ws) == 0
    b.check()
    b.ws.random_(0, 256)
    b.out.fill_(7.0)
    assert torch.equal(b.run(), first)
    assert pkv.workspace_status(b.ws) == 0


def test_pages_past_four_gigabytes():
    b = Batch(5, [(1, 300), (1, 17)], 16)
    nb, used = 260_000, b.cache.shape[0]                       # 4.8 GB
    far = torch.empty(nb, 16, D, dtype=torch.bfloat16, device="cuda")
    far[nb - used:] = b.cache
    b.cache = far
    b.bt = torch.where(b.bt < used, b.bt + (nb - used), b.bt)
    b.run()
    assert pkv.workspace_status(b.ws) == 0
    b.check()
    # the same rows gathered
    starts = torch.tensor([0, 300, 317], dtype=torch.int32, device="cuda")
    out = torch.empty(317, D, dtype=torch.bfloat16, device="cuda")
    pkv.latent_gather(out, b.cache, b.bt, b.lens, starts, 300)
    assert torch.equal(out.double().cpu(), torch.cat(b.rows))


def test_no_tokens_at_all():
    b = Batch(1, [(1, 30)], 4)
    empty = torch.zeros(2, dtype=torch.int32, device="cuda")
    pkv.latent_paged_attn(b.out[:0], b.query[:0], b.cache, b.bt, b.lens, empty, 1, 30, 1.0, b.ws)
    assert pkv.workspace_status(b.ws) == 0
    assert (b.out == 7.0).all()


def test_two_streams_with_a_workspace_each():
    bs = [Batch(30 + i, [(1, 900), (1, 64), (40, 200)], 16) for i in range(2)]
    want = []
    for b in bs:
        want.append(b.run().clone())
        b.check()
        b.out.fill_(7.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(10):
        for b, s in zip(bs, streams):
            b.run(stream=s)
    torch.cuda.synchronize()
    for b, w in zip(bs, want):
        assert torch.equal(b.out, w)


@pytest.mark.parametrize("H,q,n", [(16, 70, 150), (1, 64, 64), (5, 100, 1100), (16, 4, 64), (64, 3, 130), (128, 2, 9)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_infinities_and_nan_in_later_tokens_rows(H, q, n, what):
    """Rows of the chunk's own tokens hold infinities or NaN, in a latent dim or in a rotated one: the tokens before
    them come out as without, bit for bit; those that see one are no numbers where NaN is seen."""
    b = Batch(31, [(q, n), (1, 40)], H)
    want = b.run().clone()
    b.check()
    first = n - q + max(1, q // 3)                         # the first key with such a value
    for i, j in enumerate(range(first, n, 3)):
        page = b.bt[0, j // 16]
        b.cache[page, j % 16, (7, 511, 300, 575, 512)[i % 5]] = what
    b.out.fill_(7.0)
    b.run()
    seen = first - (n - q)                                 # query tokens before it
    assert torch.equal(b.out[:seen], want[:seen])
    assert torch.equal(b.out[q:], want[q:])
    if what != what:
        assert torch.isnan(b.out[seen:q]).all()
    assert pkv.workspace_status(b.ws) == 0
