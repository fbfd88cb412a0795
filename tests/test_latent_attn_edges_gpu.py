"""The latent attention where its parts meet, against the plain 64-bit form and the bound of test_latent_attn_gpu."""

import pytest
import torch

import paged_kv_cache_111_gb300 as pkv
from test_latent_attn_gpu import D, W, Batch

pytestmark = pytest.mark.gpu


def rewrite(b, r, rows):
    """Request r's cached rows replaced (64-bit values of bf16 numbers)."""
    n = b.reqs[r][1]
    b.rows[r] = rows
    at = torch.arange(n)
    b.cache[b.bt[r, at.cuda() // 16].long(), (at % 16).cuda()] = rows.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("H,seqs", [(128, 600), (16, 900)])
def test_scores_that_jump_where_items_meet(H, seqs):
    """Runs of many short row tiles: the scores of every second key tile jump past the softmax reference's bound, so
    that rescaling falls into the tiles behind an item's first, again and again, and the same bits come out."""
    g = torch.Generator().manual_seed(H)
    b = Batch(41, [(1, int(n)) for n in torch.randint(1, 200, (seqs,), generator=g)], H)
    for r, (q, n) in enumerate(b.reqs):
        rows = b.rows[r]
        rows[:, W:] = 0
        rows[:, W] = (torch.arange(n) // 64 * 16).double()
        rewrite(b, r, rows)
    b.query[:, :, W] = 40.0
    first = b.run().clone()
    assert pkv.workspace_status(b.ws) == 0
    b.check()
    for _ in range(20):
        b.out.fill_(7.0)
        assert torch.equal(b.run(), first)
    assert pkv.workspace_status(b.ws) == 0


@pytest.mark.parametrize("H,seqs", [(16, 3), (128, 200)])  # either form of the merge
@pytest.mark.parametrize("word", [0, 9, -1, 7])
def test_the_status_word_starts_afresh(H, seqs, word):
    b = Batch(7, [(1, 70 + r % 90) for r in range(seqs)], H)
    table, lens = b.bt.clone(), b.lens.clone()
    for code in (0, 7, 8):
        b.ws[:4].view(torch.int32).fill_(word)
        b.bt.copy_(table), b.lens.copy_(lens)
        if code == 7:
            b.bt[seqs - 1, 0] = -1
        if code == 8:
            b.lens[0] = 0
        b.run()
        assert pkv.workspace_status(b.ws) == code


@pytest.mark.parametrize("H,short,long", [(128, 63, 40000), (64, 100, 20000), (40, 160, 9000), (128, 30, 3000)])
def test_one_long_request_among_many_short_ones(H, short, long):
    """As many row tiles as make the merge one CTA a lane's tile, and among them one of many pieces."""
    g = torch.Generator().manual_seed(short)
    reqs = [(1, int(n)) for n in torch.randint(1, 70, (short,), generator=g)]
    reqs.insert(short // 3, (1, long))
    b = Batch(51, reqs, H, extra_rows=1)
    first = b.run().clone()
    assert pkv.workspace_status(b.ws) == 0
    b.check()
    b.ws.random_(0, 256)
    assert torch.equal(b.run(), first)
    # a NaN in one of the pieces makes that request's rows NaN, and no other's
    b.cache[b.bt[short // 3, long // 32].long(), 3, 5] = float("nan")
    b.out.fill_(7.0)
    b.run()
    assert torch.isnan(b.out[short // 3]).all()
    b.out[short // 3] = first[short // 3]
    assert torch.equal(b.out, first)


def off_by_16_bytes(x):
    """The same tensor, 16 bytes past where its memory begins."""
    flat = torch.empty(x.numel() + 8, dtype=x.dtype, device=x.device)
    y = flat[8:].view(x.shape)
    assert y.data_ptr() % 32 == 16
    return y.copy_(x)


@pytest.mark.parametrize("H", [16, 128])
def test_pointers_aligned_to_16_bytes_alone(H):
    b = Batch(71, [(1, 300), (40, 190), (3, 3)], H, extra_rows=1)
    first = b.run().clone()
    b.check()
    b.cache, b.query, b.out = off_by_16_bytes(b.cache), off_by_16_bytes(b.query), off_by_16_bytes(b.out)
    b.out.fill_(7.0)
    assert torch.equal(b.run(), first)
    starts = torch.tensor([0, 300, 490], dtype=torch.int32, device="cuda")
    rows = off_by_16_bytes(torch.zeros(493, D, dtype=torch.bfloat16, device="cuda"))
    pkv.latent_gather(rows, b.cache, b.bt, b.lens, starts, 300)
    assert torch.equal(rows.double().cpu(), torch.cat(b.rows))


def test_one_workspace_through_calls_of_other_shapes():
    """A workspace that other calls of other heads and lengths have left full of their pieces."""
    bs = [Batch(80 + i, reqs, H) for i, (H, reqs) in enumerate([
        (128, [(1, 3000)] * 40), (16, [(1, 9000)]), (5, [(70, 400), (1, 20)]), (64, [(2, 500)] * 90), (1, [(1, 1)])])]
    want = []
    for b in bs:
        want.append(b.run().clone())
        b.check()
    for order in ((0, 1, 2, 3, 4), (4, 3, 1, 0, 2), (1, 0, 1, 3, 2)):
        for i in order:
            bs[i].ws = bs[0].ws
            bs[i].out.fill_(7.0)
            assert torch.equal(bs[i].run(), want[i])
            assert pkv.workspace_status(bs[0].ws) == 0


def test_a_graph_replayed_with_other_lengths():
    """The captured call's bounds hold for lengths that grow from replay to replay, and for a batch padded with empty
    requests."""
    b = Batch(90, [(1, 700), (1, 333), (5, 640), (1, 64)], 16)
    lens, qsl = b.lens.clone(), b.qsl.clone()
    graph = torch.cuda.CUDAGraph()
    b.run()
    with torch.cuda.graph(graph):
        b.run()
    rows, reqs = list(b.rows), list(b.reqs)
    for n, q in (((600, 100, 600, 1), (1, 1, 5, 1)), ((601, 101, 605, 2), (1, 1, 5, 1)), ((700, 64, 0, 0), (1, 1, 0, 0)),
                 ((0, 0, 7, 0), (0, 0, 2, 0)), ((700, 333, 640, 64), (1, 1, 5, 1))):
        b.lens.copy_(torch.tensor(n, dtype=torch.int32))
        b.qsl[1:] = torch.tensor(q).cumsum(0).to(torch.int32).cuda()
        b.reqs, b.rows = list(zip(q, n)), [r[:m] for r, m in zip(rows, n)]
        b.out.fill_(7.0)
        graph.replay()
        assert pkv.workspace_status(b.ws) == 0
        b.check(what=f"{n}")
    assert torch.equal(b.lens, lens) and torch.equal(b.qsl, qsl) and b.reqs == reqs
