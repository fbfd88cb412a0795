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
