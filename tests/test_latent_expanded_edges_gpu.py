"""The expanded form where requests of one call differ, against the 64-bit form and bound of test_latent_expanded_gpu."""

import pytest
import torch

from test_latent_expanded_gpu import Ragged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [2, 16, 60])                 # shares of four, two and one CTAs a token tile
@pytest.mark.parametrize("refused", [0, 1, 2])
def test_a_refused_request_beside_good_ones_whose_keys_are_shared_out(H, refused):
    reqs = [(4, 1600), (7, 700), (6, 1300)]
    reqs[refused] = (300, reqs[refused][1])                # one more token tile, were it taken
    c = Ragged(61, reqs, H)
    c.max_q = 7
    c.run()
    assert int(c.status) == 8
    c.check(skip=(refused,))
    c.max_q, first = 300, c.out.clone()
    c.status.zero_()
    c.run()                                                # the others as before, and now that one too
    assert int(c.status) == 0
    c.check()
    t = sum(q for q, _ in reqs[:refused])
    c.out[t:t + 300] = 7.0
    assert torch.equal(c.out, first)


@pytest.mark.parametrize("H", [2, 16, 60])
def test_pointers_aligned_to_16_bytes_alone(H):
    def off(x):
        flat = torch.empty(x.numel() + 8, dtype=x.dtype, device=x.device)
        return flat[8:].view(x.shape).copy_(x)
    c = Ragged(62, [(300, 900), (3, 5)], H)
    first = c.run().clone()
    c.check()
    c.query, c.key, c.value, c.rope, c.out = (off(x) for x in (c.query, c.key, c.value, c.rope, c.out))
    c.out.fill_(7.0)
    assert torch.equal(c.run(), first)


@pytest.mark.parametrize("H", [2, 16, 60])
def test_a_graph_replayed_with_other_lengths(H):
    c = Ragged(63, [(300, 900), (40, 700), (300, 600)], H)
    c.query.nan_to_num_(), c.key.nan_to_num_(), c.value.nan_to_num_(), c.rope.nan_to_num_()
    c.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for reqs in ([(1, 200), (40, 700), (7, 7)], [(300, 300), (0, 0), (300, 900)], [(0, 0), (0, 12), (2, 900)],
                 [(300, 900), (40, 700), (300, 600)]):
        c.reqs = reqs
        c.qsl[1:] = torch.tensor([q for q, _ in reqs]).cumsum(0).to(torch.int32).cuda()
        c.ksl[1:] = torch.tensor([n for _, n in reqs]).cumsum(0).to(torch.int32).cuda()
        c.out.fill_(7.0)
        graph.replay()
        assert int(c.status) == 0
        c.check(what=f"{reqs}")
