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
