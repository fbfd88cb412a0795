"""Calls at the ends of what the latent operators take: empty batches, bounds of zero, requests without rows."""

import pytest
import torch

import paged_kv_cache_111_gb300 as pkv
from test_latent_attn_gpu import Batch

pytestmark = pytest.mark.gpu

METADATA = 8


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_a_batch_without_requests_stores_its_status():
    b = Batch(2, [(1, 40), (2, 20)], 16)
    b.lens[1] = 1                                          # fewer keys than queries
    b.run()
    assert pkv.workspace_status(b.ws) == METADATA
    before, starts = b.out.clone(), i32(0)

    def empty():
        pkv.latent_paged_attn(b.out[:0], b.query[:0], b.cache, b.bt[:0], b.lens[:0], starts, 0, 0, 1.0, b.ws)
    empty()
    assert pkv.workspace_status(b.ws) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        empty()
    b.ws[:4] = 0xFF
    graph.replay()
    assert pkv.workspace_status(b.ws) == 0
    assert torch.equal(b.out, before)


def expanded(q, n, T=None, K=None, max_q=None, max_n=None, H=2):
    """(status, output) of requests of q[r] queries and n[r] keys, in T rows and K keys."""
    T, K = sum(q) if T is None else T, sum(n) if K is None else K
    g = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    starts = [i32(0, *x).cumsum(0).to(torch.int32) for x in (q, n)]
    pkv.latent_attn_expanded(out, randn(T, H, 192), randn(K, H, 128), randn(K, 64), randn(K, H, 128), *starts,
                             max(q) if max_q is None else max_q, max(n) if max_n is None else max_n, 0.07,
                             device_status=status)
    return int(status), out


@pytest.mark.parametrize("S", [1, 3, 500])
def test_expanded_reports_requests_that_bounds_of_zero_leave_out(S):
    status, out = expanded([5] * S, [0] * S, max_n=5)      # queries, and no key at all
    assert status == METADATA and (out == 7.0).all()
    status, out = expanded([5] * S, [9] * S, max_q=0)      # a bound that no request keeps
    assert status == METADATA and (out == 7.0).all()
    status, out = expanded([0] * (S - 1) + [3], [0] * (S - 1) + [4], T=0)      # queries past the batch
    assert status == METADATA
    status, out = expanded([0] * S, [0] * (S - 1) + [4], max_n=3)              # a length past its bound
    assert status == METADATA


@pytest.mark.parametrize("S", [1, 3])
def test_expanded_with_nothing_to_do_is_no_error(S):
    assert expanded([0] * S, [0] * S, T=4, max_q=3, max_n=3)[0] == 0
    assert expanded([0] * S, [6] * S)[0] == 0
    status, out = expanded([0] * S, [6] * S, T=4)
    assert status == 0 and (out == 7.0).all()


def gather(lens, starts, rows, bound):
    """(status, output) of the cached rows of requests in `rows` rows."""
    cache = torch.ones(9, 16, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(len(lens), -(-bound // 16) + 1, dtype=torch.int32, device="cuda")
    out = torch.full((rows, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.latent_gather(out, cache, table, i32(*lens), i32(*starts), bound, device_status=status)
    return int(status), out


def test_gather_reports_requests_past_a_bound_of_zero():
    status, out = gather([0, 3], [0, 0], 5, 0)
    assert status == METADATA and (out == 7.0).all()
    assert gather([0, 0], [0, 0], 5, 0)[0] == 0


def test_gather_with_a_bound_of_zero_needs_the_lengths_alone():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, cache = torch.empty(0, 576, dtype=torch.bfloat16, device="cuda"), torch.ones(1, 16, 576).bfloat16().cuda()
    pkv.latent_gather(out, cache, torch.empty(2, 0, dtype=torch.int32, device="cuda"), i32(0, 0), i32(0, 0), 0,
                      device_status=status)
    assert int(status) == 0


def test_gather_into_no_rows():
    assert gather([0, 0], [0, 0], 0, 40)[0] == 0
    assert gather([0, 3], [0, 0], 0, 40)[0] == METADATA    # rows outside the output


def test_gather_takes_no_notice_of_where_an_empty_request_would_start():
    status, out = gather([2, 0, 0], [1, -1, 1000], 4, 40)
    assert status == 0
    assert (out[1:3] == 1.0).all() and (out[0] == 7.0).all() and (out[3] == 7.0).all()
