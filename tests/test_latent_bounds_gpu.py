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
