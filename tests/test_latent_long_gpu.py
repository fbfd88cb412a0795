"""Requests of twenty million keys, each CTA of which works on them for longer than a bounded wait lasts.

A few keys at both ends have ordinary scores and the ones between them scores lower by 66 in the log2 domain.  The
other dims spread scores by less than 20 (eight standard deviations of 2.5), so those keys add less than 2e7 * 2^-46,
2^-21, of the weights: a 2^-12th part of the bound, which is that of the ordinary keys alone (half a bf16 step of the
output and of every weight, and the fp32 score's error twice, 2^-20 of the sum of its absolute products).
"""

import pytest
import torch

import paged_kv_cache_111_gb300 as pkv
from latent_ref import BF16_HALF_STEP

pytestmark = pytest.mark.gpu

N = 20_000_000
FAR = -16.0                     # of one rotated dim, times 40 of the query's: -640 / sqrt(192) * log2(e) = -66


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(got, query, key, value, visible, scale):
    """got [R, W] of rows query [R, D] over key [K, D], value [K, W], where visible [R, K]."""
    s = (query @ key.T * scale).masked_fill(~visible, float("-inf"))
    w = torch.softmax(s, -1)
    ref, mag = w @ value, w @ value.abs()
    score = (query.abs() @ key.abs().T).amax(-1, keepdim=True) * scale
    bound = BF16_HALF_STEP * ref.abs() + mag * (BF16_HALF_STEP * (1 + BF16_HALF_STEP) + 2 * 2.0 ** -20 * score)
    assert ((got - ref).abs() <= bound).all()


def test_latent_attention():
    """One chunk of 152 row tiles of 16 heads: a row tile a CTA, against 312500 key tiles.  The pages between the ends
    are one page of the cache."""
    g = torch.Generator(device="cuda").manual_seed(1)
    H, q = 16, 608
    ends = [4, 40]                                         # pages at the start, and at the end with the chunk in them
    cache = torch.randn(sum(ends) + 1, 16, 576, generator=g, device="cuda").to(torch.bfloat16)
    cache[:, :, 512 + 5] = 0
    cache[0, :, 512 + 5] = FAR
    table = torch.zeros(1, N // 16, dtype=torch.int32, device="cuda")
    ids = torch.arange(1, sum(ends) + 1, dtype=torch.int32, device="cuda")
    table[0, :ends[0]], table[0, -ends[1]:] = ids[:ends[0]], ids[ends[0]:]
    query = torch.randn(q, H, 576, generator=g, device="cuda").to(torch.bfloat16)
    query[:, :, 512 + 5] = 40.0
    out = torch.full((q, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pkv.latent_paged_attn_workspace_size(1, q, q, N, H), dtype=torch.uint8, device="cuda")
    scale = 192 ** -0.5
    pkv.latent_paged_attn(out, query, cache, table, i32(N), i32(0, q), q, N, scale, ws)
    assert pkv.workspace_status(ws) == 0
    rows = cache[1:].view(-1, 576).double()
    at = torch.cat([torch.arange(ends[0] * 16), torch.arange(N - ends[1] * 16, N)]).cuda()
    for h in range(H):
        visible = at[None] <= torch.arange(N - q, N, device="cuda")[:, None]
        check(out[:, h].double(), query[:, h].double(), rows, rows[:, :512], visible, scale)


def test_expanded_attention():
    """One head and 153 token tiles, so that none shares its keys out: 156250 key tiles before the diagonal."""
    g = torch.Generator(device="cuda").manual_seed(2)
    q = 153 * 256
    key = torch.zeros(N, 1, 128, dtype=torch.bfloat16, device="cuda")
    rope = torch.zeros(N, 64, dtype=torch.bfloat16, device="cuda")
    value = torch.empty(N, 1, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    rope[:, 5] = FAR
    at = torch.cat([torch.arange(100), torch.arange(N - q, N, 64)]).cuda()
    rope[at, 5] = 0
    key[at] = torch.randn(at.numel(), 1, 128, generator=g, device="cuda").to(torch.bfloat16)
    query = torch.randn(q, 1, 192, generator=g, device="cuda").to(torch.bfloat16)
    query[:, :, 128 + 5] = 40.0
    out = torch.full((q, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = 192 ** -0.5
    pkv.latent_attn_expanded(out, query, key, rope, value, i32(0, q), i32(0, N), q, N, scale, device_status=status)
    assert int(status) == 0
    k = torch.cat([key[at, 0], rope[at]], -1).double()
    for r in range(0, q, 4096):
        rows = slice(r, min(q, r + 4096))
        visible = at[None] <= torch.arange(N - q, N, device="cuda")[rows, None]
        check(out[rows, 0].double(), query[rows, 0].double(), k, value[at, 0].double(), visible, scale)
