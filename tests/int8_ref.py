"""Plain forms of the int8 cache's calls (tests' helper), and the error bounds their comparisons use.

The write's scales are defined by single fp32 operations and its codes by one rounding of an exact product, so the model
here (numpy) gives them to the bit.  Attention is held against 64 bits over the values that codes and scales stand for."""

import numpy as np
import torch

BLOCK = 16
LEAST = np.float32(2.0 ** -60)
BF16_HALF_STEP = torch.finfo(torch.bfloat16).eps / 2         # 2^-8, relative
F16_HALF_STEP = torch.finfo(torch.float16).eps / 2           # 2^-11
FP32_STEP = torch.finfo(torch.float32).eps / 2               # 2^-24


def new_cache(blocks, hkv, d, seed=0):
    """A cache of arbitrary codes and scales."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-127, 128, (blocks, hkv, 2, BLOCK, d), generator=g, dtype=torch.int8)
    return codes, torch.rand(blocks, hkv, 2, generator=g) * 0.05 + 0.002


def write(cache, scales, key, value, slots, ignored=()):
    """The model of the write, in place on numpy arrays (int8, fp32); key and value fp32 [T, Hkv, d].  `ignored`: tokens
    that count for nothing."""
    t, T, blocks = 0, len(slots), cache.shape[0]
    with np.errstate(all="ignore"):
        while t < T:
            if slots[t] < 0 or slots[t] // BLOCK >= blocks:
                t += 1
                continue
            b, end = slots[t] // BLOCK, t
            while end < T and slots[end] >= 0 and slots[end] // BLOCK == b:
                end += 1
            row = {}
            for i in range(t, min(end, t + BLOCK)):          # (what follows the 16th of a stretch is skipped)
                if i not in ignored:
                    row[int(slots[i] % BLOCK)] = i           # the last of those with one slot
            t = end
            if not row:
                continue
            offs, toks = list(row), [row[o] for o in row]
            for side, x in ((0, key), (1, value)):
                new = x[toks].astype(np.float32)                                  # [n, Hkv, d]
                a = np.abs(new).max(axis=(0, 2))
                want = np.maximum(a * np.float32(1 / 127), LEAST).astype(np.float32)
                want[~np.isfinite(new).all(axis=(0, 2))] = np.nan
                old = scales[b, :, side].copy()
                s = want if 0 in row else np.where((old >= want) | np.isnan(old), old, want)
                r = (np.float32(1) / s).astype(np.float32)
                codes = np.rint(new.astype(np.float64) * r[None, :, None].astype(np.float64))
                fine = np.isfinite(s)
                if 0 not in row:
                    for h in np.nonzero(fine & (s > old))[0]:
                        kept = [o for o in range(BLOCK) if o not in row]
                        ratio = np.float32(old[h] * r[h])
                        cache[b, h, side, kept] = np.rint(cache[b, h, side, kept].astype(np.float64) * np.float64(ratio)).astype(np.int8)
                for n, o in enumerate(offs):
                    cache[b, fine, side, o] = codes[n, fine].astype(np.int8)
                scales[b, :, side] = s


def same(cache, scales, ref_cache, ref_scales):
    """Scales equal (NaN beside NaN), and codes wherever the scale is a number."""
    got_s, got_c = scales.cpu().numpy(), cache.cpu().numpy()
    assert np.array_equal(got_s, ref_scales, equal_nan=True), np.argwhere((got_s != ref_scales) & ~np.isnan(ref_scales))[:5]
    fine = ~np.isnan(ref_scales)
    bad = (got_c != ref_cache).any(axis=(3, 4)) & fine
    assert not bad.any(), f"blocks {np.argwhere(bad)[:5].tolist()} of {int(bad.sum())}"


def values(cache, scales):
    """What an int8 cache stands for, 64 bits."""
    return cache.double() * scales.double()[..., None, None]


def rows_of(cache, scales, table, n):
    """K and V of the first n tokens of a request, 64 bits [n, Hkv, d] each, on the cache's device."""
    pages = table[: -(-n // BLOCK)].long()
    x = values(cache[pages], scales[pages])                                        # [pages, Hkv, 2, 16, d]
    return [x[:, :, side].transpose(1, 2).reshape(-1, x.shape[1], x.shape[4])[:n] for side in (0, 1)]


def attention(query, cache, scales, tables, lens, qsl, scale):
    """(out, bound) in 64 bits, [T, Hq, d]; rows that no request owns are NaN in `bound`.

    The bound: the output's rounding to bf16; each weight's to f16 (2^-11 relative, and 2^-25 absolute where the largest
    weight times its V scale is one or more); and the scores' errors, which move a weight by as much relative to it: S is
    a sum of at most 8 products and a start of 1152 sum q, each accumulation good to 2^-23 of the largest term, and the
    query's parts below 2^-24 of its largest are lost; 16 such steps are taken, twice (weight and sum)."""
    T, hq, d = query.shape
    hkv = cache.shape[1]
    group = hq // hkv
    out = torch.full((T, hq, d), float("nan"), dtype=torch.float64, device=query.device)
    bound = out.clone()
    for r, n in enumerate(lens):
        q0, q1 = qsl[r], qsl[r + 1]
        if q1 == q0:
            continue
        k, v = rows_of(cache, scales, tables[r], n)
        pages = tables[r][: -(-n // BLOCK)].long()
        s = scales[pages].double().repeat_interleave(BLOCK, 0)[:n]                 # [n, Hkv, 2]
        q = query[q0:q1].double()
        seen = torch.arange(n, device=q.device)[None] < torch.arange(n - (q1 - q0) + 1, n + 1, device=q.device)[:, None]
        for h in range(hkv):
            mine = q[:, h * group:(h + 1) * group]                                 # [q, G, d]
            w = torch.einsum("qgd,nd->gqn", mine, k[:, h]) * scale
            w = torch.softmax(torch.where(seen, w, -torch.inf), -1)
            w = torch.where(seen, w, 0.0)
            vis = torch.where(torch.isfinite(v[:, h]), v[:, h], torch.zeros_like(v[:, h]))
            o = torch.einsum("gqn,nd->qgd", w, v[:, h] if torch.isfinite(v[:, h]).all() else vis)
            a = torch.einsum("gqn,nd->qgd", w, vis.abs())
            size = abs(scale) * (1152 * mine.abs().sum(-1)[..., None] * s[None, None, :, h, 0].nan_to_num()).amax(-1)   # [q, G]
            slip = 2 * 16 * 2 * FP32_STEP * size + 2.0 ** -18
            least = 127 * n * 2.0 ** -25 * (w * s[:, h, 1].nan_to_num()[None, None]).amax(-1).T                        # [q, G]
            e = (F16_HALF_STEP + slip)[..., None] * a + least[..., None]
            out[q0:q1, h * group:(h + 1) * group] = o
            bound[q0:q1, h * group:(h + 1) * group] = BF16_HALF_STEP * o.abs() + (1 + BF16_HALF_STEP) * e
    return out, bound


def check(got, ref, bound, what=""):
    owned = ~torch.isnan(bound)
    err = (got.double() - ref).abs()[owned]
    assert torch.isfinite(got[owned].float()).all(), f"{what}: not finite"
    worst = (err - bound[owned]).max().item() if err.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} past the bound (max err {err.max().item():.3e})"
