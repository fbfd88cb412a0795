"""Plain 64-bit references of the norm, rotation, latent-cache and latent-attention calls (tests' helper), and the
error bounds their comparisons use."""

import torch

BF16_HALF_STEP = torch.finfo(torch.bfloat16).eps / 2         # 2^-8, relative
FP32_STEP = torch.finfo(torch.float32).eps / 2               # 2^-24


def angles(rot, length, base=10000.0):
    """fp32 [length, rot]: cosines, then sines."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(length, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def norm_rotate(x, weight, eps, table, positions, interleaved):
    """x [T, H, d] -> (value, magnitude) in 64 bits: magnitude is the sum of the absolute terms of each output, which
    the fp32 arithmetic's error is relative to."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    rot = table.shape[1]
    row = table.double()[positions]
    c, s = row[:, None, :rot // 2], row[:, None, rot // 2:]
    if interleaved:
        i = torch.arange(0, rot, 2, device=x.device)
        j = i + 1
    else:
        i = torch.arange(rot // 2, device=x.device)
        j = i + rot // 2
    y, m = x.clone(), x.abs().clone()
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    m[..., i] = (x[..., i] * c).abs() + (x[..., j] * s).abs()
    m[..., j] = (x[..., j] * c).abs() + (x[..., i] * s).abs()
    return y, m


# The fp32 steps of an output: a sum of up to 512 squares across lanes (16 terms in a lane, 5 exchanges: 21 roundings
# of a mean, halved by the square root), rsqrt (2 ulp), the eps, two products and three of the rotation: under 20
# half steps.  32 is taken.
FP32_SLACK = 32 * FP32_STEP


def check_rounded(got, ref, mag, what):
    err = (got.double() - ref).abs()
    bound = BF16_HALF_STEP * ref.abs() + (1 + BF16_HALF_STEP) * FP32_SLACK * mag
    assert torch.isfinite(got.float()).all(), f"{what}: not finite"
    worst = (err - bound).max().item()
    assert worst <= 0, f"{what}: {worst:.3e} past the bound (max err {err.max().item():.3e})"


def attention(query, rows, limit, scale, width):
    """query [q, H, D], rows [n, D] (64 bits), limit [q] visible keys -> (out, out of |values|), [q, H, width]."""
    w = torch.einsum("qhd,nd->hqn", query, rows) * scale
    hidden = torch.arange(rows.shape[0], device=rows.device)[None] >= limit[:, None]
    w = torch.softmax(w.masked_fill(hidden[None], float("-inf")), -1)
    v = torch.where(torch.isfinite(rows[:, :width]), rows[:, :width], torch.zeros_like(rows[:, :width]))
    return torch.einsum("hqn,nd->qhd", w, v), torch.einsum("hqn,nd->qhd", w, v.abs())
