"""The operators around a paged cache: what is measured of each, its plain form and its exact value.

Five operators.  ``qk`` norms the query and key heads, rotates them to their positions and stores K and V in the
paged cache.  ``latent-write`` does the same for a cache of one latent vector a token (512 normed dims and 64 rotated
ones).  ``latent-attn`` is causal attention of every head over that cache in the latent space (the absorbed form),
``latent-gather`` reads a batch's cached rows out of their pages, and ``expanded`` is causal attention over the
per-head keys and values that an up-projection makes of such rows (128 plain and 64 shared rotated key dims, 128
value dims).  Lengths are those of the engine steps that the benchmark names: small and large decode batches, and a
mixed step of decodes and a 2046-token prefill chunk.
"""

import math

import torch

own = False

BLOCK = 16
LATENT, ROPE = 512, 64
ROW = LATENT + ROPE
NOPE, VDIM = 128, 128


# ---- cases -----------------------------------------------------------------------------------------------------

def listed():
    return [
        # a handful of interactive requests, one new token each: latency
        {"name": "qk-decode-4", "op": "qk", "tokens": 4, "hq": 8, "hkv": 8, "d": 64, "rot": 64, "inter": False,
         "fp8": False, "blocks": 64, "seed": 1},
        # a prefill step of a grouped-query model, q, k and v views of one fused projection
        {"name": "qk-chunk-8192", "op": "qk", "tokens": 8192, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "inter": False, "fp8": False, "blocks": 1024, "seed": 2},
        # the mixed step (two decodes and a 2046-token chunk) into an E4M3 cache, half of each head rotated in pairs
        {"name": "qk-fp8-2048", "op": "qk", "tokens": 2048, "hq": 64, "hkv": 8, "d": 128, "rot": 64, "inter": True,
         "fp8": True, "blocks": 512, "seed": 3},
        # one decode step of 64 requests
        {"name": "latent-write-64", "op": "latent-write", "tokens": 64, "heads": 128, "inter": True, "blocks": 4096,
         "seed": 4},
        # a prefill step of odd length
        {"name": "latent-write-8191", "op": "latent-write", "tokens": 8191, "heads": 16, "inter": False,
         "blocks": 1024, "seed": 5},
        # four requests at the start of their answers: latency
        {"name": "latent-attn-4", "op": "latent-attn", "heads": 16, "kind": "uniform", "seqs": 4, "lo": 1, "hi": 128,
         "chunk": 0, "context": 0, "seed": 6},
        # a large decode batch, every head on this GPU
        {"name": "latent-attn-256", "op": "latent-attn", "heads": 128, "kind": "lognormal", "seqs": 256, "lo": 16,
         "hi": 4096, "chunk": 0, "context": 0, "seed": 7},
        # a mixed step: two decodes and a chunk that starts after 500 cached tokens
        {"name": "latent-attn-mixed", "op": "latent-attn", "heads": 16, "kind": "uniform", "seqs": 2, "lo": 700,
         "hi": 1500, "chunk": 2046, "context": 500, "seed": 8},
        # the cached rows of a small batch, and those of a large one
        {"name": "latent-gather-4", "op": "latent-gather", "kind": "uniform", "seqs": 4, "lo": 1, "hi": 128,
         "seed": 9},
        {"name": "latent-gather-256", "op": "latent-gather", "kind": "lognormal", "seqs": 256, "lo": 16, "hi": 4096,
         "seed": 10},
        # the mixed step's chunk beside two short prompts
        {"name": "expanded-mixed", "op": "expanded", "heads": 16, "seqs": 3, "lo": 300, "hi": 2046, "context": 0,
         "seed": 11},
        # a later chunk of a long prompt, every head on this GPU
        {"name": "expanded-8192", "op": "expanded", "heads": 128, "seqs": 1, "lo": 2048, "hi": 2048,
         "context": 6144, "seed": 12},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "latent-write", "latent-attn", "latent-gather", "expanded"])
    case = {"op": op, "seed": rng.randrange(1 << 20)}
    if op == "qk":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8, 40])
        group = 1 if hkv == 40 else rng.choice([1, 3, 4, 8])
        tokens = _log_int(rng, 1, 8192 * 32 // max(32, hkv * group))
        case.update(tokens=tokens, hq=hkv * group, hkv=hkv, d=d, rot=rng.choice([16, d // 2, d]),
                    inter=rng.random() < 0.5, fp8=rng.random() < 0.5, blocks=-(-tokens // BLOCK) * 2 + 1)
    elif op == "latent-write":
        heads = rng.choice([1, 5, 16, 32, 64, 128])
        tokens = _log_int(rng, 1, 8191 * 16 // max(16, heads))
        case.update(tokens=tokens, heads=heads, inter=rng.random() < 0.5, blocks=-(-tokens // BLOCK) * 2 + 1)
    elif op == "latent-attn":
        hi = _log_int(rng, 2, 4096)
        chunk = rng.choice([0, 0, _log_int(rng, 2, 1024)])
        heads = rng.choice([5, 16, 20, 32, 64, 128]) if not chunk else rng.choice([5, 16, 20, 32])
        case.update(heads=heads, kind=rng.choice(["uniform", "lognormal"]),
                    seqs=_log_int(rng, 1, 128 if not chunk else 4), lo=rng.randint(1, hi), hi=hi, chunk=chunk,
                    context=rng.randrange(0, 700) if chunk else 0)
    elif op == "latent-gather":
        hi = _log_int(rng, 2, 4096)
        case.update(kind=rng.choice(["uniform", "lognormal"]), seqs=_log_int(rng, 1, 200), lo=rng.randint(1, hi),
                    hi=hi)
    else:
        heads = rng.choice([1, 5, 16, 32, 128])
        seqs = rng.randint(1, 4)
        most = max(2, int(math.sqrt(2048 * 8192 * 128 / (heads * seqs)) / 2))
        hi = _log_int(rng, 2, min(2048, most))
        case.update(heads=heads, seqs=seqs, lo=rng.randint(1, hi), hi=hi,
                    context=rng.randrange(0, min(6144, most)))
    return case


def _lengths(case, rng_seed):
    """The requests' lengths (uniform, or round(exp(N)) clipped, mean about 780): part of the case, not of the inputs."""
    g = torch.Generator().manual_seed(rng_seed)
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    if case.get("kind") == "lognormal":
        x = torch.exp(torch.randn(n, generator=g, dtype=torch.float64) * 0.8 + math.log(800.0) - 0.32)
        return [int(v) for v in x.round().clamp(min(lo, hi), hi)]
    return [int(v) for v in torch.randint(lo, hi + 1, (n,), generator=g)]


def _requests(case):
    """[(query tokens, keys)] of the step: decodes, then the chunk where there is one."""
    lens = _lengths(case, case["seed"])
    if case["op"] == "expanded":
        return [(n, n + case["context"]) for n in lens]
    reqs = [(1, n) for n in lens]
    if case.get("chunk"):
        reqs.append((case["chunk"], case["chunk"] + case["context"]))
    return reqs


def _pairs(reqs):
    return sum(q * (n - q) + q * (q + 1) // 2 for q, n in reqs)


def work(case):
    op = case["op"]
    if op == "qk":
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        stored = 1 if case["fp8"] else 2
        return {"bytes": t * (4 * hq * d + 2 * hkv * d * (2 + stored) + 4 * case["rot"] + 16) + 4 * d,
                "flops": t * (hq + hkv) * (4 * d + 3 * case["rot"])}
    if op == "latent-write":
        t, h = case["tokens"], case["heads"]
        return {"bytes": t * (4 * ROW + 4 * h * ROPE + 4 * ROPE + 16) + 2 * LATENT,
                "flops": t * (4 * LATENT + 3 * (h + 1) * ROPE)}
    reqs = _requests(case)
    keys, rows = sum(n for _, n in reqs), sum(q for q, _ in reqs)
    tables = 4 * sum(-(-n // BLOCK) for _, n in reqs) + 8 * len(reqs)
    if op == "latent-gather":
        return {"bytes": keys * 4 * ROW + tables, "flops": 0}
    h = case["heads"]
    if op == "latent-attn":
        return {"bytes": keys * 2 * ROW + rows * h * 2 * (ROW + LATENT) + tables,
                "flops": 2 * (ROW + LATENT) * h * _pairs(reqs)}
    return {"bytes": keys * 2 * (h * (NOPE + VDIM) + ROPE) + rows * h * 2 * (NOPE + ROPE + VDIM) + 8 * len(reqs),
            "flops": 2 * (NOPE + ROPE + VDIM) * h * _pairs(reqs)}


# ---- inputs ----------------------------------------------------------------------------------------------------

def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def _angles(rot, length):
    """fp32 [length, rot]: cosines, then sines, of position * 10000^(-2i / rot), made in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _table(g, reqs):
    """A block table of pages in random order, -1 past each request's last, and the number of pages in the pool."""
    counts = [-(-n // BLOCK) for _, n in reqs]
    total, width = sum(counts), max(counts)
    blocks = total + total // 8 + 1
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    c = torch.tensor(counts, device="cuda")
    inside = torch.arange(width, device="cuda")[None] < c[:, None]
    table = torch.full((len(reqs), width), -1, dtype=torch.int32, device="cuda")
    table[inside] = order[:total]
    return table, blocks


def _starts(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1009 + case["seed"])
    op, s = case["op"], dict(case)
    if op in ("qk", "latent-write"):
        t, blocks = case["tokens"], case["blocks"]
        s["slots"] = torch.randperm(blocks * BLOCK, generator=g, device="cuda")[:t].contiguous()
        s["positions"] = torch.randint(0, 4096, (t,), generator=g, device="cuda")
        s["eps"] = 1e-6
    if op == "qk":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        fused = _normal(g, t, hq + 2 * hkv, d)
        s["query"], s["key"], s["value"] = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
        s["wq"], s["wk"] = _normal(g, d, std=0.3) + 1, _normal(g, d, std=0.3) + 1
        s["table"] = _angles(case["rot"], 4096)
        cache = _normal(g, blocks, hkv, 2, BLOCK, d)
        s["k_scale"], s["v_scale"] = 0.0173, 0.011
        s["cache"] = cache.float().to(torch.float8_e4m3fn) if case["fp8"] else cache
        s["query_out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda")
    elif op == "latent-write":
        h = case["heads"]
        down = _normal(g, t, ROW)
        s["latent"], s["key_rope"] = down[:, :LATENT], down[:, LATENT:]
        s["weight"] = _normal(g, LATENT, std=0.3) + 1
        s["table"] = _angles(ROPE, 4096)
        s["query_rope"] = _normal(g, t, h, NOPE + ROPE)[:, :, NOPE:]
        s["query"] = _normal(g, t, h, ROW)
        s["cache"] = _normal(g, blocks, BLOCK, ROW)
    else:
        reqs = _requests(case)
        q, n = [a for a, _ in reqs], [b for _, b in reqs]
        s["max_q"], s["max_n"] = max(q), max(n)
        s["starts"], s["lens"] = _starts(q), torch.tensor(n, dtype=torch.int32, device="cuda")
        s["key_starts"] = _starts(n)
        rows, keys = sum(q), sum(n)
        # where each query token and each key stands in a padded [request, index] grid
        s["seq_of"] = torch.repeat_interleave(torch.arange(len(q), device="cuda"), torch.tensor(q, device="cuda"))
        s["at"] = torch.arange(rows, device="cuda") - s["starts"].long()[s["seq_of"]]
        s["key_seq"] = torch.repeat_interleave(torch.arange(len(n), device="cuda"), torch.tensor(n, device="cuda"))
        s["key_at"] = torch.arange(keys, device="cuda") - s["key_starts"].long()[s["key_seq"]]
        if op == "expanded":
            h = case["heads"]
            s["query"] = _normal(g, rows, h, NOPE + ROPE)
            up = _normal(g, keys, h, NOPE + VDIM)
            s["key"], s["value"] = up[:, :, :NOPE], up[:, :, NOPE:]
            s["key_rope"] = _normal(g, keys, ROPE)
            s["scale"] = 1.0 / math.sqrt(NOPE + ROPE)
            s["out"] = torch.empty(rows, h, VDIM, dtype=torch.bfloat16, device="cuda")
        else:
            s["block_table"], blocks = _table(g, reqs)
            s["cache"] = _normal(g, blocks, BLOCK, ROW)
            if op == "latent-gather":
                s["out"] = torch.empty(keys, ROW, dtype=torch.bfloat16, device="cuda")
            else:
                h = case["heads"]
                s["query"] = _normal(g, rows, h, ROW)
                s["scale"] = 1.0 / math.sqrt(NOPE + ROPE)
                s["out"] = torch.empty(rows, h, LATENT, dtype=torch.bfloat16, device="cuda")
    return s


# ---- the operators ---------------------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_qk(s):
    import paged_kv_cache_111_gb300 as pkv
    if s["fp8"]:
        pkv.qk_norm_rope_kv_write_fp8(s["query_out"], s["cache"], s["query"], s["key"], s["value"], s["wq"], s["wk"],
                                      s["eps"], s["table"], s["positions"], s["slots"], s["k_scale"], s["v_scale"],
                                      interleaved=s["inter"])
    else:
        pkv.qk_norm_rope_kv_write(s["query_out"], s["cache"], s["query"], s["key"], s["value"], s["wq"], s["wk"],
                                  s["eps"], s["table"], s["positions"], s["slots"], interleaved=s["inter"])
    return [s["query_out"], s["cache"]]


def _own_latent_write(s):
    import paged_kv_cache_111_gb300 as pkv
    pkv.latent_kv_write(s["cache"], s["latent"], s["key_rope"], s["weight"], s["eps"], s["table"], s["positions"],
                        s["slots"], query_rope_out=s["query"][:, :, LATENT:], query_rope=s["query_rope"],
                        interleaved=s["inter"])
    return [s["query"], s["cache"]]


def _own_latent_attn(s):
    import paged_kv_cache_111_gb300 as pkv
    if "workspace" not in s:
        n = pkv.latent_paged_attn_workspace_size(s["lens"].shape[0], s["query"].shape[0], s["max_q"], s["max_n"],
                                                 s["query"].shape[1])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    pkv.latent_paged_attn(s["out"], s["query"], s["cache"], s["block_table"], s["lens"], s["starts"], s["max_q"],
                          s["max_n"], s["scale"], s["workspace"])
    return s["out"]


def _own_latent_gather(s):
    import paged_kv_cache_111_gb300 as pkv
    pkv.latent_gather(s["out"], s["cache"], s["block_table"], s["lens"], s["key_starts"], s["max_n"])
    return s["out"]


def _own_expanded(s):
    import paged_kv_cache_111_gb300 as pkv
    pkv.latent_attn_expanded(s["out"], s["query"], s["key"], s["key_rope"], s["value"], s["starts"], s["key_starts"],
                             s["max_q"], s["max_n"], s["scale"])
    return s["out"]


def _rms(x, w, eps):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _turn(x, table, positions, rot, inter):
    """The first `rot` dims of x [T, H, d] (fp32) rotated by the table's row of each token's position."""
    row = table[positions]
    c, n = row[:, None, :rot // 2], row[:, None, rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    p, q = a * c - b * n, b * c + a * n
    y = torch.stack([p, q], -1).flatten(-2) if inter else torch.cat([p, q], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_qk(s):
    q = _turn(_rms(s["query"], s["wq"], s["eps"]), s["table"], s["positions"], s["rot"], s["inter"])
    k = _turn(_rms(s["key"], s["wk"], s["eps"]), s["table"], s["positions"], s["rot"], s["inter"])
    block, at = s["slots"] // BLOCK, s["slots"] % BLOCK
    v = s["value"]
    if s["fp8"]:
        k = (k / s["k_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        v = (v.float() / s["v_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
    cache = s["cache"].view(torch.uint8 if s["fp8"] else torch.int16)
    cache[block, :, 0, at] = k.to(s["cache"].dtype).view(cache.dtype)
    cache[block, :, 1, at] = v.contiguous().view(cache.dtype)
    s["query_out"].copy_(q)
    return [s["query_out"], s["cache"]]


def _plain_latent_write(s):
    row = _turn(s["key_rope"].float()[:, None], s["table"], s["positions"], ROPE, s["inter"])[:, 0]
    new = torch.cat([_rms(s["latent"], s["weight"], s["eps"]), row], -1).bfloat16()
    s["cache"].view(-1, ROW)[s["slots"]] = new
    s["query"][:, :, LATENT:] = _turn(s["query_rope"].float(), s["table"], s["positions"], ROPE, s["inter"]).bfloat16()
    return [s["query"], s["cache"]]


def _cached_rows(s):
    page = s["block_table"].long()[s["key_seq"], s["key_at"] // BLOCK]
    return s["cache"].view(-1, ROW)[page * BLOCK + s["key_at"] % BLOCK]


def _padded(s, x, seq, at, length):
    y = torch.zeros((s["lens"].shape[0], length) + tuple(x.shape[1:]), dtype=torch.float32, device="cuda")
    y[seq, at] = x.float()
    return y


def _hidden(s):
    """[request, query, key]: keys after the query's own position, and those past the request's end."""
    n, q = s["lens"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    last = (n - q)[:, None] + torch.arange(s["max_q"], device="cuda")
    return torch.arange(s["max_n"], device="cuda")[None, None] > torch.minimum(last, n[:, None] - 1)[:, :, None]


def _plain_latent_attn(s):
    c = _padded(s, _cached_rows(s), s["key_seq"], s["key_at"], s["max_n"])          # [S, N, 576]
    q = _padded(s, s["query"], s["seq_of"], s["at"], s["max_q"])                    # [S, Q, H, 576]
    b, m, h = q.shape[:3]
    scores = torch.bmm(q.view(b, m * h, ROW), c.transpose(1, 2)).view(b, m, h, -1) * s["scale"]
    scores.masked_fill_(_hidden(s)[:, :, None], -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(b, m * h, -1), c[:, :, :LATENT]).view(b, m, h, LATENT)
    return o[s["seq_of"], s["at"]].bfloat16()


def _plain_latent_gather(s):
    return _cached_rows(s)


def _plain_expanded(s):
    q = _padded(s, s["query"], s["seq_of"], s["at"], s["max_q"]).transpose(1, 2)    # [S, H, Q, 192]
    k = _padded(s, s["key"], s["key_seq"], s["key_at"], s["max_n"]).transpose(1, 2)
    v = _padded(s, s["value"], s["key_seq"], s["key_at"], s["max_n"]).transpose(1, 2)
    r = _padded(s, s["key_rope"], s["key_seq"], s["key_at"], s["max_n"])[:, None]
    scores = torch.matmul(q[..., :NOPE], k.transpose(2, 3))
    scores += torch.matmul(q[..., NOPE:], r.transpose(2, 3))
    scores *= s["scale"]
    scores.masked_fill_(_hidden(s)[:, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True)
    p = scores.exp_()
    p /= p.sum(-1, keepdim=True)
    return torch.matmul(p, v).transpose(1, 2)[s["seq_of"], s["at"]].bfloat16()


_own = {"qk": _own_qk, "latent-write": _own_latent_write, "latent-attn": _own_latent_attn,
        "latent-gather": _own_latent_gather, "expanded": _own_expanded}
_plain = {"qk": _plain_qk, "latent-write": _plain_latent_write, "latent-attn": _plain_latent_attn,
          "latent-gather": _plain_latent_gather, "expanded": _plain_expanded}


# ---- exact values ----------------------------------------------------------------------------------------------

def _spin(x, s, rot):
    """x [T, H, d] in 64 bits with its first `rot` dims turned, as products of complex numbers."""
    turn = torch.complex(s["table"][:, :rot // 2].double(), s["table"][:, rot // 2:].double())[s["positions"]][:, None]
    head, tail = x[..., :rot], x[..., rot:]
    pair = head.unflatten(-1, (rot // 2, 2)) if s["inter"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    z = z if s["inter"] else z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), tail], -1)


def _normed(x, w, eps):
    x = x.double()
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt() * w.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "latent-gather":
        return None                                        # copied bits
    if op == "qk":
        q = _spin(_normed(s["query"], s["wq"], s["eps"]), s, case["rot"])
        k = _spin(_normed(s["key"], s["wk"], s["eps"]), s, case["rot"])
        v, cache = s["value"].double(), s["cache"].to(torch.float32).double()
        if case["fp8"]:                                    # what a code stands for, in units of the scale
            k, v = (k / s["k_scale"]).clamp(-448, 448), (v / s["v_scale"]).clamp(-448, 448)
        cache[s["slots"] // BLOCK, :, 0, s["slots"] % BLOCK] = k
        cache[s["slots"] // BLOCK, :, 1, s["slots"] % BLOCK] = v
        return [q, cache]
    if op == "latent-write":
        cache, query = s["cache"].double(), s["query"].double()
        rows = cache.view(-1, ROW)
        rows[s["slots"], :LATENT] = _normed(s["latent"], s["weight"], s["eps"])
        rows[s["slots"], LATENT:] = _spin(s["key_rope"].double()[:, None], s, ROPE)[:, 0]
        query[:, :, LATENT:] = _spin(s["query_rope"].double(), s, ROPE)
        return [query, cache]
    # attention: one request (and, in the expanded form, one head) after the other
    reqs, parts = _requests(case), []
    width = ROW + LATENT if op == "latent-attn" else NOPE + ROPE + VDIM
    if 2 * width * case["heads"] * sum(q * n for q, n in reqs) > 6e12:
        return None                                        # 64-bit products of over about ten seconds
    q0 = k0 = 0
    for r, (q, n) in enumerate(reqs):
        limit = torch.arange(n - q, n, device="cuda")[:, None] >= torch.arange(n, device="cuda")[None]
        query = s["query"][q0:q0 + q].double()
        if op == "latent-attn":
            pages = s["block_table"][r, :-(-n // BLOCK)].long()
            c = s["cache"][pages].reshape(-1, ROW)[:n].double()
            w = torch.einsum("qhd,nd->hqn", query, c) * s["scale"]
            w = torch.softmax(torch.where(limit[None], w, -math.inf), -1)
            parts.append(torch.einsum("hqn,nd->qhd", w, c[:, :LATENT]))
        else:
            out = torch.empty(q, case["heads"], VDIM, dtype=torch.float64, device="cuda")
            for h in range(case["heads"]):
                k = torch.cat([s["key"][k0:k0 + n, h], s["key_rope"][k0:k0 + n]], -1).double()
                w = torch.where(limit, query[:, h] @ k.T * s["scale"], -math.inf)
                out[:, h] = torch.softmax(w, -1) @ s["value"][k0:k0 + n, h].double()
            parts.append(out)
        q0, k0 = q0 + q, k0 + n
    return torch.cat(parts)
