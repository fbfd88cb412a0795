"""The operators of a cache of 8-bit integers: what is measured of each, its plain form and its exact value.

The cache holds a code a value and an fp32 scale for each block of 16 tokens, head and side (K, V).  ``store`` quantises
a step's keys and values into it and reads the requests back; ``qk-store`` does so behind the norm and rotation of the
heads; ``attn`` is causal attention over such a cache; ``gather`` reads requests back as bf16; ``copy`` copies blocks
with their scales.  Lengths are those of the engine steps that the benchmark names: small and large decode batches, and a
mixed step of decodes and a 2046-token prefill chunk.

Writing.  a = max |x| over the rows of one block, head and side that a step writes, s' = max(a / 127, 2^-60).  A block
whose first row is written takes the scale s = s', any other s = max(old scale, s'); rows that were there are
requantised when the scale grows, code = rint(code * old scale / s).  A new code is rint(x / s).  Both quotients are products with
r = 1 / s (32 bits) that are rounded once, to the code: x * r, and code * (old scale * r) with 32 bits in the bracket.
"""

import math

import torch

own = False

BLOCK = 16
LEAST = 2.0 ** -60                       # the smallest scale


# ---- cases -----------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 requests, most of them in the middle of a block
        {"name": "store-decode-64", "op": "store", "seqs": 64, "q_lo": 1, "q_hi": 1, "context": 47, "hkv": 8, "d": 128,
         "seed": 1},
        # a prefill step of four prompts of odd lengths, some behind a cached start
        {"name": "store-prompts-4", "op": "store", "seqs": 4, "q_lo": 1500, "q_hi": 2600, "context": 33, "hkv": 8,
         "d": 128, "seed": 2},
        # a handful of interactive requests, one new token each: latency
        {"name": "qk-store-decode-4", "op": "qk-store", "seqs": 4, "q_lo": 1, "q_hi": 1, "context": 127, "hq": 8,
         "hkv": 8, "d": 64, "rot": 64, "inter": False, "seed": 3},
        # a prefill chunk of a grouped-query model, q, k and v views of one fused projection
        {"name": "qk-store-chunk-2046", "op": "qk-store", "seqs": 1, "q_lo": 2046, "q_hi": 2046, "context": 100,
         "hq": 32, "hkv": 8, "d": 128, "rot": 128, "inter": False, "seed": 4},
        # four requests at the start of their answers: latency
        {"name": "attn-decode-4", "op": "attn", "kind": "uniform", "seqs": 4, "lo": 1, "hi": 128, "q": 1, "chunk": 0,
         "context": 0, "hq": 8, "hkv": 8, "d": 64, "seed": 5},
        # a decode batch of a small grouped-query model
        {"name": "attn-decode-64", "op": "attn", "kind": "uniform", "seqs": 64, "lo": 512, "hi": 2048, "q": 1,
         "chunk": 0, "context": 0, "hq": 32, "hkv": 4, "d": 64, "seed": 6},
        # a large decode batch of a model with a key head for every query head
        {"name": "attn-decode-256", "op": "attn", "kind": "lognormal", "seqs": 256, "lo": 16, "hi": 4096, "q": 1,
         "chunk": 0, "context": 0, "hq": 40, "hkv": 40, "d": 128, "seed": 7},
        # a mixed step: two decodes and a later chunk of a long prompt
        {"name": "attn-mixed-8190", "op": "attn", "kind": "uniform", "seqs": 2, "lo": 700, "hi": 1500, "q": 1,
         "chunk": 2046, "context": 6144, "hq": 32, "hkv": 8, "d": 128, "seed": 8},
        # the keys and values of a small batch, and of a large one
        {"name": "gather-4", "op": "gather", "kind": "uniform", "seqs": 4, "lo": 1, "hi": 128, "hkv": 8, "d": 64,
         "seed": 9},
        {"name": "gather-256", "op": "gather", "kind": "lognormal", "seqs": 256, "lo": 16, "hi": 4096, "hkv": 8,
         "d": 128, "seed": 10},
        # the last blocks of eight forks; and a beam search that copies whole answers
        {"name": "copy-8", "op": "copy", "pairs": 8, "hkv": 8, "d": 128, "seed": 11},
        {"name": "copy-4095", "op": "copy", "pairs": 4095, "hkv": 40, "d": 128, "seed": 12},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "qk-store", "attn", "attn", "gather", "copy"])
    hkv, d = rng.choice([1, 2, 3, 4, 8, 40]), rng.choice([64, 128])
    case = {"op": op, "hkv": hkv, "d": d, "seed": rng.randrange(1 << 20)}
    if op in ("store", "qk-store"):
        seqs = _log_int(rng, 1, 64)
        most = max(1, 8192 * 8 // (max(8, hkv) * seqs))
        hi = rng.choice([1, _log_int(rng, 1, most)])
        case.update(seqs=seqs, q_lo=rng.randint(1, hi), q_hi=hi, context=rng.randrange(0, min(128, most)))
        if op == "qk-store":
            case.update(hq=hkv * (1 if hkv == 40 else rng.choice([1, 3, 4, 8])), rot=rng.choice([16, d // 2, d]),
                        inter=rng.random() < 0.5)
            case["q_hi"] = max(1, min(hi, 2046 * 40 // (seqs * (case["hq"] + hkv))))
            case["q_lo"] = min(case["q_lo"], case["q_hi"])
    elif op == "attn":
        group = 1 if hkv == 40 else rng.choice([1, 3, 4, 8, 16])
        chunk = rng.choice([0, 0, _log_int(rng, 2, 2046)])
        seqs = _log_int(rng, 1, 128 if not chunk else 4)
        hi = _log_int(rng, 2, min(4096, 10 ** 9 // (seqs * hkv * d)))
        if chunk:
            group = min(group, max(1, 32 // hkv))
        case.update(kind=rng.choice(["uniform", "lognormal"]), seqs=seqs, q=rng.choice([1, 1, 2, 3]),
                    lo=rng.randint(1, hi), hi=hi, chunk=chunk,
                    context=rng.randrange(0, 6144 if hkv < 40 else 2000) if chunk else 0, hq=hkv * group)
    elif op == "gather":
        seqs = _log_int(rng, 1, 200)
        hi = _log_int(rng, 2, min(4096, 2 * 10 ** 8 // (seqs * hkv * d)))
        case.update(kind=rng.choice(["uniform", "lognormal"]), seqs=seqs, lo=rng.randint(1, hi), hi=hi)
    else:
        case["pairs"] = _log_int(rng, 1, 4095)
    return case


def _lengths(case):
    """The requests' lengths (uniform, or round(exp(N)) clipped, mean about 780): part of the case, not of the inputs."""
    g = torch.Generator().manual_seed(case["seed"])
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    if case["kind"] == "lognormal":
        x = torch.exp(torch.randn(n, generator=g, dtype=torch.float64) * 0.8 + math.log(800.0) - 0.32)
        return [int(v) for v in x.round().clamp(min(lo, hi), hi)]
    return [int(v) for v in torch.randint(lo, hi + 1, (n,), generator=g)]


def _requests(case):
    """[(new tokens, keys)] of the step: decodes, then the chunk where there is one."""
    if case["op"] in ("store", "qk-store"):
        g = torch.Generator().manual_seed(case["seed"])
        q = [int(v) for v in torch.randint(case["q_lo"], case["q_hi"] + 1, (case["seqs"],), generator=g)]
        c = [int(v) for v in torch.randint(0, case["context"] + 1, (case["seqs"],), generator=g)]
        return [(a, a + b) for a, b in zip(q, c)]
    lens = _lengths(case)
    if case["op"] == "gather":
        return [(n, n) for n in lens]
    reqs = [(min(case["q"], n), n) for n in lens]
    if case["chunk"]:
        reqs.append((case["chunk"], case["chunk"] + case["context"]))
    return reqs


def _pairs(reqs):
    return sum(q * (n - q) + q * (q + 1) // 2 for q, n in reqs)


def work(case):
    op, hkv, d = case["op"], case["hkv"], case["d"]
    side = hkv * d
    if op == "copy":
        return {"bytes": case["pairs"] * (4 * BLOCK * side + 16 * hkv + 16), "flops": 0}
    reqs = _requests(case)
    rows, keys = sum(q for q, _ in reqs), sum(n for _, n in reqs)
    blocks = sum(-(-n // BLOCK) for _, n in reqs)
    tables = 4 * blocks + 8 * len(reqs)
    back = keys * 6 * side + 8 * hkv * blocks + tables                      # read as codes, written as bf16
    if op == "gather":
        return {"bytes": back, "flops": 2 * keys * side}
    if op == "attn":
        hq = case["hq"]
        return {"bytes": keys * 2 * side + 8 * hkv * blocks + rows * 4 * hq * d + tables,
                "flops": 4 * d * hq * _pairs(reqs)}
    # every new value read once and its code written once, the scales of the blocks written to
    touched = sum((n - 1) // BLOCK - (n - q) // BLOCK + 1 for q, n in reqs)
    store = rows * (6 * side + 8) + 8 * hkv * touched
    if op == "store":
        return {"bytes": store + back, "flops": rows * 6 * side + 2 * keys * side}
    hq, rot = case["hq"], case["rot"]
    return {"bytes": store + back + rows * (4 * hq * d + 4 * rot + 8) + 4 * d,
            "flops": rows * ((hq + hkv) * (4 * d + 3 * rot) + 6 * side) + 2 * keys * side}


# ---- inputs ----------------------------------------------------------------------------------------------------

def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def _angles(rot, length):
    """fp32 [length, rot]: cosines, then sines, of position * 10000^(-2i / rot), made in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _cache(g, blocks, hkv, d):
    """Codes and scales as normal values of heads of several magnitudes leave them (largest code near 127)."""
    cache = torch.empty(blocks, hkv, 2, BLOCK, d, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 28) // (hkv * 2 * BLOCK * d))
    for b in range(0, blocks, step):
        part = cache[b:b + step]
        x = torch.randn(part.shape, generator=g, device="cuda", dtype=torch.float32).mul_(36.0).round_()
        part.copy_(x.clamp_(-127, 127))
    head = torch.exp(0.4 * torch.randn(1, hkv, 2, generator=g, device="cuda"))
    block = 0.9 + 0.2 * torch.rand(blocks, hkv, 2, generator=g, device="cuda")
    return cache, (head * block / 36.0).contiguous()


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
    op, s, hkv, d = case["op"], dict(case), case["hkv"], case["d"]
    if op == "copy":
        n = case["pairs"]
        s["cache"], s["scales"] = _cache(g, 2 * n + 1, hkv, d)
        order = torch.randperm(2 * n + 1, generator=g, device="cuda")
        s["mapping"] = torch.stack([order[:n], order[n:2 * n]], 1).contiguous()
        return s
    reqs = _requests(case)
    q, n = [a for a, _ in reqs], [b for _, b in reqs]
    rows, keys = sum(q), sum(n)
    s["max_q"], s["max_n"] = max(q), max(n)
    s["starts"], s["lens"], s["key_starts"] = _starts(q), torch.tensor(n, dtype=torch.int32, device="cuda"), _starts(n)
    # where each new token and each key stands in a padded [request, index] grid
    s["seq_of"] = torch.repeat_interleave(torch.arange(len(q), device="cuda"), torch.tensor(q, device="cuda"))
    s["at"] = torch.arange(rows, device="cuda") - s["starts"].long()[s["seq_of"]]
    s["key_seq"] = torch.repeat_interleave(torch.arange(len(n), device="cuda"), torch.tensor(n, device="cuda"))
    s["key_at"] = torch.arange(keys, device="cuda") - s["key_starts"].long()[s["key_seq"]]
    s["block_table"], blocks = _table(g, reqs)
    s["cache"], s["scales"] = _cache(g, blocks, hkv, d)
    if op == "attn":
        s["query"] = _normal(g, rows, case["hq"], d)
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty(rows, case["hq"], d, dtype=torch.bfloat16, device="cuda")
        return s
    s["key_out"] = torch.empty(keys, hkv, d, dtype=torch.bfloat16, device="cuda")
    s["value_out"] = torch.empty(keys, hkv, d, dtype=torch.bfloat16, device="cuda")
    if op == "gather":
        return s
    positions = s["at"] + (s["lens"].long() - torch.tensor(q, device="cuda"))[s["seq_of"]]
    s["slots"] = (s["block_table"].long()[s["seq_of"], positions // BLOCK] * BLOCK + positions % BLOCK).contiguous()
    hq = case.get("hq", 0)
    fused = _normal(g, rows, hq + 2 * hkv, d)
    s["query"], s["key"], s["value"] = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    if op == "qk-store":
        s["positions"], s["eps"] = positions.contiguous(), 1e-6
        s["wq"], s["wk"] = _normal(g, d, std=0.3) + 1, _normal(g, d, std=0.3) + 1
        s["table"] = _angles(case["rot"], s["max_n"])
        s["query_out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")
    return s


# ---- the operators ---------------------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_gather(s):
    import paged_kv_cache_111_gb300 as pkv
    pkv.kv_gather_int8(s["key_out"], s["value_out"], s["cache"], s["scales"], s["block_table"], s["lens"],
                       s["key_starts"], s["max_n"])
    return [s["key_out"], s["value_out"]]


def _own_store(s):
    import paged_kv_cache_111_gb300 as pkv
    pkv.kv_write_int8(s["cache"], s["scales"], s["key"], s["value"], s["slots"])
    return _own_gather(s) + [s["scales"]]


def _own_qk_store(s):
    import paged_kv_cache_111_gb300 as pkv
    pkv.qk_norm_rope_kv_write_int8(s["query_out"], s["cache"], s["scales"], s["query"], s["key"], s["value"], s["wq"],
                                   s["wk"], s["eps"], s["table"], s["positions"], s["slots"], interleaved=s["inter"])
    return _own_gather(s) + [s["scales"], s["query_out"]]


def _own_attn(s):
    import paged_kv_cache_111_gb300 as pkv
    if "workspace" not in s:
        n = pkv.paged_attn_workspace_size(s["lens"].shape[0], s["query"].shape[0], s["max_q"], s["max_n"],
                                          s["query"].shape[1], s["hkv"], s["d"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    pkv.paged_attn_int8(s["out"], s["query"], s["cache"], s["scales"], s["block_table"], s["lens"], s["starts"],
                        s["max_q"], s["max_n"], s["scale"], s["workspace"])
    pkv.paged_attn_combine(s["out"], s["workspace"])
    return s["out"]


def _own_copy(s):
    import paged_kv_cache_111_gb300 as pkv
    pkv.copy_blocks_int8(s["cache"], s["scales"], s["mapping"])
    return [s["cache"], s["scales"]]


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


def _values(s):
    """K and V of every request's tokens, fp32 [keys, Hkv, d]."""
    page, at = s["block_table"].long()[s["key_seq"], s["key_at"] // BLOCK], s["key_at"] % BLOCK
    return [s["cache"][page, :, side, at].float() * s["scales"][page, :, side, None] for side in (0, 1)]


def _plain_gather(s):
    return [x.bfloat16() for x in _values(s)]


def _plain_write(s, key, value):
    """key and value fp32 [T, Hkv, d], written to the step's slots."""
    block, at = s["slots"] // BLOCK, s["slots"] % BLOCK
    fresh_or_not, which = torch.unique(block, return_inverse=True)              # the blocks written to
    n, hkv, d = fresh_or_not.shape[0], key.shape[1], key.shape[2]
    new = torch.zeros(n, hkv, 2, BLOCK, d, device="cuda")
    new[which, :, 0, at], new[which, :, 1, at] = key, value
    written = torch.zeros(n, BLOCK, dtype=torch.bool, device="cuda")
    written[which, at] = True
    old = s["scales"][fresh_or_not]                                             # [n, Hkv, 2]
    least = (new.abs().amax((-1, -2)) * torch.tensor(1 / 127, device="cuda")).clamp_min(LEAST)
    fresh = written[:, 0, None, None]
    scale = torch.where(fresh, least, torch.maximum(old, least))
    r = torch.reciprocal(scale)
    kept = s["cache"][fresh_or_not].float()
    grown = (scale > old) & ~fresh
    # (products in 64 bits: they are exact there, and next to a border between codes the last bit decides)
    moved, made = (kept.double() * (old * r).double()[..., None, None], new.double() * r.double()[..., None, None])
    kept = torch.where(grown[..., None, None], moved.round().float(), kept)
    codes = torch.where(written[:, None, None, :, None], made.round().float(), kept)
    s["cache"][fresh_or_not] = codes.to(torch.int8)
    s["scales"][fresh_or_not] = scale


def _plain_store(s):
    _plain_write(s, s["key"].float(), s["value"].float())
    return _plain_gather(s) + [s["scales"]]


def _plain_qk_store(s):
    q = _turn(_rms(s["query"], s["wq"], s["eps"]), s["table"], s["positions"], s["rot"], s["inter"])
    k = _turn(_rms(s["key"], s["wk"], s["eps"]), s["table"], s["positions"], s["rot"], s["inter"])
    _plain_write(s, k, s["value"].float())
    return _plain_gather(s) + [s["scales"], q.bfloat16()]


def _padded(s, x, seq, at, length):
    y = torch.zeros((s["lens"].shape[0], length) + tuple(x.shape[1:]), dtype=torch.float32, device="cuda")
    y[seq, at] = x.float()
    return y


def _hidden(s):
    """[request, query, key]: keys after the query's own position, and those past the request's end."""
    n, q = s["lens"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    last = (n - q)[:, None] + torch.arange(s["max_q"], device="cuda")
    return torch.arange(s["max_n"], device="cuda")[None, None] > torch.minimum(last, n[:, None] - 1)[:, :, None]


def _plain_attn(s):
    hkv, d, group = s["hkv"], s["d"], s["hq"] // s["hkv"]
    q = _padded(s, s["query"], s["seq_of"], s["at"], s["max_q"])                    # [S, Q, Hq, d]
    k, v = (_padded(s, x, s["key_seq"], s["key_at"], s["max_n"]).transpose(1, 2) for x in _values(s))
    b, m = q.shape[:2]
    q = q.view(b, m, hkv, group, d).transpose(1, 2).reshape(b, hkv, m * group, d)
    scores = torch.matmul(q, k.transpose(2, 3)).view(b, hkv, m, group, -1)
    scores *= s["scale"]
    scores.masked_fill_(_hidden(s)[:, None, :, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True)
    p = scores.exp_()
    p /= p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hkv, m * group, -1), v).view(b, hkv, m, group, d).transpose(1, 2)
    return o[s["seq_of"], s["at"]].reshape(-1, s["hq"], d).bfloat16()


def _plain_copy(s):
    source, destination = s["mapping"][:, 0], s["mapping"][:, 1]
    s["cache"][destination] = s["cache"][source]
    s["scales"][destination] = s["scales"][source]
    return [s["cache"], s["scales"]]


_own = {"store": _own_store, "qk-store": _own_qk_store, "attn": _own_attn, "gather": _own_gather, "copy": _own_copy}
_plain = {"store": _plain_store, "qk-store": _plain_qk_store, "attn": _plain_attn, "gather": _plain_gather,
          "copy": _plain_copy}


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
    op, s = case["op"], prepare(case, seed)
    if op == "copy":
        scales = s["scales"].double()
        scales[s["mapping"][:, 1]] = scales[s["mapping"][:, 0]]
        return [None, scales]                              # copied bits
    reqs, hkv, d = _requests(case), case["hkv"], case["d"]
    codes, scales = s["cache"], s["scales"].double()
    pages = [s["block_table"][r, :-(-n // BLOCK)].long() for r, (_, n) in enumerate(reqs)]

    def read(r, n):
        """K and V of a request as they stand, 64 bits, [n, Hkv, d] each."""
        c = codes[pages[r]].double() * scales[pages[r]][..., None, None]
        return [c[:, :, side].transpose(1, 2).reshape(-1, hkv, d)[:n] for side in (0, 1)]

    if op == "gather":
        both = [read(r, n) for r, (_, n) in enumerate(reqs)]
        return [torch.cat([b[0] for b in both]), torch.cat([b[1] for b in both])]
    if op in ("store", "qk-store"):
        key, value = s["key"].double(), s["value"].double()
        if op == "qk-store":
            key = _spin(_normed(s["key"], s["wk"], s["eps"]), s, case["rot"])
        keys, values, q0 = [], [], 0
        for r, (q, n) in enumerate(reqs):
            x = torch.stack(read(r, n), 2)                                       # [n, Hkv, 2, d]
            blocks, c = pages[r].shape[0], n - q
            x[c:] = torch.stack([key[q0:q0 + q], value[q0:q0 + q]], 2)
            x = torch.cat([x, torch.zeros(blocks * BLOCK - n, hkv, 2, d, dtype=x.dtype, device="cuda")])
            new = torch.arange(blocks * BLOCK, device="cuda") >= c
            x, new = x.view(blocks, BLOCK, hkv, 2, d), new.view(blocks, BLOCK, 1, 1, 1)
            largest = (x.abs() * new).amax((1, 4))                               # [blocks, Hkv, 2]
            touched = new.any(1).view(blocks, 1, 1)
            want = (largest / 127).clamp_min(LEAST)
            was = scales[pages[r]]
            scale = torch.where(touched, torch.where(new[:, 0].view(blocks, 1, 1), want, torch.maximum(was, want)), was)
            scales[pages[r]] = scale
            wide = scale[:, None, :, :, None]
            x = (x / wide).round() * wide
            x = x.reshape(-1, hkv, 2, d)[:n]
            keys.append(x[:, :, 0]), values.append(x[:, :, 1])
            q0 += q
        out = [torch.cat(keys), torch.cat(values), scales]
        return out + [_spin(_normed(s["query"], s["wq"], s["eps"]), s, case["rot"])] if op == "qk-store" else out
    # attention: one request and key head after the other
    hq = case["hq"]
    if 4 * d * hq * sum(q * n for q, n in reqs) > 6e12 or hkv * len(reqs) > 20000:
        return None                                        # 64-bit products of over about ten seconds
    parts, q0, group = [], 0, hq // hkv
    for r, (q, n) in enumerate(reqs):
        limit = torch.arange(n - q, n, device="cuda")[:, None] >= torch.arange(n, device="cuda")[None]
        k, v = read(r, n)
        query = s["query"][q0:q0 + q].double()
        out = torch.empty(q, hq, d, dtype=torch.float64, device="cuda")
        for h in range(hkv):
            mine = query[:, h * group:(h + 1) * group]
            w = torch.einsum("qgd,nd->gqn", mine, k[:, h]) * s["scale"]
            w = torch.softmax(torch.where(limit[None], w, -math.inf), -1)
            out[:, h * group:(h + 1) * group] = torch.einsum("gqn,nd->qgd", w, v[:, h])
        parts.append(out)
        q0 += q
    return torch.cat(parts)
