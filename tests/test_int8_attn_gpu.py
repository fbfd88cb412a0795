"""Attention over an int8 cache on the GPU, against 64 bits over the values that codes and scales stand for."""

import pytest
import torch

import int8_ref as ref
import latent_ref
import paged_kv_cache_111_gb300 as pkv

pytestmark = pytest.mark.gpu
BLOCK = 16


@pytest.fixture(autouse=True, scope="module")
def built():
    from paged_kv_cache_111_gb300 import _build
    _build.build()


def batch(reqs, hq, hkv, d, seed=0, spread=0.4, spare=3):
    """reqs: [(new tokens, keys)] -> a dict of device tensors; tables hold -1 past a request's pages, unused blocks have
    NaN scales, and rows behind a request's last key any code."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // BLOCK) for _, n in reqs]
    blocks = sum(counts) + spare
    codes = (torch.randn(blocks, hkv, 2, BLOCK, d, generator=g) * 36).round().clamp(-127, 127).to(torch.int8)
    scales = torch.exp(torch.randn(blocks, hkv, 2, generator=g) * spread) / 36
    order = torch.randperm(blocks, generator=g).tolist()
    tables = torch.full((len(reqs), max(counts + [1]) + 1), -1, dtype=torch.int32)
    for r, (_, n) in enumerate(reqs):
        for b in range(counts[r]):
            tables[r, b] = order.pop()
        if n % BLOCK:
            codes[tables[r, counts[r] - 1].long(), :, :, n % BLOCK:] = -128
    scales[order] = float("nan")
    q = [a for a, _ in reqs]
    T = sum(q)
    s = dict(cache=codes.cuda(), scales=scales.cuda(), tables=tables.cuda(), lens=[n for _, n in reqs],
             qsl=[sum(q[:i]) for i in range(len(q) + 1)], scale=d ** -0.5,
             query=torch.randn(T, hq, d, generator=g).bfloat16().cuda())
    s["max_q"], s["max_n"] = max(q + [0]), max(s["lens"] + [0])
    return s


def run(s, num_splits=0, ws=None, out=None, max_q=None, max_n=None, status=0, query=None, tokens=None):
    q = s["query"] if query is None else query
    T, hq, d = q.shape
    hkv = s["cache"].shape[1]
    max_q, max_n = max_q or s["max_q"], max_n or s["max_n"]
    if ws is None:
        n = pkv.paged_attn_workspace_size(len(s["lens"]), T, max_q, max_n, hq, hkv, d)
        ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((T, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    qsl = torch.tensor(s["qsl"], dtype=torch.int32, device="cuda")
    pkv.paged_attn_int8(out, q, s["cache"], s["scales"], s["tables"], lens, qsl, max_q, max_n, s["scale"], ws,
                        num_splits=num_splits)
    pkv.paged_attn_combine(out, ws)
    torch.cuda.synchronize()
    assert pkv.workspace_status(ws) == status
    return out


def check(s, out, what=""):
    want, bound = ref.attention(s["query"], s["cache"], s["scales"], s["tables"], s["lens"], s["qsl"], s["scale"])
    ref.check(out, want, bound, what)


HEADS = [(1, 1, 64), (8, 8, 128), (8, 1, 128), (32, 4, 64), (6, 2, 128), (16, 1, 64), (12, 4, 64), (40, 40, 128)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("lens", [[1], [15, 16, 17], [31, 1, 33, 700, 128], [4096, 5]])
def test_decode(hq, hkv, d, lens):
    s = batch([(1, n) for n in lens], hq, hkv, d, seed=len(lens))
    check(s, run(s))


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("reqs", [[(2, 2), (2, 40)], [(3, 17), (1, 100), (4, 260)], [(5, 5), (7, 333), (16, 16), (9, 30)]])
def test_a_few_tokens_each(hq, hkv, d, reqs):
    s = batch(reqs, hq, hkv, d, seed=3)
    check(s, run(s))


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (8, 8, 128), (8, 1, 128), (32, 4, 64), (6, 2, 128), (16, 1, 64), (5, 1, 128)])
@pytest.mark.parametrize("reqs", [[(65, 65)], [(100, 230), (1, 50)], [(300, 300), (70, 1000), (1, 16), (2, 130)],
                                  [(513, 640)]])
def test_chunks(hq, hkv, d, reqs):
    s = batch(reqs, hq, hkv, d, seed=5)
    check(s, run(s))


@pytest.mark.parametrize("hq,hkv,d", [(40, 40, 128), (80, 40, 64), (60, 60, 128)])
@pytest.mark.parametrize("reqs", [[(700, 800), (300, 300)], [(129, 129), (256, 1000), (257, 300), (1, 77)]])
def test_more_work_items_than_ctas(hq, hkv, d, reqs):
    s = batch(reqs, hq, hkv, d, seed=6)
    check(s, run(s))


@pytest.mark.parametrize("q", [17, 65, 128, 129, 256, 300])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (5, 1), (2, 2)])
def test_a_few_work_items_of_many_keys(q, hq, hkv):
    """Items cut along their keys, down to a few key tiles a piece, and cuts on the causal diagonal."""
    for n in (q, q + 1, q + 500, q + 1900, 9000):
        s = batch([(q, n)], hq, hkv, 128, seed=n)
        check(s, run(s), str(n))
    s = batch([(q, 5000), (1, 300), (q + 40, q + 40), (q + 3, 700)], hq, hkv, 64, seed=q)
    check(s, run(s))


@pytest.mark.parametrize("hq,hkv,d,reqs", [
    (40, 40, 128, [(1100, 6000)]),                            # 200 items, some of them in three runs
    (40, 40, 64, [(900, 5000), (300, 300), (1, 40)]),
    (16, 1, 64, [(2700, 4000)]),                              # 169 tiles of one kv head
    (8, 1, 128, [(2046, 3500), (700, 6000), (1, 50)]),
    (4, 2, 128, [(5000, 5200)] + [(1, 77)] * 3)])
def test_equal_runs_of_more_items_than_ctas(hq, hkv, d, reqs):
    s = batch(reqs, hq, hkv, d, seed=7)
    check(s, run(s))


def test_cut_items_with_blocks_without_a_scale():
    s = batch([(200, 6000)], 4, 2, 64, seed=4)
    want, bound = ref.attention(s["query"], s["cache"], s["scales"], s["tables"], s["lens"], s["qsl"], s["scale"])
    for page in (3, 200, 370):                          # in pieces that all rows see; one that the last rows see
        scales = s["scales"].clone()
        s["scales"][s["tables"][0, page].long(), 1] = float("nan")
        out = run(s)
        sees = torch.arange(5800, 6000, device="cuda") >= page * BLOCK
        assert torch.isnan(out[sees][:, 2:].float()).all()
        ref.check(out[:, :2], want[:, :2], bound[:, :2])
        ref.check(out[~sees], want[~sees], bound[~sees])
        s["scales"] = scales


@pytest.mark.parametrize("num_splits", [1, 2, 3, 7, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_splits(num_splits, d):
    s = batch([(1, 900), (2, 33), (1, 1), (1, 5000)], 8, 4, d, seed=2)
    check(s, run(s, num_splits=num_splits), str(num_splits))


@pytest.mark.parametrize("num_splits", [0, 1, 5])
@pytest.mark.parametrize("reqs", [[(1, 300), (1, 17)], [(2, 900), (1, 33), (2, 2)]])
def test_sixteen_rows_of_128_dims(num_splits, reqs):
    """Planned by the decode kernel itself (no splits given), and by the plan."""
    s = batch(reqs, 16 // reqs[0][0], 1, 128, seed=14)
    check(s, run(s, num_splits=num_splits))


def test_many_requests():
    g = torch.Generator().manual_seed(0)
    for S in (33, 65, 300, 1100):
        lens = torch.randint(1, 200, (S,), generator=g).tolist()
        s = batch([(1, n) for n in lens], 4, 2, 64, seed=S)
        check(s, run(s), str(S))


def test_long_request_and_window_borders():
    # pages of a chunk beyond one and two windows of 32 block ids
    for n in (16 * 31, 16 * 32 + 1, 16 * 33, 16 * 64, 16 * 65 + 3, 16 * 100):
        s = batch([(1, n)], 2, 2, 128, seed=n)
        check(s, run(s, num_splits=1), str(n))
    s = batch([(1, 40000), (1, 3)], 4, 2, 64)
    check(s, run(s))


@pytest.mark.parametrize("reqs", [[(1, 300), (3, 40)], [(200, 333)]])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 4.0])
def test_scales_of_the_softmax(reqs, scale):
    s = batch(reqs, 8, 2, 64, seed=1)
    s["scale"] = scale
    check(s, run(s))


@pytest.mark.parametrize("reqs", [[(1, 1300), (3, 40), (1, 16)], [(200, 1333), (33, 33)]])
@pytest.mark.parametrize("d", [64, 128])
def test_blocks_of_very_different_scales(reqs, d):
    s = batch(reqs, 8, 4, d, seed=1)
    g = torch.Generator().manual_seed(9)
    s["scales"][:, :, 1] = torch.exp2(torch.randint(-40, 40, s["scales"][:, :, 1].shape, generator=g).float()).cuda()
    # bounds are of a row's sums, so a row whose weight lies in small blocks has a small bound: each is held to its own
    check(s, run(s))
    s["scales"][:, :, 0] = torch.exp2(torch.randint(-20, -3, s["scales"][:, :, 0].shape, generator=g).float()).cuda()
    check(s, run(s))
    s["scales"][:, :, 1] = 0.0                                          # values of nothing
    out = run(s)
    assert (out.float().abs() < 1e-15).all()
    s = batch(reqs, 8, 4, d, seed=1)
    pick = torch.rand(s["scales"].shape[0], generator=g) < 0.5          # some blocks of zeros
    s["scales"][pick.cuda(), :, 1] = 2.0 ** -60
    check(s, run(s))
    s["scales"][pick.cuda(), :, 0] = 0.0
    check(s, run(s))


@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("reqs", [[(1, 100)], [(4, 36)], [(200, 300)], [(40, 300)]])
def test_a_block_without_a_scale(side, reqs):
    """Rows that see a key of it are NaN, the others as if it were not there."""
    s = batch(reqs, 4, 2, 64, seed=4)
    q, n = reqs[0]
    last = s["tables"][0, -(-n // BLOCK) - 1].long()
    page0 = (-(-n // BLOCK) - 1) * BLOCK
    want, bound = ref.attention(s["query"], s["cache"], s["scales"], s["tables"], s["lens"], s["qsl"], s["scale"])
    s["scales"][last, 1, side] = float("nan")
    out = run(s)
    sees = torch.arange(n - q, n) >= page0                              # position of each query
    assert torch.isnan(out[sees.cuda()][:, 2:].float()).all()
    ref.check(out[:, :2], want[:, :2], bound[:, :2])
    ref.check(out[~sees.cuda()], want[~sees.cuda()], bound[~sees.cuda()])


def test_large_and_small_queries():
    s = batch([(1, 200), (2, 64), (100, 120)], 8, 2, 128, seed=6)
    base = s["query"].clone()
    for f in (2.0 ** -100, 2.0 ** 60, 2.0 ** -130):
        s["query"] = (base.float() * f).bfloat16()
        s["scale"] = 0.09 / f if f > 2.0 ** -120 else 1e30
        check(s, run(s), str(f))
    s["query"] = base.clone()
    s["query"][:, ::2] = 0
    s["scale"] = 0.09
    check(s, run(s))


def test_rows_of_nobody_and_empty_requests():
    s = batch([(0, 20), (1, 30), (0, 0), (70, 70), (0, 5)], 4, 2, 64, seed=7)
    g = torch.Generator().manual_seed(3)
    s["query"] = torch.cat([s["query"], torch.randn(5, 4, 64, generator=g).bfloat16().cuda()])
    out = torch.full(s["query"].shape, 3.0, dtype=torch.bfloat16, device="cuda")
    run(s, out=out, max_n=96)
    check(s, out)
    assert (out[71:] == 3).all()


def test_bad_requests_and_pages():
    s = batch([(1, 40), (1, 50), (1, 30)], 4, 2, 64, seed=7)
    want, bound = ref.attention(s["query"], s["cache"], s["scales"], s["tables"], s["lens"], s["qsl"], s["scale"])
    s["lens"][1] = 1000                                                 # longer than its bound
    out = run(s, max_n=64, status=8)
    ref.check(out[[0, 2]], want[[0, 2]], bound[[0, 2]])
    assert torch.isnan(out[1].float()).all()
    # a page outside the cache reads as zeros
    s["lens"][1] = 50
    s["tables"][1, 1] = 1 << 20
    out = run(s, status=7)
    ref.check(out[[0, 2]], want[[0, 2]], bound[[0, 2]])
    assert torch.isfinite(out.float()).all()


def test_strided_query_other_stream_and_bounds_that_are_loose():
    s = batch([(1, 100), (3, 60), (90, 140)], 8, 2, 128, seed=8)
    wide = torch.randn(94, 13, 128, device="cuda").bfloat16()
    wide[:, :8] = s["query"]
    check(s, run(s, query=wide[:, :8]))
    check(s, run(s, max_q=94, max_n=144))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    n = pkv.paged_attn_workspace_size(3, 94, s["max_q"], s["max_n"], 8, 2, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.empty(94, 8, 128, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    qsl = torch.tensor(s["qsl"], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    pkv.paged_attn_int8(out, s["query"], s["cache"], s["scales"], s["tables"], lens, qsl, s["max_q"], s["max_n"],
                        s["scale"], ws, stream=stream)
    pkv.paged_attn_combine(out, ws, stream=stream)
    stream.synchronize()
    check(s, out)


def test_the_same_twice_and_a_workspace_through_other_calls():
    a = batch([(1, 700), (1, 90), (2, 300)], 8, 2, 64, seed=8)
    b = batch([(130, 400), (1, 33)], 8, 2, 64, seed=9)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    one = run(a, ws=ws)
    check(b, run(b, ws=ws))
    assert torch.equal(one, run(a, ws=ws))
    check(a, one)


@pytest.mark.parametrize("reqs", [[(1, 64), (1, 300), (1, 17)], [(1, 64), (150, 300)]])
def test_a_step_in_a_graph(reqs):
    """Norm, rotation and write, attention, merge and reading back, captured once and replayed on other inputs."""
    hq, hkv, d = 8, 2, 128
    s = batch(reqs, hq, hkv, d, seed=10)
    T = s["query"].shape[0]
    g = torch.Generator().manual_seed(1)
    fused = torch.randn(T, hq + 2 * hkv, d, generator=g).bfloat16().cuda()
    wq = (torch.randn(d, generator=g) * 0.3 + 1).bfloat16().cuda()
    positions, slots = [], []
    for r, (q, n) in enumerate(reqs):
        positions += list(range(n - q, n))
    seq = [r for r, (q, _) in enumerate(reqs) for _ in range(q)]
    tables = s["tables"].cpu()
    slots = [int(tables[r, p // BLOCK]) * BLOCK + p % BLOCK for r, p in zip(seq, positions)]
    positions, slots = torch.tensor(positions).cuda(), torch.tensor(slots).cuda()
    table = latent_ref.angles(d, 512).cuda()
    lens = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    qsl = torch.tensor(s["qsl"], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0] + s["lens"], device="cuda").cumsum(0).to(torch.int32)
    ws = torch.empty(pkv.paged_attn_workspace_size(len(reqs), T, s["max_q"], s["max_n"], hq, hkv, d), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    kv = [torch.empty(sum(s["lens"]), hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    query = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")

    def step():
        pkv.qk_norm_rope_kv_write_int8(query, s["cache"], s["scales"], fused[:, :hq], fused[:, hq:hq + hkv],
                                       fused[:, hq + hkv:], wq, wq, 1e-6, table, positions, slots)
        pkv.paged_attn_int8(out, query, s["cache"], s["scales"], s["tables"], lens, qsl, s["max_q"], s["max_n"],
                            s["scale"], ws)
        pkv.paged_attn_combine(out, ws)
        pkv.kv_gather_int8(*kv, s["cache"], s["scales"], s["tables"], lens, starts, s["max_n"])

    def look(what):
        torch.cuda.synchronize()
        assert pkv.workspace_status(ws) == 0
        s["query"] = query
        check(s, out, what)
        at = 0
        for r, n in enumerate(s["lens"]):
            for got, want in zip(kv, ref.rows_of(s["cache"], s["scales"], s["tables"][r], n)):
                assert torch.equal(got[at:at + n], want.float().bfloat16()), what
            at += n

    step()
    look("eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        fused.copy_(torch.randn(fused.shape, generator=g) * (k + 1))
        graph.replay()
        look(f"replay {k}")


def test_graphs_of_several_steps_with_one_workspace():
    """Decodes, whole chunks, and chunks cut along their keys, replayed in turn with nothing waited for between."""
    steps = [batch([(1, 64), (1, 300), (1, 17)], 8, 2, 128, seed=11), batch([(150, 300), (1, 40)], 8, 2, 128, seed=12),
             batch([(40, 6000), (1, 5)], 8, 2, 128, seed=13)]
    ws = torch.empty(max(pkv.paged_attn_workspace_size(len(s["lens"]), s["query"].shape[0], s["max_q"], s["max_n"], 8, 2,
                                                       128) for s in steps), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for s in steps:
        lens, qsl = (torch.tensor(s[k], dtype=torch.int32, device="cuda") for k in ("lens", "qsl"))
        out = torch.empty_like(s["query"])
        s["keep"] = lens, qsl

        def step():
            pkv.paged_attn_int8(out, s["query"], s["cache"], s["scales"], s["tables"], lens, qsl, s["max_q"], s["max_n"],
                                s["scale"], ws)
            pkv.paged_attn_combine(out, ws)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append(graph)
        outs.append(out)
    for order in ((0, 1, 2), (2, 0, 2, 1, 0), (1, 1, 2, 2, 0)):
        for out in outs:
            out.fill_(float("nan"))
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        assert pkv.workspace_status(ws) == 0
        for s, out in zip(steps, outs):
            check(s, out, str(order))


def test_far_blocks():
    """Pages past 2^32 bytes of the cache."""
    blocks, hkv, d = 30000, 40, 128
    cache = torch.zeros(blocks, hkv, 2, BLOCK, d, dtype=torch.int8, device="cuda")
    s = batch([(1, 100), (20, 60)], 40, hkv, d, seed=3)
    far = torch.arange(blocks - s["cache"].shape[0], blocks, device="cuda")
    cache[far] = s["cache"]
    scales = torch.zeros(blocks, hkv, 2, device="cuda")
    scales[far] = s["scales"]
    s["cache"], s["scales"] = cache, scales
    s["tables"] = torch.where(s["tables"] >= 0, s["tables"] + int(far[0]), s["tables"])
    check(s, run(s))
