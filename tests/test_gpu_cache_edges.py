"""Attention over a paged cache where it could go wrong, for every number of query rows that has a kernel of its own
(up to 8, 16, 32 with codes, 128, more) and every padded width: values that are not finite, queries and scales of all
sizes, sequences that end in every place of a tile, pools larger than 4 GiB, the same sequence twice."""

import numpy as np
import pytest

from cache_util import NAMES, Tables, finish, i32, numbers
from gpu_util import lib, need_gpu
from test_gpu_cache_attention import Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROWS = {"8": (2, 4), "16": (4, 4), "30": (6, 5), "96": (12, 8), "240": (30, 8)}  # nodes, group
KINDS = [("bf16", "bf16", 64), ("f16", "f16", 128), ("e4m3", "bf16", 96), ("i8", "f16", 256), ("bf16", "bf16", 192),
         ("e4m3", "f16", 128), ("i8", "bf16", 64)]


def plant(c, value, node, where):
    """value into a node's keys and values, of all requests: one place of a row, or its scales."""
    t = c.t
    for i, s in enumerate(c.seq):
        x = int(t.length[s]) - int(c.start[i + 1] - c.start[i]) + node
        for part in (0, 1):
            pool, scale = c.view(part)
            at = t.table[s, x // t.T], x % t.T
            if scale is not None and (c.kind == "i8" or where < 0):
                scale[at] = value
            else:
                pool[at][:, where] = value


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kind,q,width", KINDS)
def test_values_that_are_not_finite(kind, q, width, rows):
    nodes, group = ROWS[rows]
    c = Case(kind, q, 1, 16, 1, group, width, [(200, nodes), (64 - nodes // 2, nodes)], "tree", seed=nodes)
    plant(c, float("nan"), nodes - 1, 3)
    if kind != "e4m3":  # which has no infinities; its scales have
        plant(c, -float("inf"), nodes // 2, width - 1)
    else:
        plant(c, float("inf"), nodes // 2, -1)
    out, _ = c.run()
    if kind != "e4m3":  # (of which some cases have NaN among the codes that all rows see)
        assert torch.isfinite(out[c.start[0]].float()).all()  # the root sees neither


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("q,width", [("bf16", 96), ("f16", 128), ("bf16", 256)])
def test_nan_codes_among_clean_ones(q, width, rows):
    nodes, group = ROWS[rows]
    c = Case("e4m3", q, 1, 16, 1, group, width, [(200, nodes), (64 - nodes // 2, nodes)], "tree", seed=nodes)
    for pool in c.pools:
        pool.copy_(torch.nan_to_num(pool.float()).to(pool.dtype))
    plant(c, float("nan"), nodes - 1, 3)
    plant(c, float("inf"), nodes // 2, -1)
    out, _ = c.run()
    assert torch.isfinite(out[c.start[0]].float()).all()  # the root sees neither


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kind,q,width", [k for k in KINDS if k[0] in ("e4m3", "i8")])
def test_queries_and_scales_of_all_sizes(kind, q, width, rows):
    """Codes' queries and weights are f16 inside. Scales of 2^-60 to 2^60, whose keys meet queries of the inverse
    size (of 2^-12 to 2^12 in f16), rows of values much smaller than their largest, rows of zeros."""
    nodes, group = ROWS[rows]
    for power in (-60, 60) if q == "bf16" else (-9, 9):
        c = Case(kind, q, 1, 16, 1, group, width, [(150, nodes), (30, nodes)], "tree", seed=nodes)
        c.scales[0] *= 2.0**power
        c.scales[1] *= 2.0 ** (-power if q == "bf16" else 0)
        x = c.q.float() * 2.0**-power
        x[1::3] *= torch.from_numpy(2.0 ** -np.random.default_rng(2).integers(0, 9, x[1::3].shape)).float()
        x[2::7] = 0
        c.q = x.to(NAMES[q])
        c.run()


@pytest.mark.parametrize("rows", ROWS)
def test_infinite_queries(rows):
    """A query with an infinity has scores that are infinite or no numbers; its neighbours do not notice."""
    nodes, group = ROWS[rows]
    for kind, q, width in (("e4m3", "bf16", 128), ("bf16", "bf16", 64)):
        c = Case(kind, q, 1, 16, 1, group, width, [(90, nodes)], None)
        c.q[1, 0, 5], c.q[1, group - 1, 7] = float("inf"), float("nan")
        c.run()


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("width", [64, 128, 256])
def test_an_infinite_query_and_a_large_one(rows, width):
    """All scores of a row are minus infinity, by one infinite value of its query; another one, which f16 would not
    hold, does not make them anything else."""
    nodes, group = ROWS[rows]
    c = Case("e4m3", "bf16", 1, 16, 1, group, width, [(90, nodes)], None)
    c.pools[0][..., 5] = -1.0
    c.q[1, 0, 5], c.q[1, 0, 9] = float("inf"), 1e5
    out, lse = c.run()
    assert (out[1, 0] == 0).all() and lse[1, 0] == -float("inf")


def test_lengths_of_2_31_are_refused():
    """A sequence's length as it may not be, with a table that would have room for it (pages of 2^23 tokens)."""
    need_gpu()
    db = lib()
    pool = torch.zeros((2, 1 << 23, 1, 16), dtype=torch.int8, device="cuda")
    scale = torch.zeros((2, 1 << 23, 1), device="cuda")
    t = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    refs, free = torch.ones(2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    tabs = db.PageTables(torch.zeros((1, 512), dtype=torch.int32, device="cuda"), t(-(1 << 31)), refs, free, 1 << 23)
    layer = dict(k_pool=pool, v_pool=pool.clone(), k_scale=scale, v_scale=scale.clone())
    q = torch.zeros((1, 1, 16), dtype=torch.bfloat16, device="cuda")
    out, status = torch.full_like(q, 7), torch.zeros(1, dtype=torch.uint8, device="cuda")
    ws = db.workspace(db.cache_attention_workspace_size(1, 1, 1, 16, 1))
    for call in (lambda: db.cache_attention(tabs, t(0), t(0, 1), q, out=out, ws=ws, max_tokens=1, status=status, **layer),
                 lambda: db.cache_write(tabs, t(0), t(0, 1), q, q, status=status, **layer),
                 lambda: db.cache_read(tabs, t(0), t(0, 1), out, out.clone(), status=status, **layer)):
        status.zero_()
        call()
        finish()
        assert status.item() == 1 and (out == 7).all()


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kind,q,width", [("bf16", "bf16", 128), ("e4m3", "bf16", 112)])
def test_every_end_of_a_tile(kind, q, width, rows):
    nodes, group = ROWS[rows]
    before = [0, 1, 14, 15, 16, 17, 31, 33, 47, 48, 62, 63, 64, 65, 79, 127, 128, 129]
    Case(kind, q, 2, 5, 2, group, width, [(b, nodes) for b in before] + [(100, 0)], "random").run()
    Case(kind, q, 1, 24, 1, group, width, [(b, 1 + b % nodes) for b in before], None).run()


@pytest.mark.parametrize("rows", ROWS)
def test_a_zero_or_negative_scale(rows):
    nodes, group = ROWS[rows]
    for scale in (0.0, -0.125):
        for kind in ("f16", "i8"):
            Case(kind, "f16", 1, 16, 2, group, 64, [(150, nodes), (3, nodes)], "tree", scale=scale).run()


def test_the_same_sequence_twice():
    """Reading calls may name a sequence in two requests."""
    c = Case("bf16", "bf16", 1, 16, 2, 4, 64, [(100, 5), (40, 5)], "tree")
    c.seq[1] = c.seq[0]
    c.run()


def test_a_workspace_for_more_tokens_serves_less():
    need_gpu()
    db = lib()
    big = Case("e4m3", "bf16", 1, 16, 2, 8, 128, [(500, 40)], None)
    ws = big.workspace(db)
    for nodes in (40, 1, 2, 4, 12, 40):
        c = Case("e4m3", "bf16", 1, 16, 2, 8, 128, [(500, nodes), (64, nodes)], None)
        if nodes == 40:
            c = Case("e4m3", "bf16", 1, 16, 2, 8, 128, [(500, nodes)], None)
        out, lse = torch.full_like(c.q, 7.0).cuda(), torch.full(c.q.shape[:2], 7.0, device="cuda")
        c.call(db, c.t.device(), ws, c.device(), out, lse)
        finish()
        b, want = c.oracle()
        c.check(out, lse, b, want)


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_pools_larger_than_4_gib(kind):
    """Pages whose bytes, and (i8) whose scales, begin behind 2^32: written, read, attended to, kept."""
    need_gpu()
    db = lib()
    rng = np.random.default_rng(9)
    heads, width, T = 2, 64, 16
    page = heads * width * T * (2 if kind == "bf16" else 1)
    gap = 1 << 20  # bytes from page to page; the pool is a view of a larger one
    pages = (1 << 33) // gap
    store = [torch.empty((pages, gap), dtype=torch.uint8, device="cuda") for _ in range(2)]
    dtype = NAMES[kind]
    pools = [s[:, :page].view(dtype).view(pages, T, heads, width) if s[:, :page].is_contiguous() else
             torch.as_strided(s.view(dtype), (pages, T, heads, width),
                              (gap // dtype.itemsize, heads * width, width, 1)) for s in store]
    scales = [None, None] if kind == "bf16" else [
        torch.as_strided(torch.empty(pages * (gap // 4), device="cuda"), (pages, T, heads), (gap // 4, heads, 1)) for _ in range(2)]
    t = Tables(rng, [70, 33], T)
    t.table = np.where(t.table >= 0, pages - 1 - 3 * t.table, -1).astype(np.int32)  # the last ones
    t.n_pages = pages
    tabs = t.device()
    seq, start = i32([0, 1]), i32([0, 70, 103])
    rows = [torch.from_numpy(rng.standard_normal((103, heads, width)).astype(np.float32)).cuda().bfloat16() for _ in range(2)]
    layer = dict(k_pool=pools[0], v_pool=pools[1], k_scale=scales[0], v_scale=scales[1])
    db.cache_write(tabs, seq, start, *rows, **layer)
    back = [torch.zeros_like(rows[0], dtype=torch.float32) for _ in range(2)]
    db.cache_read(tabs, seq, start, *back, **layer)
    finish()
    for a, b in zip(rows, back):
        x = numbers(a)
        step = 0 if kind == "bf16" else np.abs(x).max(-1, keepdims=True) / 254 + np.abs(x) * 2.0**-21
        assert (np.abs(numbers(b) - x) <= step).all()
    # a single token of each, over what was read back
    q = torch.from_numpy(rng.standard_normal((2, heads, width)).astype(np.float32)).cuda().bfloat16()
    out = torch.zeros_like(q)
    ws = db.workspace(db.cache_attention_workspace_size(2, heads, heads, width, 1))
    db.cache_attention(tabs, seq, i32([0, 1, 2]), q, out=out, ws=ws, max_tokens=1, **layer)
    finish()
    for i, (a, e) in enumerate(((0, 70), (70, 103))):
        k, v = (numbers(b)[a:e] for b in back)
        w = np.einsum("nhd,hd->nh", k, numbers(q)[i]) * width**-0.5
        w = np.exp(w - w.max(0))
        w /= w.sum(0)
        want, spread = np.einsum("nh,nhd->hd", w, v), np.einsum("nh,nhd->hd", w, np.abs(v))
        # weights and answers of 8 bits, scores in 32
        assert (np.abs(numbers(out)[i] - want) <= spread * (2.0**-8 + 2.0**-14) + np.abs(want) * 2.0**-8 * 1.01).all()
    path, accepted = i32([0, 2, 1 + 2, -1] + [-1] * 99), i32([3, 0])
    both = torch.as_strided(store[0].view(dtype), (1, pages, T, heads, width), (0,) + pools[0].stride())
    cut = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    db.cache_keep(tabs, seq, i32([0, 4, 4]), path[:4], accepted, both, token_dim=2, cut=cut)
    finish()
    at = lambda x: pools[0][int(t.table[0, x // T]), x % T]
    assert cut.cpu().tolist() == [[0, 69], [1, 33]]
    want = numbers(back[0])
    sc = (lambda x: 1.0) if kind == "bf16" else (lambda x: scales[0][int(t.table[0, x // T]), x % T].cpu().double().numpy()[:, None])
    assert (numbers(at(67)) * sc(68) - want[68]).max() <= 2.0**-20 and (numbers(at(68)) * sc(69) - want[69]).max() <= 2.0**-20


@pytest.mark.parametrize("rows", ["8", "96"])
def test_pools_larger_than_64_gib(rows):
    """Pages 3 GiB apart, so that offsets by 16 bytes pass 32 bits."""
    need_gpu()
    db = lib()
    nodes, group = ROWS[rows]
    c = Case("e4m3", "bf16", 1, 16, 1, group, 64, [(200, nodes), (150, nodes)], "tree")
    gap = 3 << 30
    assert c.t.n_pages * gap > 1 << 36
    if torch.cuda.mem_get_info()[0] < c.t.n_pages * gap + (8 << 30):
        pytest.skip("not enough memory")
    b, want = c.oracle()
    dev = c.device()
    store = torch.empty(c.t.n_pages * gap, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    for k, name in enumerate(("k", "v")):  # values one MiB behind the keys
        dev[name] = torch.as_strided(store, dev[name].shape, (gap,) + dev[name].stride()[1:], k << 20).copy_(dev[name])
    out, lse = torch.full_like(c.q, 7.0).cuda(), torch.full(c.q.shape[:2], 7.0, device="cuda")
    c.call(db, c.t.device(), c.workspace(db), dev, out, lse)
    finish()
    c.check(out, lse, b, want)


def test_many_requests_of_all_kinds():
    rng = np.random.default_rng(12)
    for group, most in ((4, 2), (4, 8), (8, 30)):
        seqs = [(int(rng.integers(0, 90)), int(rng.integers(0, most + 1))) for _ in range(300)]
        seqs[7] = (5, most)
        Case("e4m3", "bf16", 1, 16, 1, group, 64, seqs, "tree", spare=3).run()


@pytest.mark.parametrize("kind,q,group,nodes", [("bf16", "bf16", 4, 1), ("e4m3", "bf16", 4, 4), ("i8", "f16", 4, 8), ("f16", "f16", 1, 3)])
def test_many_short_sequences_of_many_heads(kind, q, group, nodes):
    """Whole items that follow one another in a request are worked on side by side; those that a share of the work
    begins or ends in are not."""
    rng = np.random.default_rng(nodes)
    seqs = [(int(rng.choice([0, 1, 20, 63, 64, 130, 200])), int(rng.integers(1, nodes + 1))) for _ in range(260)]
    seqs[40], seqs[41] = (3000, nodes), (0, 0)
    Case(kind, q, 1, 16, 8 if group > 1 else 5, group, 64, seqs, "tree" if nodes > 1 else None).run()
