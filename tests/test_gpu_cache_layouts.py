"""Pages of keys, values and their scales at different distances, in parts of larger tensors: written, read, attended to."""

import numpy as np
import pytest

from cache_util import NAMES, Tables, finish, i32, numbers
from gpu_util import lib, need_gpu
from test_gpu_cache_attention import Case
from test_gpu_cache_edges import ROWS

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def spread(t, gap, at, fill):
    """t [pages, ...] on the GPU with `gap` elements from page to page, from element `at` on; (the store, the view)."""
    store = torch.full((t.shape[0] * gap + at,), fill, dtype=torch.float32, device="cuda").to(t.dtype)
    view = torch.as_strided(store, t.shape, (gap,) + t.stride()[1:], at)
    view.copy_(t)
    return store, view


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kind,q,width", [("bf16", "bf16", 128), ("e4m3", "bf16", 64), ("i8", "f16", 192), ("f16", "f16", 256)])
@pytest.mark.parametrize("token_dim", [1, 2])
def test_attention_over_pages_at_different_distances(kind, q, width, rows, token_dim):
    need_gpu()
    db = lib()
    nodes, group = ROWS[rows]
    c = Case(kind, q, token_dim, 16, 2, group, width, [(200, nodes), (150, nodes), (3000, nodes)], "tree", seed=nodes)
    if kind == "e4m3":
        for pool in c.pools:
            pool.copy_(torch.nan_to_num(pool.float()).to(pool.dtype))
    dev, page = c.device(), 16 * 2 * width
    for name, gap, at in (("k", 3 * page, page), ("v", 2 * page + 64, 32)):
        dev[name] = spread(dev[name], gap, at, 100.0)[1]
    if dev["ks"] is not None:
        for name, gap, at in (("ks", 33, 1), ("vs", 70, 3)):
            dev[name] = spread(dev[name], gap, at, float("nan"))[1]
    out, lse = torch.full_like(c.q, 7.0).cuda(), torch.full(c.q.shape[:2], 7.0, device="cuda")
    c.call(db, c.t.device(), c.workspace(db), dev, out, lse)
    finish()
    b, want = c.oracle()
    c.check(out, lse, b, want)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("token_dim", [1, 2])
def test_written_and_read_at_different_distances(kind, token_dim):
    """What is written in spread pages is what is written in neighbouring ones, and nothing else changes."""
    need_gpu()
    db = lib()
    rng = np.random.default_rng(23)
    heads, width, T = 3, 48, 8
    t = Tables(rng, [50, 9, 33], T)
    tabs, seq, start = t.device(), i32([2, 0, 1]), i32([0, 20, 70, 79])
    rows = [torch.from_numpy(rng.standard_normal((79, heads, width)).astype(np.float32)).cuda() for _ in range(2)]
    inner = (T, heads) if token_dim == 1 else (heads, T)
    near = [torch.zeros((t.n_pages,) + inner + (width,), dtype=NAMES[kind], device="cuda") for _ in range(2)]
    scales = [torch.zeros((t.n_pages,) + inner, device="cuda") if kind in ("e4m3", "i8") else None for _ in range(2)]
    page = T * heads * width
    stores, far = zip(*(spread(x, g * page + 16 * g, 16 * g, 7) for x, g in zip(near, (2, 3))))
    far_scales, scale_stores = [None, None], []
    if scales[0] is not None:
        pairs = [spread(x, g * T * heads + g, g, 5.0) for x, g in zip(scales, (2, 3))]
        scale_stores, far_scales = zip(*pairs)
    before = [x.clone() for x in (*stores, *scale_stores)]
    out = []
    for pools, sc in ((near, scales), (far, far_scales)):
        layer = dict(k_pool=pools[0], v_pool=pools[1], k_scale=sc[0], v_scale=sc[1], token_dim=token_dim)
        db.cache_write(tabs, seq, start, *rows, **layer)
        back = [torch.zeros_like(rows[0]) for _ in range(2)]
        db.cache_read(tabs, seq, start, *back, **layer)
        out.append(back)
    finish()
    bits = lambda x: x.contiguous().view(torch.uint8)
    for a, b in zip((*near, *scales), (*far, *far_scales)):
        assert a is None or torch.equal(bits(a), bits(b))
    assert all(torch.equal(a, b) for a, b in zip(*out)) and numbers(out[0][0]).any()
    for store, was, view in zip((*stores, *scale_stores), before, (*far, *far_scales)):
        mine = torch.as_strided(was, view.shape, view.stride(), view.storage_offset())
        mine.copy_(view)  # what was written, in its places
        assert torch.equal(bits(store), bits(was))
