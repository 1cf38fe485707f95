"""Batches whose starts do not ascend: requests that are wrong do nothing, and every other one is done, by itself."""

import numpy as np
import pytest

from cache_util import NAMES, Tables, finish, i32, numbers, raw, tokens_first
from gpu_util import lib, need_gpu
from oracle import cachedata as cd
from test_gpu_cachedata import make_layer

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BATCHES = {
    "shared rows": [0, 5, 3, 8],
    "one behind the other": [5, 8, 0, 5],
    "among good ones": [0, 1, 2, 9, 4, 6, 7, 7, 20, 21],
    "nested": [0, 100, 50, 60, 200],
    "from outside": [-3, 4, 7, 300, 2, 9],
}


def batches():
    for name, start in BATCHES.items():
        yield name, np.array(start), 240
    rng = np.random.default_rng(3)
    for n in (40, 700, 3000):
        yield f"any {n}", rng.integers(0, 240, n + 1), 240
        near = np.sort(rng.integers(0, 40000, n + 1))  # ascending but for a few
        for x in rng.integers(0, n, 3):
            near[x] = rng.integers(0, 40000)
        yield f"nearly {n}", near, 40000


ALL = {name: (start, rows) for name, start, rows in batches()}


def tables(rng, start, page=8):
    """A sequence of its own for each request, with some tokens before its rows; some are too short for them."""
    count = np.clip(np.diff(start), 0, 200)
    return Tables(rng, count + rng.integers(0, 5, len(count)), page)


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("kind,src", [("bf16", "f32"), ("i8", "bf16")])
def test_write(name, kind, src):
    need_gpu()
    db = lib()
    start, rows = ALL[name]
    rng = np.random.default_rng(5)
    t, n = tables(rng, start), len(start) - 1
    pool, scale = make_layer(rng, t, kind, 1, 2, 32)
    k = torch.from_numpy(rng.standard_normal((rows, 2, 32)).astype(np.float32)).to(NAMES[src])
    up = lambda x: None if x is None else x.cuda()  # noqa: E731
    kp, vp, ks, vs = up(pool), up(pool), up(scale), up(scale)
    status, ctr = torch.full((n,), 9, dtype=torch.uint8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    seq = rng.permutation(n)
    t.table[:n], t.length[:n] = t.table[:n][np.argsort(seq)], t.length[:n][np.argsort(seq)]
    for given in (dict(status=status, ctr=ctr), {}):
        db.cache_write(t.device(), i32(seq), i32(start), k.cuda(), k.cuda(), kp, vp, k_scale=ks, v_scale=vs, **given)
    finish()
    b = cd.Batch(t.table, t.length, t.n_pages, t.T, seq, start, rows, True)
    bits, s = raw(pool).copy(), None if scale is None else scale.numpy().copy()
    cd.write(b, k.float().numpy(), bits, s, kind, lambda r: raw(torch.from_numpy(r).to(NAMES[kind])))
    assert 0 < sum(b.status) < n
    for got, got_scale in ((kp, ks), (vp, vs)):
        assert (raw(got) == bits).all()
        if scale is not None:
            np.testing.assert_array_equal(got_scale.cpu().numpy(), s)
    assert status.cpu().tolist() == b.status and ctr.cpu().tolist() == b.counters()


@pytest.mark.parametrize("name", ALL)
def test_read(name):
    """A row that several valid requests have is one of theirs."""
    need_gpu()
    db = lib()
    start, rows = ALL[name]
    rng = np.random.default_rng(6)
    t, n = tables(rng, start), len(start) - 1
    pool, _ = make_layer(rng, t, "f16", 2, 2, 48)
    out = [torch.full((rows, 2, 48), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    status, first = torch.full((n,), 9, dtype=torch.uint8, device="cuda"), rng.integers(0, 4, n)
    seq = rng.permutation(n)
    db.cache_read(t.device(), i32(seq), i32(start), *out, pool.cuda(), pool.cuda(), first=i32(first), token_dim=2, status=status)
    finish()
    b = cd.Batch(t.table, t.length, t.n_pages, t.T, seq, start, rows, False)
    assert status.cpu().tolist() == b.status
    vals, may = tokens_first(numbers(pool), 2), [[] for _ in range(rows)]
    for i, r in enumerate(b.requests):
        for j in range(r[2] if r else 0):
            at = b.place(r[0], int(first[i]) + j) if int(first[i]) + j < r[3] else None
            may[r[1] + j].append(np.zeros((2, 48)) if at is None else vals[at])
    for got in out:
        got = numbers(got)
        for r in range(rows):  # each 8 values of a row are one request's
            if not may[r]:
                assert (got[r] == 7).all()
            else:
                pieces = [(got[r] == x).reshape(2, 6, 8).all(-1) for x in may[r]]
                assert np.any(pieces, 0).all()
