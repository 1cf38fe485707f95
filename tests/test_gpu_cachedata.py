"""Keys and values into a cache's pages and out of them, and tokens moved within, against the oracle:
codes, scales and moved bytes bit for bit, and every other byte as it was."""

import numpy as np
import pytest

from cache_util import NAMES, Tables, finish, i32, raw, tokens_first, tree
from gpu_util import lib, need_gpu
from oracle import cachedata as cd

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# (type, rows' type, token_dim, page, heads, width, [(length, new tokens)])
WRITES = [
    ("e4m3", "bf16", 1, 16, 8, 128, [(40, 5), (1, 1), (16, 16), (33, 1), (300, 257)]),
    ("e4m3", "f32", 2, 48, 5, 112, [(100, 49), (48, 1), (47, 2)]),
    ("i8", "f16", 1, 1, 1, 16, [(7, 3), (1, 1)]),
    ("i8", "bf16", 2, 3, 2, 256, [(20, 20), (9, 0), (5, 4)]),
    ("i8", "f32", 1, 64, 3, 80, [(130, 65)]),
    ("bf16", "bf16", 1, 16, 4, 64, [(1, 1), (2, 1), (50, 34)]),
    ("bf16", "f32", 2, 7, 3, 192, [(21, 8), (7, 7)]),
    ("f16", "f32", 1, 128, 1, 240, [(129, 2), (500, 131)]),
    ("f16", "bf16", 2, 16, 7, 48, [(31, 17)]),
    ("f16", "f16", 2, 16, 2, 32, [(31, 17), (4, 0)]),
]


def make_layer(rng, t, kind, token_dim, heads, width):
    """(pool, scale) of random bits that are numbers, on the host."""
    inner = (t.T, heads) if token_dim == 1 else (heads, t.T)
    shape = (t.n_pages,) + inner + (width,)
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
    if kind == "i8":
        return torch.from_numpy(rng.integers(-127, 128, shape).astype(np.int8)), torch.from_numpy(rng.random(shape[:3]).astype(np.float32))
    pool = (x * 50).to(NAMES[kind]) if kind == "e4m3" else x.to(NAMES[kind])
    return pool, torch.from_numpy(rng.random(shape[:3]).astype(np.float32)) if kind == "e4m3" else None


def new_rows(rng, n, heads, width, src):
    """Rows of many sizes: zeros, tiny ones, the type's largest, infinities and NaN among them."""
    x = rng.standard_normal((n, heads, width)) * np.exp2(rng.integers(-8, 9, (n, heads, 1)))
    for j in range(0, n, 5):
        h = j % heads
        x[j, h] = [0, 1e-40, 6e4, 3.0, -1e-7][j // 5 % 5]
    if n > 6:
        x[6, 0, width - 1], x[3, 0, 0] = np.inf, np.nan
    return torch.from_numpy(x.astype(np.float32)).to(NAMES[src])


def strided(rows, rng):
    """The rows as parts of a wider tensor, as a joint projection gives them."""
    n, h, w = rows.shape
    whole = torch.zeros((n, h + 2, w + 16), dtype=rows.dtype, device="cuda")
    whole[:, 1:h + 1, 16:] = rows.cuda()
    return whole[:, 1:h + 1, 16:]


@pytest.mark.parametrize("kind,src,token_dim,page,heads,width,seqs", WRITES)
def test_write(kind, src, token_dim, page, heads, width, seqs):
    need_gpu()
    db = lib()
    rng = np.random.default_rng(5)
    t = Tables(rng, [n for n, _ in seqs], page)
    order = rng.permutation(len(seqs))
    start = np.concatenate([[2], 2 + np.cumsum([seqs[i][1] for i in order])])  # two rows before, three behind
    rows = int(start[-1]) + 3
    k, v = new_rows(rng, rows, heads, width, src), new_rows(rng, rows, heads, width, src)
    tabs = t.device()
    pools, want = [], []
    for _ in range(2):
        pool, scale = make_layer(rng, t, kind, token_dim, heads, width)
        pools += [pool.cuda(), None if scale is None else scale.cuda()]
        want.append((pool, scale))
    status = torch.full((len(seqs),), 9, dtype=torch.uint8, device="cuda")
    ctr = torch.full((4,), 77, dtype=torch.int64, device="cuda")
    db.cache_write(tabs, i32(order), i32(start), strided(k, rng), strided(v, rng), pools[0], pools[2],
                   k_scale=pools[1], v_scale=pools[3], token_dim=token_dim, status=status, ctr=ctr)
    finish()
    b = cd.Batch(t.table, t.length, t.n_pages, page, order, start, rows, True)
    for (pool, scale), x, got, got_scale in ((want[0], k, pools[0], pools[1]), (want[1], v, pools[2], pools[3])):
        bits = raw(pool).copy()
        s = None if scale is None else scale.numpy().copy()
        narrow = lambda r: raw(torch.from_numpy(r).to(NAMES[kind]))  # noqa: E731
        cd.write(b, x.float().numpy(), tokens_first(bits, token_dim), None if s is None else tokens_first(s, token_dim),
                 kind, narrow)
        same = raw(got) == bits
        if kind in ("bf16", "f16"):
            same |= np.isnan(got.cpu().float().numpy()) & np.isnan(torch.from_numpy(bits).view(NAMES[kind]).float().numpy())
        assert same.all()
        if s is not None:
            np.testing.assert_array_equal(got_scale.cpu().numpy(), s)
    assert status.cpu().tolist() == b.status
    assert ctr.cpu().tolist() == b.counters()


READS = [
    ("e4m3", "bf16", 1, 16, 8, 128, [(40, 0, 40), (1, 0, 1), (16, 15, 5), (33, 40, 2)]),
    ("e4m3", "f32", 2, 48, 5, 112, [(100, 3, 97), (48, 47, 1), (47, 0, 0)]),
    ("i8", "f16", 2, 3, 2, 256, [(20, 7, 13), (9, 9, 4)]),
    ("i8", "f32", 1, 1, 1, 16, [(7, 0, 7), (0, 0, 3)]),
    ("bf16", "f32", 1, 7, 3, 192, [(21, 0, 21), (7, 2, 5)]),
    ("bf16", "bf16", 2, 16, 2, 64, [(300, 100, 200)]),
    ("f16", "bf16", 1, 128, 1, 240, [(129, 127, 2), (500, 0, 500)]),
    ("f16", "f16", 1, 16, 3, 48, [(129, 127, 2), (5, 0, 5)]),
]


@pytest.mark.parametrize("kind,dst,token_dim,page,heads,width,seqs", READS)
def test_read(kind, dst, token_dim, page, heads, width, seqs):
    need_gpu()
    db = lib()
    rng = np.random.default_rng(6)
    t = Tables(rng, [n for n, _, _ in seqs], page)
    order = rng.permutation(len(seqs))
    first = np.array([seqs[i][1] for i in order])
    start = np.concatenate([[1], 1 + np.cumsum([seqs[i][2] for i in order])])
    rows = int(start[-1]) + 2
    tabs = t.device()
    for positions in (first, None):
        pools, outs = [make_layer(rng, t, kind, token_dim, heads, width) for _ in range(2)], []
        for _ in range(2):
            outs.append(strided(torch.full((rows, heads, width), 3.0).to(NAMES[dst]), rng))
        c = [None if x is None else x.cuda() for pool in pools for x in pool]
        status = torch.full((len(seqs),), 9, dtype=torch.uint8, device="cuda")
        ctr = torch.full((4,), 77, dtype=torch.int64, device="cuda")
        db.cache_read(tabs, i32(order), i32(start), outs[0], outs[1], c[0], c[2], k_scale=c[1], v_scale=c[3],
                      first=None if positions is None else i32(positions), token_dim=token_dim, status=status, ctr=ctr)
        finish()
        b = cd.Batch(t.table, t.length, t.n_pages, page, order, start, rows, False)
        for (pool, scale), got in zip(pools, outs):
            # a code times a 32-bit scale, rounded to 32 bits and once more to the rows' type
            vals = pool.float() if scale is None else pool.float() * scale[..., None]
            want = np.full((rows, heads, width), 3.0)
            cd.read(b, positions, tokens_first(vals.to(NAMES[dst]).double().numpy(), token_dim), want)
            np.testing.assert_array_equal(got.cpu().double().numpy(), want)
        assert status.cpu().tolist() == b.status and ctr.cpu().tolist() == b.counters()


def test_bad_requests_and_broken_tables():
    """Requests out of place do nothing, entries that are no page are passed over, and both are reported."""
    need_gpu()
    db = lib()
    rng = np.random.default_rng(7)
    page, heads, width = 16, 2, 32
    t = Tables(rng, [40, 50, 20, 30, 17], page)
    t.table[1, 3] = t.n_pages  # no such page: tokens 48 and 49
    t.table[4, 0] = -5
    t.length[3] = (t.table.shape[1] * page) + 1  # more than a row has places for
    seq = np.array([0, 1, 99, 2, 3, -1, 4])
    start = np.array([0, 3, 8, 9, 30, 31, 33, 38])  # request 3: 21 rows of a sequence of 20
    rows = 38
    tabs = t.device()
    pool, scale = make_layer(rng, t, "e4m3", 1, heads, width)
    k = new_rows(rng, rows, heads, width, "f32")
    for call in ("write", "read"):
        got, got_scale = pool.cuda(), scale.cuda()
        out = torch.full((rows, heads, width), 3.0, device="cuda")
        status = torch.full((len(seq),), 9, dtype=torch.uint8, device="cuda")
        ctr = torch.zeros(4, dtype=torch.int64, device="cuda")
        x = k.cuda() if call == "write" else out
        getattr(db, "cache_" + call)(tabs, i32(seq), i32(start), x, x.clone(), got, got.clone(), k_scale=got_scale,
                                     v_scale=got_scale.clone(), status=status, ctr=ctr)
        finish()
        b = cd.Batch(t.table, t.length, t.n_pages, page, seq, start, rows, call == "write")
        if call == "write":
            bits, s = raw(pool).copy(), scale.numpy().copy()
            cd.write(b, k.numpy(), bits, s, "e4m3", None)
            assert (raw(got) == bits).all()
            np.testing.assert_array_equal(got_scale.cpu().numpy(), s)
        else:
            want = np.full((rows, heads, width), 3.0)
            cd.read(b, None, (pool.float() * scale[..., None]).double().numpy(), want)
            np.testing.assert_array_equal(out.cpu().double().numpy(), want)
        assert status.cpu().tolist() == b.status and ctr.cpu().tolist() == b.counters()
        assert b.broken


def test_starts_out_of_order():
    """A batch whose starts do not ascend stays in bounds: the requests that are wrong are reported, the others done."""
    need_gpu()
    db = lib()
    rng = np.random.default_rng(8)
    t = Tables(rng, [10, 10, 10], 4)
    seq, start, rows = np.array([0, 1, 2]), np.array([0, 4, 2, 100]), 8
    pool, _ = make_layer(rng, t, "bf16", 1, 1, 16)
    status = torch.zeros(3, dtype=torch.uint8, device="cuda")
    k = torch.zeros((rows, 1, 16), device="cuda", dtype=torch.bfloat16)
    db.cache_write(t.device(), i32(seq), i32(start), k, k, pool.cuda(), pool.cuda(), status=status)
    finish()
    assert status.cpu().tolist() == [0, 1, 1]


def test_many_requests():
    """Thousands of single tokens and a few long ones: every row finds its request."""
    need_gpu()
    db = lib()
    rng = np.random.default_rng(9)
    n = 5000
    lengths = rng.integers(1, 30, n)
    t = Tables(rng, lengths, 16)
    count = np.minimum(lengths, np.where(np.arange(n) % 700 == 3, 29, rng.integers(0, 3, n)))
    start = np.concatenate([[0], np.cumsum(count)])
    rows = int(start[-1])
    seq = np.arange(n)
    pool, scale = make_layer(rng, t, "i8", 1, 1, 32)
    k = new_rows(rng, rows, 1, 32, "bf16")
    kp, vp, ks, vs = pool.cuda(), pool.cuda(), scale.cuda(), scale.cuda()
    ctr = torch.zeros(4, dtype=torch.int64, device="cuda")
    db.cache_write(t.device(), i32(seq), i32(start), k.cuda(), k.cuda(), kp, vp, k_scale=ks, v_scale=vs, ctr=ctr)
    finish()
    b = cd.Batch(t.table, t.length, t.n_pages, 16, seq, start, rows, True)
    bits, s = raw(pool).copy(), scale.numpy().copy()
    cd.write(b, k.float().numpy(), bits, s, "i8", None)
    for got, got_scale in ((kp, ks), (vp, vs)):
        assert (raw(got) == bits).all()
        np.testing.assert_array_equal(got_scale.cpu().numpy(), s)
    assert ctr.cpu().tolist() == b.counters()


def test_a_written_row_reads_back_within_half_a_step():
    """Quantised and read back: i8 within half a code's step, e4m3 within 2^-4 of the value (or of its smallest normal)."""
    need_gpu()
    db = lib()
    rng = np.random.default_rng(10)
    t = Tables(rng, [64, 33], 16)
    start = np.array([0, 64, 97])
    x = rng.standard_normal((97, 3, 64)).astype(np.float32)
    for kind in ("i8", "e4m3"):
        pools = [torch.zeros((t.n_pages, 16, 3, 64), dtype=NAMES[kind], device="cuda") for _ in range(2)]
        scales = [torch.zeros((t.n_pages, 16, 3), device="cuda") for _ in range(2)]
        out = [torch.zeros((97, 3, 64), device="cuda") for _ in range(2)]
        tabs = t.device()
        rows = torch.from_numpy(x).cuda()
        db.cache_write(tabs, i32([0, 1]), i32(start), rows, rows * 2, *pools, k_scale=scales[0], v_scale=scales[1])
        db.cache_read(tabs, i32([0, 1]), i32(start), *out, *pools, k_scale=scales[0], v_scale=scales[1])
        finish()
        for got, by in zip(out, (1, 2)):
            want = x.astype(np.float64) * by
            top = np.abs(want).max(-1, keepdims=True)
            # three 32-bit roundings (L / a, the product, a / L) on top: 4 * 2^-24 relative to the largest
            step = top / 127 / 2 if kind == "i8" else np.maximum(np.abs(want), top / 448 * 2.0**-6) * 2.0**-4
            assert (np.abs(got.cpu().double().numpy() - want) <= step + top * 2.0**-22).all()


# (type, token_dim, page, planes, heads, width, [(length, tree)], pages outermost)
KEEPS = [
    ("bf16", 2, 16, 3, 2, 64, [(40, 9), (25, 25), (17, 1), (90, 48)], True),
    ("i8", 3, 48, 2, 5, 112, [(100, 30), (49, 3)], False),
    ("f32", 2, 1, 1, 1, 5, [(12, 12), (3, 2)], False),
    ("i8", 2, 5, 4, 3, 7, [(30, 20), (8, 8)], True),
    ("f16", 3, 8, 1, 3, 3, [(300, 280)], False),
]


@pytest.mark.parametrize("kind,token_dim,page,planes,heads,width,seqs,outer", KEEPS)
def test_keep(kind, token_dim, page, planes, heads, width, seqs, outer):
    need_gpu()
    db = lib()
    rng = np.random.default_rng(11)
    t = Tables(rng, [n for n, _ in seqs], page)
    inner = (page, heads) if token_dim == 2 else (heads, page)
    shape = (planes, t.n_pages) + inner + (width,)
    pool = torch.from_numpy(rng.integers(-100, 100, shape).astype(np.float32)).to(NAMES[kind])
    for turn in range(3):
        order = rng.permutation(len(seqs))
        start = np.concatenate([[1], 1 + np.cumsum([seqs[i][1] for i in order])])
        rows = int(start[-1]) + 1
        path, accepted = np.full(rows, -1), []
        for i, at in zip(order, start):
            _, sees = tree(rng, seqs[i][1], 20)
            way = np.flatnonzero(sees[rng.integers(0, len(sees))]) if turn else np.arange(len(sees))[rng.integers(0, 2):]
            path[at:at + len(way)] = way
            accepted.append(len(way))
        got = pool.transpose(0, 1).contiguous().cuda().transpose(0, 1) if outer else pool.cuda()
        cut = torch.zeros((len(seqs), 2), dtype=torch.int32, device="cuda")
        status = torch.full((len(seqs),), 9, dtype=torch.uint8, device="cuda")
        ctr = torch.full((4,), 77, dtype=torch.int64, device="cuda")
        db.cache_keep(t.device(), i32(order), i32(start), i32(path), i32(accepted), got, token_dim=token_dim, cut=cut,
                      status=status, ctr=ctr)
        finish()
        b = cd.Batch(t.table, t.length, t.n_pages, page, order, start, rows, True)
        want = pool.double().numpy().copy()
        view = want if token_dim == 2 else want.transpose(0, 1, 3, 2, 4)
        cuts = cd.keep(b, path, accepted, view)
        np.testing.assert_array_equal(got.cpu().double().numpy(), want)
        assert (cut.cpu().numpy().view(np.uint32) == np.array(cuts, np.uint64)).all()
        assert status.cpu().tolist() == b.status and ctr.cpu().tolist() == b.counters()


def test_keep_refuses_broken_paths():
    need_gpu()
    db = lib()
    rng = np.random.default_rng(12)
    t = Tables(rng, [20] * 7, 8)
    t.table[6, 2] = t.n_pages + 5
    seq, start = np.arange(7), np.arange(8) * 6
    path = np.tile([0, 2, 3, 5, -1, -1], 7)
    path[6 + 1] = 0     # named twice
    path[12 + 3] = 6    # past the request's rows
    path[18 + 2] = -4
    accepted = np.array([4, 4, 4, 4, 7, -1, 4])
    pool = torch.from_numpy(rng.standard_normal((2, t.n_pages, 8, 2, 16)).astype(np.float32))
    got = pool.cuda()
    status = torch.zeros(7, dtype=torch.uint8, device="cuda")
    cut = torch.zeros((7, 2), dtype=torch.int32, device="cuda")
    ctr = torch.zeros(4, dtype=torch.int64, device="cuda")
    db.cache_keep(t.device(), i32(seq), i32(start), i32(path), i32(accepted), got, cut=cut, status=status, ctr=ctr)
    finish()
    b = cd.Batch(t.table, t.length, t.n_pages, 8, seq, start, 42, True)
    want = pool.numpy().copy()
    cuts = cd.keep(b, path, accepted, want)
    assert b.status == [0, 1, 1, 1, 1, 1, 0] and b.broken
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert (cut.cpu().numpy().view(np.uint32) == np.array(cuts, np.uint64)).all()
    assert status.cpu().tolist() == b.status and ctr.cpu().tolist() == b.counters()


def test_empty_batches():
    need_gpu()
    db = lib()
    rng = np.random.default_rng(13)
    t = Tables(rng, [5], 4)
    tabs = t.device()
    pool = torch.ones((t.n_pages, 4, 1, 16), dtype=torch.bfloat16, device="cuda")
    none, zero = i32(np.zeros(0)), i32([0])
    rows = torch.zeros((0, 1, 16), dtype=torch.bfloat16, device="cuda")
    for call in (db.cache_write, db.cache_read):
        ctr = torch.full((4,), 77, dtype=torch.int64, device="cuda")
        call(tabs, none, zero, rows, rows, pool, pool, ctr=ctr)
        finish()
        assert ctr.cpu().tolist() == [0, 0, 0, 0]
    ctr = torch.full((4,), 77, dtype=torch.int64, device="cuda")
    db.cache_keep(tabs, none, zero, none, none, pool[None], ctr=ctr)
    db.cache_write(tabs, i32([0]), i32([0, 0]), rows, rows, pool, pool)
    finish()
    assert ctr.cpu().tolist() == [0, 0, 0, 0] and (pool == 1).all()
