"""Attention of drafted tokens over a paged cache against the formula in 64 bits.

The bound of each output follows from the kernel's roundings. A weight's relative error is e_p: the score is a sum of
`width` products in 32 bits (width + 8 roundings of 2^-24 of the sum of magnitudes, twice that for products by scales
and the change to base 2), exp2's own 2^-22, a few roundings more. Weights are then rounded to u_w = 2^-8 (bf16) or
2^-11 (f16, below 2^-14 in steps of 2^-24), so that the output is off by at most spread * (2 e_p + u_w) from them, n
tokens' sums in 32 bits by n 2^-24 of that, and by half a step of its own type."""

import numpy as np
import pytest

from cache_util import NAMES, Tables, finish, i32, numbers, tokens_first, tree, words
from gpu_util import lib, need_gpu
from oracle import cachedata as cd

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0**-8, "f16": 2.0**-11}


class Case:
    def __init__(self, kind, q, token_dim, page, heads, group, width, seqs, mask, seed=3, spare=0, scale=None):
        """seqs: (tokens before, drafted tokens); mask: None (chain), "tree", "random", "nothing"."""
        rng = self.rng = np.random.default_rng(seed)
        self.kind, self.qk, self.token_dim, self.mask_kind = kind, q, token_dim, mask
        self.t = t = Tables(rng, [a + m for a, m in seqs], page)
        self.seq = rng.permutation(len(seqs))
        counts = [seqs[i][1] for i in self.seq]
        self.start = np.concatenate([[spare], spare + np.cumsum(counts)])
        self.rows = int(self.start[-1]) + spare
        self.max_tokens = max(max(counts), 1)
        self.scale = width**-0.5 if scale is None else scale
        inner = (page, heads) if token_dim == 1 else (heads, page)
        shape = (t.n_pages,) + inner + (width,)
        self.pools, self.scales = [], []
        for _ in range(2):
            x = rng.standard_normal(shape)
            if kind == "i8":
                self.pools.append(torch.from_numpy(np.clip(np.rint(x * 40), -127, 127).astype(np.int8)))
            else:
                self.pools.append(torch.from_numpy((x * (100 if kind == "e4m3" else 1)).astype(np.float32)).to(NAMES[kind]))
            self.scales.append(torch.from_numpy(rng.uniform(0.005, 0.03, shape[:3]).astype(np.float32))
                               if kind in ("i8", "e4m3") else None)
        self.q = torch.from_numpy((rng.standard_normal((self.rows, heads * group, width)) * 2).astype(np.float32)).to(NAMES[q])
        self.mask = None
        if mask:
            n_words = -(-self.max_tokens // 32) + 1
            self.mask = np.full((self.rows, n_words), 0xFFFFFFFF, np.uint32)  # bits past a request's nodes mean nothing
            for i, m in enumerate(counts):
                sees = {"tree": lambda: tree(rng, m)[1], "random": lambda: rng.random((m, m)) < 0.3,
                        "nothing": lambda: np.zeros((m, m), bool)}[mask]()
                keep = np.zeros((m, n_words * 32), bool)
                keep[:, :m] = sees
                self.mask[self.start[i]:self.start[i] + m] = words(keep, n_words) | words(np.arange(n_words * 32) >= m + np.zeros((m, 1)), n_words)

    def view(self, part):
        """The pool's (and scales') arrays by token, for planting values: (pool tensor, scale tensor) [pages, tokens, heads...]."""
        pool, scale = self.pools[part], self.scales[part]
        if self.token_dim == 2:
            pool = pool.transpose(1, 2)
            scale = None if scale is None else scale.transpose(1, 2)
        return pool, scale

    def oracle(self):
        b = cd.Batch(self.t.table, self.t.length, self.t.n_pages, self.t.T, self.seq, self.start, self.rows, True, self.max_tokens)
        vals = [cd.values(tokens_first(numbers(p), self.token_dim),
                          None if s is None else tokens_first(s.numpy(), self.token_dim)) for p, s in zip(self.pools, self.scales)]
        return b, cd.attend(b, numbers(self.q), *vals, self.scale, self.mask)

    def call(self, db, tabs, ws, dev, out, lse, **kw):
        db.cache_attention(tabs, dev["seq"], dev["start"], dev["q"], dev["k"], dev["v"], out, ws, max_tokens=self.max_tokens,
                           scale=self.scale, mask=dev["mask"], lse=lse, k_scale=dev["ks"], v_scale=dev["vs"],
                           token_dim=self.token_dim, **kw)

    def device(self):
        up = lambda x: None if x is None else x.cuda()  # noqa: E731
        return {"seq": i32(self.seq), "start": i32(self.start), "q": up(self.q), "k": up(self.pools[0]), "v": up(self.pools[1]),
                "ks": up(self.scales[0]), "vs": up(self.scales[1]),
                "mask": None if self.mask is None else i32(self.mask.view(np.int32))}

    def workspace(self, db):
        heads = self.pools[0].shape[3 - self.token_dim]
        return db.workspace(db.cache_attention_workspace_size(len(self.seq), self.q.shape[1], heads, self.q.shape[2], self.max_tokens))

    def check(self, out, lse, b, want):
        o, l, spread, size = want
        rows = np.zeros(self.rows, bool)
        for r in b.requests:
            if r:
                rows[r[1]:r[1] + r[2]] = True
        got, got_lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
        assert (got[~rows] == 7).all() and (got_lse[~rows] == 7).all()  # as they were
        n, width = int(self.t.length.max()), self.q.shape[2]
        spread, size = np.nan_to_num(spread, nan=np.inf), np.nan_to_num(size, nan=np.inf)
        e_p = 2 * (width + 8) * 2.0**-24 * size[..., None] + 2.0**-20
        coded = self.kind in ("i8", "e4m3")
        u_w = HALF["bf16"] if coded else HALF[self.qk]
        bound = spread * (2 * e_p + u_w + n * 2.0**-24) + np.abs(o) * HALF[self.qk] * 1.01
        if self.qk == "f16":  # steps below the normal range: of the weights and of the output
            top = np.nanmax(np.abs(np.where(np.isfinite(numbers(self.pools[1])), numbers(self.pools[1]), 0)))
            bound = bound + (0 if coded else n * 2.0**-25 * top) + 2.0**-25
        ok = (np.abs(got - o) <= bound) | ((got == o) | np.isnan(got) & np.isnan(o))
        bad = ~ok & rows[:, None, None]
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], o[bad][:4], bound[bad][:4])
        finite = np.isfinite(l)
        with np.errstate(invalid="ignore"):
            apart = np.abs(got_lse - l)
        off = np.where(finite, apart, 0) <= e_p[..., 0] + (np.abs(np.where(finite, l, 0)) + 1) * 2.0**-20 + n * 2.0**-24
        same = np.where(finite, off, (got_lse == l) | (np.isnan(got_lse) & np.isnan(l)))
        assert same[rows].all()

    def run(self, **kw):
        need_gpu()
        db = lib()
        out, lse = torch.full_like(self.q, 7.0).cuda(), torch.full(self.q.shape[:2], 7.0, device="cuda")
        n = len(self.seq)
        status = torch.full((n,), 9, dtype=torch.uint8, device="cuda")
        ctr = torch.full((4,), 77, dtype=torch.int64, device="cuda")
        ws = self.workspace(db)
        self.call(db, self.t.device(), ws, self.device(), out, lse, status=status, ctr=ctr, **kw)
        finish()
        b, want = self.oracle()
        self.check(out, lse, b, want)
        assert status.cpu().tolist() == b.status and ctr.cpu().tolist() == b.counters()
        assert (ws[:4096] == 0).all()  # ready for the next call
        return out, lse


SHAPES = [
    ("bf16", "bf16", 1, 16, 2, 4, 128, [(100, 1), (0, 1), (63, 1), (64, 1), (1, 1)], None),
    ("bf16", "bf16", 1, 16, 2, 4, 128, [(200, 8), (5, 3), (0, 8)], "tree"),
    ("bf16", "bf16", 2, 48, 1, 8, 112, [(150, 25), (33, 7)], "tree"),
    ("f16", "f16", 1, 1, 3, 1, 16, [(10, 1), (130, 3), (0, 5)], "random"),
    ("f16", "f16", 2, 7, 1, 3, 48, [(300, 40), (12, 12)], "random"),
    ("f16", "f16", 1, 64, 2, 2, 256, [(70, 20), (200, 1)], None),
    ("bf16", "bf16", 1, 100, 1, 7, 192, [(350, 5), (20, 20)], "tree"),
    ("bf16", "bf16", 2, 16, 1, 1, 256, [(64, 64), (0, 64)], "random"),
    ("e4m3", "bf16", 1, 16, 2, 8, 128, [(500, 1), (64, 1), (0, 1)], None),
    ("e4m3", "f16", 2, 16, 2, 4, 64, [(120, 10), (3, 2)], "tree"),
    ("e4m3", "bf16", 1, 3, 1, 5, 80, [(90, 33), (65, 9)], "random"),
    ("i8", "f16", 2, 48, 1, 8, 112, [(200, 61), (10, 30)], "tree"),
    ("i8", "bf16", 1, 32, 3, 2, 96, [(77, 4), (0, 2)], "nothing"),
    ("i8", "bf16", 1, 16, 1, 16, 240, [(90, 9)], "random"),
    ("e4m3", "f16", 1, 128, 1, 1, 256, [(129, 40), (1000, 2)], None),
    ("bf16", "bf16", 1, 16, 1, 64, 64, [(30, 3)], None),
    ("bf16", "bf16", 1, 16, 1, 2, 32, [(40, 70), (0, 100)], "tree"),
    ("f16", "f16", 1, 16, 2, 8, 64, [(300, 30), (2000, 9), (64, 17)], None),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"{i}-{s[0]}-{s[1]}-{s[6]}-{s[8]}" for i, s in enumerate(SHAPES)])
def test_shapes(shape):
    Case(*shape, spare=2).run()


def test_long_cache_is_cut_over_the_whole_gpu():
    Case("e4m3", "bf16", 1, 16, 1, 2, 64, [(30000, 1), (7, 1)], None).run()
    Case("bf16", "bf16", 1, 16, 1, 4, 128, [(9000, 6), (100, 2)], "tree").run()


DEEP = [
    ("bf16", "bf16", 1, 16, 4, 4, 128, [(6000, 20), (3000, 33), (90, 9)], "tree"),
    ("i8", "f16", 2, 48, 2, 8, 112, [(9000, 20), (5000, 61)], "tree"),
    ("e4m3", "bf16", 1, 16, 8, 8, 64, [(20000, 16)], None),
    ("f16", "f16", 1, 7, 8, 5, 48, [(3000, 40), (2500, 9), (3, 3)], "random"),
    ("e4m3", "f16", 1, 64, 2, 4, 256, [(12000, 30)], "tree"),
    ("bf16", "bf16", 2, 128, 3, 8, 192, [(8000, 12), (777, 20)], "random"),
    ("f16", "f16", 2, 48, 2, 4, 112, [(4000, 20), (1000, 11)], "tree"),
    ("bf16", "bf16", 1, 8, 5, 8, 80, [(2000, 9), (1999, 33)], None),
    ("bf16", "bf16", 1, 64, 2, 8, 256, [(2500, 9), (1000, 17)], "tree"),
    ("i8", "bf16", 1, 33, 16, 3, 32, [(1500, 13), (1400, 11), (1300, 12), (0, 30)], "tree"),
]


@pytest.mark.parametrize("shape", DEEP, ids=[f"{i}-{s[0]}-{s[1]}-{s[6]}" for i, s in enumerate(DEEP)])
def test_many_tiles_of_many_rows(shape):
    """Several tiles and items for each CTA, so that every ring wraps."""
    Case(*shape, spare=1).run()


def test_many_requests():
    """More requests than a CTA has threads, some without rows."""
    rng = np.random.default_rng(1)
    Case("bf16", "bf16", 1, 8, 1, 2, 16, [(int(a), int(m)) for a, m in zip(rng.integers(0, 20, 400), rng.integers(0, 3, 400))],
         None, spare=1).run()


@pytest.mark.parametrize("kind,q,group", [("bf16", "bf16", 2), ("f16", "f16", 8), ("e4m3", "bf16", 4), ("i8", "f16", 16),
                                          ("bf16", "bf16", 16)])
def test_what_is_not_seen_does_not_matter(kind, q, group):
    """Infinities and NaN in slots past the end, in spare pages and in nodes off the path reach no row that does not see
    them, and those that do as in the formula."""
    c = Case(kind, q, 1, 16, 2, group, 64, [(70, 9), (0, 6), (130, 12)], "tree")
    t = c.t
    used = np.zeros((t.n_pages, t.T), bool)
    for s, n in enumerate(t.length):
        for x in range(n):
            used[t.table[s, x // t.T], x % t.T] = True
    for part in (0, 1):
        pool, scale = c.view(part)
        for p, j in np.argwhere(~used):
            if scale is not None:
                scale[p, j] = float("nan")
            if kind in ("bf16", "f16"):
                pool[p, j] = float("inf") if (p + j) % 2 else float("nan")
            elif kind == "e4m3":
                pool[p, j] = float("nan")
    for i, s in enumerate(c.seq):  # the request's third and last nodes: NaN and infinite keys and values
        m, n = int(c.start[i + 1] - c.start[i]), int(t.length[s])
        for node, value in ((2, float("nan")), (m - 1, float("inf"))):
            x = n - m + node
            for part in (0, 1):
                pool, scale = c.view(part)
                if scale is not None:
                    scale[t.table[s, x // t.T], x % t.T] = value
                else:
                    pool[t.table[s, x // t.T], x % t.T, :, 5] = value
    out, _ = c.run()
    for i in range(len(c.seq)):  # node 0 sees neither
        assert torch.isfinite(out[c.start[i]].float()).all()


def test_scores_of_minus_infinity():
    """A row that sees a single key, of minus infinity in its only place, is like one that sees nothing."""
    c = Case("bf16", "bf16", 1, 16, 1, 1, 16, [(0, 1), (3, 1)], None)
    c.q[:] = 1.0
    t = c.t
    s = 0
    c.pools[0][t.table[s, 0], 0, 0, 3] = -float("inf")
    out, lse = c.run()
    i = int(np.flatnonzero(c.seq == 0)[0])
    assert (out[c.start[i]] == 0).all() and (lse[c.start[i]] == -float("inf")).all()


def test_bad_requests_and_broken_tables():
    c = Case("bf16", "bf16", 1, 16, 2, 2, 32, [(100, 3), (40, 5), (10, 2), (64, 4)], "tree")
    c.seq[1] = 77
    c.t.table[c.seq[0], 1] = c.t.n_pages + 3
    c.t.table[c.seq[2], 0] = -2
    c.run()
    c = Case("bf16", "bf16", 1, 16, 2, 2, 32, [(100, 3), (40, 5), (10, 2)], None)
    c.max_tokens = 3  # the request of five is refused
    c.run()


def test_q_may_be_out_and_strided():
    need_gpu()
    db = lib()
    c = Case("e4m3", "bf16", 1, 16, 2, 4, 64, [(300, 6), (40, 3)], "tree")
    b, want = c.oracle()
    dev, tabs, ws = c.device(), c.t.device(), c.workspace(db)
    wide = torch.full((c.rows, 12, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10, 16:] = dev["q"]
    dev["q"] = wide[:, 2:10, 16:]
    lse = torch.zeros((c.rows, 8), device="cuda")
    c.call(db, tabs, ws, dev, dev["q"], lse)
    finish()
    c.check(dev["q"], lse, b, want)
    wide[:, 2:10, 16:] = 7
    assert (wide == 7).all()


def test_captured_and_replayed_with_grown_sequences():
    """A step in a graph: lengths, tables and rows change between replays, the workspace stays."""
    need_gpu()
    db = lib()
    c = Case("i8", "bf16", 1, 16, 2, 4, 64, [(200, 4), (1000, 2), (30, 5)], "tree")
    dev, tabs, ws = c.device(), c.t.device(), c.workspace(db)
    out, lse = torch.full_like(dev["q"], 7.0), torch.full(c.q.shape[:2], 7.0, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.call(db, tabs, ws, dev, out, lse)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.call(db, tabs, ws, dev, out, lse)
    for cut in (0, 3, 150):  # sequences lose tokens at their ends
        c.t.length[:3] = [max(n - cut, m) for n, m in zip((204, 1002, 35), (4, 2, 5))]
        tabs.length.copy_(torch.from_numpy(c.t.length))
        c.q = (c.q.float() * 0.7).bfloat16()
        dev["q"].copy_(c.q)
        out.fill_(7)
        graph.replay()
        finish()
        b, want = c.oracle()
        c.check(out, lse, b, want)


def test_two_streams_with_two_workspaces():
    need_gpu()
    db = lib()
    cases = [Case("bf16", "bf16", 1, 16, 2, 4, 128, [(700, 5), (90, 3)], "tree", seed=s) for s in (1, 2)]
    made = []
    for c in cases:
        made.append((c, c.device(), c.t.device(), c.workspace(db), torch.full_like(c.q, 7.0).cuda(),
                     torch.full(c.q.shape[:2], 7.0, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, dev, tabs, ws, out, lse, stream in made:
            c.call(db, tabs, ws, dev, out, lse, stream=stream)
    finish()
    for c, dev, tabs, ws, out, lse, stream in made:
        b, want = c.oracle()
        c.check(out, lse, b, want)


def test_the_same_bits_every_time():
    need_gpu()
    db = lib()
    c = Case("bf16", "bf16", 1, 16, 1, 4, 128, [(5000, 8), (60, 2), (900, 3)], "tree")
    dev, tabs, ws = c.device(), c.t.device(), c.workspace(db)
    got = []
    for _ in range(8):
        out, lse = torch.zeros_like(dev["q"]), torch.zeros(c.q.shape[:2], device="cuda")
        c.call(db, tabs, ws, dev, out, lse)
        got.append((out, lse))
    finish()
    assert all(torch.equal(o, got[0][0]) and torch.equal(x, got[0][1]) for o, x in got[1:])
