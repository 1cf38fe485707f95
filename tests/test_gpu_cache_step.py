"""Speculative steps on a paged cache: room for the drafts, their keys and values written, attention over the cache,
verification, the accepted tokens kept and the others' slots given back, without a host round trip between the calls;
once eagerly, step by step against the oracles, and once as a captured graph replayed."""

import numpy as np
import pytest

from cache_util import NAMES, finish, i32, numbers, tree, words
from gpu_util import lib, need_gpu
from oracle import cachedata as cd

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HEADS, GROUP, WIDTH, PAGE, COLUMNS, PAGES, VOCAB, LAYERS = 2, 4, 64, 16, 12, 200, 300, 2


class Engine:
    """Sequences 0 to n - 1 take a step of `nodes` drafted tokens each; the inputs are given from outside."""

    def __init__(self, kind, n, nodes):
        db = self.db = lib()
        self.n, self.nodes, self.kind = n, nodes, kind
        rows = n * nodes
        z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")
        self.tables = db.PageTables.empty(n + 2, COLUMNS, PAGES, PAGE)
        # [planes, pages, tokens, heads, width]: keys and values of each layer in turn
        self.pool = z(2 * LAYERS, PAGES, PAGE, HEADS, WIDTH, t=NAMES[kind])
        self.scales = z(2 * LAYERS, PAGES, PAGE, HEADS, t=torch.float32) if self.pool.element_size() == 1 else None
        self.page_ws = db.workspace(db.page_workspace_size(n + 2, PAGES))
        self.ws = db.workspace(db.cache_attention_workspace_size(n, HEADS * GROUP, HEADS, WIDTH, nodes))
        self.moves, self.n_moves = z(PAGES, 4), z(1)
        self.grow = i32([[s, nodes] for s in range(n)])
        self.seq, self.start = i32(range(n)), i32(range(0, rows + 1, nodes))
        self.k, self.v = (z(LAYERS, rows, HEADS, WIDTH, t=torch.bfloat16) for _ in range(2))
        self.q = z(LAYERS, rows, HEADS * GROUP, WIDTH, t=torch.bfloat16)
        self.out, self.mask = torch.zeros_like(self.q), z(rows, 1)
        self.parent, self.token, self.u = z(rows), z(rows), z(rows, t=torch.float32)
        self.p, self.d = z(rows, VOCAB, t=torch.float32), z(rows, VOCAB, t=torch.float32)
        self.path, self.accepted, self.next, self.cut = z(rows), z(n), z(n), z(n, 2)
        self.status = z(6, n, t=torch.uint8)

    def layer(self, x):
        ks, vs = (None, None) if self.scales is None else (self.scales[2 * x], self.scales[2 * x + 1])
        return dict(k_pool=self.pool[2 * x], v_pool=self.pool[2 * x + 1], k_scale=ks, v_scale=vs)

    def extend(self):
        self.db.page_extend(self.tables, self.grow, self.moves, self.n_moves, self.page_ws, status=self.status[0])
        for pool in (self.pool, self.scales):
            if pool is not None:
                self.db.page_copy(self.moves, self.n_moves, pool, pool, token_dim=2)

    def attend(self):
        for x in range(LAYERS):
            self.db.cache_write(self.tables, self.seq, self.start, self.k[x], self.v[x], status=self.status[1], **self.layer(x))
            self.db.cache_attention(self.tables, self.seq, self.start, self.q[x], out=self.out[x], ws=self.ws,
                                    max_tokens=self.nodes, mask=self.mask, status=self.status[2], **self.layer(x))

    def settle(self):
        self.db.draft_verify(self.start, self.parent, self.token, self.p, self.u, self.path, self.accepted, self.next, q=self.d,
                             status=self.status[3])
        for pool in (self.pool, self.scales):
            if pool is not None:
                self.db.cache_keep(self.tables, self.seq, self.start, self.path, self.accepted, pool, token_dim=2, cut=self.cut,
                                   status=self.status[4])
        self.db.page_free(self.tables, self.cut, self.page_ws, status=self.status[5])

    def step(self):
        self.extend(), self.attend(), self.settle()

    def draft(self, rng):
        """New inputs: trees, their tokens and probabilities, keys, values and queries. Returns what the oracles take."""
        n, m = self.n, self.nodes
        parents, sees = zip(*(tree(rng, m) for _ in range(n)))
        x = rng.standard_normal((2, n * m, VOCAB)) * 2
        pq = (np.exp(x) / np.exp(x).sum(-1, keepdims=True)).astype(np.float32)
        token = rng.integers(0, VOCAB, n * m).astype(np.int32)
        for r in range(n * m):  # likely drafts, so that paths are some tokens long
            if r % m:
                token[r] = int(np.argmax(pq[0, r - r % m + parents[r // m][r % m]]))
        mask = np.concatenate([words(s, 1) for s in sees])
        u = rng.random(n * m).astype(np.float32)
        given = dict(parent=np.concatenate(parents).astype(np.int32), token=token, u=u, p=pq[0], d=pq[1], mask=mask.view(np.int32))
        for name, a in given.items():
            getattr(self, name).copy_(torch.from_numpy(a))
        for t in (self.k, self.v, self.q):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)))
        return given, mask

    def state(self):
        t = self.tables
        return [x.clone() for x in (t.table, t.length, t.refs, self.pool.view(torch.uint8), self.out, self.path, self.accepted,
                                    self.next, self.cut, self.status)]


def prompts(e, rng, lengths):
    """The sequences' first tokens; sequence 1 is a fork of 0 (its last page is shared until the first step)."""
    db = e.db
    rows = sum(lengths)
    db.page_extend(e.tables, i32([[s if s < 1 else s + 1, n] for s, n in enumerate(lengths)]), e.moves, e.n_moves, e.page_ws)
    seq, start = i32([s if s < 1 else s + 1 for s in range(len(lengths))]), i32(np.concatenate([[0], np.cumsum(lengths)]))
    for x in range(LAYERS):
        k, v = (torch.from_numpy(rng.standard_normal((rows, HEADS, WIDTH)).astype(np.float32)).cuda().bfloat16() for _ in range(2))
        db.cache_write(e.tables, seq, start, k, v, **e.layer(x))
    db.page_fork(e.tables, i32([[0, 1, lengths[0], 0]]), e.page_ws)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_steps_against_the_oracles(kind):
    need_gpu()
    rng = np.random.default_rng(31)
    e = Engine(kind, 4, 7)
    prompts(e, rng, [21, 40, 3])
    longest = 0
    for _ in range(4):
        given, mask = e.draft(rng)
        e.extend(), e.attend()
        finish()
        table, length = e.tables.table.cpu().numpy(), e.tables.length.cpu().numpy()
        batch = cd.Batch(table, length, PAGES, PAGE, e.seq.cpu().numpy(), e.start.cpu().numpy(), e.n * e.nodes, True)
        scales = None if e.scales is None else e.scales.cpu().numpy()
        pool = numbers(e.pool)
        for x in range(LAYERS):
            # the new rows come back as written: off by half a step of the type (E4M3's smallest is 2^-9), and by three
            # roundings in 32 bits, of the scale, its inverse and the product
            vals = [cd.values(pool[2 * x + j], None if scales is None else scales[2 * x + j]) for j in (0, 1)]
            for j, rows in enumerate((e.k[x], e.v[x])):
                back = np.zeros((e.n * e.nodes, HEADS, WIDTH))
                first = [int(length[s]) - e.nodes for s in range(e.n)]
                cd.read(batch, first, vals[j], back)
                want = numbers(rows)
                top = np.abs(want).max(-1, keepdims=True)
                step = 0 * want if kind == "bf16" else np.abs(want) * 2.0**-4 + top * 2.0**-10 / 448 if kind == "e4m3" else top / 254
                assert (np.abs(back - want) <= step + np.abs(want) * 2.0**-21).all()
            out, _, spread, size = cd.attend(batch, numbers(e.q[x]), vals[0], vals[1], WIDTH**-0.5, mask)
            # weights and answers are rounded to 8 bits at least; scores are sums of 64 products in 32 bits (2^-18 of
            # their size), whose errors weights have once above and once below the line
            bound = spread * (2.0**-8 + (size[..., None] + 1) * 2.0**-17) + np.abs(out) * 2.0**-8 + 2.0**-40
            assert (np.abs(numbers(e.out[x]) - out) <= bound * (1 + 2.0**-6)).all()
        e.settle()
        finish()
        path, accepted, following, _ = cd.verify(e.start.cpu().numpy(), e.n * e.nodes, given["parent"], given["token"], given["p"],
                                                 given["d"], given["u"], VOCAB)
        assert e.path.cpu().tolist() == path.tolist() and e.next.cpu().tolist() == following.tolist()
        assert e.accepted.cpu().tolist() == accepted.tolist()
        cut = cd.keep(batch, path, accepted, pool)
        assert e.cut.cpu().tolist() == cut and (numbers(e.pool) == pool).all()
        assert e.tables.length.cpu().tolist()[:e.n] == [n for _, n in cut]
        assert e.status.cpu().tolist() == [[0] * e.n] * 6
        longest = max(longest, int(accepted.max()))
    assert longest > 2  # paths of some length were kept


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_a_captured_step_replayed_is_the_eager_one(kind):
    need_gpu()
    a, b = Engine(kind, 4, 7), Engine(kind, 4, 7)
    for e in (a, b):
        prompts(e, np.random.default_rng(5), [30, 11, 64])
    rng = [np.random.default_rng(6) for _ in range(2)]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    for x, r in zip((a, b), rng):
        x.draft(r), x.step()
    finish()
    with torch.cuda.graph(graph, stream=stream):
        b.step()
    for _ in range(3):
        for x, r in zip((a, b), rng):
            x.draft(r)
        a.step()
        graph.replay()
        finish()
        for p, q in zip(a.state(), b.state()):
            assert torch.equal(p, q)


def test_two_steps_on_two_streams_with_their_own_workspaces():
    need_gpu()
    engines = [Engine("e4m3", 4, 7) for _ in range(3)]
    for e in engines:
        prompts(e, np.random.default_rng(7), [30, 11, 64])
        e.draft(np.random.default_rng(8))
    finish()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for e, s in zip(engines, streams):
        with torch.cuda.stream(s):
            e.step()
    engines[2].step()
    finish()
    for x, y, z in zip(*(e.state() for e in engines)):
        assert torch.equal(x, z) and torch.equal(y, z)
