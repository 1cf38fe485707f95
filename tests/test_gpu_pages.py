"""The paged cache on the GPU against the one-request-at-a-time oracle. Everything is whole
numbers or moved bytes, so every comparison is for equality."""

import ctypes

import numpy as np
import pytest

from gpu_util import lib, need_gpu
from oracle import pages as po

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int64)).astype(dtype)).cuda()


def u32(rows, width):
    """Requests (values up to 2^32 - 1) as int32 bits."""
    a = np.asarray(rows, dtype=np.int64).reshape(-1, width)
    return torch.from_numpy(np.ascontiguousarray(a.astype(np.uint32).view(np.int32))).cuda()


def ctr():
    return torch.full((4,), -7, dtype=torch.int64, device="cuda")


class Both:
    """A cache on the GPU and in the oracle; every call is made on both and compared."""

    def __init__(self, n_seqs, columns, n_pages, page_tokens):
        self.db = lib()
        self.o = po.Cache(n_seqs, columns, n_pages, page_tokens)
        self.t = self.db.PageTables.empty(n_seqs, columns, n_pages, page_tokens)
        self.ws = self.db.workspace(self.db.page_workspace_size(n_seqs, n_pages))

    def load(self):
        """The oracle's state onto the GPU."""
        self.t.table.copy_(dev(self.o.table))
        self.t.length.copy_(torch.from_numpy(self.o.length.astype(np.uint32).view(np.int32)))
        self.t.refs.copy_(dev(self.o.refs))
        self.t.free.copy_(torch.from_numpy(po.pack_free(self.o.refs).view(np.int32)))

    def same(self, t=None):
        t = t or self.t
        torch.cuda.synchronize()
        assert (t.table.cpu().numpy() == self.o.table).all()
        assert (t.length.cpu().numpy().view(np.uint32) == self.o.length).all()
        assert (t.refs.cpu().numpy() == self.o.refs).all()
        assert (t.free.cpu().numpy().view(np.uint32) == po.pack_free(self.o.refs)).all()

    def _status(self, n):
        return torch.full((n + 1,), 99, dtype=torch.uint8, device="cuda")

    def _told(self, status, c, want_status, want_ctr):
        assert status.cpu().tolist() == list(want_status) + [99]
        assert c.cpu().tolist() == want_ctr

    def free(self, req):
        st, c = self._status(len(req)), ctr()
        self.db.page_free(self.t, u32(req, 2), self.ws, status=st, ctr=c)
        want = self.o.free(req)
        self.same()
        self._told(st, c, *want)

    def fork(self, req):
        st, c = self._status(len(req)), ctr()
        self.db.page_fork(self.t, u32(req, 4), self.ws, status=st, ctr=c)
        want = self.o.fork(req)
        self.same()
        self._told(st, c, *want)

    def extend(self, req):
        st, c = self._status(len(req)), ctr()
        moves = torch.full((len(req) + 1, 4), -9, dtype=torch.int32, device="cuda")
        n = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        self.db.page_extend(self.t, u32(req, 2), moves, n, self.ws, status=st, ctr=c)
        status, counters, want = self.o.extend(req)
        self.same()
        self._told(st, c, status, counters)
        m = int(n.cpu()[0])
        assert moves.cpu()[:m].tolist() == want
        assert (moves.cpu()[m:] == -9).all()  # nothing past them is written

    def compact(self, cap, apart=True):
        c = ctr()
        moves = torch.full((cap + 1, 4), -9, dtype=torch.int32, device="cuda")
        n = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        out = self.t
        if apart:
            out = self.db.PageTables(*(torch.full_like(x, -5) for x in (
                self.t.table, self.t.length, self.t.refs, self.t.free)), self.t.page_tokens)
            before = [x.clone() for x in (self.t.table, self.t.length, self.t.refs, self.t.free)]
        self.db.page_compact(self.t, out, moves[:cap], n, self.ws, ctr=c)
        counters, want = self.o.compact(cap)
        self.same(out)
        assert c.cpu().tolist() == counters
        got = moves.cpu().numpy().view(np.uint32).astype(np.int64)
        assert got[: len(want)].tolist() == want and int(n.cpu()[0]) == len(want)
        assert (moves.cpu()[len(want):] == -9).all()
        if apart:
            for x, y in zip((self.t.table, self.t.length, self.t.refs, self.t.free), before):
                assert torch.equal(x, y)  # the input is as it was
            self.t = out


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


SHAPES = [  # sequences, columns, pages, page tokens
    (1, 1, 1, 1),
    (5, 3, 7, 4),
    (9, 6, 33, 1),
    (12, 5, 64, 5),
    (40, 9, 129, 16),
    (33, 17, 500, 3),
    (3, 400, 1200, 2),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
@pytest.mark.parametrize("seed", range(3))
def test_random_histories(shape, seed):
    n_seqs, columns, n_pages, page = shape
    rng = np.random.default_rng([seed, n_seqs, n_pages])
    b = Both(*shape)
    for step in range(30):
        k = int(rng.integers(0, n_seqs + 1))
        op = int(rng.integers(0, 5))
        seq = rng.integers(0, n_seqs + 2, k) if rng.random() < 0.5 else rng.permutation(n_seqs)[:k]
        far = columns * page + 2
        if op <= 1:
            take = rng.integers(0, 3, k) if rng.random() < 0.6 else rng.integers(0, far, k)
            b.extend(np.stack([seq, take], 1))
        elif op == 2:
            parent = rng.integers(0, n_seqs + 1, k)
            has = np.append(b.o.length, 3)[parent]
            b.fork(np.stack([parent, seq, rng.integers(0, has + 2), seq * 7], 1))
        elif op == 3:
            b.free(np.stack([seq, np.where(rng.random(k) < 0.3, 0, rng.integers(0, far, k))], 1))
        else:
            b.compact(int(rng.integers(0, n_pages // 2 + 2)), apart=bool(rng.integers(0, 2)))
    po.check(b.o)


@pytest.mark.parametrize("n_seqs,columns,n_pages,page", [
    (1500, 4, 3001, 8),       # more requests than a CTA has threads
    (9001, 3, 20011, 4),      # more than a cluster has, and than starts are kept on chip
    (64, 700, 45056, 16),     # many pages for each request
    (7, 40, 1100003, 16),     # a pool of more than a million pages, mostly free
], ids=["n1500", "n9001", "long", "pool"])
def test_larger_batches(n_seqs, columns, n_pages, page):
    rng = np.random.default_rng(n_seqs)
    b = Both(n_seqs, columns, n_pages, page)
    far = columns * page
    half = n_seqs // 2
    b.extend(np.stack([rng.permutation(half), rng.integers(1, far // 2, half)], 1))
    child = half + rng.permutation(n_seqs - half)
    parent = rng.integers(0, half, n_seqs - half)
    b.fork(np.stack([parent, child, rng.integers(0, b.o.length[parent] + 1), child], 1))
    seq = rng.permutation(n_seqs)
    b.extend(np.stack([seq, rng.integers(0, 2 * page, n_seqs)], 1))
    b.free(np.stack([seq, rng.integers(0, far, n_seqs)], 1))
    b.compact(n_pages // 2, apart=False)
    b.extend(np.stack([seq, rng.integers(0, page, n_seqs)], 1))
    po.check(b.o)


def test_the_last_holder_keeps_a_shared_page():
    b = Both(6, 4, 30, 8)
    b.extend([[0, 13]])
    b.fork([[0, k, 13, 0] for k in (1, 2, 3)])
    b.free([[0, 0]])                                   # three holders, all of them in the batch
    b.extend([[2, 1], [1, 4], [3, 0]])                 # 3 adds nothing: two of three copy
    b.extend([[3, 1]])                                 # alone now
    b.fork([[1, 4, 9, 0], [1, 5, 9, 0]])
    b.extend([[5, 7], [4, 8], [1, 1]])                 # 1 holds 5 more tokens of the shared page


def test_a_short_batch_changes_nothing():
    b = Both(4, 8, 10, 4)
    b.extend([[0, 20], [1, 7]])
    b.fork([[1, 2, 7, 0]])
    b.extend([[2, 1], [1, 1], [3, 9], [3, 1]])         # a copy and 3 pages, of 3 free ones
    b.extend([[2, 1], [1, 1], [3, 8], [9, 1]])         # a copy and 2
    b.extend([[3, 0], [0, 0]])                         # none needed, none free
    b.extend([[3, 1]])                                 # one needed, none free


def test_rows_and_lengths_at_their_ends():
    b = Both(3, 2, 8, 4)
    b.extend([[0, 8], [1, 9]])                         # a full row; one token too many
    b.extend([[0, 1], [1, 0xFFFFFFFF], [2, 0x80000000]])
    b.fork([[0, 1, 8, 0], [0, 2, 9, 0]])
    b.fork([[0, 2, 0, 0]])                             # no tokens: nothing, and 2 stays empty
    b.free([[0, 0xFFFFFFFF], [1, 8], [0, 0]])          # named twice: the first keeps all
    b.free([[0, 7], [1, 4]])
    b.free([[0, 0], [1, 0]])
    b.free([[0, 0], [0xFFFFFFFF, 0]])


def test_no_requests_zero_the_counters():
    b = Both(3, 2, 8, 4)
    b.extend(np.zeros((0, 2)))
    b.fork(np.zeros((0, 4)))
    b.free(np.zeros((0, 2)))
    b.compact(0)
    b.compact(4)


def test_page_tokens_that_pass_32_bits():
    """Columns x page tokens above 2^32: lengths stay below it."""
    b = Both(3, 8, 20, 0x70000000)
    b.extend([[0, 0x70000001], [1, 0xFFFFFFFF], [2, 5]])
    b.extend([[0, 0x8FFFFFFE], [1, 1]])                # 2^32 - 1 tokens; one too many
    b.fork([[0, 2, 1, 0]])
    b.free([[0, 0xE0000000]])
    b.free([[0, 0xE0000000 - 1], [1, 1]])


def test_few_free_pages_far_apart():
    """The pages taken lie in more words of free bits than a CTA keeps on chip."""
    n_pages = 200003
    b = Both(3, n_pages, n_pages, 4)
    held = np.flatnonzero(np.arange(n_pages) % 1301 != 700)
    b.o.table[0, : held.size] = held
    b.o.length[0] = 4 * held.size
    b.o.refs[held] = 1
    b.load()
    b.extend([[1, 4 * 100 + 1]])
    b.extend([[2, 3], [1, 4]])
    b.extend([[2, 4 * 200]])                           # more than there are
    b.free([[1, 9], [0, 40]])
    b.extend([[1, 70000], [2, 70000]])
    b.compact(60000, apart=False)


@pytest.mark.parametrize("shift", [0, 1])
def test_compaction_of_every_array_apart_or_in_place(shift):
    """Each output may be the input's array or another one, 16-byte aligned or not."""
    db = lib()
    for mask in range(16):
        rng = np.random.default_rng(mask)
        b = Both(21, 9, 301, 4)
        b.extend(np.stack([rng.permutation(21), rng.integers(1, 36, 21)], 1))
        b.fork([[3, k, 1, 0] for k in range(21)])
        b.free([[k, 0] for k in range(0, 21, 3)])

        def other(t, k):
            if not mask >> k & 1:
                return t
            off = shift if k < 3 else 4 * shift        # free bits stay on 16 bytes
            return torch.full((t.numel() + off,), -5, dtype=torch.int32, device="cuda")[off:].view(t.shape)

        t = b.t
        out = db.PageTables(*(other(x, k) for k, x in enumerate((t.table, t.length, t.refs, t.free))), 4)
        for cap in (7, 150):
            moves, n = torch.zeros((cap, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
            db.page_compact(b.t, out, moves, n, b.ws)
            _, want = b.o.compact(cap)
            b.same(out)
            assert moves.cpu().numpy().view(np.uint32)[: int(n)].tolist() == want
            b.t = out


def test_rows_without_alignment():
    """A table, lengths and references at 4-byte addresses, a status at an odd one."""
    db = lib()
    b = Both(30, 7, 100, 8)
    at = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)
    b.t = db.PageTables(at(b.t.table), at(b.t.length), at(b.t.refs), b.t.free, 8)
    b._status = lambda n: torch.full((n + 2,), 99, dtype=torch.uint8, device="cuda")[1:]
    rng = np.random.default_rng(2)
    b.extend(np.stack([rng.permutation(15), rng.integers(1, 40, 15)], 1))
    b.fork([[k, 15 + k, int(b.o.length[k]), 0] for k in range(15)])
    b.extend(np.stack([rng.permutation(30), np.ones(30)], 1))
    b.free(np.stack([rng.permutation(30), rng.integers(0, 30, 30)], 1))


def test_workspace_is_left_as_it_was():
    b = Both(70, 5, 300, 4)
    rng = np.random.default_rng(0)
    claims = slice(256, 256 + 4 * 70)  # what a call finds must be what the first one found
    for _ in range(4):
        b.extend(np.stack([rng.integers(0, 72, 70), rng.integers(0, 6, 70)], 1))
        b.fork(np.stack([rng.integers(0, 70, 70), rng.integers(0, 72, 70), rng.integers(0, 3, 70), np.zeros(70)], 1))
        b.extend(np.stack([rng.permutation(70), np.ones(70)], 1))
        b.free(np.stack([rng.integers(0, 72, 70), rng.integers(0, 6, 70)], 1))
        assert int(b.ws[claims].sum()) == 0


def test_broken_tables_are_reported_and_stay_in_bounds():
    db = lib()
    T = 4

    def cache():
        b = Both(4, 4, 10, T)
        b.extend([[0, 9], [1, 6]])
        return b

    guard = 1 << 30
    for bad in (10, guard, 0x7FFFFFFF, -1, -5):
        b = cache()
        b.t.table[0, 1] = bad
        c = ctr()
        db.page_fork(b.t, u32([[0, 2, 9, 0]], 4), b.ws, ctr=c)
        assert c.cpu().tolist() == [3, 0, 0, db.ERR_PAGE_TABLE]
        b = cache()
        b.t.table[0, 1] = bad
        c = ctr()
        db.page_free(b.t, u32([[0, 0]], 2), b.ws, ctr=c)
        assert c.cpu().tolist() == [2, 0, 0, db.ERR_PAGE_TABLE]
        b = cache()
        b.t.table[1, 1] = bad
        c, st = ctr(), torch.zeros(2, dtype=torch.uint8, device="cuda")
        moves, n = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        db.page_extend(b.t, u32([[1, 1], [2, 1]], 2), moves, n, b.ws, status=st, ctr=c)
        assert c.cpu().tolist() == [1, 1, 0, db.ERR_PAGE_TABLE] and st.cpu().tolist() == [1, 0]
    b = cache()
    b.t.refs[1] = 0                                     # a page that no row should hold
    c = ctr()
    db.page_free(b.t, u32([[0, 0]], 2), b.ws, ctr=c)
    assert c.cpu()[3] == db.ERR_PAGE_TABLE and int(b.t.refs[1]) == 0
    b = cache()
    b.free([[1, 0]])
    b.extend([[2, 12]])
    b.free([[0, 0]])
    b.t.table[3, 3] = 99
    c = ctr()
    moves, n = torch.zeros((5, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    db.page_compact(b.t, b.t, moves, n, b.ws, ctr=c)
    assert c.cpu()[3] == db.ERR_PAGE_TABLE and int(b.t.table[3, 3]) == 99


# ------------------------------------------------------------------------ copy
def pool(rng, shape, dtype):
    a = rng.integers(0, 256, int(np.prod(shape)) * np.dtype(dtype).itemsize, dtype=np.uint8)
    return a.view(dtype).reshape(shape)


COPIES = [  # planes, pages, page, token axis (of the pool), type
    (1, 4, (1,), None, np.uint8),
    (1, 3, (1, 1), 2, np.uint8),
    (2, 9, (16, 2, 8), 2, np.int16),
    (3, 9, (5, 7, 3), 3, np.uint8),
    (3, 7, (5, 7, 3), 2, np.uint8),
    (2, 11, (5, 48, 116), 3, np.uint8),
    (2, 11, (48, 5, 116), 2, np.uint8),
    (4, 6, (8, 16, 128), 3, np.int16),
    (2, 5, (16, 8, 128), 2, np.int32),
    (5, 40, (8,), None, np.float32),
    (2, 30, (3, 6), 3, np.int16),
    (1, 5, (3, 33, 4), 3, np.int32),
    (2, 4, (2, 100, 90), 3, np.int16),
    (33, 20, (2, 3, 4), 3, np.uint8),
]


@pytest.mark.parametrize("planes,pages,page,token_dim,dtype", COPIES, ids=[str(c[:4]) for c in COPIES])
@pytest.mark.parametrize("layout", ["same", "apart", "page-major", "odd"])
def test_copy(planes, pages, page, token_dim, dtype, layout):
    db = lib()
    rng = np.random.default_rng([planes, pages, len(page), sum(page)])
    shape = (planes, pages) + page

    def place(a, how):
        t = torch.from_numpy(a.view(np.uint8).reshape(a.shape + (-1,)).copy()) if dtype != np.uint8 else torch.from_numpy(a.copy())
        t = t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[np.dtype(dtype).itemsize]).reshape(shape).cuda()
        if how == "page-major":
            return t.transpose(0, 1).contiguous().transpose(0, 1)
        if how == "odd":  # one element past an aligned base, pages 3 elements apart
            n = t[0, 0].numel()
            flat = torch.full((planes * pages * (n + 3) + 1,), 7, dtype=t.dtype, device="cuda")[1:]
            strides = t[0, 0].stride()
            v = flat.as_strided(shape, (pages * (n + 3), n + 3) + strides, flat.storage_offset())
            v.copy_(t)
            return v
        return t

    a, d = pool(rng, shape, dtype), pool(rng, shape, dtype)
    if layout == "same":
        d = a
    src = place(a, "odd" if layout == "odd" else "page-major" if layout == "page-major" else "plain")
    dst = src if layout == "same" else place(d, "odd" if layout == "odd" else "plain")
    order = rng.permutation(pages)
    k = max(1, pages // 2) if layout == "same" and pages > 1 else pages if layout != "same" else 0
    to = order[:k]
    frm = order[k:][:k] if layout == "same" else rng.integers(0, pages, k)
    to = to[: len(frm)]
    T = shape[token_dim] if token_dim is not None else 1
    tokens = rng.integers(0, T + 3, len(frm))
    tokens[rng.random(len(frm)) < 0.3] = po.ALL
    rec = np.stack([frm, to, tokens, rng.integers(0, 2**32, len(frm))], 1).astype(np.int64)
    bad = np.array([[pages, 0, po.ALL, 0], [0, pages, po.ALL, 0], [2**32 - 1, 2**31, 1, 0]], np.int64)
    rec = np.concatenate([rec, bad]) if len(rec) else bad
    rec = rec[rng.permutation(len(rec))]
    spare = np.concatenate([rec, np.array([[0, 0, po.ALL, 0]], np.int64)])  # past the count
    want = d.copy().view(dtype)
    po.copy(rec, want.copy() if layout == "same" else a, want, token_dim)
    c = ctr()
    db.page_copy(u32(spare, 4), dev([len(rec)]), src, dst, token_dim, ctr=c)
    torch.cuda.synchronize()
    got = np.ascontiguousarray(dst.cpu().numpy())
    assert (got.view(np.uint8) == np.ascontiguousarray(want).view(np.uint8).reshape(got.view(np.uint8).shape)).all()
    assert c.cpu().tolist() == [len(rec) - 3, 3, 0, 0]
    if layout == "odd":  # nothing between the pages is touched
        n = dst[0, 0].numel()
        gaps = dst.as_strided((planes * pages, 3), (n + 3, 1), dst.storage_offset() + n)
        assert (gaps == 7).all()


def test_copy_counts():
    """The count on the device bounds the list, and the list bounds the count."""
    db = lib()
    x = torch.arange(6 * 64, dtype=torch.int32, device="cuda").reshape(1, 6, 64)
    for count, done in ((0, 0), (1, 1), (2, 2), (3, 2), (0x7FFFFFFF, 2), (-1, 2)):
        y, c = torch.zeros_like(x), ctr()
        db.page_copy(u32([[5, 1, po.ALL, 0], [4, 2, 1, 0]], 4), dev([count]), x, y, None, ctr=c)
        assert c.cpu().tolist() == [done, 0, 0, 0]
        assert torch.equal(y[0, 1], x[0, 5] if done > 0 else torch.zeros_like(x[0, 1]))
        assert torch.equal(y[0, 2], x[0, 4] if done > 1 else torch.zeros_like(x[0, 1]))
    c = ctr()
    db.page_copy(u32(np.zeros((0, 4)), 4), dev([5]), x, y, None, ctr=c)
    assert c.cpu().tolist() == [0, 0, 0, 0]


def test_copy_offsets_past_32_bits():
    """A pool above 8 GiB: pages at both ends, in the last plane."""
    db = lib()
    planes, pages, words = 2, 70000, 16384  # 64 KiB pages: 4.6 GB a plane
    x = torch.zeros((planes, pages, words), dtype=torch.int32, device="cuda")
    for p in (0, 1, 40000, 69999):
        x[:, p] = torch.arange(words, dtype=torch.int32, device="cuda") + p
        x[1, p] *= -1
    db.page_copy(u32([[69999, 2, po.ALL, 0], [0, 69998, po.ALL, 0], [40000, 35000, 1, 0]], 4), dev([3]), x, x, None)
    assert torch.equal(x[:, 2], x[:, 69999]) and torch.equal(x[:, 69998], x[:, 0]) and torch.equal(x[:, 35000], x[:, 40000])
    assert int(x[:, 3].abs().sum()) == 0 and int(x[:, 69997].abs().sum()) == 0


@pytest.mark.parametrize("width", [4, 256])  # short runs, and pages of 16 KiB
def test_copy_to_and_from_pinned_host_memory(width):
    db = lib()
    rng = np.random.default_rng(1)
    x = torch.from_numpy(pool(rng, (3, 8, 16, width), np.int32)).cuda()
    h = torch.zeros((3, 5, 16, width), dtype=torch.int32).pin_memory()
    db.page_copy(u32([[7, 0, po.ALL, 0], [2, 4, 5, 0]], 4), dev([2]), x, h, 2)
    torch.cuda.synchronize()
    assert torch.equal(h[:, 0], x[:, 7].cpu()) and torch.equal(h[:, 4, :5], x[:, 2, :5].cpu())
    assert int(h[:, 4, 5:].abs().sum()) == 0 and int(h[:, 1].abs().sum()) == 0
    db.page_copy(u32([[0, 3, po.ALL, 0]], 4), dev([1]), h, x, 2)
    assert torch.equal(x[:, 3].cpu(), h[:, 0])


# ----------------------------------------------------------- streams and graphs
def beam_step(db, t, ws, cut, fork, grow, moves, n, pool_, stream=None):
    db.page_free(t, cut, ws, stream=stream)
    db.page_fork(t, fork, ws, stream=stream)
    db.page_extend(t, grow, moves, n, ws, stream=stream)
    db.page_copy(moves, n, pool_, pool_, 2, stream=stream)


def beams(seed):
    """8 parents, 24 beams behind them, and the oracle after the step."""
    rng = np.random.default_rng(seed)
    b = Both(32, 6, 250, 8)
    b.extend(np.stack([np.arange(8), rng.integers(9, 40, 8)], 1))
    parent = np.repeat(np.arange(8), 3)
    child = 8 + rng.permutation(24)
    b.fork(np.stack([parent, child, b.o.length[parent], child], 1))
    b.extend(np.stack([child, np.ones(24)], 1))
    parent = parent[rng.permutation(24)]
    cut = np.stack([child, np.zeros(24)], 1)
    fork = np.stack([parent, child, b.o.length[parent], child], 1)
    grow = np.stack([child, np.ones(24)], 1)
    data = pool(rng, (2, 250, 8, 6), np.int16)
    b.o.free(cut)
    b.o.fork(fork)
    _, _, moves = b.o.extend(grow)
    want = data.copy()
    po.copy(moves, data, want, 2)
    return b, (u32(cut, 2), u32(fork, 4), u32(grow, 2)), torch.from_numpy(data).cuda(), want, moves


@pytest.mark.parametrize("way", ["default", "stream", "graph"])
def test_a_beam_step(way):
    db = lib()
    b, req, x, want, moves = beams(11)
    m, n = torch.zeros((24, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    if way == "default":
        beam_step(db, b.t, b.ws, *req, m, n, x)
    elif way == "stream":
        s = torch.cuda.Stream()
        beam_step(db, b.t, b.ws, *req, m, n, x, stream=s)
        s.synchronize()
    else:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            beam_step(db, b.t, b.ws, *req, m, n, x)
        for _ in range(3):  # a step that finds its own result does it again
            g.replay()
    b.same()
    assert m.cpu()[: int(n)].tolist() == moves
    assert (x.cpu().numpy() == want).all()


def test_a_graph_of_larger_batches():
    """Clusters and second kernels, launched as dependents, in a captured graph."""
    db = lib()
    b = Both(3000, 40, 70001, 4)
    rng = np.random.default_rng(4)
    b.extend(np.stack([np.arange(1500), rng.integers(1, 70, 1500)], 1))
    child = 1500 + rng.permutation(1500)
    parent = rng.integers(0, 1500, 1500)
    fork = np.stack([parent, child, b.o.length[parent], child], 1)
    grow = np.stack([child, rng.integers(1, 30, 1500)], 1)
    cut = np.stack([child, np.zeros(1500)], 1)
    req = u32(cut, 2), u32(fork, 4), u32(grow, 2)
    m, n = torch.zeros((1500, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        db.page_free(b.t, req[0], b.ws)
        db.page_fork(b.t, req[1], b.ws)
        db.page_extend(b.t, req[2], m, n, b.ws)
    b.o.free(cut)
    b.o.fork(fork)
    _, _, moves = b.o.extend(grow)
    for _ in range(3):
        g.replay()
        b.same()
        assert m.cpu()[: int(n)].tolist() == moves


def test_tables_past_32_bits():
    """Rows whose entries lie beyond 2^32 of the table's first."""
    db = lib()
    columns, n_seqs, n_pages = 1 << 20, 4100, 500       # 17 GB of table
    t = db.PageTables.empty(n_seqs, columns, n_pages, 4)
    ws = db.workspace(db.page_workspace_size(n_seqs, n_pages))
    o = po.Cache(3, 100, n_pages, 4)                     # the rows that are used
    rows = np.array([0, 4097, 4099])

    def same():
        torch.cuda.synchronize()
        for k, s in enumerate(rows):
            assert (t.table[s, :100].cpu().numpy() == o.table[k]).all()
            assert int(t.length[s]) == o.length[k]
        assert (t.refs.cpu().numpy() == o.refs).all()
        assert (t.free.cpu().numpy().view(np.uint32) == po.pack_free(o.refs)).all()

    m, n = torch.zeros((250, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    db.page_extend(t, u32([[4099, 311], [0, 9]], 2), m, n, ws)
    o.extend([[2, 311], [0, 9]])
    same()
    db.page_fork(t, u32([[4099, 4097, 310, 0]], 4), ws)
    o.fork([[2, 1, 310, 0]])
    same()
    db.page_extend(t, u32([[4097, 1], [4099, 40]], 2), m, n, ws)
    _, _, moves = o.extend([[1, 1], [2, 40]])
    same()
    assert m.cpu()[: int(n)].tolist() == moves
    db.page_free(t, u32([[4099, 30], [0, 0]], 2), ws)
    o.free([[2, 30], [0, 0]])
    same()
    db.page_compact(t, t, m, n, ws)
    o.compact(250)
    same()
    assert int((t.table[1:4097, :8] != -1).sum()) == 0


def test_compaction_beside_readers_of_the_old_tables():
    """The old tables and their pages stay whole while the moves are made."""
    db = lib()
    rng = np.random.default_rng(5)
    b = Both(20, 8, 190, 4)
    b.extend(np.stack([np.arange(20), rng.integers(1, 32, 20)], 1))
    b.free([[k, 0] for k in range(0, 20, 3)])
    x = torch.from_numpy(pool(rng, (2, 190, 4, 5), np.int16)).cuda()

    def read(t):
        i = t.table.long()
        return torch.where((i >= 0)[None, :, :, None, None], x[:, i.clamp(min=0)], 0)

    before, old = read(b.t), b.t
    moves, n = torch.zeros((95, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = db.PageTables(torch.empty_like(old.table), old.length, torch.empty_like(old.refs), torch.empty_like(old.free), 4)
    db.page_compact(old, out, moves, n, b.ws)
    db.page_copy(moves, n, x, x, 2)
    assert int(n) > 0
    assert torch.equal(read(old), before) and torch.equal(read(out), before)
    assert int(out.table.max()) == int((out.refs > 0).sum()) - 1


# --------------------------------------------------------------------- refusals
def test_refusals():
    db = lib()
    b = Both(4, 3, 40, 4)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    big = u32([[k % 4, 1] for k in range(5)], 2)
    with pytest.raises(db.DescBuildError, match="-22"):  # more requests than sequences
        db.page_free(b.t, big, b.ws)
    with pytest.raises(ValueError):                      # moves shorter than the batch
        db.page_extend(b.t, big[:3], i32(2, 4), i32(1), b.ws)
    with pytest.raises(db.DescBuildError, match="-28"):  # workspace
        db.page_fork(b.t, u32([[0, 1, 0, 0]], 4), b.ws[:256])
    with pytest.raises(ValueError):
        db.page_free(b.t, big[:2], b.ws, status=torch.zeros(1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):                      # a table's type, a free word too few
        db.PageTables(b.t.table.long(), b.t.length, b.t.refs, b.t.free, 4)
    with pytest.raises(ValueError):
        db.PageTables(b.t.table, b.t.length, b.t.refs, b.t.free[:1], 4)
    other = db.PageTables.empty(4, 3, 41, 4)
    with pytest.raises(db.DescBuildError, match="-22"):  # another cache's sizes
        db.page_compact(b.t, other, i32(3, 4), i32(1), b.ws)
    x = i32(2, 6, 4, 8)
    with pytest.raises(ValueError):                      # page shapes
        db.page_copy(i32(1, 4), i32(1), x, i32(2, 6, 8, 4), 2)
    with pytest.raises(ValueError):
        db.page_copy(i32(1, 4), i32(1), x, x, 4)
    with pytest.raises(ValueError):                      # pages not contiguous
        db.page_copy(i32(1, 4), i32(1), x.transpose(2, 3), x.transpose(2, 3), 2)
    with pytest.raises(db.DescBuildError, match="-22"):  # pages over one another
        db.page_copy(i32(1, 4), i32(1), x, x[:, :1].expand(2, 6, 4, 8), 2)
    b.same()
