"""The paged cache's calls where a cluster of CTAs plans a batch (free and fork from 257 requests on,
extend from 1,025 or from 262,145 pages on) or a gang has several CTAs: sequences named twice, out of
range or by others' requests, batches that are short, tables that are broken, pages far apart. After
every call the parts of the workspace that must be zero between calls are.

Everything is whole numbers, so every comparison is for equality."""

import numpy as np
import pytest

from gpu_util import lib, need_gpu
from oracle import pages as po
from test_gpu_pages import Both, ctr, u32

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def up256(x):
    return -(-x // 256) * 256


class Kept(Both):
    """Both, with a look at the workspace after each comparison: the head's counts, and each
    sequence's claim, each page's holders and their last are zero between calls."""

    def workspace_is_zero(self):
        n_seqs, n_pages = self.o.length.size, self.o.refs.size
        end = 256 + up256(4 * n_seqs) + 2 * up256(4 * n_pages)
        assert int(self.ws[:16].count_nonzero()) == 0, "released, done, bad"
        assert int(self.ws[256:end].count_nonzero()) == 0, "claim, holders, latest"

    def same(self, t=None):
        super().same(t)
        self.workspace_is_zero()


# Requests of a batch, and what it reaches: teams of 2 to 8 CTAs with and without a second kernel
# (which the table's width decides), the gang of 1,024 threads, more requests than a cluster has
# threads (which are planned in rounds).
SHAPES = [  # sequences, columns, pages, page tokens
    (300, 12, 1800, 4),
    (1000, 6, 3000, 4),
    (1500, 6, 5000, 5),
    (2000, 40, 30000, 2),
    (9001, 3, 14000, 4),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
@pytest.mark.parametrize("seed", range(2))
def test_histories_with_requests_that_do_not_count(shape, seed):
    n_seqs, columns, n_pages, page = shape
    rng = np.random.default_rng([seed, n_seqs])
    b = Kept(*shape)
    far = columns * page
    seen = {0: set(), 1: set(), 2: set()}

    def ids(k):
        """Random sequences: about a third of them named before, some out of range."""
        seq = rng.integers(0, n_seqs, k)
        out = rng.random(k) < 0.02
        seq[out] = rng.choice([n_seqs, n_seqs + 1, 0x7FFFFFFF, 0x80000000, 0xFFFFFFFF], out.sum())
        return seq

    def told(kind, before):
        seen[kind] |= set(before)

    for step in range(4):
        k = n_seqs if step % 2 == 0 else int(rng.integers(max(257, n_seqs * 3 // 4), n_seqs + 1))
        # prompts, most of them of a page or two, some longer than a row
        take = np.where(rng.random(k) < 0.1, rng.integers(0, far + 3, k), rng.integers(0, 2 * page, k))
        seq = ids(k)
        told(0, b.o.copy().extend(np.stack([seq, take], 1))[0])
        b.extend(np.stack([seq, take], 1))
        # some end, and others fork from what is there: many children of a few parents
        cut = np.stack([ids(k), np.where(rng.random(k) < 0.6, 0, rng.integers(0, far, k))], 1)
        told(1, b.o.copy().free(cut)[0])
        b.free(cut)
        few = np.flatnonzero(b.o.length > 0)[:7]
        parent = np.where(rng.random(k) < 0.5, ids(k), rng.choice(few, k))
        has = np.append(b.o.length, 1)[np.minimum(parent, n_seqs)]
        child = ids(k)
        fork = np.stack([parent, child, rng.integers(0, has + 2), child], 1)
        told(2, b.o.copy().fork(fork)[0])
        b.fork(fork)
        # a token or two for many: copies of partly filled pages, whole or part of their holders there
        b.extend(np.stack([ids(k), rng.integers(0, 3, k)], 1))
        # a page more for each than are free: refused, and nothing changes
        short = np.stack([ids(k), np.full(k, far // 2)], 1)
        status = b.o.copy().extend(short)[0]
        told(0, status)
        b.extend(short)
    assert seen[0] == {po.OK, po.INVALID, po.SHORT} and seen[1] == seen[2] == {po.OK, po.INVALID}
    po.check(b.o)


@pytest.mark.parametrize("n,columns", [(300, 30), (1500, 40), (1500, 100)])
def test_a_team_frees_and_forks_rows_of_more_than_a_few_entries(n, columns):
    """Few entries in all, so that the team does them itself, but more a row than a thread takes."""
    rng = np.random.default_rng(n + columns)
    b = Kept(n, columns, 8000, 4)
    some = rng.permutation(n)[: n // 5]
    b.extend(np.stack([some, rng.integers(4 * 5, 4 * 12, some.size)], 1))
    cut = np.stack([rng.permutation(n), rng.integers(0, 4, n)], 1)
    assert (b.o.length > 4 * 4).sum() > 8 and b.o.refs.sum() < 8192
    b.free(cut)
    b.extend(np.stack([some[: n // 20], rng.integers(4 * 5, 4 * 12, n // 20)], 1))
    parent = some[rng.integers(0, n // 20, n)]
    b.fork(np.stack([parent, rng.permutation(n), np.minimum(b.o.length[parent], rng.integers(0, 30, n)), parent], 1))
    b.free(np.stack([rng.permutation(n), np.zeros(n)], 1))
    assert b.o.refs.sum() == 0


def test_free_pages_in_more_words_than_a_cta_keeps():
    """A pool of more than 262,144 pages, so that a cluster plans, its free pages so far apart that
    the batch's lie in more words than a CTA keeps on chip: the second kernel finds them."""
    n_pages = 300007
    b = Kept(4, n_pages, n_pages, 4)
    held = np.flatnonzero(np.arange(n_pages) % 1301 != 700)
    b.o.table[0, : held.size] = held
    b.o.length[0] = 4 * held.size
    b.o.refs[held] = 1
    b.load()
    b.extend([[1, 4 * 100 + 1], [3, 5]])                # 103 pages over 4,200 words
    assert int(b.o.table[1, 100]) > 32 * 2048
    b.free([[1, 9]])
    b.extend([[2, 3], [1, 4]])                          # two pages, in few words
    b.fork([[1, 3, 0, 0], [2, 2, 1, 0]])                # neither is empty, or another
    b.extend([[2, 4 * 240]])                            # more than there are
    b.free([[0, 40]])
    b.extend([[1, 70000], [2, 70000]])
    b.compact(20000)


def test_a_team_in_a_large_pool():
    """More than 1,024 requests on a pool of more than 262,144 pages, ids named twice among them."""
    n_pages = 300007
    rng = np.random.default_rng(9)
    b = Kept(3000, 40, n_pages, 4)
    held = np.flatnonzero(rng.random(n_pages) < 0.6)[: 2000 * 40]
    b.o.table[:2000] = held.reshape(2000, 40)
    b.o.length[:2000] = 160
    b.o.refs[held] = 1
    b.load()
    b.free(np.stack([rng.permutation(3000), rng.integers(0, 170, 3000)], 1))
    b.extend(np.stack([rng.permutation(3000), rng.integers(0, 60, 3000)], 1))
    b.extend(np.stack([rng.integers(0, 3100, 3000), rng.integers(0, 3, 3000)], 1))
    po.check(b.o)


# ------------------------------------------------------------- gangs of several CTAs
def test_gangs_of_several_ctas_leave_the_head_as_it_was():
    n, columns, n_pages = 100, 400, 40000
    rng = np.random.default_rng(3)
    b = Kept(n, columns, n_pages, 4)
    b.extend(np.stack([rng.permutation(50), rng.integers(500, 1300, 50)], 1))
    parent = rng.integers(0, 50, 50)
    b.fork(np.stack([parent, 50 + rng.permutation(50), np.minimum(b.o.length[parent], rng.integers(0, 1300, 50)), parent], 1))
    b.extend(np.stack([rng.permutation(n), rng.integers(0, 90, n)], 1))
    b.free(np.stack([rng.integers(0, 110, n), rng.integers(0, 1300, n)], 1))
    rows = np.flatnonzero(b.o.length > 1)
    b.t.table[int(rows[0]), 0] = 1 << 30
    c = ctr()
    b.db.page_free(b.t, u32(np.stack([rng.permutation(n), np.zeros(n)], 1), 2), b.ws, ctr=c)
    assert int(c[3]) == b.db.ERR_PAGE_TABLE
    b.workspace_is_zero()


# --------------------------------------------------------------- broken tables
BAD = (-1, -2, -5, 1 << 30, 0x7FFFFFFF)  # and the number of pages
BROKEN = [(300, 12, 3000), (1500, 40, 30000), (9001, 3, 27003)]  # team alone; second kernel; rounds


def broken(n, columns, n_pages):
    """A cache of exclusive pages, and the entries (row, column) that will not be pages."""
    rng = np.random.default_rng(n)
    b = Kept(n, columns, n_pages, 4)
    most = min(columns * 4, n_pages * 4 // n - 4)
    b.extend(np.stack([rng.permutation(n), rng.integers(1, most, n)], 1))
    rows = np.flatnonzero(b.o.length > 0)
    rows = rows[rng.permutation(rows.size)[: rows.size // 9]]
    return rng, b, rows


def plant(b, rows, cols, n_pages):
    bad = np.array(BAD + (n_pages,))[np.arange(rows.size) % 6]
    b.o.table[rows, cols] = bad
    at = [torch.from_numpy(x).cuda() for x in (rows, cols)]
    b.t.table[at[0], at[1]] = torch.from_numpy(bad.astype(np.int32)).cuda()


@pytest.mark.parametrize("n,columns,n_pages", BROKEN)
def test_broken_rows_are_freed_and_reported(n, columns, n_pages):
    rng, b, rows = broken(n, columns, n_pages)
    plant(b, rows, rng.integers(0, b.o.pages(1) + (b.o.length[rows] - 1) // 4), n_pages)
    keep = np.where(rng.random(n) < 0.5, 0, rng.integers(0, columns * 4, n))
    seq = rng.permutation(n)
    released, reported = 0, 0
    for s, k in zip(seq.tolist(), keep.tolist()):
        if k >= b.o.length[s]:
            continue
        for col in range(b.o.pages(k), b.o.pages(b.o.length[s])):
            p = int(b.o.table[s, col])
            b.o.table[s, col] = -1
            if 0 <= p < n_pages:
                b.o.refs[p] -= 1
                released += 1
            else:
                reported += 1
        b.o.length[s] = k
    assert reported
    c = ctr()
    b.db.page_free(b.t, u32(np.stack([seq, keep], 1), 2), b.ws, ctr=c)
    b.same()
    assert c.cpu().tolist() == [released, 0, 0, b.db.ERR_PAGE_TABLE]


@pytest.mark.parametrize("n,columns,n_pages", BROKEN)
def test_broken_rows_are_forked_and_reported(n, columns, n_pages):
    rng, b, rows = broken(n, columns, n_pages)
    kids = np.setdiff1d(rng.permutation(n)[: n - 20], rows)[: n * 2 // 3]
    b.free(np.stack([kids, np.zeros(kids.size)], 1))
    plant(b, rows, np.zeros(rows.size, np.int64), n_pages)
    parent = rows[rng.integers(0, rows.size, kids.size)]
    tokens = rng.integers(0, b.o.length[parent] + 1)
    taken = 0
    for p, k, t in zip(parent.tolist(), kids.tolist(), tokens.tolist()):
        m = b.o.pages(t)
        row = b.o.table[p, :m]
        b.o.table[k, :m] = row
        np.add.at(b.o.refs, row[(row >= 0) & (row < n_pages)], 1)
        b.o.length[k] = t
        taken += m
    c = ctr()
    b.db.page_fork(b.t, u32(np.stack([parent, kids, tokens, kids], 1), 4), b.ws, ctr=c)
    b.same()
    assert c.cpu().tolist() == [taken, 0, 0, b.db.ERR_PAGE_TABLE]


@pytest.mark.parametrize("n,columns,n_pages", BROKEN[1:])
def test_broken_last_pages_are_refused_and_reported(n, columns, n_pages):
    """A request whose row names no page where its last one should be is invalid; the others are served."""
    rng, b, rows = broken(n, columns, n_pages)
    rows = rows[b.o.length[rows] % 4 != 0]
    plant(b, rows, (b.o.length[rows] - 1) // 4, n_pages)
    seq, take = rng.permutation(n), np.ones(n, np.int64)
    gone = np.isin(seq, rows) & (b.o.length[seq] + 1 <= columns * 4)
    assert gone.any()
    status, counters, want = b.o.extend(np.stack([np.where(gone, n, seq), take], 1))
    c, st = ctr(), torch.full((n,), 99, dtype=torch.uint8, device="cuda")
    moves, m = torch.full((n, 4), -9, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    b.db.page_extend(b.t, u32(np.stack([seq, take], 1), 2), moves, m, b.ws, status=st, ctr=c)
    b.same()
    assert st.cpu().tolist() == status
    assert c.cpu().tolist() == counters[:3] + [b.db.ERR_PAGE_TABLE]
    assert moves.cpu()[: int(m)].tolist() == want


@pytest.mark.parametrize("n,columns,n_pages", BROKEN)
def test_broken_rows_stay_through_a_compaction(n, columns, n_pages):
    """In one CTA, and with moves and tables by the whole GPU."""
    rng, b, rows = broken(n, columns, n_pages)
    b.free(np.stack([np.setdiff1d(rng.permutation(n)[: n // 3], rows)] * 2, 1) * [1, 0])
    plant(b, rows, np.zeros(rows.size, np.int64), n_pages)
    c = ctr()
    cap = n_pages // 2
    moves, m = torch.full((cap, 4), -9, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    b.db.page_compact(b.t, b.t, moves, m, b.ws, ctr=c)
    counters, want = b.o.compact(cap)
    b.same()
    assert c.cpu().tolist() == counters[:3] + [b.db.ERR_PAGE_TABLE] and len(want) > 0
    assert moves.cpu().numpy().view(np.uint32)[: int(m)].tolist() == want
