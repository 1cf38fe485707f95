"""The paged cache's oracle against hand-worked cases, its invariants, and planted mistakes."""

import os

import numpy as np
import pytest

from conftest import ROOT
from oracle import pages

SRC = os.path.join(ROOT, "oracle", "pages.py")


def hand_cases(m):
    """Worked by hand on a cache of 4 sequences, 4 columns, 8 pages of 4 tokens."""
    c = m.Cache(4, 4, 8, 4)
    # 5 tokens take pages 0 and 1, 8 take 2 and 3
    assert c.extend([[0, 5], [2, 8]]) == ([0, 0], [4, 0, 0, 0], [])
    assert c.table.tolist() == [[0, 1, -1, -1], [-1] * 4, [2, 3, -1, -1], [-1] * 4]
    # 1 and 3 take sequence 0's tokens: both its pages are in three rows
    assert c.fork([[0, 1, 5, 0], [0, 3, 5, 0]]) == ([0, 0], [4, 0, 0, 0])
    assert c.refs.tolist() == [3, 3, 1, 1, 0, 0, 0, 0] and c.length.tolist() == [5, 5, 8, 5]
    # a third fork onto a sequence that holds tokens, of more than the parent has, of itself
    assert c.fork([[2, 1, 1, 0], [2, 9, 1, 0], [3, 3, 1, 0]]) == ([1, 1, 1], [0, 3, 0, 0])
    # one token each for the three holders of page 1: the first two copy its one token, the
    # last finds itself alone; sequence 2 is full to the page and takes a new one
    status, ctr, moves = c.extend([[3, 1], [0, 1], [2, 1], [1, 1]])
    assert (status, ctr) == ([0] * 4, [3, 0, 0, 0])
    assert moves == [[1, 4, 1, 0], [1, 5, 1, 0]]
    assert c.table.tolist() == [[0, 5, -1, -1], [0, 1, -1, -1], [2, 3, 6, -1], [0, 4, -1, -1]]
    assert c.refs.tolist() == [3, 1, 1, 1, 1, 1, 1, 0]
    # 11 more tokens for sequence 1 pass its 16; 8 more for 0 and 2 need four pages of one
    status, ctr, moves = c.extend([[1, 11], [0, 8], [2, 7], [7, 1], [0, 1]])
    assert (status, ctr, moves) == ([1, 2, 2, 1, 1], [3, 3, 2, 0], [])
    # the whole of 3 goes (page 0 stays with 0 and 1), and all but 4 tokens of 2 (3 and 6 go)
    assert c.free([[3, 0], [2, 4], [2, 0], [1, 6]]) == ([0, 0, 1, 0], [3, 1, 0, 0])
    assert c.refs.tolist() == [2, 1, 1, 0, 0, 1, 0, 0] and c.length.tolist() == [6, 6, 4, 0]
    assert m.pack_free(c.refs).tolist() == [0b11011000]
    # 4 live pages: page 5 is the highest, page 3 the lowest free one
    d = c.copy()
    assert d.compact(0) == ([1, 0, 1, 0], []) and (d.table == c.table).all()
    assert c.compact(4) == ([1, 0, 0, 0], [[5, 3, m.ALL, 0]])
    assert c.table.tolist() == [[0, 3, -1, -1], [0, 1, -1, -1], [2, -1, -1, -1], [-1] * 4]
    assert c.refs.tolist() == [2, 1, 1, 1, 0, 0, 0, 0]
    m.check(c)
    # two holders in the batch and one outside it: both copy
    c.fork([[0, 3, 6, 0]])
    c.free([[2, 0]])
    c.fork([[0, 2, 5, 0]])
    _, _, moves = c.extend([[2, 1], [3, 2]])
    assert moves == [[3, 2, 1, 0], [3, 4, 2, 0]]
    m.check(c)
    # a shared page that is full is not copied
    c.free([[3, 0]])
    c.fork([[0, 3, 4, 0]])
    assert c.extend([[3, 1]]) == ([0], [1, 0, 0, 0], [])
    m.check(c)
    # 4 of the 6 pages stay, among them 3 and 4 in two rows; the highest goes to the lowest place
    c = m.Cache(4, 3, 6, 4)
    c.extend([[0, 4], [1, 8], [2, 8]])
    c.fork([[2, 3, 7, 0]])
    assert c.free([[0, 0], [1, 3], [2, 6]]) == ([0] * 3, [2, 0, 0, 0])
    assert c.table.tolist() == [[-1] * 3, [1, -1, -1], [3, 4, -1], [3, 4, -1]]
    assert c.compact(2) == ([2, 0, 0, 0], [[4, 0, m.ALL, 0], [3, 2, m.ALL, 0]])
    assert c.table[1:].tolist() == [[1, -1, -1], [2, 0, -1], [2, 0, -1]]
    assert c.refs.tolist() == [2, 1, 2, 0, 0, 0]
    # short by one: of two holders the first needs a copy, the last keeps the page all the same
    c = m.Cache(3, 3, 2, 4)
    c.extend([[0, 6]])
    c.fork([[0, 1, 6, 0]])
    assert c.extend([[1, 1], [0, 1]]) == ([2, 2], [1, 0, 2, 0], [])
    m.check(c)
    # the first tokens of a page, token axis inside
    a = np.arange(2 * 3 * 2 * 4).reshape(2, 3, 2, 4)
    b = np.zeros_like(a)
    m.copy([[2, 0, 3, 0], [1, 1, m.ALL, 0], [7, 2, 1, 0]], a, b, 3)
    assert (b[:, 0, :, :3] == a[:, 2, :, :3]).all() and (b[:, 0, :, 3] == 0).all()
    assert (b[:, 1] == a[:, 1]).all() and (b[:, 2] == 0).all()


def test_hand_cases():
    hand_cases(pages)


MUTANTS = [
    ("a copied page keeps its reference", "self.refs[shared] -= 1\n", "pass\n"),
    ("every partly filled page is copied", "> 1:\n                shared", "> 0:\n                shared"),
    ("a full page is copied", "length % self.T != 0 and ", ""),
    ("pages are counted down", "return -(-int(tokens) // self.T)", "return int(tokens) // self.T"),
    ("a short batch leaves what it took", "self.table, self.length, self.refs = was.table, was.length, was.refs", "pass"),
    ("free keeps the partly kept page's column", "for c in range(self.pages(keep),", "for c in range(int(keep) // self.T,"),
    ("forked pages take no reference", "self.refs[page] += 1\n                taken", "taken"),
    ("a fork may go onto a held sequence", "and before[child] == 0", ""),
    ("a moved page has one row", "self.refs[lo], self.refs[hi] = self.refs[hi], 0", "self.refs[lo], self.refs[hi] = 1, 0"),
    ("the lowest live page moves first", "lo, hi = 0, refs.size - 1", "lo, hi = 0, live"),
    ("the tables keep a moved page's old name", "self.table[self.table == hi] = lo", "pass"),
    ("a move takes the whole page", "min(tokens, src.shape[token_dim])", "src.shape[token_dim]"),
    ("a sequence may be named twice", "or seq in seen:", "or False:"),
]


@pytest.mark.parametrize("name,old,new", MUTANTS, ids=[m[0] for m in MUTANTS])
def test_planted_mistakes_are_caught(name, old, new):
    text = open(SRC).read()
    assert text.count(old) == 1, "the mutant's anchor moved"
    mod = type(pages)("mutant")
    exec(compile(text.replace(old, new), "mutant", "exec"), mod.__dict__)
    with pytest.raises((AssertionError, IndexError, ValueError)):
        hand_cases(mod)


@pytest.mark.parametrize("seed", range(6))
def test_random_histories_keep_the_invariants(seed):
    rng = np.random.default_rng(seed)
    c = pages.Cache(9, int(rng.integers(1, 7)), int(rng.integers(1, 60)), int(rng.integers(1, 6)))
    for _ in range(60):
        k = int(rng.integers(0, 10))
        op = rng.integers(0, 4)
        seq = rng.integers(0, 10, k)
        if op == 0:
            c.extend(np.stack([seq, rng.integers(0, 9, k)], 1))
        elif op == 1:
            c.fork(np.stack([rng.integers(0, 10, k), seq, rng.integers(0, 12, k), seq], 1))
        elif op == 2:
            c.free(np.stack([seq, rng.integers(0, 12, k)], 1))
        else:
            cap = int(rng.integers(0, 8))
            ctr, moves = c.compact(cap)
            if ctr[2] == 0:  # all of them made: the live pages are the lowest
                live = int((c.refs > 0).sum())
                assert (c.refs[:live] > 0).all() and (c.refs[live:] == 0).all()
        pages.check(c)


def test_one_batch_is_its_requests_one_at_a_time():
    """An extension that is not short gives the rows, references and moves of its requests made
    one call at a time (the pages differ only by what a single call finds lowest)."""
    rng = np.random.default_rng(3)
    a = pages.Cache(8, 6, 60, 4)
    a.extend([[0, 7], [1, 13]])
    a.fork([[0, 2, 7, 0], [0, 3, 6, 0], [1, 4, 13, 0], [1, 5, 10, 0]])
    b = a.copy()
    req = np.stack([rng.permutation(6), rng.integers(1, 9, 6)], 1)
    status, ctr, moves = a.extend(req)
    each = [b.extend(r[None]) for r in req]
    assert [s for e in each for s in e[0]] == status
    assert [x for e in each for x in e[2]] == moves
    assert (a.table == b.table).all() and (a.refs == b.refs).all() and (a.length == b.length).all()
