"""The oracle of a paged cache's contents against hand-worked cases, and planted mistakes."""

import os
import types

import numpy as np
import pytest

from conftest import ROOT
from oracle import cachedata

SRC = os.path.join(ROOT, "oracle", "cachedata.py")
F = np.float32


def tables(m, seq, start, rows, fresh, length=(3, 6), **kw):
    """Two sequences on pages of 4 tokens: the first on page 2, the second on pages 0 and 3."""
    return m.Batch([[2, -1], [0, 3]], length, 4, 4, seq, start, rows, fresh, **kw)


def codes(m):
    # halves between codes go to the even one: 1.0625 lies between 1 (56) and 1.125 (57), 1.1875 between 57 and 58
    assert m.e4m3_code([0, 1, 1.0625, 1.1875, 448, 460, -1, 2.0**-9, 2.0**-10, 3 * 2.0**-10]).tolist() == [
        0, 56, 56, 58, 126, 126, 184, 1, 0, 2]
    assert m.E4M3[126] == 448 and np.isnan(m.E4M3[127]) and m.E4M3[8] == 2.0**-6
    c, s = m.quantise(F([896, 448, -2, 0]), "e4m3")
    assert s == 2 and c.tolist() == [126, 118, 184, 0]
    c, s = m.quantise(F([-254, 1, 3, 5]), "i8")  # by twos: halves 0.5, 1.5, 2.5
    assert s == 2 and c.view(np.int8).tolist() == [-127, 0, 2, 2]
    for row in ([0, 0], [1e-45, 0], [1e-40, 0]):  # of the last, 127 / 1e-40 is infinite
        c, s = m.quantise(F(row), "i8")
        assert s == 0 and c.tolist() == [0, 0]
    for row in ([np.inf, 1], [np.nan, 1], [1, -np.inf]):
        c, s = m.quantise(F(row), "e4m3")
        assert np.isnan(s) and c.tolist() == [0, 0]


def moves(m):
    pool = np.zeros((4, 4, 1, 2), F)
    b = tables(m, [1, 0], [0, 3, 4], 5, True)
    rows = np.arange(10, dtype=F).reshape(5, 1, 2)
    m.write(b, rows, pool, None, "f32", lambda x: x)
    # positions 3, 4, 5 of the second sequence and position 2 of the first
    assert pool[0, 3].tolist() == [[0, 1]] and pool[3, 0].tolist() == [[2, 3]] and pool[3, 1].tolist() == [[4, 5]]
    assert pool[2, 2].tolist() == [[6, 7]] and (pool != 0).sum() == 7
    assert b.status == [0, 0] and b.counters() == [4, 0, 0, 0]
    pool[3, 2] = 9  # behind the sequence's last token
    out = np.full((5, 1, 2), -1.0)
    b = tables(m, [1, 0], [0, 4, 5], 5, False)
    m.read(b, [4, 2], m.values(pool, None), out)
    assert out[:, 0].tolist() == [[2, 3], [4, 5], [0, 0], [0, 0], [6, 7]]
    # more rows than tokens are no new tokens; neither is a sequence that is not there, nor one longer than its table
    b = tables(m, [0, 2, 1], [0, 4, 4, 4], 4, True, length=(3, 9))
    assert b.status == [1, 1, 1] and b.counters() == [0, 3, 0, 0]
    assert tables(m, [0], [0, 3], 3, True, max_tokens=2).status == [1]
    b = m.Batch(np.zeros((1, 1 << 10), np.int64), [-(1 << 31)], 4, 1 << 22, [0], [0, 1], 1, True)
    assert b.status == [1]  # 2^31 tokens, of 2^32 places
    assert tables(m, [0, 0, 0], [2, 1, 3, 4], 3, False).status == [1, 0, 1]
    # page 9 of 4 is none: its token reads as zeros, and the counters say so
    b = m.Batch([[9]], [2], 4, 4, [0], [0, 2], 2, False)
    out[:] = 5
    m.read(b, None, pool, out)
    assert (out[:2] == 0).all() and b.counters() == [2, 0, 0, 8]


def attention(m):
    # keys 0, 0, ln 2 in one direction, values 4, 8, 1: a query of 1 weighs the tokens 1, 1, 2
    keys, vals = np.zeros((4, 4, 1, 2)), np.zeros((4, 4, 1, 2))
    keys[2, 2, 0, 0] = np.log(2)
    vals[2, :3, 0, 0] = [4, 8, 1]
    q = np.zeros((2, 2, 2))
    q[:, 0, 0], q[:, 1, 0] = 1, -1
    out, lse, spread, size = m.attend(tables(m, [0], [0, 1], 2, True), q, keys, vals, 1.0)
    assert np.allclose(out[0, :, 0], [14 / 4, (4 + 8 + 0.5) / 2.5]) and np.allclose(lse[0], np.log([4, 2.5]))
    assert np.isnan(out[1]).all() and np.allclose(size[0], np.log(2))
    # two new tokens: the first does not see the second, by the chain or by the mask
    for mask in (None, np.uint32([[1], [2]]), np.uint32([[1], [0]])):
        out, lse, *_ = m.attend(tables(m, [0], [0, 2], 2, True), q, keys, vals, 1.0, mask)
        assert np.allclose(out[0, 0, 0], 6) and np.allclose(lse[0, 0], np.log(2))
        seen = {0: [4, 8, 1], 1: [4, 1], 2: [4]}[0 if mask is None else 1 if mask[1, 0] else 2]
        w = {3: [1, 1, 2], 2: [1, 2], 1: [1]}[len(seen)]
        assert np.allclose(out[1, 0, 0], np.dot(w, seen) / sum(w))
    # a row that sees nothing
    out, lse, *_ = m.attend(tables(m, [0], [0, 3], 3, True), np.ones((3, 1, 2)), keys, vals, 1.0, np.uint32([[0], [1], [3]]))
    assert (out[0] == 0).all() and lse[0, 0] == -np.inf and out[1, 0, 0] == 4 and out[2, 0, 0] == 6


def verification(m):
    p, q = F([[0.5, 0.25, 0.25]] * 4), F([[0.25, 0.5, 0.25]] * 4)
    run = lambda parent, token, u, drafter, p=p: [x.tolist() if hasattr(x, "tolist") else x for x in m.verify(
        [0, len(parent)], len(parent), parent, token, p[:len(parent)], drafter, F(u), 3)]
    # a chain: token 0 (0.3 < 0.5) stays, token 1 (0.25 is not below 0.25) goes; of the rest 0.5, 0.25 the next is 0 or 2
    assert run([-1, 0, 1], [0, 0, 1], [0.6, 0.3, 0.25], None) == [[0, 1, -1], [2], [0], [0]]
    assert run([-1, 0, 1], [0, 0, 1], [0.67, 0.3, 0.25], None) == [[0, 1, -1], [2], [2], [0]]
    # two children of the root: the first is refused, so the second is tried on what is left: 0.34 * 0.5 < 0.25, 0.5 * 0.5 is not
    assert run([-1, 0, 0], [0, 0, 1], [0, 0.5, 0.34], None) == [[0, 2, -1], [2], [0], [0]]
    assert run([-1, 0, 0], [0, 0, 1], [0, 0.5, 0.5], None)[1] == [1]
    # with a drafter: 0.5 * 0.5 is not below 0.25, so what is left is 0.25, 0, 0, and token 0 is certain
    assert run([-1, 0], [0, 1], [0.99, 0.5], q) == [[0, -1], [1], [0], [0]]
    assert run([-1, 0], [0, 1], [0.99, 0.49], q)[1] == [2]
    # tokens of no probability are not drawn
    assert run([-1], [0], [0], None, F([[0, 0.5, 0.5]]))[2] == [1]
    # no probability at all; a NaN and a negative one count as none
    assert run([-1], [0], [0.5], None, F([[0, np.nan, -1]]))[2] == [-1]
    # parents and tokens out of place, and no rows
    assert run([-1, 1], [0, 0], [0, 0], None) == [[-1, -1], [0], [-1], [1]]
    assert run([-1, 0], [0, 3], [0, 0], None)[3] == [1]
    assert m.verify([0, 0], 0, [], [], p[:0], None, F([]), 3)[3] == [1]


def kept(m):
    pool = np.zeros((1, 4, 4, 1))
    pool[0, 0, :, 0], pool[0, 3, :, 0] = [10, 11, 12, 13], [14, 15, 16, 17]
    b = tables(m, [1], [0, 4], 4, True)  # positions 2 to 5
    assert m.keep(b, [0, 2, 3, -1], [3], pool) == [[1, 5]]
    assert pool[0, 0, :, 0].tolist() == [10, 11, 12, 14] and pool[0, 3, :2, 0].tolist() == [15, 15]
    for path, n in (([0, 0, -1, -1], 2), ([0, 4, -1, -1], 2), ([1, 0, -1, -1], 2), ([0, 1, 2, 3], 5), ([0, 1, 2, 3], -1)):
        b, before = tables(m, [1], [0, 4], 4, True), pool.copy()
        assert m.keep(b, path, [n], pool) == [[1, m.KEEP_ALL]] and (pool == before).all() and b.status == [1]
    b = tables(m, [1], [0, 4], 4, True)
    assert m.keep(b, [-1] * 4, [0], pool) == [[1, 2]]


CASES = (codes, moves, attention, verification, kept)


@pytest.mark.parametrize("case", CASES, ids=lambda f: f.__name__)
def test_hand_worked(case):
    case(cachedata)


MISTAKES = [
    ("(up == down) & (hi % 2 == 0)", "(up == down)"), ("np.float32(full / top), np.float32(top / full)", "np.float32(top / full), np.float32(full / top)"),
    ("not np.isfinite(row).all()", "np.isnan(row).all()"), ("scale == 0 or np.isinf(by)", "scale == 0"),
    ("fresh and b - a > n", "fresh and b - a > n + 1"), ("n <= self.table.shape[1] * T", "n <= self.table.shape[1] * T + 1"), ("n < 1 << 31 and", ""),
    ("b.place(s, n - m + j)", "b.place(s, j)"), ("if position < n else None", "if position <= n else None"),
    ("sees = own <= j", "sees = own < j"), ("group = q_heads // keys.shape[2]", "group = 1"), ("(kk @ qq) * scale", "(kk @ qq)  * scale * 2"),
    ("out[where] = (w @ vv) / w.sum()", "out[where] = w @ vv"), ("top + np.log(w.sum())", "np.log(w.sum())"),
    ("* by * W < float(w[t])", "* by * W <= float(w[t])"), ("W -= float(w[t])", "pass"), ("w[t] = 0", "pass"),
    ('side="right"', 'side="left"'), ("0 <= parent[a + j] < j", "0 <= parent[a + j] <= j"), ("n - m + a])", "n + a])"),
    ("x >= y for x, y", "x > y for x, y"), ("if a > m or", "if a > m + 1 or"),
]


@pytest.mark.parametrize("old,new", MISTAKES, ids=[str(i) for i in range(len(MISTAKES))])
def test_planted_mistakes_are_found(old, new):
    with open(SRC) as f:
        src = f.read()
    assert old in src
    m = types.ModuleType("wrong")
    exec(compile(src.replace(old, new), SRC, "exec"), m.__dict__)
    with pytest.raises(Exception):
        for case in CASES:
            case(m)
