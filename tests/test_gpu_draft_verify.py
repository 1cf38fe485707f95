"""Verification of drafted tokens against the oracle: paths, counts and drawn tokens are the same numbers."""

import numpy as np
import pytest

from cache_util import NAMES, finish, i32, tree
from gpu_util import lib, need_gpu
from oracle import cachedata as cd

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def probabilities(rng, rows, vocab, kind, sharp=2.0):
    x = rng.standard_normal((rows, vocab)) * sharp
    x = np.exp(x - x.max(1, keepdims=True))
    return torch.from_numpy((x / x.sum(1, keepdims=True)).astype(np.float32)).to(NAMES[kind])


def run(start, rows, parent, token, p, q, u, wide=0):
    need_gpu()
    db = lib()
    n, vocab = len(start) - 1, p.shape[1]

    def up(x):  # rows of a wider tensor
        if x is None:
            return None
        y = torch.zeros((x.shape[0], vocab + wide), dtype=x.dtype, device="cuda")
        y[:, :vocab] = x.cuda()
        return y[:, :vocab]

    path = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    accepted, following = (torch.full((n,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    status = torch.full((n,), 9, dtype=torch.uint8, device="cuda")
    ctr = torch.full((4,), 77, dtype=torch.int64, device="cuda")
    db.draft_verify(i32(start), i32(parent), i32(token), up(p), torch.from_numpy(u.astype(np.float32)).cuda(), path, accepted,
                    following, q=up(q), status=status, ctr=ctr)
    finish()
    want = cd.verify(start, rows, parent, token, p.float().numpy(), None if q is None else q.float().numpy(),
                     u.astype(np.float32), vocab)
    assert status.cpu().tolist() == want[3]
    assert accepted.cpu().tolist() == want[1].tolist()
    assert path.cpu().tolist() == want[0].tolist()
    assert following.cpu().tolist() == want[2].tolist()
    done = [int(start[i + 1] - start[i]) for i in range(n) if want[3][i] == 0]
    assert ctr.cpu().tolist() == [sum(done), n - len(done), 0, 0]
    return want


CASES = [(kind, drafter, vocab, n, nodes, shape) for kind, drafter, vocab, n, nodes, shape in (
    ("f32", True, 50, 40, 9, "tree"), ("f32", False, 50, 40, 9, "tree"), ("bf16", True, 1000, 7, 33, "tree"),
    ("f16", False, 33, 100, 5, "chain"), ("f32", True, 1, 4, 4, "tree"), ("bf16", False, 7, 9, 1, "chain"),
    ("f32", True, 20011, 3, 12, "star"), ("f16", True, 70001, 2, 7, "star"), ("f32", False, 70001, 1, 7, "star"),
    ("bf16", True, 4097, 400, 4, "chain"), ("f32", False, 9000, 30, 300, "tree"))]


@pytest.mark.parametrize("kind,drafter,vocab,n,nodes,shape", CASES)
def test_trees(kind, drafter, vocab, n, nodes, shape):
    rng = np.random.default_rng(4)
    counts = [int(rng.integers(1, nodes + 1)) for _ in range(n)]
    counts[0] = nodes
    start = np.concatenate([[1], 1 + np.cumsum(counts)])
    rows = int(start[-1]) + 2
    parent = np.full(rows, -1)
    for i, m in enumerate(counts):
        parent[start[i]:start[i] + m] = {"tree": lambda: tree(rng, m)[0], "chain": lambda: np.arange(m) - 1,
                                         "star": lambda: np.minimum(np.arange(m) - 1, 0)}[shape]()
    p = probabilities(rng, rows, vocab, kind)
    q = probabilities(rng, rows, vocab, kind) if drafter else None
    # tokens as a drafter draws them, some of them twice
    by = (p if q is None else q).double().numpy()
    first = np.repeat(start[:-1], counts)
    above = np.arange(rows)
    above[start[0]:start[-1]] = first + np.maximum(parent[start[0]:start[-1]], 0)
    pick = (np.cumsum(by[above], 1) > rng.random((rows, 1)) * by[above].sum(1, keepdims=True)).argmax(1)
    want = run(start, rows, parent, pick, p, q, rng.random(rows), wide=3)
    if nodes > 3 and n > 6 and 1 < vocab < 5000:  # of a flat target, a token alone is hardly ever accepted
        assert len(set(want[1].tolist())) > 1


def test_borders():
    """Random numbers of 0 and just below 1, probabilities of 0 and 1, p = q, and rows of nothing."""
    vocab = 64
    e = lambda *at: np.eye(vocab, dtype=np.float32)[list(at)].sum(0) / len(at)  # noqa: E731
    p = np.stack([e(3), e(5), e(9), e(1, 2), e(4), np.zeros(vocab, np.float32), e(7), e(8, 9)])
    parent, token = np.array([-1, 0, -1, 0, -1, 0, -1, 0]), np.array([0, 3, 0, 8, 0, 4, 0, 7])
    start = np.array([0, 2, 4, 6, 8])
    for u in (np.zeros(8), np.full(8, 0.99999994), np.full(8, 0.5)):
        for q in (None, p, np.stack([e(3)] * 8), np.full((8, vocab), 1 / 64, np.float32), np.zeros((8, vocab), np.float32)):
            run(start, 8, parent, token, torch.from_numpy(p), None if q is None else torch.from_numpy(q), u)


def test_numbers_that_are_no_probabilities():
    """NaN and negative ones count as 0, larger ones as 1, in the sums and in the tests alike."""
    rng = np.random.default_rng(6)
    start, rows, vocab = np.array([0, 5, 9]), 9, 300
    p, q = (rng.random((rows, vocab)).astype(np.float32) * 0.01 for _ in range(2))
    for x in (p, q):
        x[:, 5], x[:, 6], x[:, 7], x[:, 8] = np.nan, -1, 1e30, np.inf
    parent = np.array([-1, 0, 0, 1, 2, -1, 0, 1, 2])
    for token in (5, 6, 7, 8, 100):
        run(start, rows, parent, np.full(rows, token), torch.from_numpy(p), torch.from_numpy(q), rng.random(rows))
        run(start, rows, parent, np.full(rows, token), torch.from_numpy(p), None, np.array([np.nan, -1, 2, 0.5, 0.1, 5, 0, 1, 0.2]))


def test_bad_trees_are_refused():
    rng = np.random.default_rng(7)
    rows, vocab = 1100, 20
    start = np.array([0, 4, 8, 12, 12, 16, 1050, 1060, 1055, 5000])
    parent = np.concatenate([[-1, 0, 1, 2]] * 275)
    token = np.zeros(rows, np.int64)
    parent[5] = 3      # below itself?
    parent[9] = 1      # itself
    token[14] = vocab
    parent[16:1050] = np.arange(1034) - 1  # more than 1,024 nodes
    p = probabilities(rng, rows, vocab, "f32")
    want = run(start, rows, parent, token, p, None, rng.random(rows))
    assert want[3][0] == 0 and 0 < sum(want[3]) < len(want[3])


def test_drawn_as_the_target():
    """The drawn token's frequencies are the target's, whatever the drafter: 200,000 walks of one and of two children
    (a difference of 5 standard deviations would be a 1 in 10^6 event)."""
    need_gpu()
    db = lib()
    rng = np.random.default_rng(8)
    vocab, n = 6, 200000
    p = np.array([0.05, 0.3, 0.1, 0.25, 0.2, 0.1], np.float32)
    q = np.array([0.4, 0.05, 0.2, 0.05, 0.2, 0.1], np.float32)
    for m in (2, 3):
        parent = torch.from_numpy(np.tile([-1] + [0] * (m - 1), n).astype(np.int32)).cuda()
        token = torch.from_numpy(rng.choice(vocab, n * m, p=q / q.astype(np.float64).sum()).astype(np.int32)).cuda()
        P = torch.from_numpy(np.tile(p, (n * m, 1))).cuda()
        Q = torch.from_numpy(np.tile(q, (n * m, 1))).cuda()
        u = torch.from_numpy(rng.random(n * m).astype(np.float32)).clamp(max=0.99999).cuda()
        path = torch.zeros(n * m, dtype=torch.int32, device="cuda")
        accepted, following = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
        start = torch.arange(n + 1, dtype=torch.int32, device="cuda") * m
        db.draft_verify(start, parent, token, P, u, path, accepted, following, q=Q)
        finish()
        first = torch.where(accepted > 1, token.reshape(n, m).gather(1, path.reshape(n, m)[:, 1:2].clamp(min=0).long())[:, 0], following)
        freq = torch.bincount(first.long(), minlength=vocab).double().cpu().numpy() / n
        assert (np.abs(freq - p) < 5 * np.sqrt(p * (1 - p) / n)).all(), freq


def test_captured_with_two_trees():
    need_gpu()
    db = lib()
    rng = np.random.default_rng(9)
    start, rows, vocab = np.array([0, 6, 11]), 11, 5000
    parent = np.concatenate([tree(rng, 6)[0], tree(rng, 5)[0]])
    p, q = probabilities(rng, rows, vocab, "bf16"), probabilities(rng, rows, vocab, "bf16")
    tok, u = rng.integers(0, vocab, rows), rng.random(rows)
    dev = [i32(start), i32(parent), i32(tok), p.cuda(), torch.from_numpy(u.astype(np.float32)).cuda()]
    path = torch.zeros(rows, dtype=torch.int32, device="cuda")
    accepted, following = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    Q = q.cuda()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        db.draft_verify(*dev, path, accepted, following, q=Q)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        db.draft_verify(*dev, path, accepted, following, q=Q)
    for _ in range(3):
        tok, u = rng.integers(0, vocab, rows), rng.random(rows)
        tok[1], u[1] = int(p[0].argmax()), 0.0
        dev[2].copy_(i32(tok))
        dev[4].copy_(torch.from_numpy(u.astype(np.float32)))
        graph.replay()
        finish()
        want = cd.verify(start, rows, parent, tok, p.float().numpy(), q.float().numpy(), u.astype(np.float32), vocab)
        assert path.cpu().tolist() == want[0].tolist() and following.cpu().tolist() == want[2].tolist()
