"""Attention over 8-bit codes whose scales lie far apart, and its roundings of 2^-11.

Weights times scales are rounded to f16 (half a step is 2^-11 of the value, 2^-25 below the normal numbers), after
division by a power of two that puts the largest of a row, of the tokens that it sees, at 2^4 or above. So an output is
off by spread * 2^-11, by 2^-29 of that largest for each code it is summed from, and by what the scores' errors, the
sums in 32 bits and the output's own type add (test_gpu_cache_attention.py). What a row does not see has no part in it."""

import numpy as np
import pytest

from cache_util import finish, numbers, tokens_first
from gpu_util import lib, need_gpu
from oracle import cachedata as cd
from test_gpu_cache_attention import DEEP, HALF, SHAPES, Case
from test_gpu_cache_edges import ROWS

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LARGEST = {"i8": 127.0, "e4m3": 448.0}


class Codes(Case):
    """A case over codes that are numbers, compared within the bounds above."""

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        for pool in self.pools:
            if self.kind == "e4m3":
                pool.copy_(torch.nan_to_num(pool.float()).to(pool.dtype))

    def check(self, out, lse, b, want):
        super().check(out, lse, b, want)
        o, _, spread, size = want
        keys, _ = (tokens_first(numbers(p), self.token_dim) for p in self.pools)
        k_scale, v_scale = (tokens_first(s.numpy(), self.token_dim) for s in self.scales)
        scales = np.broadcast_to(np.abs(v_scale)[..., None], keys.shape)
        _, _, largest, _ = cd.attend(b, numbers(self.q), cd.values(keys, k_scale), scales, self.scale, self.mask)
        n = int(self.t.length.max())
        e_p = 2 * (self.q.shape[2] + 8) * 2.0**-24 * size[..., None] + 2.0**-20
        bound = spread * (2 * e_p + 2.0**-11 * 1.01 + n * 2.0**-24) + largest * n * LARGEST[self.kind] * 2.0**-29
        bound = bound + np.abs(o) * HALF[self.qk] * 1.01 + (2.0**-25 if self.qk == "f16" else 0)
        rows = np.isfinite(o)
        got = out.cpu().double().numpy()
        bad = rows & ~(np.abs(got - o) <= bound)
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], o[bad][:4], bound[bad][:4])

    def bits(self):
        """Outputs and sums, once."""
        need_gpu()
        db = lib()
        out, lse = torch.full_like(self.q, 7.0).cuda(), torch.full(self.q.shape[:2], 7.0, device="cuda")
        self.call(db, self.t.device(), self.workspace(db), self.device(), out, lse)
        finish()
        return out, lse

    def place(self, i, position):
        """(page, slot) of request i's position."""
        return int(self.t.table[self.seq[i], position // self.t.T]), position % self.t.T

    def nodes(self, i):
        return int(self.start[i + 1] - self.start[i])

    def hide(self, node):
        """No row sees this node of any request."""
        for i in range(len(self.seq)):
            if node < self.nodes(i):
                self.mask[self.start[i]:self.start[i + 1], node // 32] &= np.uint32(0xFFFFFFFF ^ (1 << node % 32))


KINDS = [("e4m3", "bf16", 96), ("i8", "f16", 256), ("e4m3", "f16", 128), ("i8", "bf16", 64)]
CODED = [s for s in SHAPES + DEEP if s[0] in ("e4m3", "i8")]


@pytest.mark.parametrize("shape", CODED, ids=[f"{i}-{s[0]}-{s[1]}-{s[6]}-{s[8]}" for i, s in enumerate(CODED)])
def test_roundings_of_f16(shape):
    Codes(*shape, spare=1).run()


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kind,q,width", KINDS)
def test_a_hidden_token_of_large_values(kind, q, width, rows):
    """A node that no row sees, whose values' scale is up to 2^100 times the others': the same bits as without."""
    nodes, group = ROWS[rows]
    seen = None
    for power in (0, 20, 28, 40, 100):
        c = Codes(kind, q, 1, 16, 1, group, width, [(200, nodes), (64 - nodes // 2, nodes), (3000, nodes)], "tree", seed=nodes)
        c.hide(nodes - 1)
        _, scale = c.view(1)
        for i in range(len(c.seq)):
            scale[c.place(i, int(c.t.length[c.seq[i]]) - 1)] *= 2.0**power
        got = c.run() if power in (0, 28, 100) else c.bits()
        seen = seen or got
        assert all(torch.equal(x, y) for x, y in zip(got, seen)), power


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kind,width", [("e4m3", 128), ("i8", 64), ("e4m3", 240)])
def test_later_tokens_of_a_chain_with_large_values(kind, width, rows):
    """Without a mask a node does not see those behind it, each of which has values 2^12 times the one's before."""
    nodes, group = ROWS[rows]
    c = Codes(kind, "bf16", 2, 48, 1, group, width, [(150, nodes), (63, nodes)], None, seed=nodes)
    _, scale = c.view(1)
    for i in range(len(c.seq)):
        for j in range(min(nodes, 8)):
            scale[c.place(i, int(c.t.length[c.seq[i]]) - nodes + j)] *= 2.0 ** (12 * j)
    c.run()


def plant(c, position, weight, power):
    """A token of every request whose score is that of a weight of 2^weight for all rows, and whose values' scale is
    2^power times what it was."""
    code, width = {"i8": -100.0, "e4m3": -64.0}[c.kind], c.q.shape[2]
    c.q[:, :, 0] = 4.0
    for i in range(len(c.seq)):
        at = c.place(i, position)
        for part in (0, 1):
            pool, scale = c.view(part)
            if part:
                scale[at] *= 2.0**power
            else:
                row = torch.zeros((pool.shape[2], width))
                row[:, 0] = code
                pool[at] = row.to(pool.dtype)
                scale[at] = weight * np.log(2.0) / (code * 4.0 * c.scale)
                assert weight < 0


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kind,q,width", KINDS)
@pytest.mark.parametrize("weight,power", [(-150, 40), (-150, 100), (-60, 40), (-30, 24)])
def test_a_token_of_large_values_that_hardly_counts(kind, q, width, rows, weight, power):
    """A token that all rows see, the first, one in the middle or the last before the nodes, of a weight that makes
    nothing of its large values."""
    nodes, group = ROWS[rows]
    for position in (0, 70, 149):
        c = Codes(kind, q, 1, 16, 1, group, width, [(150, nodes), (2500, nodes)], "tree", seed=nodes)
        plant(c, position, weight, power)
        c.run()


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kind,width", [("e4m3", 64), ("i8", 128), ("e4m3", 256)])
def test_scales_from_token_to_token(kind, width, rows):
    """Scales between 2^-20 and 2^20 in one sequence, in disorder, rising and falling."""
    nodes, group = ROWS[rows]
    for order in ("disorder", "rising", "falling"):
        c = Codes(kind, "bf16", 1, 16, 1, group, width, [(700, nodes), (64, nodes)], "tree", seed=nodes)
        _, scale = c.view(1)
        for i in range(len(c.seq)):
            n = int(c.t.length[c.seq[i]])
            power = np.linspace(-20, 20, n)
            power = {"disorder": c.rng.permutation(power), "rising": power, "falling": power[::-1]}[order]
            for x in range(n):
                scale[c.place(i, x)] *= 2.0 ** np.rint(power[x])
        c.run()


@pytest.mark.parametrize("rows", ROWS)
def test_parts_of_sums_with_scales_far_apart(rows):
    """A long sequence is cut into parts and these are joined: the first half's values are 2^90 times the second's, whose
    weights are 2^150 times the first's; so the products of the first are 2^-60 of the others', and its sums 2^-150."""
    nodes, group = ROWS[rows]
    c = Codes("i8", "bf16", 1, 64, 1, group, 64, [(6000, nodes)], None, seed=nodes)
    pool, scale = c.view(0)
    c.q[:, :, 0] = 4.0
    for x in range(3000):
        at = c.place(0, x)
        row = torch.zeros((1, 64), dtype=torch.int8)
        row[:, 0] = -100
        pool[at], scale[at] = row, 150 * np.log(2.0) / (400 * c.scale)
        c.view(1)[1][at] *= 2.0**90
    c.run()
