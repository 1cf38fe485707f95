"""Rows of attention that have only scores of minus infinity have an answer of 0, whatever the values are."""

import numpy as np
import pytest

from test_gpu_cache_attention import Case
from test_gpu_cache_edges import ROWS

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kind,q,width", [("bf16", "bf16", 64), ("e4m3", "bf16", 128), ("f16", "f16", 256), ("i8", "bf16", 80)])
@pytest.mark.parametrize("length", [60, 700, 9000])
def test_values_that_are_not_finite_of_scores_of_minus_infinity(kind, q, width, rows, length):
    nodes, group = ROWS[rows]
    c = Case(kind, q, 1, 16, 1, group, width, [(length, nodes)], None, seed=nodes)
    if kind == "e4m3":
        for pool in c.pools:
            pool.copy_(torch.nan_to_num(pool.float()).to(pool.dtype))
    c.pools[0][..., 5] = -1
    c.q[1, 0, 5] = float("inf")  # all its scores
    pool, scale = c.view(1)
    for position, value in ((3, float("inf")), (length // 2, -float("inf")), (length - 1, float("nan")), (length, float("inf"))):
        at = int(c.t.table[0, position // 16]), position % 16
        if scale is not None:
            scale[at] = value
        else:
            pool[at][:, 7] = value
    out, lse = c.run()
    assert (out[1, 0] == 0).all() and lse[1, 0] == -float("inf")
