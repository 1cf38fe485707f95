"""Tokens kept together in pages that begin behind 4 GiB: the bytes that move, and every other one of the sequence's."""

import numpy as np
import pytest

from cache_util import Tables, finish, i32
from gpu_util import lib, need_gpu
from oracle import cachedata as cd

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [64, 7])  # vectors of 16 bytes, and single ones
def test_kept_bytes_behind_4_gib(width):
    need_gpu()
    db = lib()
    rng = np.random.default_rng(19)
    heads, T, gap = 2, 16, 1 << 20
    pages = (6 << 30) // gap
    store = torch.empty(pages * gap, dtype=torch.int8, device="cuda")
    planes = 2
    pool = torch.as_strided(store, (planes, pages, T, heads, width), (gap // 2, gap, heads * width, width, 1))
    t = Tables(rng, [70, 33], T)
    t.table = np.where(t.table >= 0, pages - 1 - 3 * t.table, -1).astype(np.int32)
    t.n_pages = pages
    used = np.unique(t.table[t.table >= 0])
    assert int(used.min()) * gap > 1 << 32
    at = torch.from_numpy(used.astype(np.int64)).cuda()
    pool[:, at] = torch.from_numpy(rng.integers(-128, 128, (planes, len(used), T, heads, width)).astype(np.int8)).cuda()
    before = pool[:, at].cpu().numpy()
    seq, start, path, accepted = [0, 1], [0, 9, 16], [0, 2, 3, 7, 8, -1, -1, -1, -1, 1, 4, 6, -1, -1, -1, -1], [5, 3]
    cut = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    db.cache_keep(t.device(), i32(seq), i32(start), i32(path), i32(accepted), pool, token_dim=2, cut=cut)
    finish()
    small = np.searchsorted(used, t.table)  # the same pages, numbered from 0
    b = cd.Batch(np.where(t.table >= 0, small, -1), t.length, len(used), T, seq, start, 16, True)
    want = before.copy()
    assert cd.keep(b, path, accepted, want) == cut.cpu().tolist() == [[0, 66], [1, 29]]
    assert (want != before).any()
    np.testing.assert_array_equal(pool[:, at].cpu().numpy(), want)
