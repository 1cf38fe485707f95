"""Attention whose weights are held finer than the type that is multiplied: 16-bit caches of rows of up to 128 values with
up to 16 query rows, and f16 answers from codes with up to 8.

A weight is a sum of two numbers of the type, each off by half a step of what is left: by 2^-16 of itself (bf16) or
2^-22 (f16, where small parts are off by 2^-25 of what 2^8 stands for, that is by 2^-33 of the row's largest). So an
output is off by spread * (that and the scores' errors of test_gpu_cache_attention.py), and by half a step of its own."""

import numpy as np
import pytest

from cache_util import numbers, tokens_first
from oracle import cachedata as cd
from test_gpu_cache_attention import HALF, Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Fine(Case):
    def check(self, out, lse, b, want):
        super().check(out, lse, b, want)
        o, _, spread, size = want
        n, coded = int(self.t.length.max()), self.kind in ("i8", "e4m3")
        e_p = 2 * (self.q.shape[2] + 8) * 2.0**-24 * size[..., None] + 2.0**-20
        bound = spread * (2 * e_p + {"bf16": 2.0**-16, "f16": 2.0**-22}[self.qk] + n * 2.0**-24)
        bound = bound + np.abs(o) * HALF[self.qk] * 1.01
        if self.qk == "f16":
            keys, vals = (tokens_first(numbers(p), self.token_dim) for p in self.pools)
            scales = np.ones(keys.shape[:3]) if not coded else tokens_first(self.scales[1].numpy(), self.token_dim)
            k_scale = None if not coded else tokens_first(self.scales[0].numpy(), self.token_dim)
            _, _, largest, _ = cd.attend(b, numbers(self.q), cd.values(keys, k_scale),
                                         np.broadcast_to(scales[..., None], keys.shape), self.scale, self.mask)
            bound = bound + largest * n * np.abs(vals).max() * 2.0**-33 + 2.0**-25
        bad = np.isfinite(o) & ~(np.abs(out.cpu().double().numpy() - o) <= bound)
        assert not bad.any(), (np.argwhere(bad)[:4], o[bad][:4], bound[bad][:4])


FINE = [
    ("bf16", "bf16", 1, 16, 2, 4, 128, [(100, 1), (0, 1), (63, 1), (64, 1), (1, 1), (2000, 1)], None),
    ("bf16", "bf16", 2, 48, 1, 8, 112, [(150, 2), (700, 1)], None),
    ("bf16", "bf16", 1, 8, 3, 2, 64, [(300, 5), (64, 3), (0, 8)], "tree"),
    ("f16", "f16", 1, 16, 2, 8, 128, [(900, 1), (30, 1)], None),
    ("f16", "f16", 2, 7, 1, 4, 48, [(300, 4), (12, 2)], "random"),
    ("e4m3", "f16", 1, 16, 2, 8, 128, [(500, 1), (64, 1), (0, 1)], None),
    ("e4m3", "f16", 2, 16, 5, 1, 256, [(297, 1), (40, 1)], None),
    ("i8", "f16", 1, 48, 2, 2, 64, [(120, 4), (3, 2)], "tree"),
    ("i8", "f16", 1, 33, 1, 4, 80, [(3000, 2), (9, 1)], None),
    ("e4m3", "f16", 1, 64, 1, 1, 32, [(9000, 1)], None),
]


@pytest.mark.parametrize("shape", FINE, ids=[f"{i}-{s[0]}-{s[1]}-{s[6]}-{s[8]}" for i, s in enumerate(FINE)])
def test_fine_weights(shape):
    c = Fine(*shape, spare=1)
    for pool in c.pools:
        if c.kind == "e4m3":
            pool.copy_(torch.nan_to_num(pool.float()).to(pool.dtype))
    c.run()
