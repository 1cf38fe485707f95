"""Attention of requests of several hundred tokens: whole prompts, chunks of them behind a prefix, beside single tokens
and small trees in one batch; the bounds are those of test_gpu_cache_attention.py and test_gpu_cache_scales.py."""

import pytest

from test_gpu_cache_attention import Case
from test_gpu_cache_scales import Codes

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PROMPTS = [
    ("bf16", "bf16", 1, 16, 2, 4, 128, [(0, 700), (0, 301)], None),
    ("f16", "f16", 2, 48, 1, 1, 64, [(0, 1000), (513, 129)], None),
    ("bf16", "bf16", 1, 64, 1, 2, 256, [(0, 400), (900, 257)], None),
    ("e4m3", "bf16", 1, 16, 2, 4, 128, [(0, 600), (1000, 512)], None),
    ("i8", "f16", 2, 48, 1, 8, 112, [(0, 385), (64, 128)], None),
    ("e4m3", "f16", 1, 100, 1, 3, 240, [(31, 400)], None),
    ("bf16", "bf16", 1, 16, 1, 4, 64, [(0, 500), (2000, 1), (300, 0), (77, 9), (64, 64), (0, 1), (1500, 300)], None),
    ("e4m3", "bf16", 1, 16, 1, 4, 64, [(0, 500), (2000, 1), (300, 0), (77, 9), (64, 64), (0, 1), (1500, 300)], "tree"),
    ("i8", "bf16", 2, 16, 2, 2, 128, [(0, 260), (130, 1), (400, 200)], "random"),
    ("bf16", "bf16", 2, 8, 1, 1, 96, [(0, 300), (40, 177)], "random"),
]


@pytest.mark.parametrize("shape", PROMPTS, ids=[f"{i}-{s[0]}-{s[1]}-{s[6]}-{s[8]}" for i, s in enumerate(PROMPTS)])
def test_prompts(shape):
    (Codes if shape[0] in ("e4m3", "i8") else Case)(*shape, spare=2).run()
