"""A step in which a tree is refused: its sequence is as it was before the step, the root's slot given back with the
others', and the sequences beside it go on."""

import numpy as np
import pytest

from cache_util import finish, numbers
from gpu_util import need_gpu
from test_gpu_cache_step import Engine, prompts

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_refused_tree_takes_its_step_back(kind):
    need_gpu()
    rng = np.random.default_rng(41)
    e = Engine(kind, 4, 7)
    prompts(e, rng, [30, 11, 64])
    finish()
    before = e.tables.length.cpu().tolist()
    held = lambda s, n: numbers(e.pool)[:, e.tables.table[s].cpu().numpy()[np.arange(n) // e.tables.page_tokens],
                                       np.arange(n) % e.tables.page_tokens]
    first = [held(s, before[s]) for s in range(4)]
    e.draft(rng)
    e.parent[7 + 2] = 3  # the second sequence's tree: a parent that is not below its node
    e.step()
    finish()
    length, accepted = e.tables.length.cpu().tolist(), e.accepted.cpu().tolist()
    assert e.status[3].cpu().tolist() == [0, 1, 0, 0] and e.status[4].cpu().tolist() == [0] * 4
    assert accepted[1] == 0 and e.next[1].item() == -1 and e.cut[1].cpu().tolist() == [1, before[1]]
    assert [a - b for a, b in zip(length, before)][:4] == accepted and min(accepted[0], *accepted[2:]) >= 1
    for s in range(4):
        assert (held(s, before[s]) == first[s]).all()
    # and the step can be taken again
    e.draft(rng), e.step()
    finish()
    assert e.status.cpu().tolist() == [[0] * 4] * 6 and e.tables.length[1].item() > before[1]
