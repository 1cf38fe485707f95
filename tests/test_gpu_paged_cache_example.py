"""The example's cache reads back as written, and its descriptors name its pages."""

import importlib.util
import os

import numpy as np
import pytest

import oracle
from conftest import ROOT
from gpu_util import host64, lib, need_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_paged_cache_example():
    need_gpu()
    lib()
    spec = importlib.util.spec_from_file_location("paged_cache", os.path.join(ROOT, "examples", "paged_cache.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    same, c, req, prp, lut, put, rings, count = m.main()
    torch.cuda.synchronize()
    assert same
    heap_size = m.PAGES * m.PAGE_BYTES
    want = oracle.prp_build(host64(req), host64(lut), heap_size, 1 << 32, 64)
    assert (host64(prp) == want["prp"]).all()
    # the puts, in order, move the bytes of the sequence's pages to the same offsets at the peer
    n = int(count[1])
    wqe = rings[1, :n].cpu().numpy().reshape(n, 64)
    raddr, laddr = (wqe[:, k:k + 8].copy().view(np.uint64)[:, 0] for k in (0, 8))
    size = wqe[:, 16:20].copy().view(np.uint32)[:, 0]
    off = host64(put)[:, 0]
    assert (raddr == off + (1 << 41)).all() and (laddr == off + (1 << 30)).all()
    pages = c.tables.table[16, : -(-int(c.tables.length[16]) // m.TOKENS)].cpu().numpy()
    at = np.concatenate([np.arange(o, o + b, m.PAGE_BYTES) for o, b in zip(off.tolist(), size.tolist())])
    assert (at == pages.astype(np.int64) * m.PAGE_BYTES).all()
