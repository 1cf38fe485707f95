"""The paged cache's C entry points refuse bad arguments before they touch a GPU."""

import ctypes

import pytest

from test_abi import libpath  # noqa: F401  (the built library)

VP, U32, U64, SZ = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_size_t
FAKE = 1 << 20  # never dereferenced: the checks fail first


class Tables(ctypes.Structure):
    _fields_ = [("table", VP), ("length", VP), ("refs", VP), ("free", VP), ("n_seqs", U32),
                ("columns", U32), ("n_pages", U32), ("page_tokens", U32)]


class Pool(ctypes.Structure):
    _fields_ = [("base", VP), ("n_pages", U64), ("plane_stride", U64), ("page_stride", U64)]


class Shape(ctypes.Structure):
    _fields_ = [("planes", U32), ("segments", U32), ("page_tokens", U32), ("token_bytes", U32)]


@pytest.fixture()
def lib(libpath):  # noqa: F811
    lib = ctypes.CDLL(libpath)
    lib.db_page_workspace_size.argtypes = [U32, U32, ctypes.POINTER(SZ)]
    lib.db_page_extend.argtypes = [VP, VP, U32, VP, VP, VP, VP, VP, SZ, VP]
    lib.db_page_fork.argtypes = [VP, VP, U32, VP, VP, VP, SZ, VP]
    lib.db_page_free.argtypes = lib.db_page_fork.argtypes
    lib.db_page_compact.argtypes = [VP, VP, VP, U32, VP, VP, VP, SZ, VP]
    lib.db_page_copy.argtypes = [VP, U32, VP, VP, VP, VP, VP, VP]
    return lib


def tables(**kw):
    t = Tables(FAKE, FAKE, FAKE, FAKE, 8, 4, 100, 16)
    for k, v in kw.items():
        setattr(t, k, v)
    return ctypes.byref(t)


def test_workspace_size(lib):
    out = SZ()
    assert lib.db_page_workspace_size(1000, 50000, ctypes.byref(out)) == 0
    assert out.value >= 20 * 1000 + 8 * 50000
    for n_seqs, n_pages in ((0, 5), (5, 0), (1 << 31, 5), (5, 1 << 31)):
        assert lib.db_page_workspace_size(n_seqs, n_pages, ctypes.byref(out)) == -22
    assert lib.db_page_workspace_size(5, 5, None) == -22


BAD_TABLES = [dict(table=None), dict(length=None), dict(refs=None), dict(free=None),
              dict(table=FAKE + 2), dict(length=FAKE + 1), dict(refs=FAKE + 3), dict(free=FAKE + 8),
              dict(n_seqs=0), dict(columns=0), dict(n_pages=0), dict(page_tokens=0),
              dict(n_seqs=1 << 31), dict(n_pages=1 << 31)]


@pytest.mark.parametrize("bad", BAD_TABLES, ids=[str(b) for b in BAD_TABLES])
def test_tables(lib, bad):
    t, ok = tables(**bad), tables()
    assert lib.db_page_extend(t, FAKE, 2, FAKE, FAKE, None, None, FAKE, 1 << 30, None) == -22
    assert lib.db_page_fork(t, FAKE, 2, None, None, FAKE, 1 << 30, None) == -22
    assert lib.db_page_free(t, FAKE, 2, None, None, FAKE, 1 << 30, None) == -22
    assert lib.db_page_compact(t, ok, FAKE, 2, FAKE, None, FAKE, 1 << 30, None) == -22
    assert lib.db_page_compact(ok, t, FAKE, 2, FAKE, None, FAKE, 1 << 30, None) == -22


def test_requests_and_workspaces(lib):
    t = tables()
    for call, align in ((lib.db_page_fork, 16), (lib.db_page_free, 8)):
        assert call(None, FAKE, 2, None, None, FAKE, 1 << 30, None) == -22
        assert call(t, None, 2, None, None, FAKE, 1 << 30, None) == -22
        assert call(t, FAKE + align // 2, 2, None, None, FAKE, 1 << 30, None) == -22
        assert call(t, FAKE, 9, None, None, FAKE, 1 << 30, None) == -22       # > n_seqs
        assert call(t, FAKE, 2, None, FAKE + 4, FAKE, 1 << 30, None) == -22   # counters
        assert call(t, FAKE, 2, None, None, None, 1 << 30, None) == -22
        assert call(t, FAKE, 2, None, None, FAKE + 128, 1 << 30, None) == -22
        assert call(t, FAKE, 2, None, None, FAKE, 256, None) == -28
        # entries of a batch are numbered in 32 bits
        wide = tables(n_seqs=1 << 20, columns=1 << 14)
        assert call(wide, FAKE, 1 << 18, None, None, FAKE, 1 << 40, None) == -22
    ext = lib.db_page_extend
    assert ext(t, FAKE, 2, None, FAKE, None, None, FAKE, 1 << 30, None) == -22
    assert ext(t, FAKE, 2, FAKE + 8, FAKE, None, None, FAKE, 1 << 30, None) == -22
    assert ext(t, FAKE, 2, FAKE, None, None, None, FAKE, 1 << 30, None) == -22
    assert ext(t, FAKE, 2, FAKE, FAKE + 2, None, None, FAKE, 1 << 30, None) == -22
    assert ext(t, FAKE + 4, 2, FAKE, FAKE, None, None, FAKE, 1 << 30, None) == -22
    assert ext(t, FAKE, 2, FAKE, FAKE, None, None, FAKE, 256, None) == -28
    com = lib.db_page_compact
    assert com(t, None, FAKE, 2, FAKE, None, FAKE, 1 << 30, None) == -22
    assert com(t, t, None, 2, FAKE, None, FAKE, 1 << 30, None) == -22
    assert com(t, t, FAKE + 8, 2, FAKE, None, FAKE, 1 << 30, None) == -22
    assert com(t, t, FAKE, 2, None, None, FAKE, 1 << 30, None) == -22
    for other in (dict(n_seqs=9), dict(columns=5), dict(n_pages=101), dict(page_tokens=8)):
        assert com(t, tables(**other), FAKE, 2, FAKE, None, FAKE, 1 << 30, None) == -22
    assert com(t, t, FAKE, 2, FAKE, None, FAKE, 512, None) == -28


def test_copy(lib):
    pool = Pool(FAKE, 10, 1 << 20, 4096)
    shape = Shape(2, 1, 16, 256)
    ref = ctypes.byref

    def call(moves=FAKE, n=3, count=FAKE, src=pool, dst=pool, shape=shape, ctr=None):
        return lib.db_page_copy(moves, n, count, ref(src) if src else None,
                                ref(dst) if dst else None, ref(shape) if shape else None, ctr, None)

    assert call(moves=None) == -22 and call(moves=FAKE + 8) == -22
    assert call(count=None) == -22 and call(count=FAKE + 1) == -22
    assert call(src=None) == -22 and call(dst=None) == -22 and call(shape=None) == -22
    assert call(ctr=FAKE + 4) == -22
    for bad in ((0, 1, 16, 256), (2, 0, 16, 256), (2, 1, 0, 256), (2, 1, 16, 0),
                (65537, 1, 16, 256), (1, 1 << 16, 1 << 16, 1), (1, 1, 1 << 30, 4)):
        assert call(shape=Shape(*bad)) == -22
    for bad in ((None, 10, 1 << 20, 4096), (FAKE, 0, 1 << 20, 4096), (FAKE, 1 << 32, 1 << 20, 4096),
                (FAKE, 10, 4095, 4096), (FAKE, 10, 1 << 20, 4095)):
        assert call(src=Pool(*bad)) == -22 and call(dst=Pool(*bad)) == -22
    assert call(n=0, moves=None) == 0  # nothing to do, and nothing to count
