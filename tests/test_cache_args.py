"""The C entry points on a paged cache's contents refuse bad arguments before they touch a GPU."""

import ctypes

import pytest

from test_abi import libpath  # noqa: F401  (the built library)
from test_page_args import FAKE, SZ, U32, U64, VP, Pool, Shape, tables

BF16, F16, F32, E4M3, I8 = range(5)
ref = ctypes.byref


class Batch(ctypes.Structure):
    _fields_ = [("seq", VP), ("start", VP), ("n", U32), ("rows", U32)]


class Layer(ctypes.Structure):
    _fields_ = [("k", VP), ("v", VP), ("k_scale", VP), ("v_scale", VP), ("k_stride", U64), ("v_stride", U64),
                ("k_scale_stride", U64), ("v_scale_stride", U64), ("heads", U32), ("width", U32), ("type", U32),
                ("heads_first", U32)]


class Rows(ctypes.Structure):
    _fields_ = [("base", VP), ("row_stride", U64), ("head_stride", U64)]


def batch(**kw):
    return changed(Batch(FAKE, FAKE, 3, 10), kw)


def layer(**kw):  # 16 tokens a page (tables), 2 heads of 32 values in bf16
    return changed(Layer(FAKE, FAKE, None, None, 2048, 2048, 0, 0, 2, 32, BF16, 0), kw)


def codes(**kw):
    return changed(Layer(FAKE, FAKE, FAKE, FAKE, 1024, 1024, 128, 128, 2, 32, E4M3, 0), kw)


def rows(**kw):
    return changed(Rows(FAKE, 128, 64), kw)


def changed(s, kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.fixture()
def lib(libpath):  # noqa: F811
    lib = ctypes.CDLL(libpath)
    lib.db_cache_write.argtypes = [VP, VP, VP, VP, VP, U32, VP, VP, VP]
    lib.db_cache_read.argtypes = [VP, VP, VP, VP, VP, VP, U32, VP, VP, VP]
    lib.db_cache_attention_workspace_size.argtypes = [U32] * 5 + [ctypes.POINTER(SZ)]
    lib.db_cache_attention.argtypes = [VP, VP, VP, VP, VP, U32, U32, U32, ctypes.c_float, VP, U32, VP, VP, VP, VP, SZ, VP]
    lib.db_draft_verify.argtypes = [VP, U32, U32, VP, VP, VP, U64, VP, U64, U32, U32, VP, VP, VP, VP, VP, VP, VP]
    lib.db_cache_keep.argtypes = [VP] * 10
    return lib


def at(s):
    return ref(s) if isinstance(s, ctypes.Structure) else s


def write(lib, t=None, b=None, c=None, k=None, v=None, kind=BF16, ctr=None):
    return lib.db_cache_write(t or tables(), at(b or batch()), at(c or layer()), at(k or rows()), at(v or rows()), kind, None,
                              ctr, None)


def read(lib, t=None, b=None, c=None, k=None, v=None, kind=BF16, ctr=None, first=None):
    return lib.db_cache_read(t or tables(), at(b or batch()), first, at(c or layer()), at(k or rows()), at(v or rows()), kind,
                             None, ctr, None)


def attend(lib, t=None, b=None, c=None, q=None, out=None, kind=BF16, q_heads=4, most=5, scale=0.1, mask=None, words=0,
           lse=None, ctr=None, ws=FAKE, size=1 << 40):
    wide = lambda: rows(row_stride=256)
    return lib.db_cache_attention(t or tables(), at(b or batch()), at(c or layer()), at(q or wide()), at(out or wide()), kind,
                                  q_heads, most, scale, mask, words, lse, None, ctr, ws, size, None)


def keep(lib, t=None, b=None, path=FAKE, accepted=FAKE, pool=None, shape=None, cut=None, ctr=None):
    return lib.db_cache_keep(t or tables(), at(b or batch()), path, accepted, at(pool or Pool(FAKE, 100, 1 << 20, 4096)),
                             at(shape or Shape(2, 1, 16, 256)), cut, None, ctr, None)


CALLS = [write, read, attend, keep]


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_tables_and_batches(lib, call):
    for bad in (dict(table=None), dict(length=None), dict(table=FAKE + 2), dict(length=FAKE + 1), dict(n_seqs=0),
                dict(columns=0), dict(n_pages=0), dict(page_tokens=0), dict(n_seqs=1 << 31), dict(n_pages=1 << 31)):
        assert call(lib, t=tables(**bad)) == -22
    for bad in (dict(seq=None), dict(start=None), dict(seq=FAKE + 2), dict(start=FAKE + 3), dict(n=1 << 31),
                dict(rows=1 << 31)):
        assert call(lib, b=batch(**bad)) == -22
    assert call(lib, ctr=FAKE + 4) == -22
    assert call(lib, b=batch(n=0, seq=None, start=None)) == 0  # nothing to do, and nothing to count


@pytest.mark.parametrize("call", CALLS[:3], ids=lambda f: f.__name__)
def test_layers(lib, call):
    for bad in (dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 4), dict(k_stride=2040), dict(v_stride=2052),
                dict(k_stride=2032), dict(v_stride=1024), dict(heads=0), dict(heads=1 << 28), dict(width=0), dict(width=24),
                dict(width=272), dict(type=F32), dict(type=5), dict(k_scale=FAKE), dict(v_scale=FAKE)):
        assert call(lib, c=layer(**bad)) == -22
    for bad in (dict(k_scale=None), dict(v_scale=None), dict(k_scale=FAKE + 2), dict(v_scale=FAKE + 1),
                dict(k_scale_stride=126), dict(v_scale_stride=124), dict(k_stride=1008), dict(type=BF16)):
        assert call(lib, c=codes(**bad)) == -22


def test_rows(lib):
    for call in (write, read):
        for bad in (dict(base=None), dict(base=FAKE + 8), dict(row_stride=120), dict(head_stride=56)):
            assert call(lib, k=rows(**bad)) == -22
            assert call(lib, v=rows(**bad)) == -22
        assert call(lib, kind=E4M3) == -22 and call(lib, kind=7) == -22
    # two heads that are written over each other; read from, they may be
    assert read(lib, k=rows(head_stride=48)) == -22
    assert read(lib, first=FAKE + 2) == -22


def test_attention(lib):
    size = SZ()
    ask = lambda *a: lib.db_cache_attention_workspace_size(*a, ref(size))
    for bad in ((65537, 4, 2, 32, 5), (3, 0, 2, 32, 5), (3, 4, 0, 32, 5), (3, 5, 2, 32, 5), (3, 130, 2, 32, 5),
                (3, 4, 2, 0, 5), (3, 4, 2, 24, 5), (3, 4, 2, 272, 5), (3, 4, 2, 32, 0), (3, 4, 2, 32, 1 << 24)):
        assert ask(*bad) == -22
    assert lib.db_cache_attention_workspace_size(3, 4, 2, 32, 5, None) == -22
    for bad in (dict(kind=F32), dict(kind=F16), dict(kind=E4M3), dict(q_heads=5), dict(q_heads=0), dict(q_heads=130),
                dict(most=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(b=batch(n=65537)),
                dict(mask=FAKE, words=0), dict(mask=FAKE + 2, words=1), dict(mask=FAKE, words=1, most=33), dict(lse=FAKE + 2),
                dict(ws=None), dict(ws=FAKE + 128), dict(q=rows(base=None)), dict(q=rows(base=FAKE + 8)),
                dict(out=rows(row_stride=264)), dict(out=rows(row_stride=256, head_stride=48))):
        assert attend(lib, **bad) == -22, bad
    assert attend(lib, c=codes(), kind=F32) == -22


def verify(lib, start=FAKE, n=3, rows=10, parent=FAKE, token=FAKE, p=FAKE, p_stride=50, q=None, q_stride=0, kind=F32, vocab=50,
           u=FAKE, path=FAKE, accepted=FAKE, following=FAKE, ctr=None):
    return lib.db_draft_verify(start, n, rows, parent, token, p, p_stride, q, q_stride, kind, vocab, u, path, accepted,
                               following, None, ctr, None)


def test_verification(lib):
    for name in ("start", "parent", "token", "p", "u", "path", "accepted", "following"):
        assert verify(lib, **{name: None}) == -22
        assert verify(lib, **{name: FAKE + 2}) == -22
    for bad in (dict(kind=E4M3), dict(vocab=0), dict(vocab=(1 << 19) + 1, p_stride=1 << 20), dict(p_stride=49),
                dict(q=FAKE, q_stride=49), dict(q=FAKE + 2, q_stride=50), dict(p_stride=1 << 32), dict(n=1 << 28),
                dict(rows=1 << 31), dict(ctr=FAKE + 4), dict(kind=BF16, p=FAKE + 1)):
        assert verify(lib, **bad) == -22, bad
    assert verify(lib, n=0, start=None, accepted=None, following=None) == 0


def test_keep(lib):
    for bad in (dict(path=None), dict(accepted=None), dict(path=FAKE + 2), dict(accepted=FAKE + 1), dict(cut=FAKE + 4)):
        assert keep(lib, **bad) == -22, bad
    for bad in ((0, 1, 16, 256), (2, 0, 16, 256), (2, 1, 8, 256), (2, 1, 16, 0), (65537, 1, 16, 256), (1, 1 << 28, 16, 1),
                (1 << 16, 1, 16, 1 << 12)):
        assert keep(lib, shape=Shape(*bad)) == -22, bad
    for bad in ((None, 100, 1 << 20, 4096), (FAKE, 99, 1 << 20, 4096), (FAKE, 1 << 32, 1 << 20, 4096),
                (FAKE, 100, 4095, 4096), (FAKE, 100, 1 << 20, 4095)):
        assert keep(lib, pool=Pool(*bad)) == -22, bad
    assert lib.db_cache_keep(tables(), ref(batch()), FAKE, FAKE, None, ref(Shape(2, 1, 16, 256)), None, None, None, None) == -22
    assert lib.db_cache_keep(tables(), ref(batch()), FAKE, FAKE, ref(Pool(FAKE, 100, 1 << 20, 4096)), None, None, None, None,
                             None) == -22
