"""The Python calls on a paged cache's contents refuse what the GPU could not read or write, before the library
is called, and hand over the rest as the C structs say. (As in test_page_binding.py the library is a stand-in, and
the GPU's tensors are host tensors that say they are.)"""

import struct
import types

import pytest

from test_abi import libpath  # noqa: F401  (the built library)
from test_page_binding import gpu, i32

torch = pytest.importorskip("torch")

NAMES = ("write", "read", "attention", "verify", "keep")


@pytest.fixture()
def db(libpath, monkeypatch):  # noqa: F811
    import descriptor_build_gb300 as db

    calls = []
    lib = types.SimpleNamespace(**{
        name: (lambda *a, name=name: calls.append((name, a)) or 0)
        for name in ("db_cache_write", "db_cache_read", "db_cache_attention", "db_draft_verify", "db_cache_keep")})
    monkeypatch.setattr(db, "_lib", lib)
    monkeypatch.setattr(db, "calls", calls, raising=False)
    return db


def arguments(db, op, kind=torch.bfloat16, token_dim=1):
    """Each call's tensors: 3 requests of 10 rows, 2 heads of 32 values, 4 query heads."""
    tables = db.PageTables(gpu(i32(6, 5)), gpu(i32(6)), gpu(i32(40)), gpu(i32(2)), 16)
    shape = (41, 16, 2, 32) if token_dim == 1 else (41, 2, 16, 32)
    pool = lambda: gpu(torch.zeros(shape, dtype=kind))
    scale = lambda: gpu(torch.zeros(shape[:3])) if kind.itemsize == 1 else None
    rows = lambda heads: gpu(torch.zeros(10, heads, 32, dtype=torch.bfloat16))
    batch = dict(tables=tables, seq=gpu(i32(3)), start=gpu(i32(4)))
    layer = dict(k_pool=pool(), v_pool=pool(), k_scale=scale(), v_scale=scale(), token_dim=token_dim)
    last = dict(status=gpu(torch.zeros(3, dtype=torch.uint8)), ctr=gpu(torch.zeros(4, dtype=torch.int64)), stream=0)
    if op == "write":
        return dict(batch, k=rows(2), v=rows(2), **layer, **last)
    if op == "read":
        return dict(batch, k=rows(2), v=rows(2), first=gpu(i32(3)), **layer, **last)
    if op == "attention":
        return dict(batch, q=rows(4), out=rows(4), ws=gpu(torch.zeros(4096, dtype=torch.uint8)), max_tokens=5,
                    mask=gpu(i32(10, 2)), lse=gpu(torch.zeros(10, 4)), **layer, **last)
    if op == "verify":
        return dict(start=gpu(i32(4)), parent=gpu(i32(10)), token=gpu(i32(10)), p=gpu(torch.zeros(10, 50)),
                    q=gpu(torch.zeros(10, 50)), u=gpu(torch.zeros(10)), path=gpu(i32(10)), accepted=gpu(i32(3)),
                    next=gpu(i32(3)), **last)
    return dict(batch, path=gpu(i32(10)), accepted=gpu(i32(3)), pool=gpu(torch.zeros(3, 41, 16, 2, 32)), token_dim=2,
                cut=gpu(i32(3, 2)), **last)


def call(db, op, args):
    getattr(db, "draft_verify" if op == "verify" else f"cache_{op}")(**args)


def refused(db, op, match=None, **changes):
    args = arguments(db, op, changes.pop("kind", torch.bfloat16))
    args.update(changes)
    with pytest.raises(ValueError, match=match):
        call(db, op, args)
    assert db.calls == []


def test_structs_hold_what_the_header_says(db):
    for token_dim in (1, 2):
        args = arguments(db, "write", torch.float8_e4m3fn, token_dim)
        args["k"] = gpu(torch.zeros(10, 3, 40, dtype=torch.bfloat16)[:, :2, :32])  # rows with gaps
        call(db, "write", args)
        _, (tables, batch, layer, k, v, kind, status, ctr, stream) = db.calls.pop()
        at = lambda name: args[name].data_ptr()
        assert struct.unpack("=QQII", batch) == (at("seq"), at("start"), 3, 10)
        assert struct.unpack("=8Q4I", layer) == (at("k_pool"), at("v_pool"), at("k_scale"), at("v_scale"), 1024, 1024, 128,
                                                 128, 2, 32, 3, token_dim - 1)
        assert struct.unpack("=3Q", k) == (at("k"), 240, 80)
        assert struct.unpack("=3Q", v) == (at("v"), 128, 64)
        assert (kind, status, ctr, stream) == (0, at("status"), at("ctr"), 0)
    args = arguments(db, "attention")
    call(db, "attention", args)
    _, a = db.calls.pop()
    assert struct.unpack("=8Q4I", a[2])[2:4] == (0, 0)
    assert a[5:8] == (0, 4, 5) and a[8] == 32**-0.5 and a[9:11] == (args["mask"].data_ptr(), 2)
    assert a[14:] == (args["ws"].data_ptr(), 4096, 0)
    args = arguments(db, "verify")
    wide = gpu(torch.zeros(10, 64))
    args.update(p=wide[:, :50], q=None)
    call(db, "verify", args)
    _, a = db.calls.pop()
    assert a[1:3] == (3, 10) and a[5:9] == (wide.data_ptr(), 64, None, 0) and a[9:11] == (2, 50)
    call(db, "keep", arguments(db, "keep"))
    assert db.calls.pop()[0] == "db_cache_keep"


TENSORS = [(op, k) for op, ks in (
    ("write", ("seq", "start", "k", "v", "k_pool", "v_pool", "k_scale", "v_scale", "status", "ctr")),
    ("read", ("seq", "start", "first", "k", "v", "k_pool", "v_pool", "k_scale", "v_scale", "status", "ctr")),
    ("attention", ("seq", "start", "q", "out", "k_pool", "v_pool", "k_scale", "v_scale", "ws", "mask", "lse", "status", "ctr")),
    ("verify", ("start", "parent", "token", "p", "q", "u", "path", "accepted", "next", "status", "ctr")),
    ("keep", ("seq", "start", "path", "accepted", "pool", "cut", "status", "ctr"))) for k in ks]


@pytest.mark.parametrize("op,name", TENSORS, ids=["-".join(x) for x in TENSORS])
def test_ordinary_host_memory_is_refused(db, op, name):
    args = arguments(db, op, torch.int8 if "scale" in name else torch.bfloat16)
    refused(db, op, "pinned", kind=torch.int8 if "scale" in name else torch.bfloat16,
            **{name: args[name].as_subclass(torch.Tensor)})


SHORT = [x for x in TENSORS if x[1] not in ("k", "v", "q", "p", "out", "k_pool", "v_pool", "k_scale", "v_scale", "pool", "ws")]


@pytest.mark.parametrize("op,name", SHORT, ids=["-".join(x) for x in SHORT])
def test_arrays_shorter_than_what_is_read_or_written_are_refused(db, op, name):
    t = arguments(db, op)[name]
    if (op, name) == ("keep", "path"):
        return  # its length is the number of rows
    if (name, op) != ("start", "verify"):
        refused(db, op, **{name: t[:-1]})


@pytest.mark.parametrize("op", NAMES)
def test_integers_of_another_type_are_refused(db, op):
    for name in ("seq", "start", "first", "mask", "parent", "token", "path", "accepted", "next"):
        t = arguments(db, op).get(name)
        if t is not None:
            for dtype in (torch.int64, torch.float32, torch.int16):
                refused(db, op, "int32", **{name: gpu(torch.zeros(t.shape, dtype=dtype))})


def test_shapes_and_types(db):
    z = lambda *s, t=torch.bfloat16: gpu(torch.zeros(s, dtype=t))
    for op in ("write", "read"):
        refused(db, op, k=z(10, 3, 32)), refused(db, op, v=z(10, 2, 48)), refused(db, op, k=z(9, 2, 32))
        refused(db, op, "neighbours", k=z(10, 32, 2).transpose(1, 2))
        refused(db, op, "one type", k=z(10, 2, 32, t=torch.float16))
        refused(db, op, "one type", k=z(10, 2, 32, t=torch.float64), v=z(10, 2, 32, t=torch.float64))
    for op in ("write", "read", "attention"):
        refused(db, op, "tokens", token_dim=2), refused(db, op, "token_dim", token_dim=3)
        refused(db, op, "differ", v_pool=z(41, 16, 2, 48)), refused(db, op, "pages", k_pool=z(39, 16, 2, 32))
        refused(db, op, "differ", v_pool=z(41, 16, 2, 32, t=torch.float16))
        refused(db, op, "contiguous", k_pool=z(41, 16, 4, 32)[:, :, ::2])
        refused(db, op, "holds", k_pool=z(41, 16, 2, 32, t=torch.float32))
        refused(db, op, "needs scales", kind=torch.int8, k_scale=None)
        refused(db, op, "needs scales", kind=torch.int8, v_scale=z(41, 16, 2, 1, t=torch.float32))
        refused(db, op, "float32", kind=torch.int8, k_scale=z(41, 16, 2))
        refused(db, op, "only 8-bit", k_scale=z(41, 16, 2, t=torch.float32))
    refused(db, "attention", q=z(9, 4, 32)), refused(db, "attention", out=z(10, 2, 32))
    refused(db, "attention", "mask", mask=gpu(i32(20))), refused(db, "attention", "float32", lse=z(10, 4))
    refused(db, "attention", out=z(10, 4, 32, t=torch.float16))
    refused(db, "verify", "neighbouring", p=z(50, 10, t=torch.float32).t()), refused(db, "verify", q=z(10, 49, t=torch.float32))
    refused(db, "verify", "one type", q=z(10, 50)), refused(db, "verify", "float32", u=z(10))
    refused(db, "keep", "tokens", pool=z(3, 41, 8, 2, 32)), refused(db, "keep", "pages", pool=z(3, 39, 16, 2, 32))
    refused(db, "keep", "token_dim", token_dim=None)
