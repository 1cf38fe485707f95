"""The paged cache's Python calls refuse what the GPU could not read or write, before the library is
called. The library is a stand-in that records its calls, and tensors that stand for the GPU's are
host tensors that say they are."""

import types

import pytest

from test_abi import libpath  # noqa: F401  (the built library)

torch = pytest.importorskip("torch")


class OnGpu(torch.Tensor):
    is_cuda = True


def gpu(t):
    return t.as_subclass(OnGpu)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.fixture()
def db(libpath, monkeypatch):  # noqa: F811
    import descriptor_build_gb300 as db

    calls = []
    lib = types.SimpleNamespace(**{
        f"db_page_{op}": (lambda *a, op=op: calls.append((op, a)) or 0)
        for op in ("extend", "fork", "free", "compact", "copy")})
    monkeypatch.setattr(db, "_lib", lib)
    monkeypatch.setattr(db, "calls", calls, raising=False)
    return db


def arguments(db):
    """Each call's tensors, all of them where they should be."""
    g = lambda t: gpu(t)
    cache = lambda: db.PageTables(g(i32(6, 5)), g(i32(6)), g(i32(40)), g(i32(2)), 16)
    ws, ctr = (lambda: g(torch.zeros(4096, dtype=torch.uint8))), (lambda: g(torch.zeros(4, dtype=torch.int64)))
    status = lambda n: g(torch.zeros(n, dtype=torch.uint8))
    pool = lambda: g(torch.zeros(2, 40, 16, 8))
    return {
        "extend": dict(tables=cache(), req=g(i32(3, 2)), moves=g(i32(3, 4)), n_moves=g(i32(1)), ws=ws(),
                       status=status(3), ctr=ctr()),
        "fork": dict(tables=cache(), req=g(i32(3, 4)), ws=ws(), status=status(3), ctr=ctr()),
        "free": dict(tables=cache(), req=g(i32(3, 2)), ws=ws(), status=status(3), ctr=ctr()),
        "compact": dict(tables=cache(), out=cache(), moves=g(i32(7, 4)), n_moves=g(i32(1)), ws=ws(), ctr=ctr()),
        "copy": dict(moves=g(i32(7, 4)), n_moves=g(i32(1)), src=pool(), dst=pool(), token_dim=2, ctr=ctr()),
    }


OPS = ("extend", "fork", "free", "compact", "copy")
TENSORS = [(op, k) for op, ks in (
    ("extend", ("req", "moves", "n_moves", "ws", "status", "ctr")), ("fork", ("req", "ws", "status", "ctr")),
    ("free", ("req", "ws", "status", "ctr")), ("compact", ("moves", "n_moves", "ws", "ctr")),
    ("copy", ("moves", "n_moves", "src", "dst", "ctr"))) for k in ks]


def call(db, op, args):
    return getattr(db, f"page_{op}")(stream=0, **args)


@pytest.mark.parametrize("op", OPS)
def test_calls_reach_the_library(db, op):
    args = arguments(db)[op]
    call(db, op, args)
    (name, got), = db.calls
    assert name == op
    for k, t in args.items():
        if isinstance(t, torch.Tensor) and k not in ("src", "dst"):
            assert t.data_ptr() in got
    if op in ("extend", "fork", "free"):
        assert got[2] == 3
    else:
        assert 7 in got


@pytest.mark.parametrize("op,name", TENSORS, ids=["-".join(x) for x in TENSORS])
def test_ordinary_host_memory_is_refused(db, op, name):
    args = arguments(db)[op]
    args[name] = args[name].as_subclass(torch.Tensor)
    with pytest.raises(ValueError, match="pinned"):
        call(db, op, args)
    assert db.calls == []


def test_one_pool_in_ordinary_host_memory_is_refused(db):
    args = arguments(db)["copy"]
    args["src"] = args["dst"] = torch.zeros(2, 40, 16, 8)
    with pytest.raises(ValueError, match="pinned"):
        call(db, "copy", args)
    assert db.calls == []


@pytest.mark.parametrize("k", range(4), ids=["table", "length", "refs", "free"])
def test_tables_in_ordinary_host_memory_are_refused(db, k):
    arrays = [gpu(i32(6, 5)), gpu(i32(6)), gpu(i32(40)), gpu(i32(2))]
    db.PageTables(*arrays, 16)
    arrays[k] = arrays[k].as_subclass(torch.Tensor)
    with pytest.raises(ValueError, match="pinned"):
        db.PageTables(*arrays, 16)


SHORT = [(op, k) for op, k in TENSORS if k in ("n_moves", "ctr", "status")] + [("extend", "moves")]


@pytest.mark.parametrize("op,name", SHORT, ids=["-".join(x) for x in SHORT])
def test_arrays_shorter_than_what_is_written_are_refused(db, op, name):
    args = arguments(db)[op]
    args[name] = args[name][:-1]
    with pytest.raises(ValueError):
        call(db, op, args)
    assert db.calls == []


@pytest.mark.parametrize("op,name", [x for x in TENSORS if x[1] not in ("src", "dst", "n_moves")],
                         ids=["-".join(x) for x in TENSORS if x[1] not in ("src", "dst", "n_moves")])
def test_strided_arrays_are_refused(db, op, name):
    args = arguments(db)[op]
    t = args[name].as_subclass(torch.Tensor)
    args[name] = gpu(torch.cat([t, t])[::2])
    with pytest.raises(ValueError, match="contiguous"):
        call(db, op, args)
    assert db.calls == []


BATCHES = [(op, k) for op, k in TENSORS if k in ("req", "moves")]


@pytest.mark.parametrize("op,name", BATCHES, ids=["-".join(x) for x in BATCHES])
def test_batches_of_another_type_or_width_are_refused(db, op, name):
    """An int64 [[0, 7]], what torch.tensor makes of it, would be read as the records {0, 0}, {7, 0}."""
    n, width = arguments(db)[op][name].shape
    for dtype in (torch.int64, torch.float32, torch.uint8, torch.int16):
        args = arguments(db)[op]
        args[name] = gpu(torch.zeros((n, width), dtype=dtype))
        with pytest.raises(ValueError, match="int32"):
            call(db, op, args)
    for shape in ((n, 6 - width), (n, width, 1), (n * width + 1,), (n, 1), ()):
        args = arguments(db)[op]
        args[name] = gpu(i32(*shape))
        with pytest.raises(ValueError, match="int32"):
            call(db, op, args)
    assert db.calls == []


@pytest.mark.parametrize("op,name", BATCHES, ids=["-".join(x) for x in BATCHES])
def test_batches_flat_unsigned_and_empty(db, op, name):
    n, width = arguments(db)[op][name].shape
    for t in (i32(n * width), i32(1, n, width), i32(n, width).view(torch.uint32)):
        args = arguments(db)[op]
        args[name] = gpu(t)
        call(db, op, args)
    if (op, name) != ("extend", "moves"):
        for t in (i32(0), i32(0, width)):
            args = arguments(db)[op]
            args[name] = gpu(t)
            call(db, op, args)
            assert 0 in db.calls[-1][1]


@pytest.mark.parametrize("tokens", [-1, 0, -16, 1 << 32])
def test_page_tokens_out_of_range_are_refused(db, tokens):
    with pytest.raises(ValueError, match="page_tokens"):
        db.PageTables(gpu(i32(6, 5)), gpu(i32(6)), gpu(i32(40)), gpu(i32(2)), tokens)


def test_caches_of_no_or_too_many_sequences_or_pages_are_refused(db):
    many = 1 << 31  # sizes alone: nothing is allocated
    size = lambda *shape: torch.empty(shape, dtype=torch.int32, device="meta")
    for table, length, refs, free in (((many, 1), many, 40, 2), ((6, 5), 6, many, many // 32),
                                      ((0, 5), 0, 40, 2), ((6, 5), 6, 0, 0)):
        with pytest.raises(ValueError, match="at least one sequence and one page, and below 2.31"):
            db.PageTables(size(*table), size(length), size(refs), size(free), 16)
    with pytest.raises(ValueError, match="columns"):
        db.PageTables(gpu(i32(6, 0)), gpu(i32(6)), gpu(i32(40)), gpu(i32(2)), 16)


def test_free_words_off_16_bytes_are_refused(db):
    arrays = gpu(i32(6, 5)), gpu(i32(6)), gpu(i32(40))
    for shift in (1, 2, 3):
        with pytest.raises(ValueError, match="16 bytes"):
            db.PageTables(*arrays, gpu(i32(2 + shift)[shift:]), 16)
    db.PageTables(*arrays, gpu(i32(6)[4:]), 16)
