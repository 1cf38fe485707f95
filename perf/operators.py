"""The paged-cache operators, as they are timed: sizes, inputs, plain forms and 64-bit results.

A paged cache keeps a sequence's tokens in fixed-size pages of a device heap, the pages that a put or an
NVMe request moves. Five operators keep its tables and move its pages:

  extend   sequences grow by tokens: pages are taken, lowest free index first, and a partly filled
           last page that other sequences hold too is replaced by a copy of its own (copy on write)
  fork     a sequence gets the first tokens of another by sharing its pages
  free     sequences are cut back to their first tokens (or to none) and give pages back
  compact  live pages at high indices get the places of free pages at low ones, the tables follow
  copy     the bytes of listed pages, all planes of them, whole or their first tokens

A pass leaves the state such that the next one finds the same work: what it takes it has given back
first, and which pages are taken depends on the set of free ones alone.

Tables (int32): table [n_seqs, columns], -1 where no page is; length [n_seqs] tokens; refs [n_pages];
free, one bit a page, 32 in a word, set where the page is free.
"""

import numpy as np
import torch

own = False

ALL = -1  # "every token of the page" in a copy record (0xFFFFFFFF)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "u8": torch.uint8}


# --------------------------------------------------------------------------------------------- cases
def _step(name, seqs, tokens, page, columns, pages, take):
    return {"name": name, "op": "extend", "seqs": seqs, "tokens": tokens, "page": page, "columns": columns,
            "pages": pages, "take": take}


def _admit(name, seqs, ended, prompt, shared, page, columns, pages):
    return {"name": name, "op": "free", "seqs": seqs, "ended": ended, "prompt": prompt, "shared": shared,
            "page": page, "columns": columns, "pages": pages}


def _fork(name, parents, children, tokens, page, columns, pages, planes, heads, width, type):
    return {"name": name, "op": "fork", "parents": parents, "children": children, "tokens": tokens, "page": page,
            "columns": columns, "pages": pages, "planes": planes, "heads": heads, "width": width, "type": type}


def _copy(name, moved, pages, planes, page, heads, width, type, partial, heads_first, same):
    return {"name": name, "op": "copy", "moved": moved, "pages": pages, "planes": planes, "page": page, "heads": heads,
            "width": width, "type": type, "partial": partial, "heads_first": heads_first, "same": same}


def _compact(name, seqs, columns, page, pages, live, planes, bytes, limit):
    return {"name": name, "op": "compact", "seqs": seqs, "columns": columns, "page": page, "pages": pages,
            "live": live, "planes": planes, "bytes": bytes, "limit": limit}


def listed():
    return [
        # A speculative step of a small decode batch: 1 to 4 drafted tokens handed back and as many taken.
        _step("extend_decode_48", 48, 1500, 16, 256, 16384, 4),
        # The same for a large batch of longer sequences in a pool of a million pages, single tokens.
        _step("extend_decode_4096", 4096, 3000, 16, 512, 1048576, 1),
        # A chunk of prompt for each of 192 sequences: hundreds of pages each.
        _step("extend_prefill_192", 192, 3001, 16, 1024, 262144, 8192),
        # A serving slot's turnover: half the sequences end, new prompts behind one shared prefix enter.
        _admit("free_turnover_256", 512, 256, 900, 512, 16, 256, 65536),
        # Long contexts end and enter: 64 sequences of about 80,000 tokens.
        _admit("free_long_64", 64, 64, 80003, 0, 16, 8192, 1048576),
        # One step of a beam search: 32 beams dropped, forked anew from 8 sequences, and extended by a token
        # with the copies that asks for.
        _fork("fork_beams_8x4", 8, 4, 700, 16, 128, 2048, 8, 8, 128, "bf16"),
        # 1,023 samples of one long prompt, in an 8-bit cache with pages of 64 tokens.
        _fork("fork_samples_1023", 1, 1023, 65501, 64, 1100, 8192, 4, 4, 128, "u8"),
        # The copies of a few writers' shared pages: 6 pages of one layer.
        _copy("copy_6_pages", 6, 512, 2, 16, 8, 128, "bf16", True, False, True),
        # An odd 8-bit layout, heads outermost, rows of 112 codes and a 4-byte scale, fetched from a staging pool
        # whose pages hold all planes.
        _copy("copy_heads_8bit", 1501, 2048, 6, 48, 5, 116, "u8", True, True, False),
        # Whole pages of 16 planes into another place of a 4 GiB pool.
        _copy("copy_whole_4gib", 3500, 8192, 16, 16, 8, 128, "bf16", False, False, True),
        # A small pool compacted before its region is registered as one range.
        _compact("compact_4096", 64, 128, 16, 4096, 0.6, 2, 8192, 0),
        # A large one: 131,072 pages of 64 KiB, 55 % live.
        _compact("compact_131072", 1024, 512, 16, 131072, 0.55, 2, 32768, 0),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("extend", "extend", "free", "free", "fork", "copy", "copy", "compact"))
    page = rng.choice((8, 16, 16, 32, 48, 64, 128))
    if op == "extend":
        seqs = _log(rng, 1, 4096)
        take = rng.choice((1, 1, rng.randint(2, 8), _log(rng, 16, max(16, min(8192, 1500000 // seqs)))))
        tokens = _log(rng, 1, min(8000, max(2, 400000 * page // seqs)))
        columns = (2 * tokens + take) // page + rng.randint(3, 40)
        used = seqs * ((2 * tokens + take) // page + 2)
        return _step("", seqs, tokens, page, columns, int(used * rng.uniform(1.1, 1.6)) + rng.randint(1, 4000), take)
    if op == "free":
        seqs = _log(rng, 2, 2048)
        ended = rng.randint(1, seqs)
        prompt = _log(rng, 1, max(2, min(80000, 300000 * page // seqs)))
        shared = rng.choice((0, page * rng.randint(0, 64)))
        columns = (2 * prompt + shared) // page + rng.randint(3, 40)
        used = seqs * ((2 * prompt) // page + 2) + shared // page
        return _admit("", seqs, ended, prompt, shared, page, columns, int(used * rng.uniform(1.1, 1.5)) + rng.randint(1, 3000))
    if op == "fork":
        parents = _log(rng, 1, 32)
        children = _log(rng, 1, max(1, 1024 // parents))
        tokens = _log(rng, 1, max(2, min(60000, page * 1000000 // (parents * children))))
        planes, heads, type = rng.randint(1, 6), rng.choice((1, 2, 4, 5, 8)), rng.choice(("bf16", "f16", "u8", "f32"))
        width = rng.choice((64, 72, 96, 100, 128))
        used = parents * ((2 * tokens) // page + 2) + 2 * parents * children
        pages = int(used * rng.uniform(1.05, 1.4)) + rng.randint(1, 300)
        while planes > 1 and planes * pages * page * heads * width * 4 > 2 << 30:
            planes -= 1
        while pages * page * heads * width * 4 > 2 << 30 and heads > 1:
            heads -= 1
        return _fork("", parents, children, tokens, page, (2 * tokens) // page + rng.randint(3, 20), pages, planes, heads, width, type)
    if op == "copy":
        heads, width, type = rng.choice((1, 2, 4, 5, 8)), rng.choice((4, 64, 72, 100, 116, 128)), rng.choice(("bf16", "u8", "u8", "f32"))
        planes = _log(rng, 1, 32)
        one = planes * page * heads * width * TYPES[type].itemsize
        pages = max(4, min(16384, _log(rng, 8, 16384), (3 << 30) // one))
        return _copy("", rng.randint(1, max(1, pages // 2 - 1)), pages, planes, page, heads, width, type, rng.random() < 0.6,
                     rng.random() < 0.5, rng.random() < 0.5)
    seqs, bytes, planes = _log(rng, 1, 1024), rng.choice((64, 960, 4096, 8192, 32768)), rng.randint(1, 4)
    pages = min(_log(rng, 64, 131072), (6 << 30) // (bytes * planes))
    columns = max(1, pages // seqs)
    return _compact("", seqs, columns, page, pages, rng.uniform(0.1, 0.95), planes, bytes,
                    rng.choice((0, 0, rng.randint(1, max(2, pages // 8)))))


# -------------------------------------------------------------------------------------------- inputs
def _pack(free):
    words = np.zeros(-(-len(free) // 32) * 32, np.uint64)
    words[: len(free)] = free
    return (words.reshape(-1, 32) << np.arange(32, dtype=np.uint64)).sum(1).astype(np.uint32).view(np.int32)


def _lengths(rng, n, about):
    return np.maximum(1, rng.integers(about // 2, about + about // 2 + 1, n))


def _rows(rng, case, seqs, lengths, shared=0):
    """Tables of `seqs` sequences with pages at places all over the pool, the first `shared` tokens of all in the same
    pages."""
    page, columns, pages = case["page"], case["columns"], case["pages"]
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((seqs, columns), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    prefix = order[: shared // page]
    at = len(prefix)
    for i in range(seqs):
        n = -(-int(lengths[i]) // page)
        table[i, : len(prefix)] = prefix
        table[i, len(prefix) : n] = order[at : at + n - len(prefix)]
        at += n - len(prefix)
        np.add.at(refs, table[i, :n], 1)
    if at > pages:
        raise ValueError("the pool is too small for the case")
    return table, refs


def _host(case, seed):
    """The case's tables and requests as numpy arrays."""
    rng = np.random.default_rng([int(seed), 77])
    op, page = case["op"], case["page"]
    h = {}
    if op == "extend":
        n = case["seqs"]
        base = _lengths(rng, n, case["tokens"])
        take = rng.integers(1, case["take"] + 1, n) if case["take"] < 16 else np.full(n, case["take"])
        h["length"] = base + take  # as the step before left them
        h["table"], h["refs"] = _rows(rng, case, n, h["length"])
        seq = rng.permutation(n)
        h["cut"] = np.stack([seq, base[seq]], 1)
        h["grow"] = np.stack([seq, take[seq]], 1)
    elif op == "free":
        n, ended = case["seqs"], case["ended"]
        h["length"] = _lengths(rng, n, case["prompt"]) + case["shared"]
        h["table"], h["refs"] = _rows(rng, case, n, h["length"], case["shared"])
        seq = rng.permutation(n)[:ended]
        prompt = h["length"][seq] - case["shared"]  # those that end leave the shared prefix, and others enter behind it
        h["cut"] = np.stack([seq, np.full(ended, case["shared"])], 1)
        h["grow"] = np.stack([seq, prompt], 1)
    elif op == "fork":
        par, kids = case["parents"], case["parents"] * case["children"]
        length = _lengths(rng, par, case["tokens"]) if par > 1 else np.array([case["tokens"]])
        table, refs = _rows(rng, case, par, length)
        rows = np.full((par + kids, case["columns"]), -1, np.int32)
        rows[:par] = table
        parent = np.repeat(np.arange(par), case["children"])
        child = par + rng.permutation(kids)
        # the step before: every beam shares its parent's pages, and wrote a last one of its own
        old, spare = np.zeros(par + kids, np.int64), np.flatnonzero(refs == 0)
        old[:par] = length
        was = rng.permutation(parent)
        for k in range(kids):
            p, c = was[k], child[k]
            m = -(-int(length[p]) // page)
            rows[c, :m] = rows[p, :m]
            np.add.at(refs, rows[c, : m - 1], 1)
            rows[c, m - 1] = spare[k]
            refs[spare[k]] = 1
            old[c] = length[p]
        h["table"], h["refs"], h["length"] = rows, refs, old
        pick = parent[rng.permutation(kids)] if par > 1 else parent
        h["cut"] = np.stack([child, np.zeros(kids, np.int64)], 1)
        h["fork"] = np.stack([pick, child, length[pick], np.zeros(kids, np.int64)], 1)
        h["grow"] = np.stack([child, np.ones(kids, np.int64)], 1)
    elif op == "copy":
        k, pages = case["moved"], case["pages"]
        if case["same"]:
            p = rng.permutation(pages)
            src, dst = p[:k], p[k : 2 * k]
        else:
            src, dst = rng.integers(0, pages, k), rng.permutation(pages)[:k]
        tokens = rng.integers(1, page + 1, k) if case["partial"] else np.full(k, ALL)
        h["list"] = np.stack([src, dst, tokens, np.zeros(k, np.int64)], 1)
    else:
        n, pages = case["seqs"], case["pages"]
        want = int(case["live"] * pages)
        live = np.sort(rng.permutation(pages)[:want])
        held = live[rng.permutation(want)][: n * case["columns"]].astype(np.int32)
        cuts = np.minimum(np.sort(rng.integers(0, len(held) + 1, n - 1)) if n > 1 else np.zeros(0, np.int64), len(held))
        bounds = np.concatenate([[0], cuts, [len(held)]]).astype(np.int64)
        table, refs, length = np.full((n, case["columns"]), -1, np.int32), np.zeros(pages, np.int32), np.zeros(n, np.int64)
        for i in range(n):
            row = held[bounds[i] : bounds[i + 1]][: case["columns"]]
            if i and i % 4 == 0 and length[i - 1]:  # some are forks of the one before
                row = np.concatenate([table[i - 1, : max(1, length[i - 1] // page // 2)], row])[: case["columns"]]
            table[i, : len(row)] = row
            length[i] = len(row) * page
            np.add.at(refs, row, 1)
        h["table"], h["refs"], h["length"] = table, refs, length
    for k, v in h.items():
        h[k] = np.ascontiguousarray(v, dtype=np.int32)
    if "refs" in h:
        h["free"] = _pack(h["refs"] == 0)
    return h


def _fill(shape, type, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7 + 3)
    x = torch.empty(shape, dtype=TYPES[type], device="cuda")
    return x.random_(0, 256, generator=g) if type == "u8" else x.normal_(generator=g)


def _pools(case, seed):
    """(source, destination, token_dim) of the case's page pools, [planes, pages, ...]."""
    if case["op"] == "compact":
        x = _fill((case["planes"], case["pages"], case["bytes"] // 4), "f32", seed)
        return x, x, None
    inner = (case["page"], case["heads"], case["width"])
    if case["op"] == "copy" and case["heads_first"]:
        inner = (case["heads"], case["page"], case["width"])
    token_dim = 3 if case["op"] == "copy" and case["heads_first"] else 2
    shape = (case["planes"], case["pages"]) + inner
    dst = _fill(shape, case["type"], seed)
    if case["op"] == "fork" or case["same"]:
        return dst, dst, token_dim if case["op"] == "fork" or case["partial"] else None
    src = _fill((case["pages"], case["planes"]) + inner, case["type"], seed + 1).transpose(0, 1)
    return src, dst, token_dim if case["partial"] else None


def prepare(case, seed):
    s = {"case": case, "op": case["op"], "page": case["page"]}
    for k, v in _host(case, seed).items():
        s[k] = torch.from_numpy(v).cuda()
    if s["op"] in ("fork", "copy", "compact"):
        s["src"], s["dst"], s["token_dim"] = _pools(case, seed)
    n = 0
    if s["op"] == "copy":
        s["count"] = torch.tensor([len(s["list"])], dtype=torch.int32, device="cuda")
    elif s["op"] == "compact":
        n = case["limit"] or case["pages"] // 2
        s["move_ctr"] = torch.zeros(4, dtype=torch.int64, device="cuda")
        for k in ("table", "refs", "free"):
            s[k + "_out"] = torch.zeros_like(s[k])
    else:
        n = len(s["grow"])
        for k in ("cut", "fork", "grow"):
            if k in s:
                s[k + "_status"] = torch.zeros(len(s[k]), dtype=torch.uint8, device="cuda")
                s[k + "_ctr"] = torch.zeros(4, dtype=torch.int64, device="cuda")
    if n:
        s["list"] = torch.zeros((n, 4), dtype=torch.int32, device="cuda")
        s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own and "table" in s:
        import descriptor_build_gb300 as db

        s["tables"] = db.PageTables(s["table"], s["length"], s["refs"], s["free"], s["page"])
        s["ws"] = db.workspace(db.page_workspace_size(s["table"].shape[0], s["refs"].shape[0]))
        if s["op"] == "compact":
            s["after"] = db.PageTables(s["table_out"], s["length"], s["refs_out"], s["free_out"], s["page"])
    return s


# --------------------------------------------------------------------------------------- plain forms
def _bits(words, n):
    return ((words.long()[:, None] >> torch.arange(32, device=words.device)) & 1).bool().reshape(-1)[:n]


def _words(bits, words):
    x = torch.zeros(words.numel() * 32, dtype=torch.int64, device=bits.device)
    x[: bits.numel()] = bits.long()
    x = (x.reshape(-1, 32) << torch.arange(32, device=bits.device)).sum(1)
    return ((x ^ 0x80000000) - 0x80000000).int()


def _first(seq, n_seqs):
    """(seq is a sequence and no request before names it, seq or 0)."""
    n = seq.numel()
    i = torch.arange(n, device=seq.device)
    inside = (seq >= 0) & (seq < n_seqs)
    to = torch.where(inside, seq, n_seqs)
    first = torch.full((n_seqs + 1,), n, dtype=torch.int64, device=seq.device).scatter_reduce(0, to, i, "amin")
    return inside & (first[to] == i), torch.where(inside, seq, 0)


def _tell(ctr, total, n_invalid, n_overflow=0):
    zero = torch.zeros((), dtype=torch.int64, device=ctr.device)
    ctr.copy_(torch.stack([total + zero, n_invalid + zero, n_overflow + zero, zero]))


def plain_extend(s, req, status, ctr, copies, count):
    page, table, length, refs, free = s["page"], s["table"], s["length"], s["refs"], s["free"]
    (n_seqs, columns), n_pages, dev = table.shape, refs.numel(), table.device
    i = torch.arange(len(req), device=dev)
    add = req[:, 1].long()
    ok, seq = _first(req[:, 0].long(), n_seqs)
    old = length[seq].long()
    ok &= (add >= 0) & (old + add <= columns * page)
    had, now = (old + page - 1) // page, (old + add + page - 1) // page
    grow = torch.where(ok, now - had, 0)
    last = table[seq, (had - 1).clamp(min=0)].long().clamp(min=0)
    shared = ok & (add > 0) & (old % page != 0) & (refs[last] > 1)
    to = torch.where(shared, last, n_pages)
    holders = torch.zeros(n_pages + 1, dtype=torch.int64, device=dev).index_add_(0, to, torch.ones_like(to))
    latest = torch.full((n_pages + 1,), -1, dtype=torch.int64, device=dev).scatter_reduce(0, to, i, "amax")
    cow = shared & ~((holders[to] == refs[last]) & (latest[to] == i))
    need = grow + cow
    start = need.cumsum(0) - need
    total = need.sum()
    is_free = _bits(free, n_pages)
    fits = total <= is_free.sum()
    go, cow = ok & fits, cow & fits
    rank = is_free.cumsum(0) - 1
    nth = torch.zeros(n_pages + 1, dtype=torch.int64, device=dev)
    nth.scatter_(0, torch.where(is_free, rank, n_pages), torch.arange(n_pages, device=dev))
    column = torch.arange(columns, device=dev)
    rows = table[seq].long()
    new = (column >= had[:, None]) & (column < now[:, None]) & go[:, None]
    at = (start + cow - had)[:, None] + column
    delta = torch.where(new, nth[at.clamp(0, n_pages)] - rows, 0)
    fresh = nth[start.clamp(max=n_pages)]
    delta += torch.where(cow[:, None] & (column == (had - 1)[:, None]), fresh[:, None] - rows, 0)
    table.index_add_(0, seq, delta.int())
    length.index_add_(0, seq, torch.where(go, add, 0).int())
    taken = is_free & (rank < total) & fits
    refs += taken
    refs.index_add_(0, last, -cow.int())
    free.copy_(_words(is_free & ~taken, free))
    place = torch.where(cow, cow.cumsum(0) - 1, len(req))
    listed_ = torch.cat([copies, copies[:1]])
    listed_[place] = torch.stack([last, fresh, old % page, torch.zeros_like(old)], 1).int()
    copies.copy_(listed_[:-1])
    count.copy_(cow.sum().reshape(1))
    status.copy_(torch.where(ok, torch.where(fits, 0, 2), 1))
    _tell(ctr, total, (~ok).sum(), torch.where(fits, 0, ok.sum()))


def plain_fork(s, req, status, ctr):
    page, table, length, refs, free = s["page"], s["table"], s["length"], s["refs"], s["free"]
    (n_seqs, columns), n_pages, dev = table.shape, refs.numel(), table.device
    parent, tokens = req[:, 0].long(), req[:, 2].long()
    ok, child = _first(req[:, 1].long(), n_seqs)
    ok &= (parent >= 0) & (parent < n_seqs) & (parent != child)
    parent = torch.where(ok, parent, 0)
    ok &= (length[child] == 0) & (tokens >= 0) & (tokens <= length[parent])
    n = torch.where(ok, (tokens + page - 1) // page, 0)
    column = torch.arange(columns, device=dev)
    held = column < n[:, None]
    rows = table[parent]
    refs += torch.zeros(n_pages + 1, dtype=torch.int32, device=dev).index_add_(
        0, torch.where(held, rows, n_pages).reshape(-1), torch.ones(rows.numel(), dtype=torch.int32, device=dev))[:-1]
    table.index_add_(0, child, torch.where(held, rows - table[child], 0))
    length.index_add_(0, child, torch.where(ok, tokens, 0).int())
    status.copy_(torch.where(ok, 0, 1))
    _tell(ctr, n.sum(), (~ok).sum())


def plain_free(s, req, status, ctr):
    page, table, length, refs, free = s["page"], s["table"], s["length"], s["refs"], s["free"]
    (n_seqs, columns), n_pages, dev = table.shape, refs.numel(), table.device
    ok, seq = _first(req[:, 0].long(), n_seqs)
    keep = req[:, 1].long() & 0xFFFFFFFF
    old = length[seq].long()
    keep = torch.where(ok, torch.minimum(keep, old), old)
    column = torch.arange(columns, device=dev)
    gone = (column >= ((keep + page - 1) // page)[:, None]) & (column < ((old + page - 1) // page)[:, None])
    rows = table[seq]
    before = refs.clone()
    refs -= torch.zeros(n_pages + 1, dtype=torch.int32, device=dev).index_add_(
        0, torch.where(gone, rows, n_pages).reshape(-1), torch.ones(rows.numel(), dtype=torch.int32, device=dev))[:-1]
    free.copy_(_words(refs == 0, free))
    table.index_add_(0, seq, torch.where(gone, -1 - rows, 0))
    length.index_add_(0, seq, (keep - old).int())
    status.copy_(torch.where(ok, 0, 1))
    _tell(ctr, ((refs == 0) & (before > 0)).sum(), (~ok).sum())


def plain_compact(s, moves, count, ctr):
    table, refs, free, n_pages, dev = s["table"], s["refs"], s["free"], s["refs"].numel(), s["refs"].device
    cap = len(moves)
    p = torch.arange(n_pages, device=dev)
    is_free = _bits(free, n_pages)
    below = p < (~is_free).sum()
    hole, high = is_free & below, ~is_free & ~below
    total = hole.sum()
    hole_rank = hole.cumsum(0) - 1
    high_rank = total - high.cumsum(0)
    to, leaves = hole & (hole_rank < cap), high & (high_rank < cap)
    nowhere = torch.full((n_pages + 1,), 0, dtype=torch.int64, device=dev)
    dst = nowhere.scatter(0, torch.where(to, hole_rank, n_pages), p)
    src = nowhere.scatter(0, torch.where(leaves, high_rank, n_pages), p)
    k = torch.arange(cap, device=dev)
    made = torch.stack([src[:cap], dst[:cap], torch.full_like(k, ALL), torch.zeros_like(k)], 1).int()
    moves.copy_(torch.where((k < total)[:, None], made, moves))
    count.copy_(total.clamp(max=cap).reshape(1))
    place = torch.where(leaves, dst[high_rank.clamp(0, n_pages)], p)
    s["table_out"].copy_(torch.where(table >= 0, place[table.long().clamp(min=0)], -1))
    s["refs_out"].copy_(torch.where(leaves, 0, torch.where(to, refs[src[hole_rank.clamp(0, n_pages)]], refs)))
    s["free_out"].copy_(_words((is_free & ~to) | leaves, free))
    _tell(ctr, total, 0, (total - cap).clamp(min=0))


def plain_copy(records, count, src, dst, token_dim):
    r = records[torch.arange(len(records), device=records.device) < count]
    here, there = r[:, 0].long(), r[:, 1].long()
    got = src[:, here]
    if token_dim is not None:
        page = dst.shape[token_dim]
        tokens = torch.where(r[:, 2] < 0, page, r[:, 2])
        shape = [1, -1] + [1] * (dst.dim() - 2)
        at = [1] * dst.dim()
        at[token_dim] = page
        moved = torch.arange(page, device=dst.device).reshape(at) < tokens.reshape(shape)
        got = torch.where(moved, got, dst[:, there])
    dst[:, there] = got


# ----------------------------------------------------------------------------------------------- run
def _whole(x):
    """A pool's bytes as whole numbers."""
    x = x.reshape(-1)
    return x.view(torch.int64) if x.numel() * x.element_size() % 8 == 0 else x.view(torch.uint8)


def _answer(s):
    out = {k: s[k] for k in s if k.endswith(("_status", "_ctr", "_out"))}
    if s["op"] in ("extend", "free", "fork"):
        out |= {k: s[k] for k in ("table", "length", "refs", "free")}
    if s["op"] != "copy":
        out |= {"list": s["list"], "count": s["count"]}
    if "dst" in s:
        out["pool"] = _whole(s["dst"])
    return out


def run(s):
    op = s["op"]
    if own:
        import descriptor_build_gb300 as db

        if op in ("extend", "free", "fork"):
            t, ws = s["tables"], s["ws"]
            db.page_free(t, s["cut"], ws, status=s["cut_status"], ctr=s["cut_ctr"])
            if op == "fork":
                db.page_fork(t, s["fork"], ws, status=s["fork_status"], ctr=s["fork_ctr"])
            db.page_extend(t, s["grow"], s["list"], s["count"], ws, status=s["grow_status"], ctr=s["grow_ctr"])
        elif op == "compact":
            db.page_compact(s["tables"], s["after"], s["list"], s["count"], s["ws"], ctr=s["move_ctr"])
        if "dst" in s:
            db.page_copy(s["list"], s["count"], s["src"], s["dst"], s["token_dim"])
        return _answer(s)
    if op in ("extend", "free", "fork"):
        plain_free(s, s["cut"], s["cut_status"], s["cut_ctr"])
        if op == "fork":
            plain_fork(s, s["fork"], s["fork_status"], s["fork_ctr"])
        plain_extend(s, s["grow"], s["grow_status"], s["grow_ctr"], s["list"], s["count"])
    elif op == "compact":
        plain_compact(s, s["list"], s["count"], s["move_ctr"])
    if "dst" in s:
        plain_copy(s["list"], s["count"], s["src"], s["dst"], s["token_dim"])
    return _answer(s)


def work(case):
    """Bytes of one pass: requests, the table entries, references and free bits that change (read where their old value
    counts), and each moved page read and written once."""
    op, page = case["op"], case["page"]
    bits = case["pages"] / 8
    if op in ("extend", "free"):
        n = case["seqs"] if op == "extend" else case["ended"]
        take = case["take"] if op == "extend" else case["prompt"]
        take = (take + 1) / 2 if take < 16 else take
        # freed: entry read and cleared, reference read and written; taken: entry and reference written
        return {"bytes": n * (2 * (8 + 1) + 4 * 4) + n * take / page * (16 + 8) + 2 * bits, "flops": 0}
    if op == "fork":
        kids, held = case["parents"] * case["children"], -(-case["tokens"] // page)
        one = case["planes"] * (case["tokens"] % page) * case["heads"] * case["width"] * TYPES[case["type"]].itemsize
        tables = kids * (8 + 16 + 8 + 3 + 6 * 4) + kids * held * (8 + 4) + case["parents"] * held * (4 + 16) + 2 * bits
        return {"bytes": tables + (kids * 2 * one if case["tokens"] % page else 0), "flops": 0}
    if op == "copy":
        one = case["planes"] * page * case["heads"] * case["width"] * TYPES[case["type"]].itemsize
        return {"bytes": 16 * case["moved"] + case["moved"] * 2 * one * ((page + 1) / 2 / page if case["partial"] else 1), "flops": 0}
    live = int(case["live"] * case["pages"])
    moves = live * (1 - live / case["pages"])
    moves = min(moves, case["limit"]) if case["limit"] else moves
    return {"bytes": 2 * 4 * case["seqs"] * case["columns"] + 8 * case["pages"] + 2 * bits + moves * (16 + 2 * case["planes"] * case["bytes"]),
            "flops": 0}


# --------------------------------------------------------------------------------------------- exact
class _Cache:
    """The operators one request at a time, on numpy arrays of 64-bit numbers."""

    def __init__(self, h, page):
        self.page, self.table, self.length, self.refs = page, h["table"].astype(np.int64), h["length"].astype(np.int64), h["refs"].astype(np.int64)

    def free(self, req):
        seen, given, bad, status = set(), 0, 0, []
        for seq, keep in req.tolist():
            ok = 0 <= seq < len(self.length) and seq not in seen
            seen.add(seq)
            status.append(0 if ok else 1)
            bad += not ok
            if not ok or keep >= self.length[seq]:
                continue
            a, b = -(-keep // self.page), -(-int(self.length[seq]) // self.page)
            held = self.table[seq, a:b]
            self.refs[held] -= 1  # a row names a page once
            given += int((self.refs[held] == 0).sum())
            self.table[seq, a:b] = -1
            self.length[seq] = keep
        return status, [given, bad, 0, 0]

    def fork(self, req):
        before, seen, taken, bad, status = self.length.copy(), set(), 0, 0, []
        for parent, child, tokens, _ in req.tolist():
            n = len(before)
            ok = 0 <= child < n and 0 <= parent < n and parent != child and child not in seen and before[child] == 0 and 0 <= tokens <= before[parent]
            seen.add(child)
            status.append(0 if ok else 1)
            bad += not ok
            if ok:
                m = -(-tokens // self.page)
                self.table[child, :m] = self.table[parent, :m]
                self.refs[self.table[child, :m]] += 1
                self.length[child] = tokens
                taken += m
        return status, [taken, bad, 0, 0]

    def extend(self, req, room):
        was = self.table.copy(), self.length.copy(), self.refs.copy()
        spare, at = np.flatnonzero(self.refs == 0), 0
        seen, copies, status, need, bad = set(), [], [], 0, 0
        for seq, add in req.tolist():
            ok = 0 <= seq < len(self.length) and seq not in seen and add >= 0 and self.length[seq] + add <= self.page * self.table.shape[1]
            seen.add(seq)
            status.append(0 if ok else 1)
            bad += not ok
            if not ok or add == 0:
                continue
            old = int(self.length[seq])
            a, b = -(-old // self.page), -(-(old + add) // self.page)
            if old % self.page and self.refs[self.table[seq, a - 1]] > 1:
                need += 1
                p = self.table[seq, a - 1]
                self.refs[p] -= 1
                if at < len(spare):
                    copies.append([p, spare[at], old % self.page, 0])
                    self.refs[spare[at]] = 1
                    self.table[seq, a - 1] = spare[at]
                at += 1
            got = spare[at : at + b - a]
            need += b - a
            at += b - a
            self.table[seq, a : a + len(got)] = got
            self.refs[got] = 1
            self.length[seq] += add
        short = need > len(spare)
        if short:
            self.table, self.length, self.refs = was
            copies, status = [], [2 if x == 0 else x for x in status]
        made = np.zeros((room, 4), np.int64)
        if copies:
            made[: len(copies)] = copies
        return status, made, len(copies), [need, bad, (len(status) - bad) if short else 0, 0]


def exact(case, seed):
    h, page, op = _host(case, seed), case["page"], case["op"]
    out = {}
    records = h.get("list")
    if op in ("extend", "free", "fork"):
        c = _Cache(h, page)
        out["cut_status"], out["cut_ctr"] = c.free(h["cut"])
        if op == "fork":
            out["fork_status"], out["fork_ctr"] = c.fork(h["fork"])
        out["grow_status"], records, n, out["grow_ctr"] = c.extend(h["grow"], len(h["grow"]))
        out |= {"table": c.table, "length": c.length, "refs": c.refs, "free": _pack(c.refs == 0), "list": records, "count": [n]}
        records = records[:n]
    elif op == "compact":
        refs, table = h["refs"].astype(np.int64), h["table"].astype(np.int64)
        n_pages, cap = len(refs), case["limit"] or case["pages"] // 2
        live, spare = np.flatnonzero(refs > 0)[::-1], np.flatnonzero(refs == 0)
        both = min(len(live), len(spare))
        total = int((spare[:both] < live[:both]).sum())  # the lowest free page against the highest live one, and so on
        n = min(total, cap)
        made = np.zeros((cap, 4), np.int64)
        made[:n, 0], made[:n, 1], made[:n, 2] = live[:n], spare[:n], ALL
        place = np.arange(n_pages)
        place[live[:n]] = spare[:n]
        refs[spare[:n]] = refs[live[:n]]
        refs[live[:n]] = 0
        out = {"table_out": np.where(table >= 0, place[table], -1), "refs_out": refs, "free_out": _pack(refs == 0),
               "list": made, "count": [n], "move_ctr": [total, 0, total - n, 0]}
        records = made[:n]
    if op in ("fork", "copy", "compact"):
        src, dst, token_dim = _pools(case, seed)
        if dst.numel() * dst.element_size() > 1 << 30:
            out["pool"] = None  # gigabytes that are moved, not computed: the smaller cases hold them
        else:
            a, b = (x.contiguous().view(torch.uint8).cpu().numpy() for x in (src, dst))
            a = b.copy() if src is dst else a
            for x, y, tokens, _ in np.asarray(records).tolist():
                if token_dim is None:
                    b[:, y] = a[:, x]
                else:
                    m = page if tokens < 0 else min(tokens, page)
                    at = (slice(None),) * (token_dim - 2) + (slice(0, m),)
                    b[(slice(None), y) + at] = a[(slice(None), x) + at]
            b = b.reshape(-1)
            out["pool"] = b.view(np.int64) if b.size % 8 == 0 else b
    if all(v is None for v in out.values()):
        return None
    return {k: np.asarray(v) if isinstance(v, list) else v for k, v in out.items()}
