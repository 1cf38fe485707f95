"""Operators on the contents of a paged cache, as they are timed: sizes, inputs, plain forms and 64-bit results.

The paged cache's tables (perf/operators.py) say which pages hold a sequence's tokens. These operators work on what the
pages hold, and take a speculative step of a serving process from the drafted tokens to the cut that gives the rejected
ones back:

  write    new tokens' keys and values go to their slots, as they are or as 8-bit codes with a scale for each token and head
  read     tokens' keys and values come back from the pages in order, codes times scales
  attend   the drafted tokens of a tree attend to their sequence's cache and to their ancestors in the tree
  verify   drafted tokens are accepted or not by the target's probabilities and given random numbers, and one more is drawn
  keep     the accepted path's tokens move together behind the tokens before them, in every plane

A batch is seq [n] and start [n + 1], int32: rows start[i] to start[i + 1] of what comes with it (keys, queries, nodes of a
tree) belong to sequence seq[i], and are its last tokens where the call works on new ones.

Pools are [pages, tokens, heads, width] for the keys or the values of one layer, or [pages, heads, tokens, width], and their
scales the same without the width. Tables (int32): table [n_seqs, columns], -1 where no page is; length [n_seqs] tokens.
"""

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
LARGEST = {"e4m3": 448.0, "i8": 127.0}  # the largest code


# --------------------------------------------------------------------------------------------- cases
def _write(name, seqs, ctx, take, page, heads, width, src, type, heads_first):
    return {"name": name, "op": "write", "seqs": seqs, "ctx": ctx, "take": take, "page": page, "heads": heads, "width": width,
            "src": src, "type": type, "heads_first": heads_first}


def _read(name, seqs, tokens, whole, page, heads, width, type, dst, heads_first):
    return {"name": name, "op": "read", "seqs": seqs, "tokens": tokens, "whole": whole, "page": page, "heads": heads,
            "width": width, "type": type, "dst": dst, "heads_first": heads_first}


def _attend(name, seqs, ctx, nodes, tree, page, heads, group, width, type, q, heads_first):
    return {"name": name, "op": "attend", "seqs": seqs, "ctx": ctx, "nodes": nodes, "tree": tree, "page": page, "heads": heads,
            "group": group, "width": width, "type": type, "q": q, "heads_first": heads_first}


def _verify(name, seqs, nodes, tree, vocab, type, draft):
    return {"name": name, "op": "verify", "seqs": seqs, "nodes": nodes, "tree": tree, "vocab": vocab, "type": type, "draft": draft}


def _keep(name, seqs, ctx, nodes, page, planes, heads, width, type, heads_first):
    return {"name": name, "op": "keep", "seqs": seqs, "ctx": ctx, "nodes": nodes, "page": page, "planes": planes, "heads": heads,
            "width": width, "type": type, "heads_first": heads_first}


def listed():
    return [
        # A speculative step of a small decode batch: 1 to 5 new tokens for each sequence, one layer.
        _write("write_step_48", 48, 1500, 5, 16, 8, 128, "bf16", "e4m3", False),
        # Prompts of about 3,000 tokens enter an 8-bit cache, one layer.
        _write("write_prompts_64", 64, 0, 3001, 16, 8, 128, "bf16", "e4m3", False),
        # The end of a prefix comes back for a check: 8 sequences, a 16-bit cache.
        _read("read_tails_8", 8, 700, False, 16, 8, 128, "bf16", "bf16", False),
        # Long contexts leave the odd 8-bit layout (heads outermost, rows of 112 codes) for 16 bits, to be computed on elsewhere.
        _read("read_long_16", 16, 24011, True, 48, 5, 112, "i8", "f16", True),
        # The smallest step: a few short sequences, trees of up to 8 drafted tokens.
        _attend("attend_few_4", 4, 200, 8, True, 16, 8, 4, 128, "bf16", "bf16", False),
        # The speculative step of 48 sequences: trees of 25 tokens, queries in groups of 4 to a key head.
        _attend("attend_trees_48", 48, 3000, 25, True, 16, 8, 4, 128, "bf16", "bf16", False),
        # 64 long contexts of about 80,000 tokens in an 8-bit cache, one new token each.
        _attend("attend_long_64", 64, 80003, 1, False, 16, 2, 8, 128, "e4m3", "bf16", False),
        # Large trees over the odd 8-bit layout: products, not bytes, are most of this one.
        _attend("attend_wide_16", 16, 8192, 61, True, 48, 5, 8, 112, "i8", "f16", True),
        # Chains of 4 drafted tokens from a drafter without probabilities, 16-bit rows.
        _verify("verify_chains_48", 48, 5, False, 32000, "bf16", False),
        # Trees of 25 for a large batch, with the drafter's probabilities; rows of an odd length.
        _verify("verify_trees_256", 256, 25, True, 50001, "f32", True),
        # The accepted paths of the step of 48, in a small model's 8 planes.
        _keep("keep_paths_48", 48, 300, 25, 16, 8, 8, 128, "bf16", False),
        # The same for a large batch and 48 planes of the odd 8-bit layout.
        _keep("keep_paths_256", 256, 200, 25, 48, 48, 5, 112, "i8", True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "attend", "verify", "keep"))
    page, heads, width = rng.choice((8, 16, 16, 32, 48, 64, 128)), rng.choice((1, 2, 4, 5, 8)), rng.choice((64, 80, 96, 112, 128, 128, 192, 256))
    type, first = rng.choice(("bf16", "f16", "e4m3", "e4m3", "i8")), rng.random() < 0.4
    if op == "write":
        seqs = _log(rng, 1, 512)
        take = rng.choice((1, rng.randint(2, 8), _log(rng, 16, max(16, 190000 // seqs))))
        take = min(take, max(1, 190000 * 1024 // (seqs * heads * width)))
        return _write("", seqs, _log(rng, 1, 2000) if seqs < 200 else 64, take, page, heads, width, rng.choice(("bf16", "f16", "f32")), type, first)
    if op == "read":
        seqs = _log(rng, 1, 128)
        tokens = _log(rng, 1, max(2, min(30000, 380000 * 560 // (seqs * heads * width))))
        return _read("", seqs, tokens, rng.random() < 0.5, page, heads, width, type, rng.choice(("bf16", "f16", "f32")), first)
    if op == "attend":
        group, q = rng.choice((1, 2, 4, 8, 7)), type if type in ("bf16", "f16") else rng.choice(("bf16", "f16"))
        nodes = rng.choice((1, rng.randint(2, 8), rng.randint(9, 64)))
        seqs = _log(rng, 1, 128)
        # at most as many bytes as the longest contexts, and as many products as the widest trees
        most = min(5000000 * 256 // (seqs * heads * width), 130000 * 112 * 40 * 61 // (seqs * heads * group * nodes * width))
        return _attend("", seqs, _log(rng, 1, max(2, min(80003, most))), nodes, rng.random() < 0.8, page, heads, group, width, type, q, first)
    if op == "verify":
        seqs, nodes, vocab = _log(rng, 1, 256), rng.randint(1, 32), _log(rng, 500, 50001)
        return _verify("", seqs, nodes, rng.random() < 0.6, vocab, rng.choice(("bf16", "f16", "f32")), rng.random() < 0.5)
    seqs, nodes = _log(rng, 1, 256), rng.randint(2, 48)
    planes = min(_log(rng, 1, 48), max(1, 256 * 200 * 48 * 560 // (seqs * 128 * heads * width * 2)))
    return _keep("", seqs, _log(rng, 1, 128), nodes, page, planes, heads, width, type, first)


# -------------------------------------------------------------------------------------------- inputs
def _around(rng, n, about):
    return rng.integers((about + 1) // 2, about + about // 2 + 1, n)


def _parents(rng, n, tree):
    """A tree of n nodes, each after its parent, node 0 the root; the ones of a chain follow each other."""
    j = np.arange(n)
    return np.where(j == 0, -1, rng.integers(np.maximum(0, j - 9), np.maximum(j, 1))) if tree else j - 1


def _ancestors(parent):
    """[n, n] of truth values: the nodes on the way from the root to each one, itself included."""
    sees = np.eye(len(parent), dtype=bool)
    for j in range(1, len(parent)):
        sees[j] |= sees[parent[j]]
    return sees


def _sizes(case):
    """(rows, length, first token read) of each request: ragged, and the same for every seed, as outputs have one shape."""
    rng, op, n = np.random.default_rng(78), case["op"], case["seqs"]
    if op == "write":
        rows = rng.integers(1, case["take"] + 1, n) if case["take"] <= 16 else _around(rng, n, case["take"])
        return rows, rows + (_around(rng, n, case["ctx"]) if case["ctx"] else 0), 0 * rows
    if op == "read":
        length = np.maximum(1, _around(rng, n, case["tokens"]))
        first = np.zeros(n, np.int64) if case["whole"] else rng.integers(0, length)
        return length - first, length, first
    rows = rng.integers((case["nodes"] + 1) // 2, case["nodes"] + 1, n)
    return rows, rows + (_around(rng, n, case["ctx"]) if "ctx" in case else 0), 0 * rows


def _host(case, seed):
    """The case's tables, batch and trees as numpy arrays."""
    rng = np.random.default_rng([int(seed), 78])
    op, n = case["op"], case["seqs"]
    h = {}
    order = rng.permutation(n)
    rows, length, first = (x[order] for x in _sizes(case))
    if op == "read":
        h["first"] = first
    elif op != "write":
        trees = [_parents(rng, m, case["tree"] if "tree" in case else True) for m in rows]
        h["parent"] = np.concatenate(trees)
    seq = rng.permutation(n)  # the batch is in an order of its own
    h["seq"], h["start"] = seq, np.concatenate([[0], np.cumsum(rows)])
    if op == "attend" and case["tree"]:
        words = -(-case["nodes"] // 32)
        bits = np.zeros((len(h["parent"]), words * 32), np.uint64)
        for i, t in enumerate(trees):
            bits[h["start"][i] : h["start"][i + 1], : len(t)] = _ancestors(t)
        h["mask"] = (bits.reshape(-1, words, 32) << np.arange(32, dtype=np.uint64)).sum(2).astype(np.uint32).view(np.int32)
    if op == "keep":
        h["path"], h["accepted"] = np.full(len(h["parent"]), -1), np.zeros(n, np.int64)
        for i, t in enumerate(trees):  # the way from the root to some node
            way = np.flatnonzero(_ancestors(t)[rng.integers(0, len(t))])
            h["path"][h["start"][i] : h["start"][i] + len(way)] = way
            h["accepted"][i] = len(way)
    if op != "verify":
        page = case["page"]
        per = np.zeros(n, np.int64)
        per[seq] = -(-length // page)
        columns = int(per.max()) + n % 4
        total = int(per.sum())
        pages = total + total // 8 + 3
        table = np.full((n, columns), -1, np.int64)
        table[np.arange(columns) < per[:, None]] = rng.permutation(pages)[:total]
        h["table"], h["length"], h["refs"] = table, np.zeros(n, np.int64), np.zeros(pages, np.int64)
        h["length"][seq] = length
        h["refs"][table[table >= 0]] = 1
    return {k: np.ascontiguousarray(v, dtype=np.int32) for k, v in h.items()}


def _normal(shape, type, g, std=1.0):
    """Normal values; codes of 8 bits as a quantised row of them has."""
    x = torch.empty(shape, dtype=torch.float16 if type in LARGEST else TYPES[type], device="cuda").normal_(0, 1, generator=g)
    if type in LARGEST:
        x = x.mul_(LARGEST[type] / 3.2).clamp_(-LARGEST[type], LARGEST[type])
        return x.round_().to(torch.int8) if type == "i8" else x.to(TYPES[type])
    return x.mul_(std)


def _probabilities(rows, vocab, type, g):
    """(the target's, the drafter's) rows of probabilities."""
    logits = torch.empty((rows, vocab), device="cuda").normal_(0, 2.5, generator=g)
    p = torch.softmax(logits, 1).to(TYPES[type])
    logits += torch.empty_like(logits).normal_(0, 0.7, generator=g)
    return p, torch.softmax(logits, 1).to(TYPES[type])


def prepare(case, seed):
    s = {"case": case, "op": case["op"]}
    h = _host(case, seed)
    for k, v in h.items():
        s[k] = torch.from_numpy(v).cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 11 + 5)
    op, rows, n = s["op"], int(h["start"][-1]), case["seqs"]
    s["status"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    if op == "verify":
        p, q = _probabilities(rows, case["vocab"], case["type"], g)
        by = (q if case["draft"] else p).float()
        first = torch.repeat_interleave(s["start"][:-1], s["start"].diff())
        above = first + s["parent"].clamp(min=0)  # the row that a node's token is drawn from
        noise = torch.empty_like(by).exponential_(generator=g)
        s["token"] = (by[above] / noise).argmax(1).int()
        s["p"], s["q"] = p, q if case["draft"] else None
        s["u"] = torch.rand(rows, generator=g, device="cuda")
        s["path"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        s["accepted"], s["next"] = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
        return s
    page, heads, width, type = case["page"], case["heads"], case["width"], case["type"]
    s["page"], s["token_dim"], pages = page, 2 if case["heads_first"] else 1, len(h["refs"])
    inner = (heads, page) if case["heads_first"] else (page, heads)
    if op == "keep":
        # [pages, planes, ...] in memory, so that a page is one range of the heap
        s["pool"] = _normal((pages, case["planes"]) + inner + (width,), type, g).transpose(0, 1)
        s["cut"] = torch.zeros((n, 2), dtype=torch.int32, device="cuda")
    else:
        s["k_pool"], s["v_pool"] = (_normal((pages,) + inner + (width,), type, g) for _ in range(2))
        s["k_scale"] = s["v_scale"] = None
        if type in LARGEST:
            s["k_scale"], s["v_scale"] = (torch.empty((pages,) + inner, device="cuda").uniform_(2.5, 4, generator=g) / LARGEST[type] for _ in range(2))
    if op == "write":
        new = torch.empty((rows, 3 * heads, width), dtype=TYPES[case["src"]], device="cuda").normal_(generator=g)
        s["k"], s["v"] = new[:, heads : 2 * heads], new[:, 2 * heads :]  # parts of a joint projection
    elif op == "read":
        s["k"], s["v"] = (torch.zeros((rows, heads, width), dtype=TYPES[case["dst"]], device="cuda") for _ in range(2))
    elif op == "attend":
        s["q"] = _normal((rows, heads * case["group"], width), case["q"], g, 2.0)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(s["q"].shape[:2], device="cuda")
        s["scale"] = width**-0.5
        s.setdefault("mask", None)
    if own:
        import descriptor_build_gb300 as db

        free = torch.zeros((pages + 31) // 32, dtype=torch.int32, device="cuda")  # these calls take no pages
        s["tables"] = db.PageTables(s["table"], s["length"], s["refs"], free, page)
        if op == "attend":
            s["ws"] = db.workspace(db.cache_attention_workspace_size(n, heads * case["group"], heads, width, case["nodes"]))
    return s


# --------------------------------------------------------------------------------------- plain forms
def _requests(s):
    """(request of each row, its first row, its number of rows)."""
    count = s["start"].diff().long()
    i = torch.repeat_interleave(torch.arange(count.numel(), device=count.device), count)
    return i, s["start"].long()[i], count[i]


def _at(s, seq, position):
    """(page, slot) of a sequence's position."""
    return s["table"][seq, position // s["page"]].long(), position % s["page"]


def _slots(pool, token_dim, page, slot):
    """The rows [..., heads, width] (scales: [..., heads]) of a pool [pages, ...]."""
    return pool[page, slot] if token_dim == 1 else pool[page, :, slot]


def _bytes(x):
    return x.view(torch.int8) if x.element_size() == 1 else x


def plain_write(s):
    i, first, count = _requests(s)
    seq = s["seq"].long()[i]
    position = s["length"].long()[seq] - count + torch.arange(i.numel(), device=i.device) - first
    page, slot = _at(s, seq, position)
    at = (page, slot) if s["token_dim"] == 1 else (page, slice(None), slot)
    type = s["case"]["type"]
    for new, pool, scale in ((s["k"], s["k_pool"], s["k_scale"]), (s["v"], s["v_pool"], s["v_scale"])):
        x = new.float()
        if type in LARGEST:
            top = x.abs().amax(-1)
            full = torch.full_like(top, LARGEST[type])  # a tensor: by a number it would be a product with its reciprocal
            scale[at] = top / full
            x = (x * (full / top)[..., None]).clamp(-LARGEST[type], LARGEST[type])
            x = x.round() if type == "i8" else x
        _bytes(pool)[at] = _bytes(x.to(TYPES[type]))
    s["status"].zero_()


def plain_read(s):
    i, first, count = _requests(s)
    seq = s["seq"].long()[i]
    page, slot = _at(s, seq, s["first"].long()[i] + torch.arange(i.numel(), device=i.device) - first)
    for out, pool, scale in ((s["k"], s["k_pool"], s["k_scale"]), (s["v"], s["v_pool"], s["v_scale"])):
        x = _slots(_bytes(pool), s["token_dim"], page, slot).view(pool.dtype).float()
        if scale is not None:
            x = x * _slots(scale, s["token_dim"], page, slot)[..., None]
        out.copy_(x)
    s["status"].zero_()


def _held(s, pool, scale, seq, most):
    """A batch's keys or values in 32 bits, [n, heads, most tokens, width]."""
    page = s["page"]
    rows = s["table"][seq, : -(-most // page)].long().clamp(min=0)
    x = _bytes(pool)[rows].view(pool.dtype).float()
    if scale is not None:
        x = x * scale[rows][..., None]
    x = x.permute(0, 3, 1, 2, 4) if s["token_dim"] == 1 else x.permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])[:, :, :most]


def plain_attend(s):
    case, q, n = s["case"], s["q"], s["seq"].numel()
    heads, group, width, nodes = case["heads"], case["group"], case["width"], case["nodes"]
    most = s["table"].shape[1] * s["page"]
    i, first, count = _requests(s)
    seq = s["seq"].long()
    node = torch.arange(i.numel(), device=i.device) - first
    # queries of a request side by side, those that it lacks see the first token and are not read
    rows = torch.zeros((n, nodes, heads * group, width), device=q.device)
    rows[i, node] = q.float()
    rows = rows.reshape(n, nodes, heads, group, width).permute(0, 2, 1, 3, 4).reshape(n, heads, nodes * group, width)
    length = s["length"].long()[seq]
    position = torch.arange(most, device=q.device)
    of = position - (length - s["start"].diff())[:, None]  # a position's node, negative before them
    if s["mask"] is None:
        sees = of[i] <= node[:, None]
    else:
        word = s["mask"].long().gather(1, (of[i].clamp(0, nodes - 1) // 32))
        sees = (of[i] < 0) | (((word >> (of[i].clamp(min=0) % 32)) & 1) != 0) & (of[i] < nodes)
    sees &= position < length[i][:, None]
    visible = (position < 1).expand(n, nodes, most).clone()
    visible[i, node] = sees
    visible = visible[:, None, :, None].expand(n, heads, nodes, group, most).reshape(n, heads, nodes * group, most)
    scores = (rows * s["scale"]) @ _held(s, s["k_pool"], s["k_scale"], seq, most).transpose(2, 3)
    scores.masked_fill_(~visible, -torch.inf)
    del visible
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == -torch.inf, 0, top)
    weights = scores.sub_(top).exp_()
    total = weights.sum(3, keepdim=True)
    # values of places that no row sees count as zeros, whatever they hold
    v = _held(s, s["v_pool"], s["v_scale"], seq, most).masked_fill_(~(position < length[:, None])[:, None, :, None], 0)
    out = (weights @ v) / torch.where(total == 0, 1, total)
    lse = total.log() + top
    back = lambda x: x.reshape(n, heads, nodes, group, -1).permute(0, 2, 1, 3, 4).reshape(n, nodes, heads * group, -1)[i, node]  # noqa: E731
    s["out"].copy_(back(out))
    s["lse"].copy_(back(lse)[..., 0])
    s["status"].zero_()


def plain_verify(s):
    n, p, q = s["seq"].numel(), s["p"], s["q"]
    start, count, parent, token, u = s["start"].long(), s["start"].diff().long(), s["parent"].long(), s["token"].long(), s["u"].double()
    dev, all_ = p.device, torch.arange(n, device=p.device)
    here = torch.zeros(n, dtype=torch.int64, device=dev)  # the node that a request has come to
    accepted = torch.ones_like(here)
    path = torch.full((n, s["case"]["nodes"]), -1, dtype=torch.int64, device=dev)
    path[:, 0] = 0
    left = p[start[:-1]].double()  # what is left of the target's probabilities there
    total = torch.ones(n, dtype=torch.float64, device=dev)
    for j in range(1, s["case"]["nodes"]):
        row = (start[:-1] + j).clamp(max=p.shape[0] - 1)
        child = (j < count) & (parent[row] == here)
        t = token[row]
        by = q[start[:-1] + here].double() if q is not None else None
        against = u[row] * total * (by[all_, t] if q is not None else 1)
        yes = child & (against < left[all_, t])
        no = child & ~yes
        path[all_, torch.where(yes, accepted, 0)] = torch.where(yes, j, 0)
        accepted += yes
        here = torch.where(yes, j, here)
        if q is not None:
            less = (left / torch.where(total > 0, total, 1)[:, None] - by).clamp(min=0)
            now = less.sum(1)
        else:
            less = left.clone()
            less[all_, t] = 0
            now = total - left[all_, t]
        left = torch.where(yes[:, None], p[start[:-1] + here].double(), torch.where(no[:, None], less, left))
        total = torch.where(yes, 1, torch.where(no, now, total))
    left = torch.where((left.sum(1) > 0)[:, None], left, p[start[:-1] + here].double())
    upto = left.cumsum(1)
    s["next"].copy_((upto > (u[start[:-1]] * upto[:, -1])[:, None]).int().argmax(1))
    s["accepted"].copy_(accepted)
    i, first, _ = _requests(s)
    s["path"].copy_(path[i, torch.arange(i.numel(), device=dev) - first])
    s["status"].zero_()


def plain_keep(s):
    i, first, count = _requests(s)
    k = torch.arange(i.numel(), device=i.device) - first
    base = (s["length"].long()[s["seq"].long()] - s["start"].diff())[i]
    seq, kept = s["seq"].long()[i], k < s["accepted"][i]
    here = torch.where(kept, s["path"].long(), k)  # what is not accepted stays where it is
    (a, b), (c, d) = _at(s, seq, base + here), _at(s, seq, base + k)
    pool = _bytes(s["pool"])
    if s["token_dim"] == 1:
        pool[:, c, d] = torch.where(kept[:, None, None], pool[:, a, b], pool[:, c, d])
    else:
        pool[:, c, :, d] = torch.where(kept[:, None, None, None], pool[:, a, :, b], pool[:, c, :, d])
    cut = torch.stack([s["seq"].long(), s["length"].long()[s["seq"].long()] - s["start"].diff() + s["accepted"]], 1)
    s["cut"].copy_(cut)
    s["status"].zero_()


# ----------------------------------------------------------------------------------------- the calls
def own_calls(s):
    import descriptor_build_gb300 as db

    op = s["op"]
    if op == "write":
        db.cache_write(s["tables"], s["seq"], s["start"], s["k"], s["v"], s["k_pool"], s["v_pool"], k_scale=s["k_scale"],
                       v_scale=s["v_scale"], token_dim=s["token_dim"], status=s["status"])
    elif op == "read":
        db.cache_read(s["tables"], s["seq"], s["start"], s["k"], s["v"], s["k_pool"], s["v_pool"], k_scale=s["k_scale"],
                      v_scale=s["v_scale"], first=s["first"], token_dim=s["token_dim"], status=s["status"])
    elif op == "attend":
        db.cache_attention(s["tables"], s["seq"], s["start"], s["q"], s["k_pool"], s["v_pool"], s["out"], s["ws"],
                           max_tokens=s["case"]["nodes"], scale=s["scale"], mask=s["mask"], lse=s["lse"], k_scale=s["k_scale"],
                           v_scale=s["v_scale"], token_dim=s["token_dim"], status=s["status"])
    elif op == "verify":
        db.draft_verify(s["start"], s["parent"], s["token"], s["p"], s["u"], s["path"], s["accepted"], s["next"], q=s["q"],
                        status=s["status"])
    else:
        db.cache_keep(s["tables"], s["seq"], s["start"], s["path"], s["accepted"], s["pool"], token_dim=s["token_dim"] + 1,
                      cut=s["cut"], status=s["status"])


PLAIN = {"write": plain_write, "read": plain_read, "attend": plain_attend, "verify": plain_verify, "keep": plain_keep}
OUTPUTS = {"write": ("k_pool", "v_pool", "k_scale", "v_scale"), "read": ("k", "v"), "attend": ("out", "lse"),
           "verify": ("path", "accepted", "next"), "keep": ("pool", "cut")}


def run(s):
    if own:
        own_calls(s)
    else:
        PLAIN[s["op"]](s)
    return {k: s[k] for k in OUTPUTS[s["op"]] + ("status",)}


def work(case):
    """Bytes and operations of one pass: what is written and read, once; the products of the visible part of the cache."""
    op, (rows, length, _) = case["op"], _sizes(case)
    size = lambda t: TYPES[t].itemsize  # noqa: E731
    if op == "verify":
        return {"bytes": int(case["seqs"] * (case["vocab"] * size(case["type"]) * (2 if case["draft"] else 1) + 16) + rows.sum() * 24), "flops": 0}
    heads, width = case["heads"], case["width"]
    held = heads * (width * size(case["type"]) + (4 if case["type"] in LARGEST else 0))  # a token's keys or values in the cache
    if op in ("write", "read"):
        return {"bytes": int(2 * rows.sum() * (heads * width * size(case["src" if op == "write" else "dst"]) + held)), "flops": 0}
    if op == "keep":
        h = _host(case, 0)
        place = np.arange(len(h["path"])) - np.repeat(h["start"][:-1], np.diff(h["start"]))
        moved = int(((h["path"] >= 0) & (h["path"] != place)).sum())
        return {"bytes": 2 * moved * case["planes"] * heads * width * size(case["type"]) + 4 * len(place) + 20 * case["seqs"], "flops": 0}
    queries = rows * heads * case["group"]
    return {"bytes": int(2 * length.sum() * held + queries.sum() * (2 * width * size(case["q"]) + 4)),
            "flops": int((4 * queries * (length - rows / 2) * width).sum())}


# --------------------------------------------------------------------------------------------- exact
def _rows_of(h, i):
    return range(h["start"][i], h["start"][i + 1])


def _tokens(case, h, seq, first, count):
    """(page, slot) of a sequence's tokens, one after the other."""
    at = np.arange(first, first + count)
    return torch.from_numpy(h["table"][seq, at // case["page"]].astype(np.int64)).cuda(), torch.from_numpy(at % case["page"]).cuda()


def _exact_values(case, s, h, i, part, first, count):
    """Keys or values of request i's tokens in 64 bits, [count, heads, width]."""
    page, slot = _tokens(case, h, h["seq"][i], first, count)
    pool, scale = s[part + "_pool"], s[part + "_scale"]
    raw = pool.view(torch.int8) if pool.element_size() == 1 else pool
    got = (raw[page, :, slot] if case["heads_first"] else raw[page, slot]).view(pool.dtype).double()
    if scale is not None:
        got *= (scale[page, :, slot] if case["heads_first"] else scale[page, slot]).double()[..., None]
    return got


def _exact_write(case, s, h):
    out = {}
    for part in ("k", "v"):
        pool, scale = s[part + "_pool"].double(), s[part + "_scale"]
        scale = scale.double() if scale is not None else None
        for i in range(case["seqs"]):
            rows, seq = _rows_of(h, i), h["seq"][i]
            page, slot = _tokens(case, h, seq, h["length"][seq] - len(rows), len(rows))
            x = s[part][rows.start : rows.stop].double()
            if scale is not None:
                top = x.abs().amax(-1, keepdim=True)
                x = x * LARGEST[case["type"]] / top
                x = x.round() if case["type"] == "i8" else x.float().to(torch.float8_e4m3fn).double()
                if case["heads_first"]:
                    scale[page, :, slot] = top[..., 0] / LARGEST[case["type"]]
                else:
                    scale[page, slot] = top[..., 0] / LARGEST[case["type"]]
            if case["heads_first"]:
                pool[page, :, slot] = x
            else:
                pool[page, slot] = x
        out[part + "_pool"], out[part + "_scale"] = None if case["type"] == "i8" else pool, scale
    return out


def _exact_attend(case, s, h):
    out, lse = torch.zeros_like(s["q"], dtype=torch.float64), torch.zeros_like(s["lse"], dtype=torch.float64)
    group = case["group"]
    for i in range(case["seqs"]):
        rows, seq = _rows_of(h, i), h["seq"][i]
        length, m = int(h["length"][seq]), len(rows)
        sees = np.ones((m, length), bool)
        sees[:, length - m :] = _ancestors(h["parent"][rows.start : rows.stop])
        hidden = torch.from_numpy(~sees).cuda()
        k, v = (_exact_values(case, s, h, i, part, 0, length) for part in ("k", "v"))
        for head in range(case["heads"]):
            q = s["q"][rows.start : rows.stop, head * group : (head + 1) * group].double()
            scores = (q @ k[:, head].T) * s["scale"]
            scores.masked_fill_(hidden[:, None], -torch.inf)
            norm = torch.logsumexp(scores, 2)
            out[rows.start : rows.stop, head * group : (head + 1) * group] = torch.exp(scores - norm[..., None]) @ v[:, head]
            lse[rows.start : rows.stop, head * group : (head + 1) * group] = norm
    return {"out": out, "lse": lse}


def _exact_verify(case, s, h):
    path, accepted, following = np.full(len(h["parent"]), -1), [], []
    u, token = s["u"].double().cpu().numpy(), s["token"].cpu().numpy()
    row = lambda x, r: x[r].double().cpu().numpy()  # noqa: E731
    for i in range(case["seqs"]):
        a, m = h["start"][i], len(_rows_of(h, i))
        here, way = 0, [0]
        p = target = row(s["p"], a)
        total = 1.0
        for j in range(1, m):
            if h["parent"][a + j] != here:
                continue
            t = token[a + j]
            q = row(s["q"], a + here) if case["draft"] else (np.arange(case["vocab"]) == t) * 1.0
            if u[a + j] * q[t] * total < p[t]:
                here, total = j, 1.0
                way.append(j)
                p = target = row(s["p"], a + j)
            elif case["draft"]:
                p = np.maximum(p / total - q, 0)
                total = p.sum()
            else:
                total -= p[t]
                p = p * (q == 0)
        p = p if p.sum() > 0 else target
        upto = np.cumsum(p)
        path[a : a + len(way)] = way
        accepted.append(len(way))
        following.append(int(np.searchsorted(upto, u[a] * upto[-1], side="right")))
    return {"path": path, "accepted": np.array(accepted), "next": np.array(following)}


def _exact_keep(case, s, h):
    pool = (s["pool"].view(torch.int8) if case["type"] in LARGEST else s["pool"]).clone()
    cut = []
    for i in range(case["seqs"]):
        rows, seq, a = _rows_of(h, i), h["seq"][i], h["accepted"][i]
        base = int(h["length"][seq]) - len(rows)
        to, at = _tokens(case, h, seq, base, a)
        page, slot = _tokens(case, h, seq, base, len(rows))
        way = torch.from_numpy(h["path"][rows.start : rows.start + a].astype(np.int64)).cuda()
        if case["heads_first"]:
            pool[:, to, :, at] = pool[:, page[way], :, slot[way]]
        else:
            pool[:, to, at] = pool[:, page[way], slot[way]]
        cut.append([seq, base + a])
    return {"pool": pool.view(s["pool"].dtype).double() if case["type"] != "i8" else pool, "cut": np.array(cut)}


def exact(case, seed):
    s, h = prepare(case, seed), _host(case, seed)
    if case["op"] == "read":
        parts = {part: torch.cat([_exact_values(case, s, h, i, part, int(h["first"][i]), len(_rows_of(h, i))) for i in range(case["seqs"])])
                 for part in ("k", "v")}
        return parts | {"status": None}
    made = {"write": _exact_write, "attend": _exact_attend, "verify": _exact_verify, "keep": _exact_keep}[case["op"]](case, s, h)
    return made | {"status": np.zeros(case["seqs"], np.int64)}
