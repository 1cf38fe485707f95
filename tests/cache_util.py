"""Caches, batches and trees for the tests of what a paged cache's pages hold."""

import numpy as np

from gpu_util import lib

try:
    import torch
except ImportError:  # pragma: no cover
    torch = None

NAMES = {} if torch is None else {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
                                  "e4m3": torch.float8_e4m3fn, "i8": torch.int8}


class Tables:
    """Sequences of the given lengths with pages all over a pool, one page and one column more than they need."""

    def __init__(self, rng, lengths, page, spare_seqs=1):
        self.T = page
        lengths = list(lengths) + [0] * spare_seqs
        per = [-(-n // page) for n in lengths]
        self.n_pages = sum(per) + 1
        self.table = np.full((len(lengths), max(per) + 1), -1, np.int32)
        order, at = rng.permutation(self.n_pages), 0
        for i, n in enumerate(per):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.length = np.array(lengths, np.int32)

    def device(self):
        db = lib()
        t = lambda a: torch.from_numpy(a.copy()).cuda()
        refs = torch.ones(self.n_pages, dtype=torch.int32, device="cuda")
        free = torch.zeros((self.n_pages + 31) // 32, dtype=torch.int32, device="cuda")
        return db.PageTables(t(self.table), t(self.length), refs, free, self.T)


def numbers(t):
    """A pool's values as float64: 8-bit codes stand for themselves."""
    return t.detach().cpu().double().numpy() if t.dtype != torch.float8_e4m3fn else t.detach().cpu().float().double().numpy()


def raw(t):
    """A tensor's bits as integers of its own size."""
    size = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]
    return t.detach().cpu().view(size).numpy()


def tokens_first(x, token_dim):
    """A pool [pages, ...] as [pages, tokens, heads, ...] (a view)."""
    return x if token_dim == 1 else x.transpose(0, 2, 1, *range(3, x.ndim))


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def tree(rng, m, back=5):
    """Parents of a random tree of m nodes and its ancestors' mask [m, m]."""
    parent = np.array([-1] + [int(rng.integers(max(0, j - back), j)) for j in range(1, m)], np.int64)[:m]
    sees = np.eye(m, dtype=bool)
    for j in range(1, m):
        sees[j] |= sees[parent[j]]
    return parent, sees


def words(bits, n_words):
    """Rows of truth values as 32-bit words."""
    out = np.zeros((len(bits), n_words), np.uint32)
    for j, row in enumerate(bits):
        for b in np.flatnonzero(row):
            out[j, b // 32] |= np.uint32(1 << (b % 32))
    return out


def finish():
    torch.cuda.synchronize()
