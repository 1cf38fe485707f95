"""A paged cache in the device heap, from prompts to descriptors.

Sequences of a small model are admitted, forked into beams, extended token by
token and cut back, all on the device; the pool is compacted; then one
sequence is written to an NVMe drive (PRP lists for its pages) and another is
put to a peer (work-queue entries for its pages). Run on a GPU:

    python examples/paged_cache.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import descriptor_build_gb300 as db  # noqa: E402

# A page holds 16 tokens of every layer: 4 layers x (keys, values) x 16 tokens
# x 4 heads x 32 values of 16 bits = 32 KiB, half a 64 KiB granule of the heap.
LAYERS, TOKENS, HEADS, WIDTH = 4, 16, 4, 32
PLANES = 2 * LAYERS
PAGES, SEQS, COLUMNS = 1024, 64, 40
PAGE_BYTES = PLANES * TOKENS * HEADS * WIDTH * 2


class Cache:
    """The tables, the pool and what the calls need, allocated once."""

    def __init__(self, device="cuda"):
        self.tables = db.PageTables.empty(SEQS, COLUMNS, PAGES, TOKENS, device)
        # [pages, planes, ...] in memory, so that a page is one range of the heap
        self.heap = torch.zeros((PAGES, PLANES, TOKENS, HEADS, WIDTH), dtype=torch.bfloat16, device=device)
        self.pool = self.heap.transpose(0, 1)
        self.ws = db.workspace(db.page_workspace_size(SEQS, PAGES), device)
        self.moves = torch.zeros((PAGES, 4), dtype=torch.int32, device=device)
        self.n_moves = torch.zeros(1, dtype=torch.int32, device=device)
        self.ctr = torch.zeros(4, dtype=torch.int64, device=device)
        self.device = device

    def _req(self, rows):
        return torch.tensor(rows, dtype=torch.int32, device=self.device)

    def extend(self, rows):
        """[[sequence, tokens], ...]: room for the tokens, shared pages copied first."""
        db.page_extend(self.tables, self._req(rows), self.moves, self.n_moves, self.ws, ctr=self.ctr)
        db.page_copy(self.moves, self.n_moves, self.pool, self.pool, token_dim=2)

    def fork(self, rows):
        """[[parent, child, tokens, 0], ...]"""
        db.page_fork(self.tables, self._req(rows), self.ws)

    def free(self, rows):
        """[[sequence, tokens kept], ...]"""
        db.page_free(self.tables, self._req(rows), self.ws)

    def compact(self):
        db.page_compact(self.tables, self.tables, self.moves, self.n_moves, self.ws)
        db.page_copy(self.moves, self.n_moves, self.pool, self.pool)

    def write(self, seq, first, values):
        """The model's part: keys and values [planes, tokens, heads, width] of tokens from `first` on."""
        at = torch.arange(first, first + values.shape[1], device=self.device)
        page = self.tables.table[seq, at // TOKENS].long()
        self.heap[page, :, at % TOKENS] = values.transpose(0, 1)

    def read(self, seq):
        """What the model's attention reads: [planes, length, heads, width]."""
        n = int(self.tables.length[seq])
        at = torch.arange(n, device=self.device)
        return self.heap[self.tables.table[seq, at // TOKENS].long(), :, at % TOKENS].transpose(0, 1)

    def ranges(self, seq):
        """The heap ranges {offset, bytes} of a sequence's pages, neighbours merged."""
        n = -(-int(self.tables.length[seq]) // TOKENS)
        page = self.tables.table[seq, :n].long()
        new = torch.ones(n, dtype=torch.bool, device=self.device)
        new[1:] = page[1:] != page[:-1] + 1
        run = new.cumsum(0) - 1
        count = torch.bincount(run)
        return torch.stack([page[new] * PAGE_BYTES, count * PAGE_BYTES], 1)


def main():
    torch.manual_seed(0)
    c = Cache()
    values = lambda n: torch.randn((PLANES, n, HEADS, WIDTH), device="cuda").bfloat16()
    kept = {}  # what each sequence must read back as

    def grow(rows):
        c.extend(rows)
        for seq, n in rows:
            v = values(n)
            have = kept.get(seq)
            c.write(seq, 0 if have is None else have.shape[1], v)
            kept[seq] = v if have is None else torch.cat([have, v], 1)

    # eight prompts, each decoded by four beams for twenty steps
    grow([[s, 37 + 29 * s] for s in range(8)])
    beams = [(8 + 4 * s + k, s) for s in range(8) for k in range(4)]
    c.fork([[s, b, kept[s].shape[1], 0] for b, s in beams])
    for b, s in beams:
        kept[b] = kept[s].clone()
    for step in range(20):
        grow([[b, 1] for b, _ in beams])
        if step % 5 == 4:  # the worst beam of each four is dropped for a fork of the best
            c.free([[8 + 4 * s + 3, 0] for s in range(8)])
            c.fork([[8 + 4 * s, 8 + 4 * s + 3, kept[8 + 4 * s].shape[1], 0] for s in range(8)])
            for s in range(8):
                kept[8 + 4 * s + 3] = kept[8 + 4 * s].clone()
    # prompts and losing beams end; two rejected tokens are taken back from a winner
    over = list(range(8)) + [b for b, _ in beams if b % 4]
    c.free([[s, 0] for s in over] + [[8, kept[8].shape[1] - 2]])
    for s in over:
        del kept[s]
    kept[8] = kept[8][:, :-2]
    before = {s: c.ranges(s).shape[0] for s in kept}
    used = int((c.tables.refs > 0).sum())
    c.compact()
    top = int(c.tables.table.max()) + 1
    same = all(torch.equal(c.read(s), v) for s, v in kept.items())
    print(f"{used} pages in use, highest page {top - 1} after compaction; contents "
          f"{'as written' if same else 'DIFFER'}")

    # sequence 12 goes to a drive: PRP lists for its ranges of the heap
    heap_size = PAGES * PAGE_BYTES
    lut = (torch.randperm(1 << 20, device="cuda")[: heap_size >> 16] + 1) << 16
    req = c.ranges(12)
    prp = torch.zeros((req.shape[0], 2), dtype=torch.int64, device="cuda")
    arena = torch.zeros((64, 512), dtype=torch.int64, device="cuda")
    ctr = torch.zeros(4, dtype=torch.int64, device="cuda")
    ws = db.workspace(db.prp_workspace_size(req.shape[0]))
    db.prp_build(req, lut, heap_size, 1 << 32, 64, arena, prp, ws, ctr=ctr)
    # sequence 16 goes to peer 1 on queue pair 0
    put = c.ranges(16)
    put[:, 1] |= 1 << 32  # {u32 bytes; u16 pe; u16 qp}
    rings = torch.zeros((2, 64, 64), dtype=torch.uint8, device="cuda")
    head = torch.zeros(2, dtype=torch.int64, device="cuda")
    count = torch.zeros(2, dtype=torch.int32, device="cuda")
    peers = torch.tensor([1 << 40, 1 << 41], device="cuda")
    wws = db.workspace(db.wqe_workspace_size(put.shape[0], 2))
    db.wqe_bucket(put, peers, torch.tensor([7, 8], dtype=torch.int32, device="cuda"), 2, 1, 1 << 30, 3,
                  heap_size, rings, 64, head, count, wws)
    print(f"sequence 12: {req.shape[0]} requests (before compaction {before[12]}), "
          f"{int(ctr[0])} list pages; sequence 16: {int(count[1])} puts (before {before[16]})")
    return same, c, req, prp, lut, put, rings, count


if __name__ == "__main__":
    sys.exit(0 if main()[0] else 1)
