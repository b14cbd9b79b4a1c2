"""A paged cache for serving: sequences that grow, share pages, are cut back and
leave, over the paged entry points of ``ops``.

:class:`Pages` keeps the books (which page holds which tokens of which sequence,
and who shares it) without touching a device; :class:`PagedCache` owns the pools
of every layer and carries the books' decisions out with ``ops.page_copy``,
``ops.rope``, ``ops.paged_append`` and ``ops.paged_attn``.
"""
from __future__ import annotations

import dataclasses

import torch

from . import ops


class OutOfPages(RuntimeError):
    """The pool has too few free pages; nothing has changed."""


class Pages:
    """Page lists of sequences over a pool of ``num_pages`` pages of ``page_size``
    tokens.  A page may belong to several sequences; only a page of a single one is
    ever written.  Methods that need page contents moved return (source,
    destination) pairs; sources and destinations never meet."""

    def __init__(self, num_pages: int, page_size: int):
        if num_pages < 1 or page_size < 1:
            raise ValueError("num_pages and page_size must be positive")
        self.num_pages, self.page_size = num_pages, page_size
        self._free = list(range(num_pages - 1, -1, -1))
        self._owners = [0] * num_pages
        self._pages: dict[int, list] = {}
        self._length: dict[int, int] = {}
        self._next = 0

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def length(self, seq: int) -> int:
        return self._length[seq]

    def pages(self, seq: int) -> tuple:
        return tuple(self._pages[seq])

    def sequences(self) -> tuple:
        return tuple(self._pages)

    def new(self) -> int:
        """An empty sequence."""
        seq, self._next = self._next, self._next + 1
        self._pages[seq], self._length[seq] = [], 0
        return seq

    def _take(self) -> int:
        page = self._free.pop()
        self._owners[page] = 1
        return page

    def _drop(self, page: int):
        self._owners[page] -= 1
        if self._owners[page] == 0:
            self._free.append(page)

    def extend(self, counts: dict) -> list:
        """Room for ``counts[seq]`` more tokens of each sequence.  A shared page that
        would be written is replaced by a copy."""
        need, copied = 0, {}
        for seq, n in counts.items():
            if n < 0:
                raise ValueError("a sequence grows by a number of tokens of at least 0")
            length, pages = self._length[seq], self._pages[seq]
            need += max(0, -(-(length + n) // self.page_size) - len(pages))
            at = length // self.page_size
            if n and at < len(pages):
                copied[seq] = pages[at]
        # of a page's owners that write now, all copy it but one if nobody else holds it
        writers: dict = {}
        for seq, page in copied.items():
            writers.setdefault(page, []).append(seq)
        moves = []
        for page, seqs in writers.items():
            moves += seqs[1:] if self._owners[page] == len(seqs) else seqs
        need += len(moves)
        if need > len(self._free):
            raise OutOfPages(f"{need} pages needed, {len(self._free)} free")
        copies = []
        for seq in moves:
            at = self._length[seq] // self.page_size
            old, page = self._pages[seq][at], self._take()
            self._pages[seq][at] = page
            self._drop(old)
            copies.append((old, page))
        for seq, n in counts.items():
            self._length[seq] += n
            while len(self._pages[seq]) * self.page_size < self._length[seq]:
                self._pages[seq].append(self._take())
        return copies

    def undo_extend(self, counts: dict, copies: list):
        """Takes back the last :meth:`extend`, which returned ``copies``."""
        for seq in reversed(counts):
            pages = self._pages[seq]
            self._length[seq] -= counts[seq]
            while len(pages) * self.page_size >= self._length[seq] + self.page_size:
                self._drop(pages.pop())
        where = {}  # of each copy, whose it is
        for seq in counts:
            at = self._length[seq] // self.page_size
            if at < len(self._pages[seq]):
                where[self._pages[seq][at]] = seq, at
        for old, page in reversed(copies):
            seq, at = where[page]
            self._pages[seq][at] = old
            self._owners[old] += 1
            self._drop(page)

    def fork(self, seq: int) -> int:
        """Another sequence with the same tokens, sharing every page; the first of
        them to write the last, partly filled one gets a copy then."""
        new = self.new()
        self._pages[new], self._length[new] = list(self._pages[seq]), self._length[seq]
        for page in self._pages[new]:
            self._owners[page] += 1
        return new

    def truncate(self, seq: int, length: int):
        """Keeps the first ``length`` tokens (a rejected speculation, an edit)."""
        if not 0 <= length <= self._length[seq]:
            raise ValueError(f"length must lie in [0, {self._length[seq]}]")
        keep = -(-length // self.page_size)
        for page in self._pages[seq][keep:]:
            self._drop(page)
        del self._pages[seq][keep:]
        self._length[seq] = length

    def free(self, seq: int):
        self.truncate(seq, 0)
        del self._pages[seq], self._length[seq]

    def compaction(self) -> list:
        """What :meth:`compact` will move, into pages that are free until then."""
        live = self.num_pages - len(self._free)
        holes = sorted(p for p in self._free if p < live)
        high = sorted(p for p in range(live, self.num_pages) if self._owners[p])
        return list(zip(high, holes))

    def compact(self) -> list:
        """Moves live pages to the lowest numbers; afterwards the live pages are
        0 .. live - 1."""
        live = self.num_pages - len(self._free)
        where = dict(self.compaction())
        for pages in self._pages.values():
            pages[:] = [where.get(p, p) for p in pages]
        for src, dst in where.items():
            self._owners[dst], self._owners[src] = self._owners[src], 0
        self._free = list(range(self.num_pages - 1, live - 1, -1))
        return list(where.items())


@dataclasses.dataclass
class Batch:
    """The new tokens of one step: what the calls of every layer share."""
    seqs: tuple
    page_table: torch.Tensor   # [seqs, max_pages] int32
    cu_new: torch.Tensor       # [seqs + 1] int32
    cache_lens: torch.Tensor   # [seqs] int32
    positions: torch.Tensor    # [total] int32
    max_new: int
    total: int


class PagedCache:
    """Keys, values and pooled keys of ``layers`` layers in pages.

    A step: ``batch = cache.extend({seq: new_tokens, ...})``, then for each layer
    ``cache.attend(layer, batch, q, k, v, topk)`` with the packed new tokens'
    q [total, Hq, D] and k, v [total, Hkv, D] bf16 in the order of ``batch.seqs``.
    Calls are enqueued on the current stream; one stream at a time."""

    def __init__(self, layers: int, num_pages: int, Hkv: int, D: int, page_size: int = 64,
                 block_size: int = 512, device="cuda", pooling=ops.POOL_MEAN):
        if block_size % page_size:
            raise ValueError("block_size must be a multiple of page_size")
        self.books = Pages(num_pages, page_size)
        self.block_size, self.pooling = block_size, pooling
        shape = (layers, num_pages, Hkv)
        # (zeros, not what the memory held: a cache is inspected and saved whole)
        self.k_pages = torch.zeros(*shape, page_size, D, dtype=torch.bfloat16, device=device)
        self.v_pages = torch.zeros_like(self.k_pages)
        self.kbar_pages = torch.zeros(*shape, D, dtype=torch.float32, device=device)

    @property
    def device(self):
        return self.k_pages.device

    def _ints(self, x):
        return torch.tensor(x, dtype=torch.int32).to(self.device)

    def _move(self, pairs):
        for i in range(0, len(pairs), 65536):  # (what one call takes)
            src, dst = zip(*pairs[i:i + 65536])
            ops.page_copy(self.k_pages, self.v_pages, self.kbar_pages, self._ints(src), self._ints(dst))

    def new(self) -> int:
        return self.books.new()

    def fork(self, seq: int) -> int:
        return self.books.fork(seq)

    def truncate(self, seq: int, length: int):
        self.books.truncate(seq, length)

    def free(self, seq: int):
        self.books.free(seq)

    def compact(self) -> int:
        """Moves the live pages to the front of the pools; how many moved.  A
        batch made before names the old pages: finish its step first."""
        pairs = self.books.compaction()
        self._move(pairs)
        self.books.compact()  # (a copy that fails changes nothing)
        return len(pairs)

    def extend(self, counts: dict) -> Batch:
        """Room for ``counts[seq]`` new tokens of each sequence, and the tables of the
        step that writes and attends them.  A call that fails changes nothing
        (:class:`OutOfPages`, or what copying shared pages or making the tables raises)."""
        if not counts:
            raise ValueError("a step needs a sequence")
        copies = self.books.extend(counts)
        try:
            self._move(copies)
            return self._batch(counts)
        except BaseException:  # (pages that were copied to are free again)
            self.books.undo_extend(counts, copies)
            raise

    def _batch(self, counts: dict) -> Batch:
        seqs = tuple(counts)
        cu, positions, lens, rows = [0], [], [], []
        for seq in seqs:
            n = self.books.length(seq)
            cu.append(cu[-1] + counts[seq])
            lens.append(n)
            positions.extend(range(n - counts[seq], n))
            rows.append(list(self.books.pages(seq)))
        width = max(1, max(len(r) for r in rows))
        table = [r + [-1] * (width - len(r)) for r in rows]
        return Batch(seqs, self._ints(table), self._ints(cu), self._ints(lens), self._ints(positions),
                     max(1, max(counts.values())), cu[-1])

    def attend(self, layer: int, batch: Batch, q, k, v, topk: int, freqs=None,
               interleaved: bool = False, magnitude: float = 1.0, stream=None, **kw):
        """One layer of a step: q and k rotated to the tokens' positions (with
        ``freqs``, see ``ops.rope_frequencies``), k and v appended, and the attention
        -> (out, lse, idx) of ``ops.paged_attn`` (further arguments go to it), all on
        ``stream`` (None: the current one)."""
        if freqs is not None:
            q, k = ops.rope(q, k, batch.positions, freqs, interleaved, magnitude, stream=stream)
        pools = self.k_pages[layer], self.v_pages[layer], self.kbar_pages[layer]
        ops.paged_append(k, v, *pools, batch.page_table, batch.cu_new, batch.cache_lens,
                         batch.max_new, self.block_size, pooling=self.pooling, stream=stream)
        return ops.paged_attn(q, *pools, batch.page_table, batch.cu_new, batch.cache_lens,
                              batch.max_new, self.block_size, topk, stream=stream, **kw)
