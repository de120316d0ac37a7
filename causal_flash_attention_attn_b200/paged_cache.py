"""The books of a paged KV cache: which pages each sequence holds, how many sequences share a
page, which are free. Bookkeeping is host work on plain integers; the pages themselves move
through the library's kernels (paged_append, paged_copy, attention_decode_paged)."""
from __future__ import annotations

import heapq
from array import array


class PagedCache:
    """Pools of `num_pages` pages for `num_layers` layers, and the sequences in them.

        cache = PagedCache(num_pages=512, num_kv_heads=8, head_dim=128, num_layers=2)
        a = cache.new()
        starts = cache.extend([a], [100])             # room for 100 tokens; positions to append at
        for layer in range(2):
            cache.append(layer, k[layer], v[layer], [a], starts, cu_seqlens)
        b = cache.fork(a)                             # shares a's pages
        ...
        starts = cache.extend([a, b], [1, 1])         # a step: one token each
        now = cache.tables([a, b])                    # once, for all layers
        for layer in range(2):
            cache.append(layer, k[layer], v[layer], [a, b], starts, tables=now)
            o, lse = cache.decode(layer, q[layer], [a, b], tables=now)

    A page is shared by the forks of a sequence until one of them writes into it: extend() then
    gives that sequence a copy (its last, partly filled page only, in every layer). free() and compact()
    return pages and close the gaps. Page tables are built on the host; tables() sends them to the
    device, and append() and decode() do it themselves where they are given none. No call waits for the
    device.

    k_pages, v_pages: [num_layers, num_pages, num_kv_heads, page_size, head_dim]; they may be given
    (pages=(k, v)) instead of being allocated.
    """

    def __init__(self, num_pages, num_kv_heads, head_dim, page_size=64, num_layers=1, dtype=None, device="cuda",
                 pages=None):
        if min(num_pages, num_kv_heads, head_dim, page_size, num_layers) < 1:
            raise ValueError("PagedCache: every size must be at least 1")
        if page_size % 16:
            raise ValueError(f"PagedCache: page_size must be a multiple of 16, got {page_size}")
        import torch
        shape = (num_layers, num_pages, num_kv_heads, page_size, head_dim)
        if pages is None:
            dtype = torch.bfloat16 if dtype is None else dtype
            self._check_kind(torch.device(device), dtype, head_dim)
            pages = tuple(torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        k, v = pages
        for t in (k, v):
            if tuple(t.shape) != shape:
                raise ValueError(f"PagedCache: pages of shape {tuple(t.shape)}, expected {shape}")
            # (strides of dimensions of size 1 do not matter)
            if any(n > 1 and s != w for n, s, w in zip(shape[2:], t.stride()[2:], (page_size * head_dim, head_dim, 1))):
                raise ValueError(f"PagedCache: pages must be contiguous (strides {t.stride()})")
        if (k.dtype, k.device) != (v.dtype, v.device) or (dtype is not None and k.dtype != dtype):
            raise ValueError(f"PagedCache: pages of {k.dtype} on {k.device} and {v.dtype} on {v.device}"
                             f"{'' if dtype is None else f', expected {dtype}'}")
        if k.stride() != v.stride():
            raise ValueError(f"PagedCache: pages with strides {k.stride()} and {v.stride()}, expected the same")
        self._check_kind(k.device, k.dtype, head_dim)
        self.k_pages, self.v_pages = k, v
        self.num_pages, self.page_size, self.num_layers = num_pages, page_size, num_layers
        self._free = list(range(num_pages))   # a heap: the lowest page first
        self._refs = [0] * num_pages
        self._pages = {}                      # sequence -> its pages in order
        self._lens = {}                       # sequence -> tokens
        self._next = 0

    @staticmethod
    def _check_kind(device, dtype, head_dim):
        """What the library's calls take: found out here, and not when a shared page is to be copied."""
        import torch
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"PagedCache: unsupported dtype {dtype}")
        if device.type == "cuda" and head_dim not in (64, 128, 256):
            raise ValueError(f"PagedCache: head_dim must be 64, 128 or 256, got {head_dim}")

    # ------------------------------------------------------------------ the books
    @property
    def free_pages(self):
        return len(self._free)

    def length(self, seq):
        return self._lens[seq]

    def pages(self, seq):
        return list(self._pages[seq])

    def new(self):
        """A new, empty sequence's handle."""
        seq = self._next
        self._next += 1
        self._pages[seq], self._lens[seq] = [], 0
        return seq

    def fork(self, seq):
        """A new sequence with the same tokens. Shares seq's pages; nothing is copied yet."""
        pages, length = list(self._pages[seq]), self._lens[seq]
        new = self.new()
        self._pages[new], self._lens[new] = pages, length
        for p in self._pages[new]:
            self._refs[p] += 1
        return new

    def free(self, seq):
        """Forget a sequence; pages that no other sequence holds become free."""
        for p in self._pages.pop(seq):
            self._drop(p)
        del self._lens[seq]

    def _drop(self, page):
        self._refs[page] -= 1
        if self._refs[page] == 0:
            heapq.heappush(self._free, page)

    def _take(self):
        page = heapq.heappop(self._free)
        self._refs[page] = 1
        return page

    def extend(self, seqs, counts, stream=None):
        """Make room for counts[i] more tokens of seqs[i] (each sequence once). A partly filled last page
        that is shared is copied first, in every layer. Returns the old lengths: the positions to append
        at. All or nothing: MemoryError if the free pages do not suffice, and if a copy fails the books stay
        as they were."""
        seqs, counts = list(seqs), list(counts)
        if len(seqs) != len(counts) or len(set(seqs)) != len(seqs):
            raise ValueError("PagedCache.extend: one count for each sequence, each sequence once")
        if any(n < 0 for n in counts):
            raise ValueError("PagedCache.extend: a negative count")
        ps = self.page_size
        need, shared, refs = 0, [], {}
        for s, n in zip(seqs, counts):
            held = self._lens[s]
            need += -(-(held + n) // ps) - len(self._pages[s])
            if n and held % ps:
                # the last sequence left on a page writes into it as it is
                last = self._pages[s][-1]
                if refs.setdefault(last, self._refs[last]) > 1:
                    refs[last] -= 1
                    shared.append(s)
        if need + len(shared) > len(self._free):
            raise MemoryError(f"PagedCache: {need + len(shared)} pages needed, {len(self._free)} free")
        # the copies come first: they write free pages only, and may fail
        copies = [heapq.heappop(self._free) for _ in shared]
        try:
            self._copy([(self._pages[s][-1], page) for s, page in zip(shared, copies)], stream)
        except BaseException:
            for page in copies:
                heapq.heappush(self._free, page)
            raise
        for s, page in zip(shared, copies):
            old, self._pages[s][-1], self._refs[page] = self._pages[s][-1], page, 1
            self._drop(old)
        starts = []
        for s, n in zip(seqs, counts):
            starts.append(self._lens[s])
            self._lens[s] += n
            while len(self._pages[s]) * ps < self._lens[s]:
                self._pages[s].append(self._take())
        return starts

    def compact(self, stream=None):
        """Move pages down until the held ones are 0 .. n - 1, in every layer. Returns the moves
        [(from, to), ..]; tables made before are stale after it."""
        held = sorted(p for p in range(self.num_pages) if self._refs[p])
        holes = [p for p in range(len(held)) if not self._refs[p]]
        moves = list(zip(reversed(held[len(held) - len(holes):]), holes)) if holes else []
        to = dict(moves)
        self._copy(moves, stream)  # into free pages: if it fails, the books stay as they were
        for old, new in moves:
            self._refs[new], self._refs[old] = self._refs[old], 0
        for s, pages in self._pages.items():
            self._pages[s] = [to.get(p, p) for p in pages]
        self._free = list(range(len(held), self.num_pages))
        return moves

    def _copy(self, moves, stream):
        if moves:
            from . import paged_copy
            paged_copy(self.k_pages, self.v_pages, [a for a, _ in moves], [b for _, b in moves], stream=stream)

    # ------------------------------------------------------------------ on the device
    def tables(self, seqs, stream=None):
        """(page_table int32 [len(seqs), width], seq_lens int32 [len(seqs)]) on the pools' device, for append()
        and decode() of every layer. Valid until the books change (extend, fork, free, compact). They are made on
        `stream` (the current one), for calls on that stream."""
        seqs = list(seqs)
        rows, width = self._rows(seqs)
        rows.extend(self._lens[s] for s in seqs)
        with self._on(stream):
            t = self._send(rows)
        return t[:len(seqs) * width].view(len(seqs), width), t[len(seqs) * width:]

    def _rows(self, seqs):
        """The page table's rows one after the other, and their width."""
        width = max([1] + [len(self._pages[s]) for s in seqs])
        rows = array("i")
        for s in seqs:
            pages = self._pages[s]
            rows.extend(pages)
            rows.extend([0] * (width - len(pages)))
        return rows, width

    def _send(self, ints):
        """An array of ints as an int32 tensor on the pools' device: through pinned memory, so that
        the host does not wait for the stream. (torch gives the pinned block away again only when the
        copy is done.)"""
        import torch
        device = self.k_pages.device
        host = torch.frombuffer(ints, dtype=torch.int32) if len(ints) else torch.empty(0, dtype=torch.int32)
        if device.type != "cuda":
            return host.clone()
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("PagedCache: a graph that is captured would send this moment's tables for ever: build them "
                               "before, with tables(), and give them to append() and decode()")
        return torch.empty(len(ints), dtype=torch.int32, pin_memory=True).copy_(host).to(device, non_blocking=True)

    def _on(self, stream):
        """The scope in which a call's tables are made: they belong to the stream that reads them, or
        the memory could be given away before the call has run."""
        from . import _NOTHING, _scope
        return _NOTHING if stream is None else _scope(self.k_pages.device, stream)

    @staticmethod
    def _given(what, seqs, tables):
        if seqs is not None and len(seqs) != tables[0].shape[0]:
            raise ValueError(f"PagedCache.{what}: tables of {tables[0].shape[0]} sequences for {len(seqs)}")
        return tables

    def append(self, layer, k, v, seqs, starts, cu_seqlens=None, stream=None, tables=None):
        """Write new tokens of one layer at the positions that extend() returned (paged_append). tables: what
        tables(seqs) returned, so that nothing is built and sent again for another layer (seqs may be None
        then). starts: a list, or an int32 tensor on the pools' device, which is taken as it is."""
        import torch
        from . import paged_append
        ready = isinstance(starts, torch.Tensor) and starts.device == self.k_pages.device and starts.dtype == torch.int32
        with self._on(stream):
            if tables is not None:
                table = self._given("append", seqs, tables)[0]
                starts = starts if ready else self._send(array("i", starts))
            else:
                seqs = list(seqs)
                rows, width = self._rows(seqs)
                at = len(rows)
                if not ready:
                    rows.extend(starts)
                t = self._send(rows)
                table, starts = t[:at].view(len(seqs), width), starts if ready else t[at:]
        paged_append(k, v, self.k_pages[layer], self.v_pages[layer], table, starts, cu_seqlens, stream)

    def decode(self, layer, q, seqs, stream=None, tables=None, **options):
        """attention_decode_paged of one new query per sequence; tables as in append(); options: scale, window,
        softcap, sink."""
        from . import attention_decode_paged
        table, lens = self.tables(seqs, stream) if tables is None else self._given("decode", seqs, tables)
        return attention_decode_paged(q, self.k_pages[layer], self.v_pages[layer], table, lens, stream=stream, **options)
