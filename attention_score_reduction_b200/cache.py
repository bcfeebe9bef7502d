"""The paged K/V cache of a compressed context: filled with the kept rows, grown
by new tokens, attended over (include/kvzip.h, "paged cache").

``kvzip.compact`` leaves each head's kept rows packed end to end, which no new
row can join.  ``PagedCache`` holds them in pages instead, as bf16 or quantised
to 8 or 4 bits as they are written:

    cache = PagedCache.allocate("int4", units, d, n_pages, page_rows, max_pages)
    cache.reserve(rows)                     # pages for each unit (host numbers)
    cache.write(out.k, out.v, offsets=out.offsets)   # the kept rows of a Compressed
    cache.write(k_new, v_new)               # a chunk's rows, appended
    o = cache.attend(q)                     # attention of that chunk, or of one token

A unit is one KV head of one sequence, so a layer of a batch has sequences *
heads units and each keeps its own number of rows.
"""
from __future__ import annotations

import contextlib

import torch

from . import kvzip as kz


# the current stream's handle without the Stream object around it (1.2 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class PagedCache:
    """Pools, page table and lengths of one layer's cache, on one GPU.

    The tensors given are used as they are (they may be views of a serving
    engine's pool) and kept alive; ``status`` is a zeroed int32 word.  Calls run
    on the current stream or on ``stream``, which has to wait for whatever made
    their inputs; those may be dropped right after the call.
    """

    def __init__(self, fmt: str, k_pages, v_pages, k_params, v_params, page_table, lens,
                 status=None):
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=lens.device)
        self.fmt, self.k_pages, self.v_pages = fmt, k_pages, v_pages
        self.k_params, self.v_params = k_params, v_params
        self.page_table, self.lens, self.status = page_table, lens, status
        self._c = kz.cache_struct(fmt, k_pages, v_pages, k_params, v_params, page_table, lens,
                                  status)
        self.device = k_pages.device
        self._index = self.device.index
        self.units, self.d = int(self._c.units), int(self._c.d)
        self.page_rows, self.n_pages = int(self._c.page_rows), int(self._c.n_pages)
        self.max_pages = int(self._c.max_pages)
        self._free = None      # host page lists, for caches made by allocate()
        self._owned = None
        self._ws_sizes = {}

    @classmethod
    def allocate(cls, fmt: str, units: int, d: int, n_pages: int, page_rows: int = 64,
                 max_pages: int | None = None, device="cuda") -> "PagedCache":
        """An empty cache with its own pool; ``reserve`` hands out its pages."""
        if fmt not in kz.CACHE_FORMATS:
            raise ValueError(f"cache format must be one of {sorted(kz.CACHE_FORMATS)}, got {fmt!r}")
        max_pages = max_pages or n_pages
        dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
        width = d if fmt == "bf16" else kz.cache_row_bytes(fmt, d)
        pool = lambda: torch.zeros(n_pages, page_rows, width, dtype=dt, device=device)  # noqa: E731
        par = lambda: (None if fmt == "bf16" else  # noqa: E731
                       torch.zeros(n_pages, page_rows, dtype=torch.int32, device=device))
        table = torch.full((units, max_pages), -1, dtype=torch.int32, device=device)
        lens = torch.zeros(units, dtype=torch.int32, device=device)
        c = cls(fmt, pool(), pool(), par(), par(), table, lens)
        c._free = list(range(n_pages - 1, -1, -1))
        c._owned = [0] * units
        return c

    # ------------------------------------------------------------ pages

    def reserve(self, rows):
        """Give every unit pages for at least ``rows`` rows in all: an int, or a
        host sequence of one number per unit.  Pages a unit has stay its own.  The
        table changes on the current stream."""
        if self._free is None:
            raise ValueError("reserve() needs a cache made by PagedCache.allocate")
        rows = [int(rows)] * self.units if isinstance(rows, int) else [int(r) for r in rows]
        if len(rows) != self.units:
            raise ValueError("one number of rows per unit")
        need = [max(0, -(-r // self.page_rows) - have) for r, have in zip(rows, self._owned)]
        if any(n + have > self.max_pages for n, have in zip(need, self._owned)):
            raise ValueError("a unit would need more than max_pages pages")
        if sum(need) > len(self._free):
            raise ValueError(f"the pool has {len(self._free)} free pages, {sum(need)} are needed")
        if not any(need):
            return
        us, js, ps = [], [], []
        for u, n in enumerate(need):
            for j in range(self._owned[u], self._owned[u] + n):
                us.append(u)
                js.append(j)
                ps.append(self._free.pop())
            self._owned[u] += n
        at = torch.tensor([us, js], dtype=torch.int64).to(self.device)
        self.page_table[at[0], at[1]] = torch.tensor(ps, dtype=torch.int32).to(self.device)

    def clear(self):
        """Drop every row; pages go back to the pool."""
        self.lens.zero_()
        if self._free is not None:
            self.page_table.fill_(-1)
            self._free = list(range(self.n_pages - 1, -1, -1))
            self._owned = [0] * self.units

    # ------------------------------------------------------------ calls

    @contextlib.contextmanager
    def _on(self, stream):
        """The cache's device and the call's stream current, so that what the
        call allocates belongs to the stream that uses it."""
        with torch.cuda.device(self.device):
            if stream is None:
                yield torch.cuda.current_stream(self.device).cuda_stream
            else:
                with torch.cuda.stream(stream):
                    yield stream.cuda_stream

    def _run(self, stream, call, *args):
        """call(*args, raw stream) on the cache's device and the given stream.  The
        usual case, both current already, costs no context switches: a decoding
        step's calls are short enough for the host's time to show."""
        if stream is None and torch.cuda.current_device() == self._index:
            return call(*args, _raw_stream(self._index))
        with self._on(stream) as st:
            if stream is not None:
                # the caller may drop what it gave before that stream has used it
                held = (self.k_pages, self.v_pages, self.k_params, self.v_params, self.page_table,
                        self.lens, self.status)
                for t in (*args, *held):
                    if isinstance(t, torch.Tensor) and t.is_cuda:
                        t.record_stream(stream)
            return call(*args, st)

    def _aux(self, name, t, dtype, n):
        if t is None:
            return
        if t.dtype is dtype and t.device == self.device and t.shape == (n,) and t.is_contiguous():
            return
        kz._dev_contig(name, t, dtype)
        raise ValueError(f"{name} must hold {n} numbers on {self.device}")

    def _rows(self, name, t, dims):
        if t.dtype is not torch.bfloat16:
            raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}")
        shape = t.shape
        if len(shape) != dims or shape[-1] != self.d or (t.stride(-1) != 1 and t.numel()):
            raise ValueError(f"{name} must have {dims} dimensions, the last of {self.d} "
                             "contiguous elements")
        return shape

    def write(self, k, v, starts=None, counts=None, offsets=None, stream=None):
        """Rows into the cache, at positions ``starts`` (int32 [units]; None:
        after the rows held); lengths move on to the end of what was written.

        Dense: k, v [units][n][d] bf16 (d contiguous, rows on 16-byte boundaries), of which unit
        u brings ``counts[u]`` rows (int32 [units]; None: n).  Packed, with
        ``offsets`` (int64 [units + 1]): k, v [rows][d], unit u's at
        offsets[u]:offsets[u + 1].
        """
        dims = 2 if offsets is not None else 3
        shape = self._rows("k", k, dims)
        if self._rows("v", v, dims) != shape:
            raise ValueError("k and v must have the same shape")
        if dims == 3 and shape[0] != self.units:
            raise ValueError("k and v must hold every unit")
        if offsets is not None and counts is not None:
            raise ValueError("counts go with dense rows, offsets with packed ones")
        self._aux("starts", starts, torch.int32, self.units)
        self._aux("counts", counts, torch.int32, self.units)
        self._aux("offsets", offsets, torch.int64, self.units + 1)
        ks, vs = k.stride(), v.stride()
        ks, vs = ((0, ks[0]), (0, vs[0])) if dims == 2 else (ks[:2], vs[:2])
        self._run(stream, kz.cache_write, self._c, k, v, shape[-2], ks, vs, starts, counts, offsets)

    def read(self, offsets=None, n_rows: int | None = None, starts=None, k_out=None, v_out=None,
             stream=None):
        """Rows back as bf16 from positions ``starts`` (None: 0).  Packed, with
        ``offsets`` (int64 [units + 1]) and n_rows = offsets[-1]: k, v [n_rows][d]
        as ``kvzip.decode_attention`` takes them.  Dense: [units][n_rows][d].
        Rows a unit does not hold are left as they were (outputs made here: zeros
        where dense, unspecified where packed).
        """
        if n_rows is None:
            raise ValueError("n_rows is needed: rows per unit, or with offsets of all units")
        self._aux("starts", starts, torch.int32, self.units)
        self._aux("offsets", offsets, torch.int64, self.units + 1)
        shape = (n_rows, self.d) if offsets is not None else (self.units, n_rows, self.d)
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            if t is not None:
                kz._dev_contig(name, t, torch.bfloat16)
                if t.shape != shape or t.device != self.device:
                    raise ValueError(f"{name} must be {shape} on {self.device}")
        return self._run(stream, self._read, shape, n_rows, starts, offsets, k_out, v_out)

    def _read(self, shape, n_rows, starts, offsets, k_out, v_out, st):
        make = torch.zeros if offsets is None else torch.empty
        if k_out is None:
            k_out = make(shape, dtype=torch.bfloat16, device=self.device)
        if v_out is None:
            v_out = make(shape, dtype=torch.bfloat16, device=self.device)
        kz.cache_read(self._c, k_out, v_out, n_rows, starts, offsets, st)
        return k_out, v_out

    def attend(self, q, q_lens=None, out=None, scale: float = 0.0, out_dtype=torch.bfloat16,
               stream=None):
        """Causal attention of each unit's newest tokens over its rows (their own
        K and V written before): q [units][G][n_q][d] bf16 (d contiguous, rows on
        16-byte boundaries), ``q_lens`` (int32 [units]) of the n_q tokens are a unit's own.
        Returns out [units][G][n_q][d] bf16 or float32; rows past q_lens[u] are
        left as they were (fresh outputs: zeros).
        """
        shape = self._rows("q", q, 4)
        if shape[0] != self.units:
            raise ValueError("q must hold every unit")
        self._aux("q_lens", q_lens, torch.int32, self.units)
        if out is not None:
            if out.shape != shape or out.device != self.device or (
                    out.dtype not in (torch.bfloat16, torch.float32)):
                raise ValueError(f"out must be bf16 or float32 {tuple(shape)} on {self.device}")
            if not out.is_contiguous() and not _rows_apart(out):
                raise ValueError("out's last dimension must be contiguous and its rows apart")
        return self._run(stream, self._attend, q, q_lens, out, out_dtype, scale)

    def _attend(self, q, q_lens, out, out_dtype, scale, st):
        if out is None:
            make = torch.empty if q_lens is None else torch.zeros
            out = make(q.shape, dtype=out_dtype, device=self.device)
        key = (q.shape[1], q.shape[2])
        n = self._ws_sizes.get(key)
        if n is None:
            n = self._ws_sizes[key] = max(
                kz.cache_attention_workspace_size(self._c, *key), 256)
        # scratch of this call alone: two captured graphs never share it
        ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        kz.cache_attention(self._c, q, out, ws, q_lens, scale, st)
        return out

    def check_status(self, stream=None):
        """Synchronise; raise if a call since the last check met a length, count,
        offset or page id out of range, or a kernel gave up waiting."""
        s = self._run(stream, kz.workspace_status, self.status)
        if s != kz.OK:
            raise kz.KvzipError(s, "paged cache")


def _rows_apart(t) -> bool:
    """Whether the rows along the last (contiguous) dimension never overlap."""
    if t.stride(-1) != 1:
        return False
    end = t.shape[-1]
    for st, n in sorted(zip(t.stride()[:-1], t.shape[:-1])):
        if n > 1:
            if st < end:
                return False
            end = st * (n - 1) + end
    return True
