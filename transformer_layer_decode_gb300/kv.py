"""A paged key/value cache of many sequences (the dec_kv_ calls of include/dec.h).

:class:`KVCache` holds the tensors of one cache and marshals the calls: rows
written and read (bf16, 8-bit or 4-bit blocks; keys rotated on the way), attention
of one query per sequence with a sliding window and first rows that stay visible,
and pages allocated, shared, freed and made dense.  Every call is queued on a stream and waits for
nothing; :meth:`KVCache.sync_status` reports what the kernels refused.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import dec

DEC_KV_BF16, DEC_KV_Q4B32, DEC_KV_Q8T16 = 0, 1, 3
DEC_IO_F32, DEC_IO_BF16 = 0, 1
DEC_KV_BAD_INDEX, DEC_KV_NO_PAGES, DEC_KV_BAD_LIST, DEC_KV_BAD_BOUNDS = 1, 2, 4, 8

FORMATS = {"bf16": DEC_KV_BF16, "q4": DEC_KV_Q4B32, "q8": DEC_KV_Q8T16}
_TYPES = {torch.float32: DEC_IO_F32, torch.bfloat16: DEC_IO_BF16}

# what torch.cuda.current_stream(), current_device() and is_current_stream_capturing() ask, without their
# objects: a decode step makes a few short calls per layer, and the host has to keep ahead of them
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_capturing = torch._C._cuda_isCurrentStreamCapturing


class KVCacheDesc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_rows", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("n_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("format", ctypes.c_int32),
                ("pool", ctypes.c_void_p), ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("status", ctypes.c_void_p), ("scratch", ctypes.c_void_p)]


_LARGE = 1 << 31
_PER_THREAD = 2  # the handle that is another stream in every host thread


def _int32(**numbers):
    """Refuses what ctypes would cut off to 32 bits: a window of 2^32 + 5 rows is not one of 5.  (Calls of a
    decode step look themselves first, which takes less than this call.)"""
    for name, x in numbers.items():
        if not -_LARGE <= x < _LARGE:
            raise ValueError(f"{name} {x}: 32 bits are wanted")


def default_page_rows(head_dim: int) -> int:
    """Rows of a page unless asked otherwise: those of one attention chunk of the decoder."""
    return 64 if head_dim == 128 else 128


class KVCache:
    """One cache: a pool of pages for every layer, and the tables of its sequences.

    n_layers, n_kv_heads, head_dim (64 or 128), page_rows (a multiple of 16)
    and fmt ("bf16", "q8" or "q4") fix the shape of a page.  The tensors are made
    empty here from n_pages, n_seqs and max_pages (pages of one sequence), or
    taken as they are: pool uint8 [n_layers, n_pages, page_bytes], table int32
    [n_seqs, max_pages], lens int32 [n_seqs], refs int32 [n_pages].

    The calls are for serving: autograd does not see them, and results have no gradients.

    Host threads may share a cache: a call's launches are queued without another's
    between them.  On the GPU the calls keep the order that include/dec.h asks for.

    The calls of a decode step are marshalled by the module of dec.load_calls() where their arguments are
    plainly right, and here where they are not, or have a stream of their own.
    """

    _context = None  # what that module knows of a cache, if it is there

    def __init__(self, *, n_layers: int, n_kv_heads: int, head_dim: int, page_rows: int | None = None,
                 fmt: str = "bf16", n_pages: int | None = None, n_seqs: int | None = None,
                 max_pages: int | None = None, pool=None, table=None, lens=None, refs=None,
                 device=None, lib_path: str | None = None):
        if fmt not in FORMATS:
            raise ValueError(f"fmt {fmt!r}: one of {sorted(FORMATS)}")
        self.lib = dec.load_library(lib_path or dec.LIB_PATH)
        given = [t for t in (pool, table, lens, refs) if t is not None]
        if given:
            if len(given) != 4:
                raise ValueError("pool, table, lens and refs are given together")
            n_pages, (n_seqs, max_pages) = refs.numel(), table.shape
            device = pool.device
        elif None in (n_pages, n_seqs, max_pages):
            raise ValueError("n_pages, n_seqs and max_pages are needed to make a cache")
        page_rows = default_page_rows(head_dim) if page_rows is None else page_rows
        _int32(n_layers=n_layers, n_kv_heads=n_kv_heads, head_dim=head_dim, page_rows=page_rows, n_pages=n_pages,
               n_seqs=n_seqs, max_pages=max_pages)
        self.desc = KVCacheDesc(n_layers, n_kv_heads, head_dim, page_rows, n_pages, n_seqs, max_pages,
                                FORMATS[fmt])
        self._ref = ctypes.byref(self.desc)
        page_bytes, ints = ctypes.c_size_t(), ctypes.c_size_t()
        self._check(self.lib.dec_kv_sizes(self._ref, ctypes.byref(page_bytes), ctypes.byref(ints)))
        self.page_bytes = page_bytes.value
        if given:
            self._tensor("pool", pool, torch.uint8, (n_layers, n_pages, self.page_bytes), device)
            self._tensor("lens", lens, torch.int32, (n_seqs,), device)
            self._tensor("refs", refs, torch.int32, (n_pages,), device)
            self._tensor("table", table, torch.int32, (n_seqs, max_pages), device)
        else:
            device = torch.device("cuda") if device is None else torch.device(device)
            pool = torch.empty(n_layers, n_pages, self.page_bytes, dtype=torch.uint8, device=device)
            if fmt == "q8":  # (what a block's scale was counts where it is not begun at its first row)
                pool.view(n_layers, n_pages, 2, -1)[..., n_kv_heads * page_rows * head_dim:] = 0
            table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=device)
            lens = torch.zeros(n_seqs, dtype=torch.int32, device=device)
            refs = torch.zeros(n_pages, dtype=torch.int32, device=device)
        if pool.device.type != "cuda":
            raise ValueError("the cache's tensors must be on a CUDA device")
        self.device = pool.device
        self._index, self._d = pool.device.index, head_dim
        self.pool, self.table, self.lens, self.refs = pool, table, lens, refs
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.scratch = torch.empty(ints.value, dtype=torch.int32, device=self.device)
        for name in ("pool", "table", "lens", "refs", "status", "scratch"):
            setattr(self.desc, name, getattr(self, name).data_ptr())
        self._lock = threading.Lock()  # of the launches of a call, which hand a workspace or the scratch on
        self._status_lock = threading.Lock()  # of a reading of the status, which waits for its stream
        self._workspaces: dict = {}  # of a stream's attention calls, which run one after another
        self._captured_workspaces: list = []  # of captures that keep no memory themselves
        self._fast = dec.load_calls()
        if self._fast is not None:
            self._context = self._fast.context(ctypes.addressof(self.desc), self._index, n_kv_heads, head_dim, *(
                dec.address_of(f) for f in (self.lib.dec_kv_append, self.lib.dec_kv_read, self.lib.dec_kv_attention,
                                            self.lib.dec_kv_append_rotated)))

    # ---- marshalling ----------------------------------------------------------

    def _check(self, rc: int):
        if rc != dec.DEC_OK:
            raise dec.DecError(rc, self.lib.dec_last_error(None).decode())

    @staticmethod
    def _tensor(name, t, dtype, shape, device):
        if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or t.device != device:
            raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {shape} on {device} is wanted, "
                             f"not {t.dtype} {tuple(t.shape)} on {t.device}")

    def _ints(self, name, t, n=None):
        """(address, length) of a device int32 list."""
        if t is None:
            return None, n
        if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.device != self.device:
            raise ValueError(f"{name}: a contiguous one-dimensional int32 tensor on {self.device} is wanted")
        if n is not None and t.shape[0] != n:
            raise ValueError(f"{name}: {t.shape[0]} entries for {n}")
        return t.data_ptr(), t.shape[0]

    def _rows(self, name, t, heads=None):
        """(address, type, elements from row to row) of a [n, heads, head_dim] tensor with whole rows."""
        shape, d = t.shape, self._d
        if len(shape) == 3 and shape[2] == d and (heads is None or shape[1] == heads) and t.device == self.device:
            step, type_ = t.stride(), _TYPES.get(t.dtype)
            if type_ is not None and step[2] == 1 and (step[1] == d or shape[1] == 1):
                return t.data_ptr(), type_, step[0] if shape[0] > 1 else shape[1] * d
        raise ValueError(f"{name}: a float32 or bfloat16 tensor [n, {heads or 'heads'}, {d}] on {self.device} "
                         "with contiguous rows is wanted")

    def _captured(self):
        """Whether the current stream of the cache's device is being captured."""
        if _current_device() == self._index:
            return _capturing()
        with torch.cuda.device(self.device):
            return _capturing()

    def _in_private_pool(self, t):
        """Whether t's memory is from a pool that is no one else's, as in a capture of torch.cuda.graph."""
        try:
            segments = torch.cuda.memory_snapshot()
        except RuntimeError:  # an allocator that does not say
            return False
        at = t.data_ptr()
        return any(s["device"] == self._index and s["address"] <= at < s["address"] + s["total_size"]
                   and tuple(s["segment_pool_id"]) != (0, 0) for s in segments)

    def _new(self, make, shape, dtype, stream):
        """make(shape) for a call on `stream`: its memory, and what fills it, belong to that stream."""
        if stream is None:
            return make(shape, dtype=dtype, device=self.device)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.device)
        with torch.cuda.stream(stream):
            return make(shape, dtype=dtype, device=self.device)

    def _call(self, fn, *args, stream=None, lock=None):
        handle = _raw_stream(self._index) if stream is None else \
            stream if isinstance(stream, int) else stream.cuda_stream
        if _current_device() == self._index:
            with lock or self._lock:
                rc = fn(self._ref, *args, handle)
        else:
            with torch.cuda.device(self.device), lock or self._lock:
                rc = fn(self._ref, *args, handle)
        if rc:
            self._check(rc)

    # ---- rows -----------------------------------------------------------------

    def append(self, layer: int, k, v, *, seqs=None, positions=None, stream=None):
        """Writes row t of k and v ([n, n_kv_heads, head_dim], keys already rotated) as row positions[t]
        of sequence seqs[t]; without positions, as the sequence's last row; without seqs, of sequence t.
        8-bit pages: rows of a block of 16 behind the first that is written, and not written, are given up."""
        if stream is None and self._context is not None:
            with self._lock:
                rc = self._fast.append(self._context, layer, k, v, seqs, positions)
            if rc is not None:
                return self._check(rc) if rc else None
        if not 0 <= layer < _LARGE:
            _int32(layer=layer)
        kp, kt, ks = self._rows("k", k, self.desc.n_kv_heads)
        vp, vt, vs = self._rows("v", v, self.desc.n_kv_heads)
        if k.shape[0] != v.shape[0] or kt != vt or ks != vs:
            raise ValueError("k and v: the same type, rows and row stride are wanted")
        n = k.shape[0]
        sp, _ = self._ints("seqs", seqs, n)
        pp, _ = self._ints("positions", positions, n)
        self._call(self.lib.dec_kv_append, layer, kp, vp, kt, ks, sp, pp, n, stream=stream)

    def read(self, layer: int, seqs, positions=None, *, k_out=None, v_out=None, dtype=torch.float32, stream=None):
        """Rows positions[t] of sequences seqs[t] as values: (k, v), each [n, n_kv_heads, head_dim].
        Rows of skipped entries keep what k_out and v_out hold (zeros where these are made here)."""
        if stream is None and self._context is not None and k_out is not None and v_out is not None:
            with self._lock:
                rc = self._fast.read(self._context, layer, k_out, v_out, seqs, positions)
            if rc is not None:
                if rc:
                    self._check(rc)
                return k_out, v_out
        if not 0 <= layer < _LARGE:
            _int32(layer=layer)
        sp, n = self._ints("seqs", seqs)
        pp, _ = self._ints("positions", positions, n)
        shape = (n, self.desc.n_kv_heads, self.desc.head_dim)
        if k_out is None:
            k_out = self._new(torch.zeros, shape, dtype if v_out is None else v_out.dtype, stream)
        if v_out is None:
            v_out = self._new(torch.zeros, shape, k_out.dtype, stream)
        kp, kt, ks = self._rows("k_out", k_out, shape[1])
        vp, vt, vs = self._rows("v_out", v_out, shape[1])
        if k_out.shape[0] != n or v_out.shape[0] != n or kt != vt or ks != vs:
            raise ValueError(f"k_out and v_out: the same type and row stride and {n} rows are wanted")
        self._call(self.lib.dec_kv_read, layer, kp, vp, kt, ks, sp, pp, n, stream=stream)
        return k_out, v_out

    def append_rotated(self, layer: int, rotary, q, k, v, *, seqs=None, positions=None, q_out=None, stream=None):
        """append() of keys that `rotary` (rope.Rotary) has yet to rotate, each by its position, and row t of
        q ([n, n_q_heads, head_dim]; None: no queries) rotated the same way: returns q_out, which may be q.
        Rows of skipped entries keep what q_out holds (zeros where it is made here)."""
        if stream is None and self._context is not None and (q is None) == (q_out is None):
            with self._lock:
                rc = self._fast.append_rotated(self._context, layer, k, v, seqs, positions, rotary._context, q, q_out)
            if rc is not None:
                if rc:
                    self._check(rc)
                return q_out
        if not 0 <= layer < _LARGE:
            _int32(layer=layer)
        if rotary.device != self.device:
            raise ValueError(f"rotary: a rotation on {self.device} is wanted, not on {rotary.device}")
        kp, kt, ks = self._rows("k", k, self.desc.n_kv_heads)
        vp, vt, vs = self._rows("v", v, self.desc.n_kv_heads)
        if k.shape[0] != v.shape[0] or kt != vt or ks != vs:
            raise ValueError("k and v: the same type, rows and row stride are wanted")
        n = k.shape[0]
        qp, op, qs, os_, heads = None, None, 0, 0, 0
        if q is not None:
            qp, qt, qs = self._rows("q", q)
            heads = q.shape[1]
            if q_out is None:
                q_out = self._new(torch.zeros, q.shape, q.dtype, stream)
            op, ot, os_ = self._rows("q_out", q_out, heads)
            if qt != kt or ot != kt or q.shape[0] != n or q_out.shape[0] != n:
                raise ValueError("q and q_out: the type and rows of k are wanted")
        elif q_out is not None:
            raise ValueError("q_out without q")
        sp, _ = self._ints("seqs", seqs, n)
        pp, _ = self._ints("positions", positions, n)
        self._call(self.lib.dec_kv_append_rotated, layer, rotary._ref, qp, op, qs, os_, heads, kp, vp, kt, ks, sp, pp, n,
                   stream=stream)
        return q_out

    # ---- attention ------------------------------------------------------------

    def workspace(self):
        """A workspace for attention calls on this cache: one call at a time may use it."""
        size = ctypes.c_size_t()
        with torch.cuda.device(self.device):
            self._check(self.lib.dec_kv_attention_workspace(self._ref, ctypes.byref(size)))
        return torch.empty(size.value, dtype=torch.uint8, device=self.device)

    def attention(self, layer: int, q, *, seqs=None, window: int = 0, sinks: int = 0, scale: float = 0.0,
                  out=None, workspace=None, stream=None):
        """softmax(scale q K^T) V of one query per entry of seqs over its sequence's visible rows: the last
        `window` ones (0: all) and the first `sinks` ones.  q and out: [n, n_q_heads, head_dim].  Rows of
        skipped entries keep what out holds (zeros where it is made here).  Without a workspace the calls of
        the current stream share one, and a captured call gets its own, which the graph's memory pool keeps or,
        where the capture was not begun by torch.cuda.graph, this cache; `stream` needs one to be given."""
        if not (0 <= layer < _LARGE and 0 <= window < _LARGE and 0 <= sinks < _LARGE):
            _int32(layer=layer, window=window, sinks=sinks)
        if out is not None and stream is None and self._context is not None:
            ws = self._workspace(workspace, None)
            with self._lock:
                rc = self._fast.attention(self._context, layer, q, out, seqs, window, sinks, scale, ws[0], ws[1])
            if rc is not None:
                if rc:
                    self._check(rc)
                return out
        else:
            ws = None
        qp, qt, qs = self._rows("q", q)
        n, heads = q.shape[0], q.shape[1]
        sp, _ = self._ints("seqs", seqs, n)
        if out is None:
            out = self._new(torch.zeros, q.shape, q.dtype, stream)  # (a length out of range skips any of them)
        op, ot, os_ = self._rows("out", out, heads)
        if ot != qt or out.shape[0] != n:
            raise ValueError("out: the type and rows of q are wanted")
        if ws is None:
            ws = self._workspace(workspace, stream)
        self._call(self.lib.dec_kv_attention, layer, qp, op, qt, qs, os_, sp, n, heads, window, sinks, scale,
                   ws[0], ws[1], stream=stream)
        return out

    def _workspace(self, workspace, stream):
        """(address, bytes, what holds it) of an attention call's workspace: the one given, the stream's or the graph's."""
        if workspace is None:
            if stream is not None:
                raise ValueError("a call with a stream of its own needs a workspace of its own")
            if self._captured():  # a graph keeps its own: it may be replayed beside other calls
                workspace = self.workspace()
                if not self._in_private_pool(workspace):
                    self._captured_workspaces.append(workspace)
                return workspace.data_ptr(), workspace.numel(), workspace
            key = _raw_stream(self._index)
            if key == _PER_THREAD:
                key = key, threading.get_ident()
            ws = self._workspaces.get(key)
            if ws is None:
                workspace = self.workspace()
                ws = workspace.data_ptr(), workspace.numel(), workspace
                self._workspaces[key] = ws
            return ws
        if workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace: contiguous memory on {self.device} is wanted")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace

    # ---- pages ----------------------------------------------------------------

    def extend(self, seqs=None, n_new=None, *, stream=None):
        """Makes sequences longer (by n_new[i] rows, or one), with the pages that takes: all or nothing."""
        sp, n = self._ints("seqs", seqs)
        if seqs is None:
            n = self.desc.n_seqs if n_new is None else n_new.shape[0]
        np_, _ = self._ints("n_new", n_new, n)
        self._call(self.lib.dec_kv_extend, sp, np_, n, stream=stream)

    def fork(self, parents, children, *, stream=None):
        """Makes the empty sequences `children` copies of `parents`: full pages shared, a partly filled
        last page copied.  All or nothing."""
        pp, n = self._ints("parents", parents)
        cp, _ = self._ints("children", children, n)
        self._call(self.lib.dec_kv_fork, pp, cp, n, stream=stream)

    def release(self, seqs=None, *, window: int = 0, sinks: int = 0, stream=None):
        """Empties sequences and frees their pages; with a window, frees only the pages that a query
        with this window and these sinks no longer sees."""
        _int32(window=window, sinks=sinks)
        sp, n = self._ints("seqs", seqs)
        self._call(self.lib.dec_kv_release, sp, self.desc.n_seqs if seqs is None else n, window, sinks,
                   stream=stream)

    def compact(self, *, stream=None):
        """Moves live pages to the lowest numbers; tables and counts follow."""
        self._call(self.lib.dec_kv_compact, stream=stream)

    def sync_status(self, stream=None):
        """Waits for the stream and raises DecError if a kernel refused something since the last call."""
        bits = ctypes.c_int()
        self._call(self.lib.dec_kv_status, ctypes.byref(bits), stream=stream, lock=self._status_lock)
