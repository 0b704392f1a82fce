"""The paged cache of liblittlebit.so (include/littlebit.h): rotary positions,
rows of tokens in pages, page bookkeeping, and attention over the pages of a
batch that shares a prefix.

Argument marshalling only, as in ``littlebit``: tensors are torch CUDA tensors,
every step runs in the CUDA library, and nothing here waits for the GPU.  All
calls take ``stream`` (a torch.cuda.Stream, default the current one of the
tensors' device); tensors that a call makes belong to that stream.  What the
bookkeeping cannot do (no free page, an index outside the cache) is left out
and reported by ``littlebit.device_status()``, bits 1 << 8 and 1 << 9.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import littlebit as lb

_lib = lb.library()
_P, _I, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


class LbPlane(ctypes.Structure):
    _fields_ = [("data", _P), ("stride_page", _L), ("stride_head", _L), ("stride_row", _L), ("heads", _I),
                ("width", _I), ("dt", _I)]


class LbCache(ctypes.Structure):
    _fields_ = [("planes", ctypes.POINTER(LbPlane)), ("n_planes", _I), ("n_pages", _I), ("page_size", _I),
                ("n_slots", _I), ("max_pages", _I), ("table_stride", _L), ("table", _P), ("length", _P),
                ("refs", _P)]


class LbRows(ctypes.Structure):
    _fields_ = [("data", _P), ("stride_token", _L), ("stride_head", _L), ("heads", _I), ("width", _I)]


class LbRotary(ctypes.Structure):
    _fields_ = [("phases", _P), ("rotary_dim", _I), ("interleaved", _I), ("scale", ctypes.c_float)]


for _name, _args in {
    "rotary_phases": [_I] + [ctypes.c_double] * 5 + [_I, _P],
    "rotary": [_P, _P, _I, _I, _I, _P, _P, _I, _P],
    "cache_extend": [_P, _P, _P, _I, _I, _I, _P, _P, _P],
    "cache_locate": [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P],
    "cache_write": [_P, _P, _P, _I, _I, _P, _P, _P, ctypes.c_uint, _P, _P, _P],
    "cache_read": [_P, _P, _P, _I, _I, _P, _P],
    "cache_fork": [_P, _P, _P, _I, _P, _P],
    "cache_free": [_P, _P, _I, _P],
    "cache_compact": [_P, _P, _P, _P, _P, _P],
    "cache_copy": [_P, _P, _P, _I, _P],
    "cache_attend": [_P, _I, _I, _P, _I, _P, _P, _I, _I, _I, ctypes.c_float, _P, _P, ctypes.c_size_t, _P],
}.items():
    getattr(_lib, "littlebit_" + _name).restype = _I
    getattr(_lib, "littlebit_" + _name).argtypes = _args
for _name, _args in {"cache_fork_work": [_I], "cache_compact_work": [_I],
                     "cache_attend_work": [_P, _I, _I, _I, _I, _I, _I]}.items():
    getattr(_lib, "littlebit_" + _name).restype = ctypes.c_size_t
    getattr(_lib, "littlebit_" + _name).argtypes = _args


def _call(name: str, device: torch.device, stream, *args) -> None:
    """The library call on ``stream``, with ``device`` current as it has to be."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"the stream is of {stream.device}, the tensors of {device}")
    fn = getattr(_lib, name)
    if torch.cuda.current_device() == device.index:
        code = fn(*args, stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            code = fn(*args, stream.cuda_stream)
    if code:
        raise lb.LittleBitError(code, name)


def _making(stream):
    """Tensors made inside belong to ``stream``."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _tensor(t, device, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")


def _list(t, device, name: str, n: int | None = None, dtype=torch.int32) -> int:
    """A contiguous index tensor; its address."""
    _tensor(t, device, name)
    if t.dtype != dtype or t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {'n' if n is None else n} entries, got "
                         f"{t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _rows(t, device, name: str, tokens: int | None = None, dtype=None) -> LbRows:
    """Rows (tokens, heads, width), or (tokens, width) for one head, unit stride within a row."""
    _tensor(t, device, name)
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        shape, stride = (shape[0], 1, shape[1]), (stride[0], 0, stride[1])
    if len(shape) != 3 or stride[2] != 1 or (tokens is not None and shape[0] != tokens):
        raise ValueError(f"{name} must be (tokens, heads, width) or (tokens, width) with unit stride in its rows and "
                         f"{'any' if tokens is None else tokens} tokens, got {tuple(t.shape)}, strides {t.stride()}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return LbRows(t.data_ptr(), stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0, shape[1], shape[2])


def _dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype not in lb._DTYPE:
        raise ValueError(f"{name}: {t.dtype} is not supported")
    return lb._DTYPE[t.dtype]


class Rotary:
    """Rotary positions of heads whose first ``rotary_dim`` elements are turned
    (a multiple of 16): pair i by position * base^(-2i / rotary_dim).

    interleaved: pairs are elements (2i, 2i + 1), else (i, i + rotary_dim/2).
    factor: frequencies divided by it (a context stretched by that factor);
    bands = (original, slow, fast): only pairs that turn few times over the
    ``original`` context are stretched, fully up to ``slow`` turns and not at
    all from ``fast`` turns on, with a ramp in turns between them (log_ramp: in
    their logarithm).  scale multiplies the turned elements."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, interleaved: bool = False, factor: float = 1.0,
                 bands: tuple | None = None, log_ramp: bool = False, scale: float = 1.0, device="cuda"):
        original, slow, fast = bands if bands is not None else (0.0, 0.0, 0.0)
        if bands is not None and not original > 0:
            raise ValueError("bands: the original context must be positive")
        host = (ctypes.c_uint64 * max(rotary_dim // 2, 1))()
        code = _lib.littlebit_rotary_phases(rotary_dim, base, factor, original, slow, fast, int(log_ramp), host)
        if code:
            raise lb.LittleBitError(code, "littlebit_rotary_phases")
        self.rotary_dim, self.interleaved, self.scale = rotary_dim, bool(interleaved), float(scale)
        self.phases = torch.frombuffer(bytearray(host), dtype=torch.int64).to(device)
        self.device = self.phases.device
        self._c = LbRotary(self.phases.data_ptr(), rotary_dim, int(self.interleaved), self.scale)
        self._ref = ctypes.addressof(self._c)


def rotate(xs: list, positions: torch.Tensor, rope: Rotary, outs: list | None = None, inverse: bool = False,
           stream=None) -> list:
    """Rotated rows of up to eight tensors (tokens, heads, width), fp16, bf16 or
    fp32, one dtype, in one launch.  ``outs`` may be ``xs`` (in place).
    inverse turns back; with scale 1 that is also the gradient of the rotation."""
    if not xs:
        raise ValueError("xs must not be empty")
    n, device, dtype = len(xs), rope.device, xs[0].dtype
    tokens = positions.shape[0] if isinstance(positions, torch.Tensor) and positions.dim() == 1 else None
    pos = _list(positions, device, "positions")
    src = (LbRows * n)(*[_rows(x, device, f"xs[{i}]", tokens, dtype) for i, x in enumerate(xs)])
    if outs is None:
        with _making(stream):
            outs = [torch.empty(x.shape, dtype=dtype, device=device) for x in xs]
    elif len(outs) != n:
        raise ValueError("outs must have as many tensors as xs")
    dst = (LbRows * n)(*[_rows(x, device, f"outs[{i}]", tokens, dtype) for i, x in enumerate(outs)])
    _call("littlebit_rotary", device, stream, src, dst, n, tokens, _dtype(xs[0], "xs"), pos, rope._ref, int(inverse))
    return outs


class Cache:
    """A paged cache over tensors of the caller.

    planes: list of (n_pages, heads, page_size, width) views, unit stride in the
    last dimension and any order of the others (K and V of every layer, or
    latent rows with one head).  table (n_slots, max_pages), length (n_slots,)
    and refs (n_pages,) are int32; ``Cache.empty`` makes them all."""

    def __init__(self, planes: list, table: torch.Tensor, length: torch.Tensor, refs: torch.Tensor):
        if not planes:
            raise ValueError("a cache has at least one plane")
        _tensor(planes[0], None, "planes[0]")
        device = planes[0].device
        if planes[0].dim() != 4:
            raise ValueError("planes are (n_pages, heads, page_size, width)")
        n_pages, _, page_size, _ = planes[0].shape
        arr = (LbPlane * len(planes))()
        for i, p in enumerate(planes):
            _tensor(p, device, f"planes[{i}]")
            if p.dim() != 4 or p.shape[0] != n_pages or p.shape[2] != page_size or p.stride(3) != 1:
                raise ValueError(f"planes[{i}] must be ({n_pages}, heads, {page_size}, width) with unit stride in its "
                                 f"rows, got {tuple(p.shape)}, strides {p.stride()}")
            st = [p.stride(d) if p.shape[d] > 1 else 0 for d in (0, 1, 2)]
            arr[i] = LbPlane(p.data_ptr(), st[0], st[1], st[2], p.shape[1], p.shape[3], _dtype(p, f"planes[{i}]"))
        _tensor(table, device, "table")
        if table.dtype != torch.int32 or table.dim() != 2 or table.stride(1) != 1 and table.shape[1] > 1:
            raise ValueError("table must be an int32 tensor (n_slots, max_pages) with unit stride in its rows")
        n_slots, max_pages = table.shape
        self.planes, self.table, self.length, self.refs = list(planes), table, length, refs
        self.device, self.n_pages, self.page_size = device, n_pages, page_size
        self.n_slots, self.max_pages = n_slots, max_pages
        self._planes = arr
        self._c = LbCache(arr, len(planes), n_pages, page_size, n_slots, max_pages,
                          table.stride(0) if n_slots > 1 else max_pages, table.data_ptr(),
                          _list(length, device, "length", n_slots), _list(refs, device, "refs", n_pages))
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, shapes: list, n_pages: int, page_size: int, n_slots: int, max_pages: int, dtype=torch.float16,
              device="cuda") -> "Cache":
        """A new empty cache; shapes: (heads, width) of every plane."""
        planes = [torch.empty((n_pages, h, page_size, w), dtype=dtype, device=device) for h, w in shapes]
        return cls(planes, torch.full((n_slots, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(n_slots, dtype=torch.int32, device=device),
                   torch.zeros(n_pages, dtype=torch.int32, device=device))

    # ---- bookkeeping
    def _places(self, tokens: int, stream, out):
        if out is not None:
            where, positions = out
        else:
            with _making(stream):
                where = torch.empty(tokens, dtype=torch.int64, device=self.device)
                positions = torch.empty(tokens, dtype=torch.int32, device=self.device)
        return (where, positions, _list(where, self.device, "where", tokens, torch.int64),
                _list(positions, self.device, "positions", tokens))

    def extend(self, slots: torch.Tensor, starts: torch.Tensor, tokens: int, prefix: int = -1, out=None, stream=None):
        """Room for new tokens: slots[i] grows by starts[i+1] - starts[i].
        Returns (where, positions) of the step's ``tokens`` tokens: their rows
        in the cache (int64, -1: none) and their places in their sequences,
        behind slot ``prefix``'s tokens if it is given (int32)."""
        n = slots.shape[0]
        where, positions, w, p = self._places(tokens, stream, out)
        _call("littlebit_cache_extend", self.device, stream, self._ref, _list(slots, self.device, "slots"),
              _list(starts, self.device, "starts", n + 1), n, tokens, prefix, w, p)
        return where, positions

    def locate(self, slots: torch.Tensor, starts: torch.Tensor, tokens: int, first: torch.Tensor | None = None,
               prefix: int = -1, out=None, stream=None):
        """(where, positions), as ``extend`` gives them, of tokens held: the
        tokens from first[i] (default 0) of slots[i] on."""
        n = slots.shape[0]
        where, positions, w, p = self._places(tokens, stream, out)
        _call("littlebit_cache_locate", self.device, stream, self._ref, _list(slots, self.device, "slots"),
              _list(starts, self.device, "starts", n + 1),
              None if first is None else _list(first, self.device, "first", n), n, tokens, prefix, w, p)
        return where, positions

    def fork(self, parents: torch.Tensor, children: torch.Tensor, stream=None) -> None:
        """Makes each (empty) slot children[i] a copy of slot parents[i]: full
        pages are shared, a partly filled last page is copied."""
        n = parents.shape[0]
        with _making(stream):
            work = torch.empty(_lib.littlebit_cache_fork_work(n), dtype=torch.uint8, device=self.device)
        _call("littlebit_cache_fork", self.device, stream, self._ref, _list(parents, self.device, "parents"),
              _list(children, self.device, "children", n), n, work.data_ptr())

    def free(self, slots: torch.Tensor, stream=None) -> None:
        """Empties the slots; pages that no other slot holds become free."""
        _call("littlebit_cache_free", self.device, stream, self._ref, _list(slots, self.device, "slots"),
              slots.shape[0])

    def compact(self, into: bool = False, stream=None):
        """Moves the pages in use to the lowest numbers.  Returns (table, refs,
        count of pages in use): the cache's own tensors, updated, or with
        ``into`` new ones, the cache's staying as they are (and the rows they
        lead to good until a page is taken)."""
        with _making(stream):
            work = torch.empty(_lib.littlebit_cache_compact_work(self.n_pages), dtype=torch.uint8, device=self.device)
            count = torch.empty(1, dtype=torch.int32, device=self.device)
            table = torch.empty_strided(self.table.shape, self.table.stride(), dtype=torch.int32,
                                        device=self.device) if into else self.table
            refs = torch.empty_like(self.refs) if into else self.refs
        _call("littlebit_cache_compact", self.device, stream, self._ref, table.data_ptr(), refs.data_ptr(),
              count.data_ptr(), work.data_ptr())
        return table, refs, count

    def copy(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Copies page src[i] to page dst[i] in every plane."""
        n = src.shape[0]
        _call("littlebit_cache_copy", self.device, stream, self._ref, _list(src, self.device, "src"),
              _list(dst, self.device, "dst", n), n)

    # ---- rows
    def write(self, planes: list, rows: list, where: torch.Tensor, rope: Rotary | None = None,
              positions: torch.Tensor | None = None, rotated=(), q: torch.Tensor | None = None,
              q_out: torch.Tensor | None = None, stream=None):
        """Writes rows[i] (tokens, heads, width) to plane planes[i] at the rows
        ``where``, one launch.  The planes whose place i is in ``rotated`` get
        their rows rotated by ``rope`` at ``positions``; q is rotated beside
        them and returned."""
        n, tokens = len(planes), where.shape[0]
        if n == 0 or len(rows) != n:
            raise ValueError("planes and rows must be lists of the same length, not empty")
        if (rotated or q is not None) and (rope is None or positions is None):
            raise ValueError("rotating needs rope and positions")
        if rope is not None and rope.device != self.device:
            raise ValueError(f"rope is on {rope.device}, not {self.device}")
        bits = 0
        for i in rotated:
            if not 0 <= i < n:
                raise ValueError(f"rotated: {i} is not a place in planes")
            bits |= 1 << i
        dtype = rows[0].dtype
        _dtype(rows[0], "rows")
        src = (LbRows * n)(*[_rows(r, self.device, f"rows[{i}]", tokens, dtype) for i, r in enumerate(rows)])
        qs = qd = None
        if q is not None:
            qs = ctypes.byref(_rows(q, self.device, "q", tokens, dtype))
            if q_out is None:
                with _making(stream):
                    q_out = torch.empty(q.shape, dtype=dtype, device=self.device)
            qd = ctypes.byref(_rows(q_out, self.device, "q_out", tokens, dtype))
        elif q_out is not None:
            raise ValueError("q_out without q")
        for i in planes:
            if not 0 <= i < len(self.planes) or self.planes[i].dtype != dtype:
                raise ValueError(f"plane {i}: there is none, or its dtype is not the rows' {dtype}")
        _call("littlebit_cache_write", self.device, stream, self._ref, (_I * n)(*planes), src, n, tokens,
              _list(where, self.device, "where", None, torch.int64), None if rope is None else rope._ref,
              None if positions is None else _list(positions, self.device, "positions", tokens), bits, qs, qd)
        return q_out

    def read(self, planes: list, where: torch.Tensor, outs: list | None = None, stream=None) -> list:
        """The rows ``where`` of the planes, (tokens, heads, width) each; rows
        whose ``where`` is -1 are left as ``outs`` has them (undefined in
        tensors made here).  Up to eight planes of one dtype."""
        n, tokens = len(planes), where.shape[0]
        for i in planes:
            if not 0 <= i < len(self.planes):
                raise ValueError(f"there is no plane {i}")
        if n == 0 or outs is not None and len(outs) != n:
            raise ValueError("planes must not be empty, and outs as long")
        dtype = self.planes[planes[0]].dtype
        if outs is None:
            with _making(stream):
                outs = [torch.empty((tokens, self.planes[i].shape[1], self.planes[i].shape[3]),
                                    dtype=self.planes[i].dtype, device=self.device) for i in planes]
        dst = (LbRows * n)(*[_rows(r, self.device, f"outs[{i}]", tokens, dtype) for i, r in enumerate(outs)])
        _call("littlebit_cache_read", self.device, stream, self._ref, (_I * n)(*planes), dst, n, tokens,
              _list(where, self.device, "where", None, torch.int64))
        return outs

    # ---- attention
    def attend(self, q: torch.Tensor, slots: torch.Tensor, starts: torch.Tensor, k: int = 0, v: int = 1,
               prefix: int = -1, most_q: int = 1, scale: float | None = None, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
        """Attention of the newest tokens over slot ``prefix`` (shared by the
        whole batch, read once for it) and their own slots.  q: (tokens, query
        heads, width), sequence i holding its rows starts[i] .. starts[i+1],
        the last tokens of slots[i], each of which sees the prefix and its own
        slot up to itself.  most_q bounds the tokens of one sequence.  k and v:
        planes (fp16 or bf16, width 64 or 128).  scale: default width^-0.5.
        Rows in no sequence are left as ``out`` has them (undefined in one made
        here)."""
        tokens, n = q.shape[0], slots.shape[0]
        cq = _rows(q, self.device, "q", None, self.planes[k].dtype if 0 <= k < len(self.planes) else None)
        if out is None:
            with _making(stream):
                out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
        co = _rows(out, self.device, "out", tokens, q.dtype)
        if scale is None:
            scale = 1.0 / math.sqrt(cq.width)
        size = _lib.littlebit_cache_attend_work(self._ref, k, cq.heads, tokens, n, most_q, prefix >= 0)
        with _making(stream):
            work = torch.empty(size, dtype=torch.uint8, device=self.device)
        _call("littlebit_cache_attend", self.device, stream, self._ref, k, v, ctypes.byref(cq), tokens,
              _list(slots, self.device, "slots"), _list(starts, self.device, "starts", n + 1), n, prefix, most_q,
              scale, ctypes.byref(co), work.data_ptr(), size)
        return out
