"""The paged cache of liblittlebit.so (include/littlebit.h): rotary positions,
rows of tokens in pages, page bookkeeping, and attention over the pages of a
batch that shares a prefix.

Tensors are torch CUDA tensors, every step runs in the CUDA library, and
nothing here waits for the GPU.  The marshalling of the arguments is compiled
(csrc/cache_binding.cpp, ``_cache.so``): a call takes a few microseconds, as
the kernels of a decode step do.  Arguments that do not fit raise ValueError,
what the library refuses ``littlebit.LittleBitError``.

All calls take ``stream`` (a torch.cuda.Stream, default the current one of the
tensors' device); tensors that a call makes belong to that stream.  What the
bookkeeping cannot do (no free page, an index outside the cache) is left out
and reported by ``littlebit.device_status()``, bits 1 << 8 and 1 << 9.
Autograd does not see these calls.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import littlebit as lb

BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_cache.so")
if not os.path.exists(BINDING_PATH):
    raise ImportError(
        f"{BINDING_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
        "(the paged cache has no CPU implementation)"
    )
_loader = importlib.machinery.ExtensionFileLoader("_cache", BINDING_PATH)
_b = importlib.util.module_from_spec(importlib.util.spec_from_loader("_cache", _loader))
_loader.exec_module(_b)
_b.on_fail(lb._check)

_phases = lb.library().littlebit_rotary_phases
_phases.restype = ctypes.c_int
_phases.argtypes = [ctypes.c_int] + [ctypes.c_double] * 5 + [ctypes.c_int, ctypes.c_void_p]


def _on(stream, device: torch.device):
    """``stream`` as the current one of ``device`` (the binding takes the current)."""
    if stream.device != device:
        raise ValueError(f"the stream is of {stream.device}, the tensors of {device}")
    return torch.cuda.stream(stream)


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
        lb._check(_phases(rotary_dim, base, factor, original, slow, fast, int(log_ramp), host),
                  "littlebit_rotary_phases")
        self.rotary_dim, self.interleaved, self.scale = rotary_dim, bool(interleaved), float(scale)
        self.phases = torch.frombuffer(bytearray(host), dtype=torch.int64).to(device)
        self.device = self.phases.device
        self._h = _b.rotary(self.phases, rotary_dim, self.interleaved, self.scale)


def rotate(xs: list, positions: torch.Tensor, rope: Rotary, outs: list | None = None, inverse: bool = False,
           stream=None) -> list:
    """Rotated rows of up to eight tensors (tokens, heads, width), fp16, bf16 or
    fp32, one dtype, in one launch.  ``outs`` may be ``xs`` (in place).
    inverse turns back; with any scale it is also the transpose, i.e. the
    gradient of the rotation."""
    if stream is not None:
        with _on(stream, rope.device):
            return _b.rotate(rope._h, xs, positions, outs, inverse)
    return _b.rotate(rope._h, xs, positions, outs, inverse)


class Cache:
    """A paged cache over tensors of the caller.

    planes: list of (n_pages, heads, page_size, width) views, unit stride in the
    last dimension and any order of the others (K and V of every layer, or
    latent rows with one head).  table (n_slots, max_pages), length (n_slots,)
    and refs (n_pages,) are int32; ``Cache.empty`` makes them all."""

    def __init__(self, planes: list, table: torch.Tensor, length: torch.Tensor, refs: torch.Tensor):
        self._h = _b.cache(planes, table, length, refs)
        self._tensors = tuple(planes), table, length, refs   # the handle holds their addresses
        self.device = table.device
        self.n_pages, self.page_size = planes[0].shape[0], planes[0].shape[2]
        self.n_slots, self.max_pages = table.shape

    @classmethod
    def empty(cls, shapes: list, n_pages: int, page_size: int, n_slots: int, max_pages: int, dtype=torch.float16,
              device="cuda") -> "Cache":
        """A new empty cache; shapes: (heads, width) of every plane, whose
        contents are undefined until they are written."""
        planes = [torch.empty((n_pages, h, page_size, w), dtype=dtype, device=device) for h, w in shapes]
        return cls(planes, torch.full((n_slots, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(n_slots, dtype=torch.int32, device=device),
                   torch.zeros(n_pages, dtype=torch.int32, device=device))

    # the cache's tensors; to go on with others (as compact(into=True) gives), make another Cache
    planes = property(lambda self: self._tensors[0])
    table = property(lambda self: self._tensors[1])
    length = property(lambda self: self._tensors[2])
    refs = property(lambda self: self._tensors[3])

    # ---- bookkeeping
    def extend(self, slots: torch.Tensor, starts: torch.Tensor, tokens: int, prefix: int = -1, out=None, stream=None):
        """Room for new tokens: slots[i] grows by starts[i+1] - starts[i].
        Returns (where, positions) of the step's ``tokens`` tokens: their rows
        in the cache (int64, -1: none) and their places in their sequences,
        behind slot ``prefix``'s tokens if it is given (int32)."""
        if stream is not None:
            with _on(stream, self.device):
                return _b.extend(self._h, slots, starts, tokens, prefix, out)
        return _b.extend(self._h, slots, starts, tokens, prefix, out)

    def locate(self, slots: torch.Tensor, starts: torch.Tensor, tokens: int, first: torch.Tensor | None = None,
               prefix: int = -1, out=None, stream=None):
        """(where, positions), as ``extend`` gives them, of tokens held: the
        tokens from first[i] (default 0) of slots[i] on."""
        if stream is not None:
            with _on(stream, self.device):
                return _b.locate(self._h, slots, starts, tokens, first, prefix, out)
        return _b.locate(self._h, slots, starts, tokens, first, prefix, out)

    def fork(self, parents: torch.Tensor, children: torch.Tensor, stream=None) -> None:
        """Makes each (empty) slot children[i] a copy of slot parents[i]: full
        pages are shared, a partly filled last page is copied."""
        if stream is not None:
            with _on(stream, self.device):
                return _b.fork(self._h, parents, children)
        return _b.fork(self._h, parents, children)

    def free(self, slots: torch.Tensor, stream=None) -> None:
        """Empties the slots; pages that no other slot holds become free."""
        if stream is not None:
            with _on(stream, self.device):
                return _b.free(self._h, slots)
        return _b.free(self._h, slots)

    def compact(self, into: bool = False, stream=None):
        """Moves the pages in use to the lowest numbers.  Returns (table, refs,
        count of pages in use): the cache's own tensors, updated, or with
        ``into`` new ones, the cache's staying as they are (and the rows they
        lead to good until a page is taken); go on with a Cache of the new."""
        if stream is not None:
            with _on(stream, self.device):
                return _b.compact(self._h, self.table, self.refs, into)
        return _b.compact(self._h, self.table, self.refs, into)

    def copy(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Copies page src[i] to page dst[i] in every plane."""
        if stream is not None:
            with _on(stream, self.device):
                return _b.copy(self._h, src, dst)
        return _b.copy(self._h, src, dst)

    # ---- rows
    def write(self, planes: list, rows: list, where: torch.Tensor, rope: Rotary | None = None,
              positions: torch.Tensor | None = None, rotated=(), q: torch.Tensor | None = None,
              q_out: torch.Tensor | None = None, stream=None):
        """Writes rows[i] (tokens, heads, width) to plane planes[i] at the rows
        ``where``, one launch.  The planes whose place i is in ``rotated`` get
        their rows rotated by ``rope`` at ``positions``; q is rotated beside
        them and returned."""
        h = None if rope is None else rope._h
        if stream is not None:
            with _on(stream, self.device):
                return _b.write(self._h, planes, rows, where, h, positions, rotated, q, q_out)
        return _b.write(self._h, planes, rows, where, h, positions, rotated, q, q_out)

    def read(self, planes: list, where: torch.Tensor, outs: list | None = None, stream=None) -> list:
        """The rows ``where`` of the planes, (tokens, heads, width) each; rows
        whose ``where`` is -1 are left as ``outs`` has them (undefined in
        tensors made here).  Up to eight planes of one dtype."""
        if stream is not None:
            with _on(stream, self.device):
                return _b.read(self._h, planes, where, outs)
        return _b.read(self._h, planes, where, outs)

    # ---- attention
    def attend(self, q: torch.Tensor, slots: torch.Tensor, starts: torch.Tensor, k: int = 0, v: int = 1,
               prefix: int = -1, most_q: int | None = None, scale: float | None = None,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of the newest tokens over slot ``prefix`` (shared by the
        whole batch, read once for it) and their own slots.  q: (tokens, query
        heads, width), sequence i holding its rows starts[i] .. starts[i+1],
        the last tokens of slots[i], each of which sees the prefix and its own
        slot up to itself.  most_q: the tokens of the longest of these sequences,
        which decides how the work is done, not what comes out (default: their
        mean, right for steps of single tokens and for prompts of one size).
        k and v: planes (fp16 or bf16, width 64 or 128).  scale: default
        width^-0.5.
        Rows in no sequence are left as ``out`` has them (undefined in one made
        here)."""
        if stream is not None:
            with _on(stream, self.device):
                return _b.attend(self._h, q, slots, starts, k, v, prefix, most_q, scale, out)
        return _b.attend(self._h, q, slots, starts, k, v, prefix, most_q, scale, out)
