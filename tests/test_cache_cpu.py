"""The paged cache without a GPU: what the entry points refuse (host checks,
before any CUDA call), the host function behind rotary positions, and the
oracle against its own invariants."""
import ctypes
import math

import numpy as np
import pytest

from oracle import cache_oracle as orc

ARG, ALIGN, SHAPE, UNSUPPORTED = 1, 2, 3, 6


_P, _I, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


class _C:
    """The C structures and entry points of include/littlebit.h."""

    class LbPlane(ctypes.Structure):
        _fields_ = [("data", _P), ("stride_page", _L), ("stride_head", _L), ("stride_row", _L), ("heads", _I),
                    ("width", _I), ("dt", _I)]

    class LbRows(ctypes.Structure):
        _fields_ = [("data", _P), ("stride_token", _L), ("stride_head", _L), ("heads", _I), ("width", _I)]

    class LbRotary(ctypes.Structure):
        _fields_ = [("phases", _P), ("rotary_dim", _I), ("interleaved", _I), ("scale", ctypes.c_float)]


class _LbCache(ctypes.Structure):
    _fields_ = [("planes", ctypes.POINTER(_C.LbPlane)), ("n_planes", _I), ("n_pages", _I), ("page_size", _I),
                ("n_slots", _I), ("max_pages", _I), ("table_stride", _L), ("table", _P), ("length", _P), ("refs", _P)]


_C.LbCache = _LbCache
_ARGS = {
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
    "cache_attend_work": [_P, _I, _I, _I, _I, _I, _I],
}


@pytest.fixture(scope="module")
def cm():
    from latent_binary_factorization_b200 import build_ext
    _C._lib = ctypes.CDLL(build_ext.build())
    for name, args in _ARGS.items():
        f = getattr(_C._lib, "littlebit_" + name)
        f.argtypes, f.restype = args, ctypes.c_size_t if name.endswith("_work") else ctypes.c_int
    return _C


def test_the_python_module_imports_without_a_gpu(cm):
    from latent_binary_factorization_b200 import build_ext
    build_ext.build_binding()
    import torch
    from latent_binary_factorization_b200 import cache
    cpu = torch.zeros(1, 1, 8, 16, dtype=torch.float16)
    ints = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        cache.Cache([cpu], ints.view(1, 1), ints, ints)
    with pytest.raises(ValueError):
        cache.Cache([], ints.view(1, 1), ints, ints)
    with pytest.raises(ValueError):
        cache.Rotary(16, bands=(0, 1, 2), device="cpu")


def _cache(cm, dt=0, width=128, heads=8, page=16, **over):
    planes = (cm.LbPlane * 2)(*[cm.LbPlane(4096 * (i + 1), heads * page * width, page * width, width, heads, width, dt)
                                for i in range(2)])
    c = cm.LbCache(planes, 2, 64, page, 4, 8, 8, 256, 512, 768)
    for k, v in over.items():
        setattr(c, k, v)
    c._keep = planes
    return c


def _rows(cm, heads=8, width=128, data=8192, token=None, head=None):
    return cm.LbRows(data, heads * width if token is None else token, width if head is None else head, heads, width)


@pytest.mark.parametrize("over,code", [
    (dict(page_size=12), SHAPE), (dict(page_size=4), SHAPE), (dict(page_size=2048), SHAPE), (dict(n_planes=0), SHAPE),
    (dict(n_pages=0), SHAPE), (dict(n_slots=0), SHAPE), (dict(max_pages=0), SHAPE), (dict(table_stride=7), SHAPE),
    (dict(max_pages=1 << 27, table_stride=1 << 27), SHAPE), (dict(table=None), ARG), (dict(length=None), ARG),
    (dict(refs=None), ARG),
])
def test_bad_caches_are_refused_everywhere(cm, over, code):
    lib, c = cm._lib, _cache(cm, **over)
    r, ref = ctypes.byref(_rows(cm)), ctypes.byref(c)
    pl = (ctypes.c_int * 1)(0)
    assert lib.littlebit_cache_extend(ref, 16, 16, 1, 1, -1, 16, 16, None) == code
    assert lib.littlebit_cache_locate(ref, 16, 16, None, 1, 1, -1, 16, 16, None) == code
    assert lib.littlebit_cache_write(ref, pl, r, 1, 1, 16, None, None, 0, None, None, None) == code
    assert lib.littlebit_cache_read(ref, pl, r, 1, 1, 16, None) == code
    assert lib.littlebit_cache_fork(ref, 16, 16, 1, 16, None) == code
    assert lib.littlebit_cache_free(ref, 16, 1, None) == code
    assert lib.littlebit_cache_compact(ref, 16, 16, 16, 16, None) == code
    assert lib.littlebit_cache_copy(ref, 16, 16, 1, None) == code
    assert lib.littlebit_cache_attend(ref, 0, 1, r, 1, 16, 16, 1, -1, 1, 0.1, r, 256, 1 << 40, None) == code
    assert lib.littlebit_cache_attend_work(ref, 0, 8, 1, 1, 1, 0) == 0


def test_bad_lists_and_rows_are_refused(cm):
    lib, c = cm._lib, _cache(cm)
    ref = ctypes.byref(c)
    ext = lib.littlebit_cache_extend
    assert ext(ref, None, 16, 1, 1, -1, 16, 16, None) == ARG
    assert ext(ref, 16, None, 1, 1, -1, 16, 16, None) == ARG
    assert ext(ref, 16, 16, 0, 1, -1, 16, 16, None) == SHAPE
    assert ext(ref, 16, 16, 4097, 1, -1, 16, 16, None) == SHAPE
    assert ext(ref, 16, 16, 1, -1, -1, 16, 16, None) == SHAPE
    assert ext(ref, 16, 16, 1, 1, 4, 16, 16, None) == ARG          # no such prefix slot
    assert ext(ref, 16, 16, 1, 1, -2, 16, 16, None) == ARG
    assert ext(ref, 16, 16, 1, 1, -1, None, 16, None) == ARG
    assert lib.littlebit_cache_free(ref, None, 1, None) == ARG
    assert lib.littlebit_cache_free(ref, 16, 4097, None) == SHAPE
    assert lib.littlebit_cache_fork(ref, 16, 16, 1, None, None) == ARG
    assert lib.littlebit_cache_fork(ref, 16, 16, 1, 8, None) == ALIGN
    assert lib.littlebit_cache_compact(ref, 16, 16, 16, 8, None) == ALIGN
    assert lib.littlebit_cache_copy(ref, 16, 16, (1 << 20) + 1, None) == SHAPE
    pl, bad = (ctypes.c_int * 1)(0), (ctypes.c_int * 1)(2)
    wr = lib.littlebit_cache_write

    def write(rows, planes=pl, n=1, rope=None, pos=None, bits=0, q=None, qo=None):
        return wr(ref, planes, ctypes.byref(rows), n, 1, 16, rope, pos, bits, q, qo, None)

    assert write(_rows(cm), planes=bad) == ARG
    assert write(_rows(cm, heads=4)) == SHAPE
    assert write(_rows(cm, width=64)) == SHAPE
    assert write(_rows(cm, data=8200)) == ALIGN
    assert write(_rows(cm, token=1028)) == ALIGN
    assert write(_rows(cm, data=None)) == ARG
    assert write(_rows(cm), n=8) == SHAPE
    assert write(_rows(cm), bits=1) == ARG                          # rotated without rope
    assert write(_rows(cm), bits=2) == SHAPE                        # no such place
    assert write(_rows(cm), q=ctypes.byref(_rows(cm))) == ARG       # q without q_out
    rope = cm.LbRotary(64, 144, 0, 1.0)
    assert write(_rows(cm), rope=ctypes.byref(rope), pos=16, bits=1) == SHAPE   # wider than the rows
    assert wr(ctypes.byref(_cache(cm, dt=3)), pl, ctypes.byref(_rows(cm)), 1, 1, 16, None, None, 0, None, None,
              None) == UNSUPPORTED
    assert lib.littlebit_cache_read(ref, bad, ctypes.byref(_rows(cm)), 1, 1, 16, None) == ARG


def test_bad_rotations_are_refused(cm):
    lib, r = cm._lib, ctypes.byref(_rows(cm))
    rot = lib.littlebit_rotary

    def call(rope, src=r, dst=r, n=1, tokens=1, dt=0, pos=16):
        return rot(src, dst, n, tokens, dt, pos, ctypes.byref(rope), 0, None)

    good = cm.LbRotary(64, 64, 0, 1.0)
    assert call(cm.LbRotary(None, 64, 0, 1.0)) == ARG
    assert call(cm.LbRotary(64, 64, 2, 1.0)) == ARG
    for dim in (0, 8, 24, 1040):
        assert call(cm.LbRotary(64, dim, 0, 1.0)) == SHAPE
    assert call(cm.LbRotary(64, 144, 0, 1.0)) == SHAPE
    assert call(good, pos=None) == ARG
    assert call(good, dt=3) == ARG
    assert call(good, n=0) == SHAPE
    assert call(good, n=9) == SHAPE
    assert call(good, tokens=-1) == SHAPE
    assert call(good, dst=ctypes.byref(_rows(cm, heads=4))) == SHAPE
    assert call(good, dst=ctypes.byref(_rows(cm, data=8))) == ALIGN
    assert call(good, tokens=0) == 0                                # nothing to do, no CUDA call


def test_bad_attention_calls_are_refused(cm):
    lib, c = cm._lib, _cache(cm)
    att = lib.littlebit_cache_attend

    def call(c=c, k=0, v=1, q=None, out=None, tokens=1, n=1, prefix=-1, most=1, scale=0.1, work=256, size=1 << 40):
        q = _rows(cm, heads=16) if q is None else q
        out = q if out is None else out
        return att(ctypes.byref(c), k, v, ctypes.byref(q), tokens, 16, 16, n, prefix, most, scale, ctypes.byref(out),
                   work, size, None)

    assert call(k=2) == ARG
    assert call(v=-1) == ARG
    assert call(q=_rows(cm, heads=12)) == SHAPE                     # not a multiple of 8
    assert call(q=_rows(cm, heads=16, width=64)) == SHAPE
    assert call(q=_rows(cm, heads=16, data=8)) == ALIGN
    assert call(out=_rows(cm, heads=8)) == SHAPE
    assert call(c=_cache(cm, dt=2)) == UNSUPPORTED
    assert call(c=_cache(cm, width=96)) == UNSUPPORTED
    assert call(prefix=4) == ARG
    assert call(most=0) == SHAPE
    assert call(n=0) == SHAPE
    assert call(scale=float("nan")) == ARG
    assert call(work=None) == ARG
    assert call(work=128) == ALIGN
    assert call(size=64) == SHAPE                                   # too little work memory
    assert call(tokens=0) == 0
    mixed = _cache(cm)
    mixed.planes[1].dt = 1
    assert call(c=mixed) == ARG
    mixed = _cache(cm)
    mixed.planes[1].heads = 4
    assert call(c=mixed) == SHAPE


@pytest.mark.parametrize("dim,how", [(128, {}), (64, dict(factor=8.0)), (96, dict(factor=8.0, bands=(4096, 1.0, 32.0))),
                                     (128, dict(factor=4.0, bands=(8192, 1.0, 4.0), log_ramp=True)),
                                     (16, dict(base=500000.0))])
def test_phases_are_the_frequencies(cm, dim, how):
    original, slow, fast = how.get("bands", (0.0, 0.0, 0.0))
    out = (ctypes.c_uint64 * (dim // 2))()
    assert cm._lib.littlebit_rotary_phases(dim, how.get("base", 10000.0), how.get("factor", 1.0), original, slow, fast,
                                           int(how.get("log_ramp", False)), out) == 0
    got = np.array([x / 2.0 ** 64 for x in out]) * 2 * math.pi
    # both sides go through a power and a logarithm or two in double precision or better
    assert np.allclose(got, orc.frequencies(dim, **how), rtol=1e-13, atol=0)


def test_bad_phases_are_refused(cm):
    f, out = cm._lib.littlebit_rotary_phases, (ctypes.c_uint64 * 8)()
    assert f(16, 1e4, 1.0, 0, 0, 0, 0, None) == ARG
    assert f(16, 0.0, 1.0, 0, 0, 0, 0, out) == ARG
    assert f(16, 1e4, -1.0, 0, 0, 0, 0, out) == ARG
    assert f(16, 1e4, float("nan"), 0, 0, 0, 0, out) == ARG
    assert f(16, 1e4, 2.0, 4096, 4.0, 4.0, 0, out) == ARG
    assert f(16, 1e4, 2.0, 4096, 0.0, 4.0, 1, out) == ARG
    assert f(15, 1e4, 1.0, 0, 0, 0, 0, out) == SHAPE
    assert f(0, 1e4, 1.0, 0, 0, 0, 0, out) == SHAPE


def test_oracle_rotation_depends_on_distance_alone():
    rng = np.random.default_rng(3)
    x, y = rng.standard_normal((2, 1, 1, 32))
    for inter in (False, True):
        def score(p, q):
            return float((orc.rotate(x, [p], 32, inter) * orc.rotate(y, [q], 32, inter)).sum())
        assert score(7, 3) == pytest.approx(score(1007, 1003), rel=1e-10)
        back = orc.rotate(orc.rotate(x, [123], 32, inter), [123], 32, inter, inverse=True)
        assert np.allclose(back, x, atol=1e-12)


def test_oracle_attention_joins_prefix_and_own():
    rng = np.random.default_rng(4)
    k = {0: rng.standard_normal((2, 5, 16)), 1: rng.standard_normal((2, 3, 16))}
    q = rng.standard_normal((1, 4, 16))
    both = {0: k[0], 1: np.concatenate((k[0], k[1]), 1)}
    a = orc.attend(q, lambda s: k[s], lambda s: 2 * k[s], [1], [0, 1], prefix=0)[0]
    b = orc.attend(q, lambda s: both[s], lambda s: 2 * both[s], [1], [0, 1])[0]
    assert np.allclose(a, b, atol=1e-12)


def test_oracle_pages_are_counted():
    """However a cache is used, refs[] counts the slots that hold each page."""
    rng = np.random.default_rng(5)
    m = orc.Model(24, 8, 6, 6)
    for _ in range(200):
        what = rng.integers(4)
        s, p = int(rng.integers(6)), int(rng.integers(6))
        if what == 0:
            m.extend([s], [0, int(rng.integers(1, 12))], 12)
        elif what == 1:
            m.fork([p], [s])
        elif what == 2:
            m.free([s])
        else:
            m.compact()
        held = np.zeros(24, dtype=np.int64)
        for x in range(6):
            for k in range(m.pages(int(m.length[x]))):
                held[m.table[x, k]] += 1
        assert np.array_equal(held, m.refs)
