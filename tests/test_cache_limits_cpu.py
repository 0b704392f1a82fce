"""The paged cache without a GPU: what its kernels' sources and numbers have to
hold, and refusals at the ends of the ranges."""
import ctypes
import os
import re

import pytest

from latent_binary_factorization_b200 import build_ext
from oracle import cache_oracle as orc


def _source(name):
    with open(os.path.join(build_ext.CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name", ["cache.cu", "attend.cu"])
def test_dependent_kernels_promise_nothing_about_their_inputs(name):
    """These kernels start while the one before them may still write what they
    read; a const __restrict__ pointer would let loads pass their wait."""
    code = re.sub(r"//.*", "", _source(name))
    assert "dependent_begin" in code
    assert "__restrict__" not in code and "__ldg" not in code and "ld.global.nc" not in code


def test_a_block_that_gave_up_waits_for_all_that_it_began():
    """The many-rows kernel's way out after a wait that ran out cannot be run
    without a hang, so its source is looked at: it drains both rings up to the
    copies that were begun (of K one more than of V may be), and the products."""
    code = _source("attend.cu")
    ring = code[code.index("if (dead && lane == 0)"):]
    ring = ring[: ring.index("\n      }\n")]
    assert re.search(r"k = loads\[0\], v = loads\[1\]", ring)
    assert re.search(r"x < k; \+\+x\) mbar_wait\(&k_full", ring) and re.search(r"x < v; \+\+x\) mbar_wait\(&v_full", ring)
    out = code[code.index("if (dead && issuer)"):]
    out = out[: out.index("\n    }\n")]
    assert "tc_commit(&quiet[gg])" in out and "mbar_wait(&quiet[gg], 0)" in out
    assert code.index("if (dead && issuer)") < code.index("tcgen05.dealloc")


def test_scores_do_not_rely_on_the_order_of_products():
    """Products with different accumulators are promised no order: where P
    shares S's columns, the next scores' products follow a wait for the PV
    that reads it; where it does not, the columns of S, O and P are disjoint."""
    code = _source("attend.cu")
    score = code[code.index("auto score = "):]
    score = score[: score.index("mma_ss(")]
    assert "if (!kWeights<D> && after && !dead)" in score and "mbar_wait(&p_free[gg]" in score
    at = {128: 0, 64: 256 + 64}                              # kWeights
    assert "kWeights = D == 128 ? 0 : 256 + D" in code
    for d, p in at.items():
        used = []
        for g in range(2):
            used += [*range(128 * g, 128 * g + 128), *range(256 + 128 * g, 256 + 128 * g + d)]
            if p:
                used += range(128 * g + p, 128 * g + p + 64)
        assert len(used) == len(set(used)) and max(used) < 512


def test_oracle_a_refused_sequence_asks_for_nothing():
    m = orc.Model(3, 8, 3, 16)
    where, _ = m.extend([0, 1, 2], [0, 80, 88, 93], 93)
    assert m.status == orc.PAGES and m.length.tolist() == [0, 8, 5]
    assert where[80:].tolist() == [*range(8), *range(8, 13)] and (where[:80] == -1).all()


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf"), 2.4e38, -3.4e38])
def test_scales_that_overflow_are_refused(scale):
    """Scores are in units of log 2: a finite scale times log2 e may not be."""
    lib = ctypes.CDLL(build_ext.build())

    class Plane(ctypes.Structure):
        _fields_ = [("data", ctypes.c_void_p), ("strides", ctypes.c_int64 * 3), ("heads", ctypes.c_int),
                    ("width", ctypes.c_int), ("dt", ctypes.c_int)]

    class Cache(ctypes.Structure):
        _fields_ = [("planes", ctypes.POINTER(Plane)), ("n", ctypes.c_int * 5), ("table_stride", ctypes.c_int64),
                    ("arrays", ctypes.c_void_p * 3)]

    class Rows(ctypes.Structure):
        _fields_ = [("data", ctypes.c_void_p), ("strides", ctypes.c_int64 * 2), ("heads", ctypes.c_int), ("width", ctypes.c_int)]

    plane = Plane(4096, (16 * 64, 16 * 64, 64), 1, 64, 0)
    c = Cache(ctypes.pointer(plane), (1, 4, 16, 2, 2), 2, (256, 512, 768))
    q = Rows(8192, (64, 64), 1, 64)
    f = lib.littlebit_cache_attend
    f.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                  ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                  ctypes.c_void_p]
    args = [ctypes.byref(c), 0, 0, ctypes.byref(q), 1, 16, 16, 1, -1, 1]
    assert f(*args, scale, ctypes.byref(q), 256, 1 << 40, None) == 1    # LB_ERR_ARG
    assert f(*args, 2.3e38, ctypes.byref(q), None, 0, None) == 1        # the largest go on to the next refusal: no work memory
    assert f(*args, 2.3e38, ctypes.byref(q), 256, 0, None) == 3         # LB_ERR_SHAPE: too little of it
