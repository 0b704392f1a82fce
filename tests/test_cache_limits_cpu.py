"""The paged cache without a GPU: what its kernels' sources and numbers have to
hold, and refusals at the ends of the ranges."""
import os
import re

import pytest

from latent_binary_factorization_b200 import build_ext


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
