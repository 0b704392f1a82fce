"""The paged cache at the ends of its ranges: what cannot be done is reported
and nothing else is lost to it, against the fp64 oracle and by construction."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latent_binary_factorization_b200 import cache, littlebit
    littlebit.device_status()
    return cache


@pytest.fixture
def status():
    """The bits raised since the test began, at each call."""
    from latent_binary_factorization_b200 import littlebit
    littlebit.device_status()
    return littlebit.device_status


def _ints(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _cache(cm, n_pages, page, n_slots, max_pages, shapes, seed=0, dtype=torch.float16):
    planes = [_randn((n_pages, h, page, w), dtype, seed + i) for i, (h, w) in enumerate(shapes)]
    return cm.Cache(planes, torch.full((n_slots, max_pages), -1, dtype=torch.int32, device="cuda"), _ints([0] * n_slots),
                    _ints([0] * n_pages))


# ------------------------------------------------------------------ page copies
@pytest.mark.parametrize("planes", [1, 2, 3])
@pytest.mark.parametrize("at", [0, 1, 2, 3, 4, 5, 6, 7, 1299])
def test_a_bad_page_among_many_copies_is_reported(cm, status, planes, at):
    """Copies enough for a warp each: whichever warp meets the bad number says so."""
    n = 1300
    c = _cache(cm, 2 * n, 8, 1, 1, [(1, 8)] * planes)
    src, dst = np.arange(n), n + np.arange(n)
    src[at] = 2 * n
    want = [p.clone() for p in c.planes]
    for p in want:
        keep = p[n + at].clone()
        p[n:] = p[:n]
        p[n + at] = keep
    c.copy(_ints(src), _ints(dst))
    assert status() == orc.INDEX
    assert all(torch.equal(p, w) for p, w in zip(c.planes, want))
