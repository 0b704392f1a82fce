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


def _np(t):
    return t.detach().double().cpu().numpy()


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _cache(cm, n_pages, page, n_slots, max_pages, shapes, seed=0, dtype=torch.float16):
    planes = [_randn((n_pages, h, page, w), dtype, seed + i) for i, (h, w) in enumerate(shapes)]
    return cm.Cache(planes, torch.full((n_slots, max_pages), -1, dtype=torch.int32, device="cuda"), _ints([0] * n_slots),
                    _ints([0] * n_pages))


HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


class Sequences:
    """Slots of the given lengths in pages of random order, with the fp64 rows that they hold."""

    def __init__(self, cm, lengths, heads, width, page, dtype, seed=0):
        need = [-(-n // page) for n in lengths]
        self.cache = _cache(cm, sum(need) + 2, page, len(lengths), max(need + [1]), [(heads, width)] * 2, seed, dtype)
        order = np.random.default_rng(seed).permutation(sum(need) + 2)
        self.rows, at = ({}, {}), 0
        for s, n in enumerate(lengths):
            pages = order[at: at + need[s]].tolist()
            at += need[s]
            self.cache.table[s, : need[s]] = _ints(pages)
            for plane, rows in zip(self.cache.planes, self.rows):
                rows[s] = _np(plane[pages].transpose(0, 1).reshape(heads, -1, width)[:, :n])
        self.cache.length.copy_(_ints(lengths))
        self.dtype, self.width = dtype, width

    def check(self, got, q, slots, starts, prefix=-1):
        out, reach, size = orc.attend(_np(q), self.rows[0].__getitem__, self.rows[1].__getitem__, slots, starts, prefix)
        tol = orc.attend_tolerance(out, reach, size, HALF_STEP[self.dtype], self.width)
        assert (np.abs(_np(got) - out) <= tol).all()

    def check_token(self, got, q, t, seen):
        """Token t of slot 0's, which sees its first `seen` rows."""
        one = Sequences.__new__(Sequences)
        one.rows, one.dtype, one.width = [{0: r[0][:, :seen]} for r in self.rows], self.dtype, self.width
        one.check(got[t: t + 1], q[t: t + 1], [0], [0, 1])


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


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("bad", [-2, -(1 << 40), 16])
def test_rows_before_and_behind_the_cache_are_reported(cm, status, bad):
    """Only -1 means no row; any other number outside is an error, of rows written and of rows read."""
    c = _cache(cm, 2, 8, 1, 2, [(1, 16)])
    before = c.planes[0].clone()
    rows, where = _randn((3, 16), torch.float16, 1), torch.tensor([-1, 3, bad], device="cuda")
    c.write([0], [rows], where)
    assert status() == orc.INDEX
    before[0, 0, 3] = rows[1]
    assert torch.equal(c.planes[0], before)
    back = c.read([0], where, outs=[torch.full((3, 1, 16), 7.0, dtype=torch.float16, device="cuda")])[0]
    assert status() == orc.INDEX
    assert torch.equal(back[1, 0], rows[1]) and (back[[0, 2]] == 7).all()
    c.write([0], [rows[:2]], where[:2])
    assert status() == 0


# ------------------------------------------------------------------ too few pages
def _same(c, m):
    for name in ("table", "length", "refs"):
        assert np.array_equal(getattr(c, name).cpu().numpy(), getattr(m, name)), name


def test_a_refused_sequence_takes_no_pages_from_others(cm, status):
    """Three pages are free: the sequence that asks for ten is left out, and the two behind it get theirs."""
    c = _cache(cm, 3, 8, 3, 16, [(1, 8)])
    where, positions = c.extend(_ints([0, 1, 2]), _ints([0, 80, 88, 93]), 93)
    assert status() == orc.PAGES
    assert c.length.tolist() == [0, 8, 5] and c.refs.tolist() == [1, 1, 0]
    assert where.tolist() == [-1] * 80 + list(range(8)) + list(range(8, 13))
    assert positions.tolist() == [-1] * 80 + list(range(8)) + list(range(5))


@pytest.mark.parametrize("n_pages,n_slots,most", [(7, 5, 30), (40, 30, 60), (5000, 2500, 60), (9000, 4096, 100)])
def test_shortages_follow_the_model(cm, status, n_pages, n_slots, most):
    """Steps that ask for more than there is, of sequences with and without a partly filled page, a slot named twice and
    padding among them: who gets pages, which, and what stays as it was."""
    rng = np.random.default_rng(n_pages)
    c = _cache(cm, n_pages, 8, n_slots, 16, [(1, 8)])
    m = orc.Model(n_pages, 8, n_slots, 16)
    short = 0
    for step in range(8):
        slots = rng.permutation(n_slots)
        slots[rng.random(n_slots) < 0.1] = -1
        slots[-1] = slots[0]
        grow = rng.integers(0, 3, n_slots) * rng.integers(0, most, n_slots)
        starts = np.concatenate(([0], np.cumsum(grow)))
        tokens = int(starts[-1])
        got = c.extend(_ints(slots), _ints(starts), tokens, prefix=0)
        want = m.extend(slots.tolist(), starts.tolist(), tokens, prefix=0)
        assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(got, want)), step
        _same(c, m)
        assert status() == m.status, step
        short += bool(m.status & orc.PAGES) and not c.refs.eq(0).any().item()
        m.status = 0
        gone = rng.permutation(n_slots)[: n_slots // 3].tolist()
        c.free(_ints(gone))
        m.free(gone)
    assert short   # some step took the last page


@pytest.mark.parametrize("bad", [-1, -7, 12, 1 << 30])
def test_a_fork_of_a_lost_last_page_is_refused(cm, status, bad):
    """A parent whose partly filled page is a number outside the cache: no child of rows that nobody wrote, and the
    slot stays free for another parent of the same call."""
    c = _cache(cm, 12, 8, 5, 3, [(1, 8)])
    m = orc.Model(12, 8, 5, 3, [c.planes[0].cpu().numpy().copy()])
    for t, f in ((c, _ints), (m, list)):
        t.extend(f([0, 1]), f([0, 13, 24]), 24)
        t.table[0, 1] = bad
        t.fork(f([0, 0, 1, 1]), f([2, 3, 2, 4]))
    assert status() == orc.INDEX == m.status
    _same(c, m)
    assert c.length.tolist() == [13, 11, 11, 0, 11]
    assert np.array_equal(c.planes[0].cpu().numpy(), m.planes[0])


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("most_q", [None, 1, 2, 40, 1000])
@pytest.mark.parametrize("new,heads_q,heads", [([40, 130, 1], 4, 2), ([40, 130, 1], 8, 1), ([1, 1, 33, 1, 1, 1], 16, 2),
                                               ([300], 2, 2), ([2, 2], 4, 4)])
@pytest.mark.parametrize("with_prefix", [False, True])
def test_most_q_decides_no_output(cm, status, new, heads_q, heads, most_q, with_prefix):
    """However long the sequences are said to be (None: nothing is said), every token gets its output."""
    lengths = [n + 17 * i for i, n in enumerate(new)] + [90]
    s = Sequences(cm, lengths, heads, 64, 16, torch.float16, seed=len(new))
    starts = np.concatenate(([0], np.cumsum(new)))
    q = _randn((int(starts[-1]), heads_q, 64), torch.float16, 3)
    prefix = len(new) if with_prefix else -1
    out = torch.full_like(q, float("nan"))
    s.cache.attend(q, _ints(range(len(new))), _ints(starts), prefix=prefix, most_q=most_q, out=out)
    s.check(out, q, list(range(len(new))), starts, prefix)
    assert status() == 0


def test_a_prompt_without_most_q_is_not_cut(cm):
    """The call as it is written without the argument."""
    s = Sequences(cm, [70], 2, 128, 16, torch.bfloat16)
    q = _randn((70, 8, 128), torch.bfloat16, 4)
    s.check(s.cache.attend(q, _ints([0]), _ints([0, 70])), q, [0], [0, 70])


@pytest.mark.parametrize("most_q", [1, 5000])
def test_a_long_prompt_said_to_be_short(cm, most_q):
    """Thousands of tokens in the kernel for few rows, and single tokens in the one for many."""
    s = Sequences(cm, [3000, 700, 700], 1, 64, 64, torch.float16, seed=5)
    q = _randn((2002, 4, 64), torch.float16, 6)
    got = s.cache.attend(q, _ints([0, 1, 2]), _ints([0, 2000, 2001, 2002]), prefix=-1, most_q=most_q)
    for t in (0, 1, 15, 16, 500, 1998, 1999):
        s.check_token(got, q, t, 1000 + t + 1)
    s.check(got[2000:], q[2000:], [1, 2], [0, 1, 2])


@pytest.mark.parametrize("most_q", [1, 200])
def test_values_not_seen_weigh_nothing(cm, most_q):
    """Later tokens with V of 2^126: a weight of 2^-126 in their masked places would add 1 each."""
    s = Sequences(cm, [200], 1, 64, 32, torch.bfloat16, seed=8)
    for r in range(150, 200):
        s.cache.planes[1][int(s.cache.table[0, r // 32]), :, r % 32] = 2.0 ** 126
    q = _randn((200, 4, 64), torch.bfloat16, 9)
    got = s.cache.attend(q, _ints([0]), _ints([0, 200]), most_q=most_q)
    for t in (0, 1, 17, 127, 128, 149):
        s.check_token(got, q, t, t + 1)


@pytest.mark.parametrize("most_q", [1, 60])
@pytest.mark.parametrize("starts", [[0, 30, 10, 60], [0, 60, 0, 60], [9, 0, 12, 60], [-5, 20, 40, 60], [0, 20, 40, 61],
                                    [60, 0, 60, 0]])
def test_starts_that_descend_are_reported(cm, status, starts, most_q):
    """Lists that no step has: reported by attention and by locate, nothing is written outside the outputs."""
    s = Sequences(cm, [70, 80, 90, 300], 2, 64, 16, torch.float16, seed=10)
    q = _randn((60, 8, 64), torch.float16, 11)
    room = torch.full((70, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    for _ in range(3):
        s.cache.attend(q, _ints([0, 1, 2]), _ints(starts), prefix=3, most_q=most_q, out=room[5:65])
    assert status() == orc.INDEX
    assert (room[:5] == 7).all() and (room[65:] == 7).all()
    s.cache.locate(_ints([0, 1, 2]), _ints(starts), 60)
    assert status() == orc.INDEX
    out = torch.full_like(q, 7.0)
    s.cache.attend(q, _ints([0, 1, 2]), _ints([0, 20, 40, 60]), prefix=3, most_q=most_q, out=out)   # and the next call is right
    s.check(out, q, [0, 1, 2], [0, 20, 40, 60], 3)
    assert status() == 0


# ------------------------------------------------------------------ together
def test_attention_over_a_cache_of_latent_rows(cm, status):
    """K and V projections kept as latent rows in one paged cache: located, read, expanded, rotated into a second cache
    of K and V heads and attended there; the expanded rows are those of the projections' own latents."""
    from latent_binary_factorization_b200 import layers, littlebit as lb, synth
    d, heads, width, n = 256, 4, 64, 48
    kv = [layers.upload(synth.layer(d, heads * width, 48, False, seed=i), d, heads * width, 48) for i in (1, 2)]
    latent = cm.Cache.empty([(1, lb.latent_row_elems(x)) for x in kv], 8, 16, 2, 4)
    x = torch.randn((n, d), generator=torch.Generator().manual_seed(2)).half().cuda()
    parts = [lb.latent_forward(kv, [x[a: a + 16]] * 2) for a in range(0, n, 16)]
    slot, rope = _ints([1]), cm.Rotary(width)
    for p in parts:                                           # as three steps of 16 tokens bring them
        where, _ = latent.extend(slot, _ints([0, 16]), 16)
        latent.write([0, 1], list(p), where)
    heads_cache = cm.Cache.empty([(heads, width)] * 2, 4, 16, 1, 4)
    for a, p in zip(range(0, n, 16), parts):
        at, positions = latent.locate(slot, _ints([0, 16]), 16, first=_ints([a]))
        rows = latent.read([0, 1], at)
        for r, t, layer in zip(rows, p, kv):
            assert torch.equal(r[:, 0, : layer.s], t[:, : layer.s])
        k, v = lb.latent_expand(kv, [r[:, 0].contiguous() for r in rows])
        where, _ = heads_cache.extend(_ints([0]), _ints([0, 16]), 16)
        heads_cache.write([0, 1], [y.view(16, heads, width) for y in (k, v)], where, rope=rope, positions=positions, rotated=[0])
    q = _randn((3, 8, width), torch.float16, 3)
    q = cm.rotate([q], _ints(range(n - 3, n)), rope)[0]
    out = heads_cache.attend(q, _ints([0]), _ints([0, 3]))
    at, _ = heads_cache.locate(_ints([0]), _ints([0, n]), n)
    k, v = (_np(r).transpose(1, 0, 2) for r in heads_cache.read([0, 1], at))
    want, reach, size = orc.attend(_np(q), lambda s: k, lambda s: v, [0], [0, 3])
    assert (np.abs(_np(out) - want) <= orc.attend_tolerance(want, reach, size, 2.0 ** -11, width)).all()
    assert status() == 0
