"""GPU parity of the paged cache's rows and bookkeeping against the fp64 oracle:
rotary positions, rows into and out of pages, extend, locate, fork, free,
compact and copy, and a graph of a serving step."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def cm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latent_binary_factorization_b200 import cache, littlebit
    littlebit.device_status()
    return cache


def _randn(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _ints(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")


def _rotary_tolerance(x, y, dim, interleaved, dtype, scale=1.0):
    """One rounding of the result; cos and sin are off by at most 2^-22 (half a
    step of the argument and of each function), the three fp32 operations by
    2^-24 of their magnitudes each: 2^-21 (|a| + |b|) in all.  Values below
    fp16's normal range are off by at most 2^-25."""
    x = np.abs(x)
    mag = np.zeros_like(x)
    for i in range(dim // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + dim // 2)
        mag[..., a] = mag[..., b] = x[..., a] + x[..., b]
    return HALF_STEP[dtype] * np.abs(y) + abs(scale) * 2.0 ** -21 * mag + 2.0 ** -25


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,heads,width,dim,interleaved", [
    (1, 1, 16, 16, False), (1, 32, 128, 128, True), (5, 3, 96, 96, False), (7, 14, 128, 64, True), (33, 2, 80, 48, False),
    (2500, 4, 64, 32, False), (2501, 3, 64, 64, True), (3, 2, 1024, 1024, False), (3, 2, 1032, 1024, True)])
def test_rotate(cm, dtype, tokens, heads, width, dim, interleaved):
    x, y = _randn((tokens, heads, width), dtype, 1), _randn((tokens, 2 * heads, width), dtype, 2)
    pos = np.random.default_rng(3).integers(0, 1 << 20, tokens)
    pos[:4] = [0, 2 ** 31 - 1, -5, 1][:min(tokens, 4)]
    rope = cm.Rotary(dim, interleaved=interleaved, scale=1.25)
    got = cm.rotate([x, y], _ints(pos), rope)
    for a, b in zip((x, y), got):
        ref = orc.rotate(_np(a), pos, dim, interleaved, scale=1.25)
        # the oracle's own angles in double precision: pos * f is off by 2^-53 of up to 2^31
        tol = _rotary_tolerance(_np(a), ref, dim, interleaved, dtype, 1.25) + 2.0 ** -20 * (np.abs(pos) > 2 ** 30)[:, None, None]
        assert (np.abs(_np(b) - ref) <= tol).all()
        assert torch.equal(b[..., dim:], a[..., dim:])


@pytest.mark.parametrize("how", [dict(factor=8.0), dict(factor=8.0, bands=(4096, 1.0, 32.0)),
                                 dict(factor=4.0, bands=(8192, 1.0, 4.0), log_ramp=True), dict(base=500000.0)])
def test_rotate_stretched(cm, how):
    x = _randn((64, 2, 128), torch.float32, 4)
    pos = np.arange(64) * 16411
    got = cm.rotate([x], _ints(pos), cm.Rotary(128, **how))[0]
    ref = orc.rotate(_np(x), pos, 128, **how)
    assert (np.abs(_np(got) - ref) <= _rotary_tolerance(_np(x), ref, 128, False, torch.float32)).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_views_in_place_and_back(cm, interleaved):
    """q and k as views of one projection, turned in place; the inverse is the
    transpose, hence the gradient: <rotate(x), g> = <x, inverse(g)>, and equals
    the change of <rotate(x), g> along any direction (the map is linear)."""
    qkv = _randn((9, 12, 64), torch.float32, 5)
    q, k = qkv[:, :8], qkv[:, 8:10]
    before = qkv.clone()
    rope = cm.Rotary(32, interleaved=interleaved)
    pos = _ints(range(100, 109))
    outs = cm.rotate([q, k], pos, rope, outs=[q, k])
    assert outs[0] is q
    ref = orc.rotate(_np(before[:, :10]), range(100, 109), 32, interleaved)
    assert (np.abs(_np(qkv[:, :10]) - ref) <= _rotary_tolerance(_np(before[:, :10]), ref, 32, interleaved, torch.float32)).all()
    assert torch.equal(qkv[:, 10:], before[:, 10:])
    g = _randn((9, 8, 64), torch.float32, 6)
    grad = cm.rotate([g], pos, rope, inverse=True)[0]
    ref = orc.rotate(_np(g), range(100, 109), 32, interleaved, inverse=True)
    assert (np.abs(_np(grad) - ref) <= _rotary_tolerance(_np(g), ref, 32, interleaved, torch.float32)).all()
    d = _randn((9, 8, 64), torch.float32, 7)
    up, down = (cm.rotate([(before[:, :8] + s * d).contiguous()], pos, rope)[0] for s in (0.5, -0.5))
    # 4608 products of O(1) values, each off by less than 2^-20
    assert float(((up - down).double() * g.double()).sum() - (d.double() * grad.double()).sum()) == pytest.approx(0, abs=4608 * 2.0 ** -20 * 10)


def _plane(n_pages, heads, page, width, dtype, order, seed):
    """A plane whose memory order is one of the orders of (page, head, row)."""
    if order == "phr":
        return _randn((n_pages, heads, page, width), dtype, seed)
    if order == "prh":
        return _randn((n_pages, page, heads, width), dtype, seed).transpose(1, 2)
    if order == "hpr":
        return _randn((heads, n_pages, page, width), dtype, seed).transpose(0, 1)
    wide = _randn((n_pages, heads, page, 3 * width), dtype, seed)   # K, V and something else side by side
    return wide[..., width:2 * width]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("order", ["phr", "prh", "hpr", "wide"])
@pytest.mark.parametrize("tokens,heads,page,width,dim,interleaved", [
    (1, 1, 8, 192, 32, False), (17, 4, 16, 64, 64, True), (300, 2, 64, 128, 48, False), (2400, 1, 1024, 64, 32, True)])
def test_write_and_read(cm, dtype, order, tokens, heads, page, width, dim, interleaved):
    n_pages = -(-tokens // page) + 3
    planes = [_plane(n_pages, heads, page, width, dtype, order, 10 + i) for i in range(3)]
    c = cm.Cache(planes, torch.full((1, 1), -1, dtype=torch.int32, device="cuda"), _ints([0]), _ints([0] * n_pages))
    rng = np.random.default_rng(11)
    where = rng.permutation(n_pages * page)[:tokens]
    where[rng.random(tokens) < 0.2] = -1
    pos = rng.integers(0, 10000, tokens)
    k, v, q = (_randn((tokens, h, width), dtype, 12 + i) for i, h in enumerate((heads, heads, 3 * heads)))
    before = [p.clone() for p in planes]
    rope = cm.Rotary(dim, interleaved=interleaved)
    w = torch.tensor(where, device="cuda")
    q_out = c.write([2, 0], [k, v], w, rope=rope, positions=_ints(pos), rotated=[0], q=q)
    ref = orc.rotate(_np(q), pos, dim, interleaved)
    assert (np.abs(_np(q_out) - ref) <= _rotary_tolerance(_np(q), ref, dim, interleaved, dtype)).all()
    kr = orc.rotate(_np(k), pos, dim, interleaved)
    got_k, got_v = c.read([2, 0], w, outs=[torch.zeros_like(k), torch.zeros_like(v)])
    at = where >= 0
    assert (np.abs(_np(got_k) - kr)[at] <= _rotary_tolerance(_np(k), kr, dim, interleaved, dtype)[at]).all()
    assert torch.equal(got_v[torch.tensor(at)], v[torch.tensor(at)])
    assert not got_k[torch.tensor(~at)].any() and not got_v[torch.tensor(~at)].any()
    # nothing but the rows named has changed
    assert torch.equal(planes[1], before[1])
    for p, b in ((planes[2], before[2]), (planes[0], before[0])):
        same = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
        same[w[w >= 0]] = False
        flat = [x.permute(0, 2, 1, 3).reshape(-1, heads, width) for x in (p, b)]
        assert torch.equal(flat[0][same], flat[1][same])


def test_rows_outside_the_cache_are_skipped_and_reported(cm):
    from latent_binary_factorization_b200 import littlebit as lb
    plane = _randn((2, 1, 8, 16), torch.float16, 20)
    before = plane.clone()
    c = cm.Cache([plane], torch.full((1, 2), -1, dtype=torch.int32, device="cuda"), _ints([0]), _ints([0, 0]))
    rows = _randn((3, 16), torch.float16, 21)            # one head: two dimensions will do
    c.write([0], [rows], torch.tensor([16, 3, 1 << 40], device="cuda"))
    assert lb.device_status() == orc.INDEX
    before[0, 0, 3] = rows[1]
    assert torch.equal(plane, before)
    assert lb.device_status() == 0


def _compare(c, m, tag):
    for name in ("table", "length", "refs"):
        assert np.array_equal(getattr(c, name).cpu().numpy(), getattr(m, name)), f"{tag}: {name}"
    for i, (p, r) in enumerate(zip(c.planes, m.planes)):
        assert np.array_equal(p.cpu().numpy(), r), f"{tag}: plane {i}"


def _pair(cm, n_pages, page, n_slots, max_pages, shapes, seed=30, pad=0):
    planes = [_randn((n_pages, h, page, w), torch.float16, seed + i) for i, (h, w) in enumerate(shapes)]
    table = torch.full((n_slots, max_pages + pad), -1, dtype=torch.int32, device="cuda")[:, :max_pages]
    c = cm.Cache(planes, table, _ints([0] * n_slots), _ints([0] * n_pages))
    return c, orc.Model(n_pages, page, n_slots, max_pages, [p.cpu().numpy().copy() for p in planes])


@pytest.mark.parametrize("n_pages,page,n_slots,max_pages,pad", [
    (20, 8, 5, 6, 0), (5000, 16, 40, 200, 3), (4097, 1024, 3, 8, 0), (1, 8, 2, 1, 1), (97, 32, 300, 4, 0)])
def test_bookkeeping_follows_the_model(cm, n_pages, page, n_slots, max_pages, pad):
    """Random calls, asked-too-much ones and wrong ones among them: tables, rows,
    places and status bits are the model's after every call."""
    from latent_binary_factorization_b200 import littlebit as lb
    shapes = [(1, 8), (2, 16)] if n_pages * page < 100000 else [(1, 8)]
    c, m = _pair(cm, n_pages, page, n_slots, max_pages, shapes, pad=pad)
    rng = np.random.default_rng(n_pages)
    lb.device_status()
    for step in range(60):
        what = int(rng.integers(6))
        n = int(rng.integers(1, min(2 * n_slots, 60) + 1))
        slots = rng.integers(-1, n_slots, n).tolist()
        if rng.random() < 0.1:
            slots[0] = n_slots + 7
        if what <= 1:
            if rng.random() < 0.7:   # mostly each slot once
                slots = rng.permutation(n_slots)[:n].tolist()
            n = len(slots)
            most = int(rng.choice([1, 2, page, 3 * page]))
            starts = np.concatenate(([0], np.cumsum(rng.integers(0, most + 1, n))))
            tokens = int(starts[-1]) + int(rng.integers(3))
            prefix = int(rng.integers(-1, n_slots))
            got = c.extend(_ints(slots), _ints(starts), tokens, prefix)
            want = m.extend(slots, starts.tolist(), tokens, prefix)
        elif what == 2:
            parents = rng.integers(0, n_slots, n).tolist()
            got = want = ()
            c.fork(_ints(parents), _ints(slots))
            m.fork(parents, slots)
        elif what == 3:
            got = want = ()
            slots = slots[: max(1, n // 3)]
            c.free(_ints(slots))
            m.free(slots)
        elif what == 4:
            got, want = (c.compact()[2],), (np.array([m.compact()]),)
        else:
            starts = np.concatenate(([0], np.cumsum(rng.integers(0, 5, n))))
            first = rng.integers(0, page, n)
            got = c.locate(_ints(slots), _ints(starts), int(starts[-1]) + 1, first=_ints(first), prefix=0)
            want = m.locate(slots, starts.tolist(), int(starts[-1]) + 1, first=first, prefix=0)
        for x, y in zip(got, want):
            assert np.array_equal(x.cpu().numpy(), y), (step, what)
        _compare(c, m, f"step {step}, call {what}")
        assert lb.device_status() == m.status, (step, what)
        m.status = 0


def test_extend_refuses_a_shared_last_page(cm):
    """Tables whose partly filled last page two slots hold (not made by fork)."""
    from latent_binary_factorization_b200 import littlebit as lb
    c, m = _pair(cm, 8, 8, 2, 4, [(1, 8)])
    for t in (c, m):
        t.table[0, 0], t.table[1, 0], t.refs[3] = 3, 3, 2
        t.length[0] = t.length[1] = 5
    where, positions = c.extend(_ints([0, 1]), _ints([0, 1, 2]), 2)
    assert where.tolist() == [-1, -1] and positions.tolist() == [-1, -1]
    _compare(c, m, "shared")
    assert lb.device_status() == orc.INDEX


def test_lists_that_descend_are_cut(cm):
    """starts out of order or past the tokens: reported, and nothing outside the tables is touched."""
    from latent_binary_factorization_b200 import littlebit as lb
    c, _ = _pair(cm, 64, 8, 4, 16, [(1, 8)])
    where, positions = c.extend(_ints([0, 1, 2]), _ints([0, 9, 4, 400]), 12)
    assert lb.device_status() & orc.INDEX
    assert int(where.max()) < 64 * 8
    c.locate(_ints([0, 1, 2]), _ints([-7, 9, 4, 400]), 12)
    lb.device_status()


@pytest.mark.parametrize("order", ["phr", "prh", "hpr", "wide"])
def test_fork_compact_and_copy_in_every_order(cm, order):
    planes = [_plane(12, 3, 16, 64, torch.float16, order, 40), _plane(12, 1, 16, 192, torch.bfloat16, "phr", 41)]
    c = cm.Cache(planes, torch.full((4, 3), -1, dtype=torch.int32, device="cuda"), _ints([0] * 4), _ints([0] * 12))
    m = orc.Model(12, 16, 4, 3, [planes[0].cpu().numpy().copy(), planes[1].view(torch.int16).cpu().numpy().copy()])

    def same():
        assert np.array_equal(planes[0].cpu().numpy(), m.planes[0])
        assert np.array_equal(planes[1].view(torch.int16).cpu().numpy(), m.planes[1])

    for t, f in ((c, _ints), (m, list)):
        t.extend(f([0, 1]), f([0, 37, 60]), 60)
        t.fork(f([0, 1]), f([2, 3]))
        t.free(f([0]))
    same()
    c.copy(_ints([5, -1, 0]), _ints([11, -1, 10]))
    for p in m.planes:
        p[11], p[10] = p[5], p[0]
    same()
    # into new tables first: the cache's own stay as they are, then in place
    old = c.table.clone(), c.refs.clone()
    table, refs, count = c.compact(into=True)
    assert torch.equal(c.table, old[0]) and torch.equal(c.refs, old[1])
    n = m.compact()
    assert int(count) == n and np.array_equal(table.cpu().numpy(), m.table) and np.array_equal(refs.cpu().numpy(), m.refs)
    same()
    c.compact()
    assert torch.equal(c.table, table) and torch.equal(c.refs, refs)
    same()


def test_many_planes(cm):
    """More planes than one launch takes."""
    c, m = _pair(cm, 6, 8, 3, 4, [(1, 8 * (1 + i % 3)) for i in range(150)])
    for t, f in ((c, _ints), (m, list)):
        t.extend(f([0]), f([0, 21]), 21)
        t.fork(f([0]), f([2]))
        t.free(f([0]))
        t.compact()
    _compare(c, m, "many planes")


def test_bad_pages_in_copy_are_reported(cm):
    from latent_binary_factorization_b200 import littlebit as lb
    c, m = _pair(cm, 4, 8, 1, 2, [(1, 8)])
    c.copy(_ints([0, 4, 1, -2]), _ints([-3, 1, 2, 3]))
    m.planes[0][2] = m.planes[0][1]
    _compare(c, m, "copy")
    assert lb.device_status() == orc.INDEX


def test_python_refusals(cm):
    c, _ = _pair(cm, 8, 8, 2, 4, [(2, 16), (2, 16)])
    rows = _randn((3, 2, 16), torch.float16, 50)
    where = torch.tensor([0, 1, 2], device="cuda")
    rope = cm.Rotary(16)
    bad = [
        lambda: cm.Cache([], c.table, c.length, c.refs),
        lambda: cm.Cache([c.planes[0].cpu()], c.table, c.length, c.refs),
        lambda: cm.Cache([c.planes[0].transpose(2, 3)], c.table, c.length, c.refs),
        lambda: cm.Cache(c.planes, c.table.long(), c.length, c.refs),
        lambda: cm.Cache(c.planes, c.table, c.length[:1], c.refs),
        lambda: cm.Cache(c.planes, c.table, c.length, c.refs[:4]),
        lambda: c.extend(_ints([0]).long(), _ints([0, 1]), 1),
        lambda: c.extend(_ints([0]), _ints([0]), 1),
        lambda: c.free(_ints([0, 1])[::2].cpu()),
        lambda: c.fork(_ints([0]), _ints([1, 1])),
        lambda: c.write([0], [rows.float()], where),
        lambda: c.write([0, 1], [rows], where),
        lambda: c.write([2], [rows], where),
        lambda: c.write([0], [rows[:2]], where),
        lambda: c.write([0], [rows], where.int()),
        lambda: c.write([0], [rows], where, rotated=[0]),
        lambda: c.write([0], [rows], where, rope=rope, positions=_ints([1, 2, 3]), rotated=[1]),
        lambda: c.write([0], [rows], where, q_out=rows),
        lambda: c.read([], where),
        lambda: c.read([3], where),
        lambda: cm.rotate([], _ints([1]), rope),
        lambda: cm.rotate([rows], _ints([1, 2]), rope),
        lambda: cm.rotate([rows, rows.float()], _ints([1, 2, 3]), rope),
        lambda: cm.rotate([rows.int()], _ints([1, 2, 3]), rope),
        lambda: cm.Rotary(16, bands=(0, 1, 2)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, Exception)) as e:
            f()
        assert type(e.value).__name__ in ("ValueError", "LittleBitError"), (i, e.value)


def test_nothing_to_do(cm):
    """No tokens, empty lists: calls that change nothing."""
    from latent_binary_factorization_b200 import littlebit as lb
    c, m = _pair(cm, 8, 8, 2, 4, [(2, 64), (2, 64)])
    none, slots, starts = _ints([]), _ints([0]), _ints([0, 0])
    where, positions = c.extend(slots, starts, 0)
    rows = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    rope = cm.Rotary(64)
    assert c.write([0, 1], [rows, rows], where, rope=rope, positions=positions, rotated=[0], q=rows).shape == rows.shape
    assert c.read([0], where)[0].shape == rows.shape
    assert cm.rotate([rows], none, rope)[0].shape == rows.shape
    assert c.attend(rows, slots, starts).shape == rows.shape
    c.fork(none, none)
    c.free(none)
    c.copy(none, none)
    _compare(c, m, "nothing")
    assert lb.device_status() == 0


def test_tensors_of_a_cache_are_read_only(cm):
    c, _ = _pair(cm, 8, 8, 2, 4, [(2, 16)])
    for name in ("planes", "table", "length", "refs"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))


def test_another_stream(cm):
    """Calls on a stream of the caller's: their tensors belong to it."""
    s = torch.cuda.Stream()
    c, m = _pair(cm, 16, 8, 2, 8, [(1, 16)])
    x = _randn((5, 2, 32), torch.float16, 60)
    pos, slots, starts = _ints(range(5)), _ints([1]), _ints([0, 5])
    torch.cuda.synchronize()
    y = cm.rotate([x], pos, cm.Rotary(32), stream=s)[0]
    where, _ = c.extend(slots, starts, 5, stream=s)
    s.synchronize()
    m.extend([1], [0, 5], 5)
    _compare(c, m, "stream")
    assert torch.equal(y, cm.rotate([x], pos, cm.Rotary(32))[0])
    assert where.tolist() == [0, 1, 2, 3, 4]


def test_bookkeeping_in_a_graph(cm):
    """free, fork, extend and compact captured once and replayed: each replay
    does what the calls would do on what the cache holds then."""
    c, m = _pair(cm, 64, 8, 6, 8, [(2, 16)])
    kids, parents, starts = _ints([2, 3, 4]), _ints([0, 1, 0]), _ints([0, 2, 3, 9])
    grow, one = _ints([0, 1]), _ints([0, 3, 5])

    def step(t, f):
        t.free(f([2, 3, 4]) if f is list else kids)
        t.extend(f([0, 1]) if f is list else grow, f([0, 3, 5]) if f is list else one, 5)
        t.fork(f([0, 1, 0]) if f is list else parents, f([2, 3, 4]) if f is list else kids)
        w = t.extend(f([2, 3, 4]) if f is list else kids, f([0, 2, 3, 9]) if f is list else starts, 9)
        t.compact()
        return w

    step(c, None)
    step(m, list)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        where, positions = step(c, None)
    for _ in range(4):
        g.replay()
        w, p = step(m, list)
        assert np.array_equal(where.cpu().numpy(), w) and np.array_equal(positions.cpu().numpy(), p)
        _compare(c, m, "replay")
