"""GPU parity of attention over the paged cache against the fp64 oracle, and a
run of the cache's operators behind LittleBit projections, as a serving step
uses them."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc
from oracle import littlebit_oracle as lorc
from latent_binary_factorization_b200 import synth

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def cm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latent_binary_factorization_b200 import cache, littlebit
    littlebit.device_status()
    return cache


def _ints(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")


def _np(t):
    return t.detach().double().cpu().numpy()


def _plane(n_pages, heads, page, width, dtype, order, gen):
    def r(*shape):
        return torch.randn(shape, generator=gen).to(dtype).cuda()
    if order == "phr":
        return r(n_pages, heads, page, width)
    if order == "prh":
        return r(n_pages, page, heads, width).transpose(1, 2)
    return r(heads, n_pages, page, width).transpose(0, 1)


class Setup:
    """Sequences of given lengths (slot i: lengths[i]) in shuffled pages, the
    rows behind their ends full of NaN and infinities."""

    def __init__(self, cm, lengths, heads, width, page, dtype, order="phr", seed=0, spare=3, gain=1.0):
        gen = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lengths]
        n_pages = sum(need) + spare
        perm = torch.randperm(n_pages, generator=gen).tolist()
        planes = [_plane(n_pages, heads, page, width, dtype, order, gen) for _ in range(2)]
        planes[0].mul_(gain)
        table = np.full((len(lengths), max(need + [1]) + 1), -1)
        at = 0
        self.k, self.v = {}, {}
        for s, n in enumerate(lengths):
            pages = perm[at: at + need[s]]
            at += need[s]
            table[s, :need[s]] = pages
            for p, keep in zip(planes, (self.k, self.v)):
                rows = p[pages].transpose(0, 1).reshape(heads, -1, width)[:, :n]
                keep[s] = _np(rows)
            if n % page:
                for p, junk in zip(planes, (float("nan"), float("inf"))):
                    p[pages[-1], :, n % page:] = junk
        for p in planes:
            p[perm[at:]] = float("nan")
        self.cache = cm.Cache(planes, torch.tensor(table, dtype=torch.int32, device="cuda"), _ints(lengths),
                              _ints([0] * n_pages))
        self.gen, self.dtype, self.width = gen, dtype, width

    def q(self, tokens, heads):
        return torch.randn((tokens, heads, self.width), generator=self.gen).to(self.dtype).cuda()

    def check(self, got, q, slots, starts, prefix=-1, scale=None):
        out, reach, size = orc.attend(_np(q), self.k.__getitem__, self.v.__getitem__, slots, starts, prefix, scale)
        tol = orc.attend_tolerance(out, reach, size, HALF_STEP[self.dtype], self.width)
        a, b = int(starts[0]), int(starts[-1])
        off = np.abs(_np(got) - out)[a:b]
        assert np.isfinite(off).all()
        assert (off <= tol[a:b]).all(), f"{float((off / tol[a:b]).max()):.2f} times the tolerance"


CASES = [
    # lengths (prefix last), new tokens, query heads, heads, page, with prefix
    ([1], [1], 1, 1, 8, False),                              # one key
    ([0, 5], [1], 1, 1, 8, True),                            # nothing of its own yet
    ([1, 0], [1], 2, 1, 16, True),                           # an empty prefix
    ([0, 0], [1], 2, 2, 16, True),                           # nothing at all: zeros
    ([63, 64, 65, 200, 7], [1, 1, 1, 1], 8, 2, 16, True),
    ([15, 16, 17, 129, 1000], [1, 1, 1, 1], 4, 4, 32, True),
    ([300, 1, 0, 77], [1, 1, 1, 1], 7, 1, 64, False),
    ([40, 50, 60, 300], [3, 0, 5], 8, 2, 8, True),           # several tokens, one sequence with none
    ([40, 200, 31], [40, 130, 1], 16, 2, 128, False),        # prompts: tokens see the ones before them
    ([5, 9, 700], [5, 9], 64, 8, 256, True),
    ([3, 70, 90], [7, 70], 6, 2, 16, True),                  # more new tokens than the slot holds: the first see the prefix alone
    ([2000, 1500, 2600], [1, 1], 32, 4, 16, True),
    ([600], [600], 4, 1, 1024, False),
    ([500, 900], [4], 8, 1, 16, True),                       # two tiles of the few-rows kernel
    ([1100, 3], [9], 16, 1, 32, True),                       # 144 rows: a wide tile, a short prefix
    ([0, 400, 0, 300, 200], [0, 33, 0, 70], 8, 2, 64, True), # empty sequences between others
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("width", [64, 128])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attend(cm, case, width, dtype):
    lengths, new, hq, h, page, with_prefix = CASES[case]
    s = Setup(cm, lengths, h, width, page, dtype, order=("phr", "prh", "hpr")[case % 3], seed=case)
    n = len(new)
    starts = np.concatenate(([0], np.cumsum(new)))
    q = s.q(int(starts[-1]), hq)
    prefix = len(lengths) - 1 if with_prefix else -1
    got = s.cache.attend(q, _ints(range(n)), _ints(starts), prefix=prefix, most_q=max(new))
    s.check(got, q, list(range(n)), starts, prefix)
    again = s.cache.attend(q, _ints(range(n)), _ints(starts), prefix=prefix, most_q=max(new))
    assert torch.equal(got, again)


@pytest.mark.parametrize("n,most", [(300, 1), (300, 4), (300, 64), (900, 1), (900, 12)])
def test_attend_many_sequences(cm, n, most):
    """More sequences than a block of either kernel has threads, in another order than their slots, some of them padding."""
    rng = np.random.default_rng(most)
    lengths = rng.integers(0, 40, n).tolist() + [150]
    s = Setup(cm, lengths, 1, 64, 8, torch.float16, seed=9)
    slots = rng.permutation(n)
    slots[rng.random(n) < 0.1] = -1
    new = rng.integers(0, 2, n) * rng.integers(1, most + 1, n)
    starts = np.concatenate(([0], np.cumsum(new)))
    q = s.q(int(starts[-1]), 4)
    got = s.cache.attend(q, _ints(slots), _ints(starts), prefix=n, most_q=most)
    s.check(got, q, slots.tolist(), starts, n)


@pytest.mark.parametrize("tokens", [1, 40])
def test_rows_in_no_sequence_are_left(cm, tokens):
    s = Setup(cm, [100, 60], 2, 128, 16, torch.bfloat16, seed=3)
    q = s.q(tokens + 9, 4)
    q[:2], q[tokens + 2:] = float("nan"), float("nan")      # nothing may come of the rows outside
    out = torch.full_like(q, 7.0)
    starts = [2, tokens + 2]
    got = s.cache.attend(q, _ints([0]), _ints(starts), prefix=1, most_q=tokens, out=out)
    assert got is out
    assert (out[:2] == 7).all() and (out[tokens + 2:] == 7).all()
    s.check(out, q, [0], starts, 1)


def test_strided_queries_scales_and_planes(cm):
    """q and out as views of one projection's rows; a scale of its own, also negative; K and V planes named."""
    s = Setup(cm, [100, 260], 2, 64, 16, torch.float16, seed=4)
    qkv = torch.randn((6, 12, 64), generator=s.gen).half().cuda()
    q, out = qkv[:, 2:10], torch.zeros((6, 20, 64), dtype=torch.float16, device="cuda")[:, 4:12]
    for scale in (0.3, -0.2):
        s.cache.attend(q, _ints([0]), _ints([0, 6]), prefix=1, most_q=6, scale=scale, out=out)
        s.check(out, q, [0], [0, 6], 1, scale)
    s.cache.attend(q, _ints([0]), _ints([0, 6]), k=1, v=0, prefix=1, most_q=6, out=out)
    s.k, s.v = s.v, s.k
    s.check(out, q, [0], [0, 6], 1)


@pytest.mark.parametrize("tokens", [1, 200])
def test_large_scores(cm, tokens):
    """Scores of hundreds, whose maximum comes late or early: no overflow, and the small weights vanish."""
    s = Setup(cm, [400, 900], 2, 128, 32, torch.bfloat16, seed=5, gain=40.0)
    q = s.q(tokens, 8)
    got = s.cache.attend(q, _ints([0]), _ints([0, tokens]), prefix=1, most_q=tokens)
    s.check(got, q, [0], [0, tokens], 1)


@pytest.mark.parametrize("tokens", [1, 60])
@pytest.mark.parametrize("where", ["q", "k", "inf"])
def test_non_finite_scores(cm, where, tokens):
    """A NaN of a query spoils its own row alone, a NaN or an infinity of a key that is seen every row that sees it."""
    s = Setup(cm, [300, 200], 1, 64, 16, torch.float16, seed=12)
    q = s.q(tokens, 4).abs() + 0.5                           # so that the infinite key's scores are +inf
    if where == "q":
        q[0, 1, 3] = float("nan")
    else:
        page, row = int(s.cache.table[0, 2]), 5               # own key 37: before every new token
        s.cache.planes[0][page, 0, row, 7] = float("nan") if where == "k" else float("inf")
    got = _np(s.cache.attend(q, _ints([0]), _ints([0, tokens]), prefix=1, most_q=tokens))
    bad = np.isnan(got)
    if where == "q":
        assert bad[0, 1].all() and bad.sum() == bad[0, 1].size
    else:
        assert bad.all()


def test_equal_work_in_two_calls_at_once(cm):
    """Two calls on two streams, each with its own work memory."""
    s = Setup(cm, [500, 300, 700], 2, 128, 32, torch.bfloat16, seed=13)
    qs = [s.q(80, 8), s.q(2, 8)]
    lists = [(_ints([0, 1]), _ints([0, 40, 80]), 40), (_ints([0, 1]), _ints([0, 1, 2]), 1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs = [s.cache.attend(q, a, b, prefix=2, most_q=m, stream=st) for q, (a, b, m), st in zip(qs, lists, streams)]
    torch.cuda.synchronize()
    for out, q, (a, b, m) in zip(outs, qs, lists):
        s.check(out, q, [0, 1], b.tolist(), 2)


@pytest.mark.parametrize("tokens", [1, 20])
def test_a_long_cache(cm, tokens):
    """More rows than 2^31 bytes of a plane span: offsets need 64 bits, in both kernels."""
    page, width, n_pages = 1024, 128, 9000
    planes = [torch.empty((n_pages, 1, page, width), dtype=torch.float16, device="cuda") for _ in range(2)]
    pages = [n_pages - 1, 3, n_pages - 2]
    gen = torch.Generator().manual_seed(6)
    k, v = (torch.randn((3, 1, page, width), generator=gen).half().cuda() for _ in range(2))
    for p, x in zip(planes, (k, v)):
        p[pages] = x
    c = cm.Cache(planes, torch.tensor([pages], dtype=torch.int32, device="cuda"), _ints([2500]), _ints([0] * n_pages))
    q = torch.randn((tokens, 4, width), generator=gen).half().cuda()
    got = c.attend(q, _ints([0]), _ints([0, tokens]), most_q=tokens)
    flat = [_np(x).reshape(1, -1, width)[:, :2500] for x in (k, v)]
    out, reach, size = orc.attend(_np(q), lambda s: flat[0], lambda s: flat[1], [0], [0, tokens])
    assert (np.abs(_np(got) - out) <= orc.attend_tolerance(out, reach, size, HALF_STEP[torch.float16], width)).all()


@pytest.mark.parametrize("lengths,tokens,hq,h,width,page", [([2500, 1100], 2500, 8, 1, 64, 16),
                                                            ([5000, 0], 4000, 16, 4, 128, 64)])
def test_a_long_prompt(cm, lengths, tokens, hq, h, width, page):
    """A prompt of thousands of tokens, each seeing the ones before it: rows here and there against fp64."""
    s = Setup(cm, lengths, h, width, page, torch.bfloat16, seed=14)
    q = s.q(tokens, hq)
    got = s.cache.attend(q, _ints([0]), _ints([0, tokens]), prefix=1, most_q=tokens)
    for t in (0, 1, 15, 16, 31, 127, 128, 1000, 1999, tokens - 2, tokens - 1):
        seen = lengths[0] - tokens + t + 1
        k, v = ({0: x[0][:, :seen], 1: x[1]}.__getitem__ for x in (s.k, s.v))
        out, reach, size = orc.attend(_np(q[t: t + 1]), k, v, [0], [0, 1], 1)
        tol = orc.attend_tolerance(out, reach, size, HALF_STEP[torch.bfloat16], width)
        assert (np.abs(_np(got[t: t + 1]) - out) <= tol).all(), t


@pytest.mark.parametrize("most", [1, 100])
def test_bad_pages_and_slots_are_reported(cm, most):
    """Page numbers and slots outside the cache: the other sequences' outputs stay right."""
    from latent_binary_factorization_b200 import littlebit as lb
    s = Setup(cm, [100, 130, 50], 2, 64, 16, torch.float16, seed=7)
    good = s.cache.table[0].clone()
    s.cache.table[0, 1] = 100000
    s.cache.table[0, 2] = -4
    starts = [0, most, 2 * most, 3 * most]
    q = s.q(3 * most, 2)
    lb.device_status()
    got = s.cache.attend(q, _ints([0, 1, 3]), _ints(starts), prefix=2, most_q=most)
    assert lb.device_status() == orc.INDEX
    s.check(got[most:2 * most], q[most:2 * most], [1], [0, most], 2)
    s.k[3], s.v[3] = s.k[0][:, :0], s.v[0][:, :0]            # a slot outside: nothing of its own
    s.check(got[2 * most:], q[2 * most:], [3], [0, most], 2)
    s.cache.table[0] = good


def test_two_graphs_and_a_growing_cache(cm):
    """Attention captured twice, replayed on two streams at once while the cache
    has grown since the capture: each has its own work memory."""
    s = Setup(cm, [40, 30, 500], 4, 64, 16, torch.float16, seed=8)
    q = s.q(2, 8)
    slots, starts = _ints([0, 1]), _ints([0, 1, 2])
    s.cache.attend(q, slots, starts, prefix=2)
    graphs, outs, streams = [], [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.cache.attend(q, slots, starts, prefix=2))
        graphs.append(g)
        streams.append(torch.cuda.Stream())
    s.cache.length[0], s.cache.length[1] = 37, 9             # other lengths than at the capture
    for x in (s.k, s.v):
        x[0], x[1] = x[0][:, :37], x[1][:, :9]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        s.check(out, q, [0, 1], [0, 1, 2], 2)


def test_attend_refusals(cm):
    s = Setup(cm, [20, 30], 2, 64, 16, torch.float16, seed=1)
    q, slots, starts = s.q(1, 4), _ints([0]), _ints([0, 1])
    for f in (lambda: s.cache.attend(q.bfloat16(), slots, starts), lambda: s.cache.attend(q[:, :3], slots, starts),
              lambda: s.cache.attend(q, slots, starts, k=2), lambda: s.cache.attend(q, slots, starts, v=2),
              lambda: s.cache.attend(q, slots, starts, prefix=2), lambda: s.cache.attend(q, slots, starts, most_q=0),
              lambda: s.cache.attend(q, slots, _ints([0])), lambda: s.cache.attend(q, slots.long(), starts),
              lambda: s.cache.attend(q, slots, starts, out=q.float()), lambda: s.cache.attend(q.cpu(), slots, starts),
              lambda: s.cache.attend(q[..., :32], slots, starts)):
        with pytest.raises(Exception) as e:
            f()
        assert type(e.value).__name__ in ("ValueError", "LittleBitError")


# ------------------------------------------------------------------ together
def test_serving_run_of_a_littlebit_layer(cm):
    """A LittleBit attention layer served from the cache: a shared prompt, two
    samples forked from one continuation of it, tokens decoded one by one with
    pages compacted in between, against the layer computed whole in fp64 from
    the same projections' inputs."""
    from latent_binary_factorization_b200 import layers, littlebit as lb
    d, hq, h, width, page = 512, 8, 2, 64, 16
    shapes = {"q": (d, hq * width), "k": (d, h * width), "v": (d, h * width)}
    host = {n: synth.layer(a, b, 48, True, seed=i) for i, (n, (a, b)) in enumerate(shapes.items())}
    dev = {n: layers.upload(host[n], *shapes[n], 48) for n in shapes}
    rope = cm.Rotary(width)
    c = cm.Cache.empty([(h, width), (h, width)], 40, page, 6, 12)
    prefix = 5
    history = {s: [] for s in range(6)}                      # the layer's inputs, token by token
    gen = torch.Generator().manual_seed(0)

    def step(slots, new, shared):
        starts = np.concatenate(([0], np.cumsum(new)))
        T = int(starts[-1])
        x = torch.randn((T, d), generator=gen).half()
        q, k, v = (lb.forward(dev[n], x.cuda()).view(T, -1, width) for n in "qkv")
        where, positions = c.extend(_ints(slots), _ints(starts), T, prefix=prefix if shared else -1)
        qr = c.write([0, 1], [k, v], where, rope=rope, positions=positions, rotated=[0], q=q)
        out = c.attend(qr, _ints(slots), _ints(starts), prefix=prefix if shared else -1, most_q=max(new))
        for i, s in enumerate(slots):
            history[s] += [x[t] for t in range(starts[i], starts[i + 1])]
        # whole: every sequence from its first input on, in fp64
        for i, s in enumerate(slots):
            xs = torch.stack((history[prefix] if shared else []) + history[s]).double().numpy()
            n = len(xs)
            proj = {m: lorc.factored_forward(xs, host[m]).reshape(n, -1, width) for m in "qkv"}
            kq = {m: orc.rotate(proj[m], np.arange(n), width) for m in "qk"}
            last = new[i]
            ref, reach, size = orc.attend(kq["q"][n - last:], lambda _: kq["k"].transpose(1, 0, 2),
                                          lambda _: proj["v"].transpose(1, 0, 2), [0], [0, last])
            got = _np(out[starts[i]: starts[i + 1]])
            # the projections carry the layer's own tolerance (rel-L2 2e-3): an error of that size of q and k
            # moves a score by 2 * 2e-3 of its size, and the weights by twice that
            size_l2 = np.abs(size[..., 1]).max()
            bound = (2e-3 + 2 * 2 * 2e-3 * size_l2 + 3 * 2.0 ** -11) * np.linalg.norm(reach)
            assert np.linalg.norm(got - ref) <= bound, (s, np.linalg.norm(got - ref) / np.linalg.norm(ref))
            assert np.linalg.norm(got - ref) <= 2e-2 * np.linalg.norm(ref)

    step([prefix], [45], shared=False)                       # the shared prompt
    step([0, 1], [7, 20], shared=True)                       # two users' own prompts
    step([0, 1], [1, 1], shared=True)
    c.fork(_ints([1, 1]), _ints([2, 3]))                     # two more samples of the second
    history[2], history[3] = list(history[1]), list(history[1])
    step([0, 1, 2, 3], [1, 1, 1, 1], shared=True)
    c.free(_ints([1]))
    history[1] = []
    c.compact()
    for _ in range(3):
        step([3, 0, 2], [1, 1, 1], shared=True)
    assert lb.device_status() == 0


def test_latent_rows_in_pages(cm):
    """A K projection kept as its latent rows in the paged cache, forked and
    compacted, read back and expanded: the projection of the same inputs."""
    from latent_binary_factorization_b200 import layers, littlebit as lb
    layer = layers.upload(synth.layer(512, 256, 94, False, seed=3), 512, 256, 94)
    row = lb.latent_row_elems(layer)
    c = cm.Cache.empty([(1, row)], 12, 16, 3, 6)
    x = torch.randn((16, 512), generator=torch.Generator().manual_seed(1)).half().cuda()
    (t,) = lb.latent_forward([layer], [x])
    for a in (0, 16):
        where, _ = c.extend(_ints([0]), _ints([0, 16 if a == 0 else 5]), 16 if a == 0 else 5)
        c.write([0], [t[: where.shape[0]]], where)
    c.fork(_ints([0]), _ints([2]))
    c.free(_ints([0]))
    c.compact()
    where, positions = c.locate(_ints([2]), _ints([0, 16]), 16, first=_ints([5]))
    assert positions.tolist() == list(range(5, 21))
    (back,) = c.read([0], where)
    want = torch.cat((t[5:], t[:5]))
    assert torch.equal(back[:, 0, : layer.s], want[:, : layer.s])
    (y,) = lb.latent_expand([layer], [back[:, 0].contiguous()])
    (z,) = lb.latent_expand([layer], [want])
    assert torch.equal(y, z)
    assert lb.device_status() == 0
