"""Cases of the paged cache's operators: rotary positions, rows written into
pages, pages forked and compacted, and attention over pages whose sequences
share a prefix.

With ``own`` false ``run`` is the plain form of an operator (elementary torch
operations, 32-bit sums, 64-bit angles); with ``own`` true it makes the calls
of ``latent_binary_factorization_b200.cache``.  ``exact`` is the operator's
definition in 64 bits.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # q and k of a 4096-wide attention layer (32 heads of 128), one new token of each of 8 sequences
        dict(name="rotary decode", op="rotary", dtype="f16", tokens=8, q_heads=32, k_heads=32, dim=128, rotary=128,
             interleaved=False, factor=1.0, bands=False, far=4096),
        # a prompt of an 8192-wide layer with grouped heads (64 and 8): interleaved pairs, half of each head,
        # stretched to a long context whose positions need 64-bit angles
        dict(name="rotary prompt", op="rotary", dtype="bf16", tokens=2048, q_heads=64, k_heads=8, dim=128, rotary=64,
             interleaved=True, factor=8.0, bands=True, far=1 << 20),
        # one decode step of 16 sequences: k rotated and written with v into pages, q rotated beside it
        dict(name="write decode", op="write", dtype="f16", tokens=16, q_heads=32, kv_heads=32, dim=128, rotary=128,
             interleaved=False, page=16, pages=256),
        # a prompt's rows of a grouped-head layer
        dict(name="write prompt", op="write", dtype="bf16", tokens=4096, q_heads=64, kv_heads=8, dim=128, rotary=128,
             interleaved=False, page=64, pages=256),
        # four samples of one prompt, in a cache of latent rows (K and V of one layer, rank 188 in rows of 192)
        dict(name="fork samples", op="fork", dtype="f16", parents=1, each=4, longest=500, grow=1, page=16, pages=512,
             layers=1, heads=1, width=192),
        # a search step over 32 layers: 8 beams kept, each continued by 8
        dict(name="fork beams", op="fork", dtype="f16", parents=8, each=8, longest=2000, grow=3, page=32, pages=1024,
             layers=32, heads=1, width=192),
        # a small cache with every other sequence gone
        dict(name="compact latents", op="compact", dtype="f16", sequences=16, longest=300, page=16, pages=512,
             layers=1, heads=1, width=192),
        # a large cache of grouped heads, 8 layers
        dict(name="compact layers", op="compact", dtype="bf16", sequences=40, longest=1500, page=32, pages=2048,
             layers=8, heads=8, width=128),
        # two users of one short system prompt: latency
        dict(name="attend two", op="attend", dtype="f16", sequences=2, q_heads=32, kv_heads=32, dim=128, prefix=512,
             longest=64, most_q=1, page=16),
        # eight long conversations over a long shared document, a K and V head for every query head
        dict(name="attend long", op="attend", dtype="f16", sequences=8, q_heads=32, kv_heads=32, dim=128,
             prefix=32000, longest=4000, most_q=1, page=16),
        # a serving batch over one prompt, 8 query heads to a K and V head
        dict(name="attend batch", op="attend", dtype="bf16", sequences=48, q_heads=64, kv_heads=8, dim=128,
             prefix=8192, longest=1000, most_q=1, page=32),
        # pieces of prompts of 16 sequences behind the shared one
        dict(name="attend pieces", op="attend", dtype="bf16", sequences=16, q_heads=64, kv_heads=8, dim=128,
             prefix=12000, longest=700, most_q=130, page=64),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "write", "fork", "compact", "attend", "attend"])
    half = rng.choice(["f16", "bf16"])
    if op == "rotary":
        dim = rng.choice([64, 96, 128, 192])
        return dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), tokens=_log(rng, 1, 2048),
                    q_heads=rng.choice([8, 14, 32, 64]), k_heads=rng.choice([1, 2, 8]), dim=dim,
                    rotary=rng.choice([dim, dim // 2, 32]), interleaved=rng.random() < 0.5,
                    factor=rng.choice([1.0, 4.0, 8.0]), bands=rng.random() < 0.5, far=_log(rng, 100, 1 << 20))
    if op == "write":
        dim = rng.choice([64, 128])
        return dict(op=op, dtype=half, tokens=_log(rng, 1, 4096), q_heads=rng.choice([16, 32, 64]),
                    kv_heads=rng.choice([1, 4, 8, 16]), dim=dim, rotary=rng.choice([dim, dim // 2]),
                    interleaved=rng.random() < 0.5, page=rng.choice([16, 32, 64, 128]), pages=256)
    if op == "fork":
        page = rng.choice([16, 32, 64])
        return dict(op=op, dtype=half, parents=_log(rng, 1, 8), each=_log(rng, 1, 8), longest=_log(rng, 20, 2000),
                    grow=_log(rng, 1, 40), page=page, pages=32768 // page, layers=_log(rng, 1, 32), heads=1,
                    width=8 * _log(rng, 4, 24))
    if op == "compact":
        return dict(op=op, dtype=half, sequences=_log(rng, 2, 40), longest=_log(rng, 20, 600),
                    page=rng.choice([16, 32, 64]), pages=_log(rng, 1800, 2048), layers=_log(rng, 1, 8),
                    heads=rng.choice([1, 4, 8]), width=rng.choice([64, 96, 128]))
    kv = rng.choice([1, 4, 8])
    return dict(op=op, dtype=half, sequences=_log(rng, 1, 64), q_heads=kv * rng.choice([1, 4, 7, 8]), kv_heads=kv,
                dim=rng.choice([64, 128]), prefix=rng.choice([0, _log(rng, 1, 12000)]), longest=_log(rng, 1, 1500),
                most_q=rng.choice([1, 1, 2, _log(rng, 2, 60)]), page=rng.choice([16, 32, 64, 128]))


def _spread(n, lo, hi):
    """n whole numbers between lo and hi, the same for every seed (the work of a case does not depend on it)."""
    return [lo + int((hi - lo + 1) * ((0.6180339887 * (i + 1)) % 1.0)) for i in range(n)]


def _lengths(c):
    """Tokens per sequence and new tokens among them (attend); every fourth sequence of a mixed batch decodes one."""
    new = [1 if i % 4 == 3 else v for i, v in enumerate(_spread(c["sequences"], max(1, c["most_q"] // 2), c["most_q"]))]
    new = new if len(new) > 1 else [c["most_q"]]
    length = [max(n, v) for n, v in zip(new, reversed(_spread(c["sequences"], 1, c["longest"])))]
    return new, length


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(counts):
    return _ints([sum(counts[:i]) for i in range(len(counts) + 1)])


def _frequencies(c):
    """Radians per token of each pair, in 64 bits."""
    i = torch.arange(0, c["rotary"], 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-i / c["rotary"])
    if c.get("bands"):  # pairs that turn often over the trained length keep their pace, slow ones are stretched
        keep = ((4096 * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f / c["factor"] * (1 - keep) + f * keep
    return f / c.get("factor", 1.0)


def _rope(c):
    from latent_binary_factorization_b200 import cache
    return cache.Rotary(c["rotary"], base=10000.0, interleaved=c["interleaved"], factor=c.get("factor", 1.0),
                        bands=(4096, 1.0, 32.0) if c.get("bands") else None)


def _tables(g, lengths, page, pages, slots):
    """Page tables of sequences in slots 0, 1, ...: pages taken in random order, as after some time of use."""
    need = [-(-n // page) for n in lengths]
    most = max(max(need), 1) + 4
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((slots, most), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(most, device="cuda")
    first = _ints([sum(need[:i]) for i in range(len(need))]).long()
    used = at[None, :] < _ints(need)[:, None]
    table[: len(need)] = torch.where(used, order[(first[:, None] + at).clamp(max=pages - 1)], table[: len(need)])
    length = torch.zeros(slots, dtype=torch.int32, device="cuda")
    length[: len(need)] = _ints(lengths)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[: sum(need)].long()] = 1
    return table, length, refs


def _handle(s):
    from latent_binary_factorization_b200 import cache
    return cache.Cache(list(s["planes"]), s["table"], s["length"], s["refs"])


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    dt = _DT[c["dtype"]]
    if c["op"] == "rotary":
        s["q"] = _normal(g, (c["tokens"], c["q_heads"], c["dim"]), dt)
        s["k"] = _normal(g, (c["tokens"], c["k_heads"], c["dim"]), dt)
        s["positions"] = torch.randint(0, c["far"], (c["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        s["frequencies"] = _frequencies(c)
        s["rope"] = _rope(c) if own else None
    elif c["op"] == "write":
        T, H, D = c["tokens"], c["kv_heads"], c["dim"]
        s["planes"] = _normal(g, (2, c["pages"], H, c["page"], D), dt)
        s["q"], s["k"], s["v"] = (_normal(g, (T, h, D), dt) for h in (c["q_heads"], H, H))
        s["where"] = torch.randperm(c["pages"] * c["page"], generator=g, device="cuda")[:T].contiguous()
        s["positions"] = torch.randint(0, 4096, (T,), generator=g, device="cuda", dtype=torch.int32)
        s["frequencies"] = _frequencies(c)
        s["table"], s["length"], s["refs"] = _tables(g, [0], c["page"], c["pages"], 1)
        s["rope"] = _rope(c) if own else None
        s["cache"] = _handle(s) if own else None
    elif c["op"] in ("fork", "compact"):
        n = c["parents"] if c["op"] == "fork" else c["sequences"]
        lengths = _spread(n, max(1, c["longest"] // 2), c["longest"])
        slots = n * (1 + c["each"]) if c["op"] == "fork" else n
        s["planes"] = _normal(g, (2 * c["layers"], c["pages"], c["heads"], c["page"], c["width"]), dt)
        s["table"], s["length"], s["refs"] = _tables(g, lengths, c["page"], c["pages"], slots)
        if c["op"] == "fork":
            s["parents"] = torch.randint(0, n, (n * c["each"],), generator=g, device="cuda", dtype=torch.int32)
            s["children"] = torch.arange(n, slots, device="cuda", dtype=torch.int32)
            s["starts"] = torch.arange(0, n * c["each"] + 1, device="cuda", dtype=torch.int32) * c["grow"]
            s["tokens"] = n * c["each"] * c["grow"]
        else:  # every other sequence has ended
            _plain_free(s, torch.arange(0, n, 2, device="cuda", dtype=torch.int32))
        s["cache"] = _handle(s) if own else None
    else:
        new, length = _lengths(c)
        B, T, H, D = c["sequences"], sum(new), c["kv_heads"], c["dim"]
        pages = sum(-(-n // c["page"]) for n in length + [c["prefix"]]) + 8
        s["planes"] = _normal(g, (2, pages, H, c["page"], D), dt)
        s["table"], s["length"], s["refs"] = _tables(g, length + [c["prefix"]], c["page"], pages, B + 1)
        s["q"] = (2.0 * _normal(g, (T, c["q_heads"], D), torch.float32)).to(dt)
        s["slots"] = torch.arange(B, device="cuda", dtype=torch.int32)
        s["starts"] = _starts(new)
        s["prefix"] = B if c["prefix"] else -1
        s["most_q"] = max(new)
        s["cache"] = _handle(s) if own else None
    return s


# ------------------------------------------------------------------ plain forms
def _plain_rotary(x, positions, frequencies, rotary, interleaved):
    angle = positions.double()[:, None] * frequencies
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = x[..., :rotary].float()
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rotary // 2], r[..., rotary // 2:])
    p, q = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((p, q), -1).flatten(-2) if interleaved else torch.cat((p, q), -1)
    return torch.cat((turned.to(x.dtype), x[..., rotary:]), -1)


def _plain_put(planes, where, rows):
    """Rows (planes, tokens, heads, width) to row `where` of the pages."""
    page = planes.shape[3]
    planes[:, where // page, :, where % page] = rows.transpose(0, 1)


def _plain_free(s, slots):
    table, length, refs, page = s["table"], s["length"], s["refs"], s["planes"].shape[3]
    i = slots.long()
    used = torch.arange(table.shape[1], device=table.device) < ((length[i] + page - 1) // page)[:, None]
    refs.scatter_add_(0, table[i].clamp(min=0).long().flatten(), -used.to(torch.int32).flatten())
    table[i] = -1
    length[i] = 0


def _plain_fork(s, parents, children):
    table, length, refs, planes = s["table"], s["length"], s["refs"], s["planes"]
    page, p, c = planes.shape[3], parents.long(), children.long()
    n, most = length[p], table.shape[1]
    full, rest = n // page, n % page
    free = torch.argsort((refs != 0).to(torch.int32), stable=True)
    fresh = free[(torch.cumsum((rest > 0).to(torch.int64), 0) - 1).clamp(min=0)]
    at = torch.arange(most, device=table.device)
    rows = torch.where((at == full[:, None]) & (rest > 0)[:, None], fresh.to(torch.int32)[:, None], table[p])
    refs.scatter_add_(0, rows.clamp(min=0).long().flatten(), (at < ((n + page - 1) // page)[:, None]).to(torch.int32).flatten())
    last = table[p].gather(1, full.clamp(max=most - 1).long()[:, None])[:, 0].clamp(min=0).long()
    some = (rest > 0).nonzero()[:, 0]
    dst, src = fresh[some], last[some]
    held = torch.arange(page, device=table.device)[:, None] < rest[some].view(-1, 1, 1, 1)
    planes[:, dst] = torch.where(held, planes[:, src], planes[:, dst])
    table[c] = rows
    length[c] = n


def _plain_extend(s, slots, starts, tokens):
    table, length, refs = s["table"], s["length"], s["refs"]
    page, i = s["planes"].shape[3], slots.long()
    n = starts[1:] - starts[:-1]
    have, want = (length[i] + page - 1) // page, (length[i] + n + page - 1) // page
    free = torch.argsort((refs != 0).to(torch.int32), stable=True)
    first = torch.cumsum(want - have, 0) - (want - have)
    at = torch.arange(table.shape[1], device=table.device)
    fresh = (at >= have[:, None]) & (at < want[:, None])
    pick = free[(first[:, None] + at - have[:, None]).clamp(0, refs.numel() - 1)]
    table[i] = torch.where(fresh, pick.to(torch.int32), table[i])
    refs.scatter_add_(0, pick.flatten(), fresh.to(torch.int32).flatten())
    length[i] += n
    t = torch.arange(tokens, device=table.device, dtype=torch.int32)
    b = torch.searchsorted(starts, t, right=True) - 1
    position = length[i][b] - n[b] + t - starts[b]
    where = table[i[b], (position // page).long()].long() * page + position % page
    return where, position


def _plain_compact(s):
    table, refs, planes = s["table"], s["refs"], s["planes"]
    live, at = refs > 0, torch.arange(refs.numel(), device=refs.device)
    count = live.sum()
    free = torch.argsort(live.to(torch.int32), stable=True)
    moves = live & (at >= count)
    to = torch.where(moves, free[(torch.cumsum(moves.to(torch.int64), 0) - 1).clamp(min=0)], at)
    src = moves.nonzero()[:, 0]
    planes[:, to[src]] = planes[:, src]
    table = torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table)
    refs = torch.zeros_like(refs).scatter_add_(0, to, torch.where(live, refs, torch.zeros_like(refs)))
    return table, refs, count.to(torch.int32).reshape(1)


def _plain_attend(s):
    c, planes, q = s["case"], s["planes"], s["q"].float()
    starts, slots, page = s["starts"].long(), s["slots"].long(), s["planes"].shape[3]
    B, most, Q = slots.numel(), s["table"].shape[1], s["most_q"]
    H, G, D = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["dim"]
    n, length = starts[1:] - starts[:-1], s["length"][slots].long()
    # queries padded to (B, Q); every sequence's pages in a row
    j = torch.arange(Q, device=q.device)
    token = (starts[:-1, None] + j).clamp(max=q.shape[0] - 1)
    x = q[token].view(B, Q, H, G, D)
    own_pages = min(most, -(-max(c["longest"], Q) // page))
    k, v = (planes[w][s["table"][slots, :own_pages].clamp(min=0).long()].transpose(1, 2).reshape(B, H, own_pages * page, D).float()
            for w in (0, 1))
    at = torch.arange(own_pages * page, device=q.device)
    held = at < length[:, None]
    v = torch.where(held[:, None, :, None], v, torch.zeros((), device=q.device))
    seen = held[:, None] & (at <= (length - n)[:, None, None] + j[None, :, None])          # B, Q, keys
    score = torch.einsum("bqhgd,bhkd->bhgqk", x, k) / math.sqrt(D)
    score = torch.where(seen[:, None, None], score, torch.full((), -math.inf, device=q.device))
    top = score.amax(-1, keepdim=True)
    if s["prefix"] >= 0:
        N = c["prefix"]
        pages = s["table"][s["prefix"], : -(-N // page)].long()
        pk, pv = (planes[w][pages].transpose(0, 1).reshape(H, -1, D)[:, :N].float() for w in (0, 1))
        ps = torch.einsum("bqhgd,hkd->bhgqk", x, pk) / math.sqrt(D)
        top = torch.maximum(top, ps.amax(-1, keepdim=True))
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(score - top)
    total, out = e.sum(-1, keepdim=True), torch.einsum("bhgqk,bhkd->bhgqd", e, v)
    if s["prefix"] >= 0:
        e = ps.sub_(top).exp_()
        total, out = total + e.sum(-1, keepdim=True), out + torch.einsum("bhgqk,hkd->bhgqd", e, pv)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    t = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(starts, t, right=True) - 1
    return out.permute(0, 3, 1, 2, 4)[b, t - starts[b]].reshape(s["q"].shape).to(s["q"].dtype)


def _bits(planes):
    """Pages as the bit patterns that they hold: copies have to be equal."""
    return planes.view(torch.int16)


def run(state):
    s, c = state, state["case"]
    if c["op"] == "rotary":
        if own:
            from latent_binary_factorization_b200 import cache
            return cache.rotate([s["q"], s["k"]], s["positions"], s["rope"])
        return [_plain_rotary(x, s["positions"], s["frequencies"], c["rotary"], c["interleaved"]) for x in (s["q"], s["k"])]
    if c["op"] == "write":
        if own:
            q = s["cache"].write([0, 1], [s["k"], s["v"]], s["where"], rope=s["rope"], positions=s["positions"],
                                 rotated=[0], q=s["q"])
            return {"planes": s["planes"], "q": q}
        q, k = (_plain_rotary(x, s["positions"], s["frequencies"], c["rotary"], c["interleaved"]) for x in (s["q"], s["k"]))
        _plain_put(s["planes"], s["where"], torch.stack((k, s["v"])))
        return {"planes": s["planes"], "q": q}
    if c["op"] == "fork":  # last step's children end, the chosen parents are continued
        if own:
            s["cache"].free(s["children"])
            s["cache"].fork(s["parents"], s["children"])
            where, positions = s["cache"].extend(s["children"], s["starts"], s["tokens"])
        else:
            _plain_free(s, s["children"])
            _plain_fork(s, s["parents"], s["children"])
            where, positions = _plain_extend(s, s["children"], s["starts"], s["tokens"])
        return {"planes": _bits(s["planes"]), "table": s["table"], "length": s["length"], "refs": s["refs"],
                "where": where, "positions": positions}
    if c["op"] == "compact":  # into new tables: the old ones stay good for work that is under way
        table, refs, count = s["cache"].compact(into=True) if own else _plain_compact(s)
        return {"planes": _bits(s["planes"]), "table": table, "refs": refs, "count": count}
    if own:
        return s["cache"].attend(s["q"], s["slots"], s["starts"], prefix=s["prefix"], most_q=s["most_q"])
    return _plain_attend(s)


# ------------------------------------------------------------------ 64 bits
def _exact_rotary(x, positions, c):
    """Each pair as a complex number, turned by e^(i angle)."""
    f = _frequencies(c)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), positions.double()[:, None] * f)[:, None]
    y, n = x.double().clone(), c["rotary"]
    first = torch.arange(0, n, 2) if c["interleaved"] else torch.arange(n // 2)
    second = first + (1 if c["interleaved"] else n // 2)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    c = case
    if c["op"] in ("fork", "compact"):
        return None  # whole numbers and copies
    s = prepare(c, seed)
    if c["op"] == "rotary":
        return [_exact_rotary(s[x], s["positions"], c) for x in ("q", "k")]
    if c["op"] == "write":
        planes, page = s["planes"].double(), c["page"]
        for plane, rows in ((0, _exact_rotary(s["k"], s["positions"], c)), (1, s["v"].double())):
            flat = planes[plane].transpose(1, 2).reshape(-1, c["kv_heads"], c["dim"])
            flat[s["where"]] = rows
            planes[plane] = flat.view(-1, page, c["kv_heads"], c["dim"]).transpose(1, 2)
        return {"planes": planes, "q": _exact_rotary(s["q"], s["positions"], c)}
    new, length = _lengths(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, first = c["q_heads"] // c["kv_heads"], 0

    def rows(slot, count, plane, head):
        pages = s["table"][slot, : -(-count // c["page"])].long()
        return s["planes"][plane][pages, head].reshape(-1, c["dim"])[:count].double()

    for h in range(c["kv_heads"]):
        pk, pv = (rows(c["sequences"], c["prefix"], w, h) for w in (0, 1))
        first = 0
        for b in range(c["sequences"]):
            k, v = (torch.cat((p, rows(b, length[b], w, h))) for w, p in ((0, pk), (1, pv)))
            q = s["q"][first: first + new[b], h * group: (h + 1) * group].double()
            score = torch.matmul(q, k.T) / math.sqrt(c["dim"])
            last = c["prefix"] + length[b] - new[b] + torch.arange(new[b], device="cuda")
            hidden = torch.arange(k.shape[0], device="cuda") > last[:, None]
            weight = torch.softmax(score.masked_fill(hidden[:, None], -math.inf), -1)
            out[first: first + new[b], h * group: (h + 1) * group] = torch.matmul(weight, v)
            first += new[b]
    return out


# ------------------------------------------------------------------ what cannot be done without
def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rotary":
        rows = c["tokens"] * (c["q_heads"] + c["k_heads"])
        return {"bytes": 2 * rows * c["dim"] * size + 4 * c["tokens"], "flops": 3 * rows * c["rotary"]}
    if c["op"] == "write":
        rows = c["tokens"] * (c["q_heads"] + 2 * c["kv_heads"])
        turned = c["tokens"] * (c["q_heads"] + c["kv_heads"])
        return {"bytes": 2 * rows * c["dim"] * size + 12 * c["tokens"], "flops": 3 * turned * c["rotary"]}
    if c["op"] in ("fork", "compact"):
        n = c["parents"] if c["op"] == "fork" else c["sequences"]
        lengths = _spread(n, max(1, c["longest"] // 2), c["longest"])
        row = 2 * c["layers"] * c["heads"] * c["width"] * size
        if c["op"] == "fork":  # the rows of each child's last page, the tables
            rest = sum(v % c["page"] for v in lengths) / n
            entries = n * c["each"] * (sum(lengths) / n / c["page"] + 1)
            return {"bytes": int(2 * n * c["each"] * rest * row + 12 * entries + 12 * n * c["each"] * c["grow"]), "flops": 0}
        live = sum(-(-v // c["page"]) for v in lengths[1::2])
        moved = live * (1 - live / c["pages"])
        return {"bytes": int(2 * moved * c["page"] * row + 8 * c["pages"] + 8 * live), "flops": 0}
    new, length = _lengths(c)
    keys = sum(length) + c["prefix"]
    pairs = sum(n * (m + c["prefix"]) - n * (n - 1) // 2 for n, m in zip(new, length))
    return {"bytes": 2 * size * keys * c["kv_heads"] * c["dim"] + 2 * size * sum(new) * c["q_heads"] * c["dim"],
            "flops": 4 * pairs * c["q_heads"] * c["dim"]}
