"""The paged cache operators' cases: what is timed, on which sizes, and what the answers are.

Three operators work on a cache that is held in the model's own type, in pages of ``page`` tokens:

    k, v [L][n_pages][H][page][d]

and ``pages`` [B][max_pages] lists each sequence's pages in the order of its tokens.

append  tokens start[b] .. start[b] + count[b] of every sequence b enter their pages; with a table of rotations
        the keys come as a projection leaves them and are rotated on the way, pair (i, i + d/2) of the token at
        position p by the angle p * theta^(-2i/d).
read    those tokens come back; with a table the keys are rotated back (what the mapping works in).
attend  softmax(scale * q k^T) v over the cache with query heads in groups that share a KV head; the n_q
        queries of a sequence are its last tokens, and row i sees the keys up to its own position.  With a
        table the queries come as a projection leaves them and are rotated at their positions.

A module-level ``own`` selects the library's kernels; where it is false the same is computed from elementary
tensor operations in 32 bits (the angles, which reach 10^5, in 64).
"""

import math
import random

import torch

own = False

SPREAD = 0.6180339887498949
THETA = 1.0e6

_held = {}


def _context():
    """The library's context, made once and kept, as a serving program keeps it."""
    if "ctx" not in _held:
        from cross_model_kv_amd import kvmap
        _held["kvmap"] = kvmap
        _held["ctx"] = kvmap.Context(0)
    return _held["ctx"]


def listed():
    return [
        # one new token of one sequence enters one layer's cache: a single-user decode step, latency
        dict(name="append token", op="append", L=1, B=1, n=1, start=1000, H=8, d=128, page=64, dtype="bf16",
             ragged=False, layout="tokens", rope=True),
        # one new token each of 64 sequences of unequal lengths, one layer: a serving batch's decode step
        dict(name="append batch step", op="append", L=1, B=64, n=1, start=8000, H=8, d=128, page=64, dtype="bf16",
             ragged=True, layout="tokens", rope=True),
        # the keys and values of four prompts' projections enter one layer, rotated at far positions
        dict(name="append prompts", op="append", L=1, B=4, n=2048, start=100000, H=8, d=128, page=64, dtype="bf16",
             ragged=False, layout="tokens", rope=True),
        # a whole mapped cache of 64 layers enters the pages at once, rotated already by the mapping
        dict(name="append mapped cache", op="append", L=64, B=1, n=8192, start=0, H=8, d=128, page=64, dtype="bf16",
             ragged=False, layout="heads", rope=False),
        # prompts of unequal lengths continue sequences inside their pages, 32-bit values, small heads
        dict(name="append ragged f32", op="append", L=3, B=5, n=777, start=90, H=3, d=64, page=32, dtype="f32",
             ragged=True, layout="heads", rope=True),
        # a few tokens of one layer read back, to look at them
        dict(name="read few", op="read", L=1, B=1, n=17, start=100, H=8, d=128, page=64, dtype="bf16", ragged=False,
             rope=False),
        # a source cache of 40 layers read back with its rotation stripped, to be mapped or moved
        dict(name="read stripped", op="read", L=40, B=1, n=4096, start=0, H=8, d=128, page=64, dtype="bf16",
             ragged=False, rope=True),
        # a decode step right after a short prompt: latency
        dict(name="decode short", op="attend", B=1, n_q=1, len=130, H=8, G=2, d=128, page=64, dtype="bf16", ragged=False,
             rope=True),
        # a decode step over the mapped cache of a 32,768-token prompt, one user
        dict(name="decode long", op="attend", B=1, n_q=1, len=32768, H=8, G=8, d=128, page=64, dtype="bf16", ragged=False,
             rope=True),
        # a decode step of 64 sequences, 1 to 16,384 tokens each
        dict(name="decode batch", op="attend", B=64, n_q=1, len=16384, H=8, G=8, d=128, page=64, dtype="bf16", ragged=True,
             rope=False),
        # four drafted tokens checked at once in 16 sequences, an odd group, small heads and pages
        dict(name="draft check", op="attend", B=16, n_q=4, len=5003, H=4, G=5, d=64, page=16, dtype="bf16", ragged=True,
             rope=True),
        # 32-bit decode steps of unequal sequences, an odd number of heads, one sequence empty
        dict(name="decode f32", op="attend", B=4, n_q=1, len=7091, H=3, G=3, d=128, page=32, dtype="f32", ragged=True,
             rope=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = dict(op=rng.choice(["append", "append", "read", "attend", "attend", "attend"]), B=_log(rng, 1, 64),
                 H=rng.choice([1, 2, 3, 4, 5, 8, 16]), d=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]),
                 dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), ragged=rng.random() < 0.6, rope=rng.random() < 0.7)
        size = 2 if c["dtype"] == "f32" else 1
        if c["op"] == "attend":
            c.update(n_q=rng.choice([1, 1, 1, rng.randint(2, 16)]), len=_log(rng, 1, 131072), G=rng.randint(1, 16))
            if c["G"] * c["H"] > 128 or c["B"] * c["n_q"] * c["G"] * c["H"] * (c["len"] + c["page"]) > 64 * 64 * 16384:
                continue
            if c["B"] * c["H"] * c["len"] * c["d"] * size > 64 * 8 * 16384 * 128:
                continue
        else:
            c.update(L=_log(rng, 1, 64), n=rng.choice([1, _log(rng, 1, 8192), _log(rng, 1, 8192)]),
                     start=rng.choice([0, _log(rng, 1, 131072)]))
            if c["L"] * c["B"] * c["H"] * c["d"] * (c["n"] + c["start"] + c["page"]) * size > 64 * 8 * 128 * 8192:
                continue
            if c["op"] == "append":
                c["layout"] = rng.choice(["heads", "tokens"])
        return c


def _spread(top, B, ragged):
    """B whole numbers from top down over the range, the same for every seed; the first is top."""
    return [top - int(top * ((b * SPREAD) % 1.0)) if ragged else top for b in range(B)]


def _extent(case):
    """(start, count) of every sequence: the tokens that the call writes or reads, or (0, length)."""
    B, ragged = case["B"], case["ragged"]
    if case["op"] == "attend":
        lens = _spread(case["len"], B, ragged)
        if ragged and B > 2:
            lens[-1] = 0
        return [0] * B, lens
    start = _spread(case["start"], B, ragged)
    count = [case["n"]] * B if case["n"] == 1 else _spread(case["n"], B, ragged)
    if ragged and case["n"] > 1 and B > 2:
        count[-1] = 0
    return start, count


def _positions(case):
    """The number of positions that a table of rotations covers."""
    start, count = _extent(case)
    return max(1, max(a + (n if case["op"] == "attend" else case["n"]) for a, n in zip(start, count)))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _angles(pos, d):
    """[..., d/2] angles in 64 bits."""
    i = torch.arange(d // 2, dtype=torch.float64, device=pos.device)
    return pos.double()[..., None] * THETA ** (-2.0 * i / d)


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev).manual_seed(seed)
    host = random.Random(seed)
    L, B, H, d, P, dt = case.get("L", 1), case["B"], case["H"], case["d"], case["page"], _dtype(case)
    start, count = _extent(case)
    used = [-(-(a + n) // P) if n or case["op"] == "append" else 0 for a, n in zip(start, count)]
    n_pages, max_pages = sum(used) + 1, max(max(used), 1)
    ids = list(range(n_pages))
    host.shuffle(ids)
    rows, at = [], 0
    for u in used:
        rows.append(ids[at:at + u] + [-1] * (max_pages - u))
        at += u
    s = dict(op=case["op"], case=case, pages=torch.tensor(rows, dtype=torch.int32, device=dev))

    def drawn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # what the pages hold before the call
    chan_k = torch.exp(0.5 * drawn(L, 1, H, 1, d))
    chan_v = torch.exp(0.5 * drawn(L, 1, H, 1, d))
    s["k"] = torch.zeros((L, n_pages, H, P, d), dtype=dt, device=dev)
    s["v"] = torch.zeros((L, n_pages, H, P, d), dtype=dt, device=dev)
    if case["op"] != "append" or case["start"]:
        for l in range(L):
            s["k"][l] = (drawn(n_pages, H, P, d) * chan_k[l]).to(dt)
            s["v"][l] = (drawn(n_pages, H, P, d) * chan_v[l]).to(dt)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    if case["op"] == "attend":
        s["q"] = (1.5 * drawn(B, case["n_q"], H * case["G"], d)).to(dt)
        s["lens"] = ints(count)
    else:
        s["start"], s["n"] = ints(start), case["n"]
        s["count"] = ints(count) if case["ragged"] and case["n"] > 1 else None
    if case["op"] == "append":
        if case["layout"] == "tokens":   # the two parts of one projection's output
            both = drawn(L, B, case["n"], 2 * H, d)
            both = (both * torch.cat([chan_k, chan_v], 2).transpose(2, 3)).to(dt)
            s["new_k"], s["new_v"] = both[:, :, :, :H].transpose(2, 3), both[:, :, :, H:].transpose(2, 3)
        else:
            s["new_k"] = (drawn(L, B, H, case["n"], d) * chan_k).to(dt)
            s["new_v"] = (drawn(L, B, H, case["n"], d) * chan_v).to(dt)
        # the tokens that enter, known on the host where the lengths are: (sequence, its token of this call)
        s["enter"] = torch.cat([torch.stack([torch.full((n,), b), torch.arange(n)]) for b, n in enumerate(count)], 1).to(dev)
    if own:
        ctx = _context()
        s["cache"] = _held["kvmap"].PagedCache(s["k"], s["v"])
        s["table"] = ctx.rope_table(_positions(case), d, theta=THETA) if case["rope"] else None
        if case["op"] == "attend":
            ctx.paged_reserve(s["cache"], B, case["n_q"], H * case["G"], case["len"])
    elif case["rope"]:
        a = _angles(torch.arange(_positions(case), device=dev), d)
        s["table"] = torch.stack([a.cos(), a.sin()], -1).float()
    return s


# ---- the plain forms -------------------------------------------------------------------

def _rotated(x, cs):
    """x [..., d] in 32 bits, its pairs (i, i + d/2) turned by the angles whose cosines and sines are cs [..., d/2, 2]."""
    lo, hi = x.chunk(2, -1)
    c, s = cs[..., 0], cs[..., 1]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def _append(s):
    b, i = s["enter"]
    P = s["k"].shape[3]
    pos = s["start"].long()[b] + i
    ids, off = s["pages"].long()[b, pos // P], pos % P
    for name in ("k", "v"):
        x = s["new_" + name][:, b, :, i]                              # [tokens][L][H][d]
        if name == "k" and s["case"]["rope"]:
            x = _rotated(x.float(), s["table"][pos][:, None, None]).to(s["k"].dtype)
        s[name][:, ids, :, off] = x
    return {"k": s["k"], "v": s["v"]}


def _read(s):
    pages = s["pages"].long()
    i = torch.arange(s["n"], device=pages.device)
    pos = s["start"].long()[:, None] + i                              # [B][n]
    P = s["k"].shape[3]
    slot, off = (pos // P).clamp(max=pages.shape[1] - 1), pos % P
    ids = pages[torch.arange(pos.shape[0], device=pages.device)[:, None], slot].clamp(min=0)
    got = {}
    for name in ("k", "v"):
        x = s[name][:, ids, :, off]                                   # [B][n][L][H][d]
        if name == "k" and s["case"]["rope"]:
            back = s["table"][pos] * torch.tensor([1.0, -1.0], device=pos.device)
            x = _rotated(x.float(), back[:, :, None, None]).to(x.dtype)
        if s["count"] is not None:
            x = torch.where((i < s["count"][:, None])[:, :, None, None, None], x, torch.zeros((), dtype=x.dtype, device=x.device))
        got[name] = x.permute(2, 0, 3, 1, 4).contiguous()             # [L][B][H][n][d]
    return got


def _gathered(cache, pages):
    """[B][H][max_pages * page][d] in 32 bits of one layer's cache [n_pages][H][page][d]."""
    x = cache[pages]
    B, N, H, P, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, N * P, d).float()


def _attend(s):
    q, lens, pages = s["q"].float(), s["lens"].long(), s["pages"].long().clamp(min=0)
    B, n, Hq, d = q.shape
    H = s["k"].shape[2]
    G = Hq // H
    at = lens[:, None] - n + torch.arange(n, device=q.device)         # the queries' positions
    if s["case"]["rope"]:
        q = _rotated(q, s["table"][at.clamp(min=0)][:, :, None])
    k, v = _gathered(s["k"][0], pages), _gathered(s["v"][0], pages)
    t = torch.arange(k.shape[2], device=q.device)
    v = v.masked_fill_((t >= lens[:, None])[:, None, :, None], 0.0)
    rows = q.view(B, n, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, d) * (1.0 / math.sqrt(d))
    x = torch.matmul(rows, k.transpose(-1, -2))
    hidden = (t > at[..., None]).repeat_interleave(G, 1)[:, None]     # [B][1][n * G][T]
    x.masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    lse = (m + torch.log(l)).view(B, H, n, G).permute(0, 2, 1, 3).reshape(B, n, Hq)
    o = o.view(B, H, n, G, d).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, d)
    return {"out": o.to(s["q"].dtype), "lse": lse.contiguous()}


def run(s):
    if own:
        ctx, cache = _held["ctx"], s["cache"]
        if s["op"] == "append":
            ctx.paged_append(cache, s["new_k"], s["new_v"], s["pages"], s["start"], count=s["count"], rope=s["table"])
            return {"k": cache.k, "v": cache.v}
        if s["op"] == "read":
            k, v = ctx.paged_read(cache, s["pages"], s["start"], s["n"], count=s["count"], rope=s["table"])
            return {"k": k, "v": v}
        out, lse = ctx.paged_attend(cache, s["q"], s["pages"], s["lens"], s["case"]["len"], rope=s["table"], lse=True)
        return {"out": out, "lse": lse}
    return {"append": _append, "read": _read, "attend": _attend}[s["op"]](s)


def work(case):
    start, count = _extent(case)
    B, H, d = case["B"], case["H"], case["d"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attend":
        n, Hq = case["n_q"], case["H"] * case["G"]
        seen = sum(max(0, l - n + i + 1) for l in count for i in range(n))
        turned = sum(min(l, n) for l in count) if case["rope"] else 0
        return {"bytes": 2 * sum(count) * H * d * size + 2 * B * n * Hq * d * size + 4 * B * n * Hq + 4 * d * turned,
                "flops": 4 * seen * Hq * d + 3 * turned * Hq * d}
    L, tokens = case["L"], sum(count)
    moved = tokens if case["op"] == "append" else B * case["n"]   # rows past a sequence's count read back as zeros
    turned = tokens if case["rope"] else 0
    return {"bytes": 2 * L * H * d * size * (moved + tokens) + 4 * d * turned, "flops": 3 * L * H * d * turned}


# ---- the definitions in 64 bits ----------------------------------------------------------

def _turn(x, first, sign):
    """Rows x [..., T, d] in 64 bits of the positions first .. first + T, turned by sign times their angles."""
    h = x.shape[-1] // 2
    pos = torch.arange(first, first + x.shape[-2], dtype=torch.float64, device=x.device)
    freq = torch.tensor([math.pow(THETA, -i / h) for i in range(h)], dtype=torch.float64, device=x.device)
    z = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), sign * pos[:, None] * freq)
    y = torch.complex(x[..., :h].contiguous(), x[..., h:].contiguous()) * z
    return torch.cat([y.real, y.imag], -1)


def _tokens(s, name, layer, ids, upto):
    """Tokens 0 .. upto of the pages `ids` of one layer, [H][upto][d] in 64 bits."""
    return s[name][layer][ids].double().transpose(0, 1).flatten(1, 2)[:, :upto]


def exact(case, seed):
    s = prepare(case, seed)
    (start, count), P, H, d = _extent(case), case["page"], case["H"], case["d"]
    ids = [s["pages"][b, :-(-(a + n) // P)].long() for b, (a, n) in enumerate(zip(start, count))]
    if case["op"] == "append":
        got = {}
        for name in ("k", "v"):
            got[name] = s[name].double()
            for l in range(case["L"]):
                for b in range(case["B"]):
                    x = s["new_" + name][l, b, :, :count[b]].double()
                    if name == "k" and case["rope"]:
                        x = _turn(x, start[b], 1.0)
                    for at in range(start[b] // P * P, start[b] + count[b] if count[b] else 0, P):
                        first, last = max(start[b], at), min(start[b] + count[b], at + P)
                        got[name][l, ids[b][at // P], :, first - at:last - at] = x[:, first - start[b]:last - start[b]]
            s.pop("new_" + name)
        return got
    if case["op"] == "read":
        got = {n: torch.zeros((case["L"], case["B"], H, case["n"], d), dtype=torch.float64, device="cuda") for n in ("k", "v")}
        for name in got:
            for l in range(case["L"]):
                for b in range(case["B"]):
                    if count[b]:
                        skip = start[b] // P
                        x = _tokens(s, name, l, ids[b][skip:], start[b] + count[b] - skip * P)[:, start[b] - skip * P:]
                        got[name][l, b, :, :count[b]] = _turn(x, start[b], -1.0) if name == "k" and case["rope"] else x
        return got
    n, G = case["n_q"], case["G"]
    out = torch.zeros((case["B"], n, H * G, d), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], n, H * G), -math.inf, dtype=torch.float64, device="cuda")
    for b, upto in enumerate(count):
        a = max(0, n - upto)                  # rows before it see nothing
        if a == n:
            continue
        k, v = _tokens(s, "k", 0, ids[b], upto), _tokens(s, "v", 0, ids[b], upto)
        q = s["q"][b, a:].double().transpose(0, 1)                    # [Hq][rows][d]
        if case["rope"]:
            q = _turn(q, upto - n + a, 1.0)
        ahead = torch.arange(upto, device="cuda") > torch.arange(upto - n + a, upto, device="cuda")[:, None]
        for h in range(H):
            x = torch.matmul(q[h * G:(h + 1) * G].reshape(-1, d), k[h].t()).view(G, n - a, upto) / math.sqrt(d)
            x = x.masked_fill(ahead, -math.inf)
            w = torch.logsumexp(x, -1, keepdim=True)
            lse[b, a:, h * G:(h + 1) * G] = w[..., 0].t()
            o = torch.matmul(torch.exp(x - w).view(-1, upto), v[h])
            out[b, a:, h * G:(h + 1) * G] = o.view(G, n - a, d).transpose(0, 1)
    return {"out": out, "lse": lse}
