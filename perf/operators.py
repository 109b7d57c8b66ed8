"""The 8-bit cache operators' cases: what is timed, on which sizes, and what the answers are.

Three operators work on one cache.  A cache is held in pages of ``page`` tokens, as e4m3 codes with one
power-of-two scale for each (layer, page, KV head), keys and values apart:

    k [L][n_pages][H][page][d]      k_scale [L][n_pages][H]
    v [L][n_pages][H][d][page]      v_scale [L][n_pages][H]     (a page of values is held dim-major)

and ``pages`` [B][max_pages] lists each sequence's pages in the order of its tokens.

write   tokens start[b] .. start[b] + count[b] of every sequence b enter their pages.  A page's scale is the
        smallest power of two 2^e (e in [-110, 119]) with amax <= 448 * 2^e over the finite values written and,
        where the page held earlier tokens of the sequence, at least the scale it had; the earlier tokens are
        rounded to the new scale.
read    those tokens come back as scale * code.
attend  softmax(scale * q k^T) v over the cache with query heads in groups that share a KV head; the n_q
        queries of a sequence are its last tokens, and row i sees the keys up to its own position.

A module-level ``own`` selects the library's kernels; where it is false the same is computed from elementary
tensor operations in 32 bits.
"""

import math
import random

import torch

own = False

E_MIN, E_MAX = -110, 119     # exponents of the scales
TOP = 448.0                  # largest e4m3 value
F8 = torch.float8_e4m3fn
SPREAD = 0.6180339887498949

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
        # one new token of one sequence enters one layer's cache: the write of a single-user decode step
        dict(name="write token", op="write", L=1, B=1, n=1, start=1000, H=8, d=128, page=64, dtype="bf16",
             ragged=False, layout="tokens"),
        # one new token each of 64 sequences of unequal lengths, one layer: a serving batch's decode step
        dict(name="write batch step", op="write", L=1, B=64, n=1, start=8000, H=8, d=128, page=64, dtype="bf16",
             ragged=True, layout="tokens"),
        # a whole mapped cache of 64 layers enters the pages at once, as the mapping writes it
        dict(name="write mapped cache", op="write", L=64, B=1, n=8192, start=0, H=8, d=128, page=64, dtype="bf16",
             ragged=False, layout="heads"),
        # prompts of unequal lengths continue sequences inside their pages, 32-bit values, small heads
        dict(name="write ragged f32", op="write", L=3, B=5, n=777, start=90, H=3, d=64, page=32, dtype="f32",
             ragged=True, layout="heads"),
        # a few tokens of one layer read back, to look at them
        dict(name="read few", op="read", L=1, B=1, n=17, start=100, H=8, d=128, page=64, dtype="bf16", ragged=False),
        # a source cache of 40 layers read back to be mapped
        dict(name="read cache", op="read", L=40, B=1, n=4096, start=0, H=8, d=128, page=64, dtype="bf16", ragged=False),
        # a decode step right after a short prompt: latency
        dict(name="decode short", op="attend", B=1, n_q=1, len=130, H=8, G=2, d=128, page=64, dtype="bf16", ragged=False),
        # a decode step over the mapped cache of a 32,768-token prompt, one user
        dict(name="decode long", op="attend", B=1, n_q=1, len=32768, H=8, G=8, d=128, page=64, dtype="bf16", ragged=False),
        # a decode step of 64 sequences, 1 to 16,384 tokens each
        dict(name="decode batch", op="attend", B=64, n_q=1, len=16384, H=8, G=8, d=128, page=64, dtype="bf16", ragged=True),
        # four drafted tokens checked at once in 16 sequences, an odd group, small heads and pages
        dict(name="draft check", op="attend", B=16, n_q=4, len=5003, H=4, G=5, d=64, page=16, dtype="bf16", ragged=True),
        # a user's question of 1,024 tokens read on top of a mapped 32,768-token prompt
        dict(name="prompt on mapped", op="attend", B=1, n_q=1024, len=33792, H=8, G=8, d=128, page=64, dtype="bf16",
             ragged=False),
        # short prompts in 32 bits, some shorter than the queries given, one sequence empty
        dict(name="prompt f32", op="attend", B=4, n_q=333, len=709, H=3, G=3, d=128, page=32, dtype="f32", ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = dict(op=rng.choice(["write", "read", "attend", "attend", "attend"]), B=_log(rng, 1, 64), H=rng.choice([1, 2, 3, 4, 5, 8, 16]),
                 d=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]),
                 dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), ragged=rng.random() < 0.6)
        if c["op"] == "attend":
            c.update(n_q=rng.choice([1, 1, rng.randint(2, 16), _log(rng, 17, 1024)]), len=_log(rng, 1, 33792), G=rng.randint(1, 16))
            if c["G"] * c["H"] > 128 or c["B"] * c["n_q"] * c["G"] * c["H"] * (c["len"] + c["page"]) > 64 * 1024 * 33792:
                continue
            if c["B"] * c["H"] * c["len"] * c["d"] > 64 * 8 * 16384 * 128:
                continue
        else:
            c.update(L=_log(rng, 1, 64), n=_log(rng, 1, 8192), start=rng.choice([0, _log(rng, 1, 8192)]))
            if c["L"] * c["B"] * c["H"] * c["d"] * c["n"] * (2 if c["dtype"] == "f32" else 1) > 64 * 8 * 128 * 8192:
                continue
            if c["L"] * c["B"] * c["H"] * c["d"] * (c["n"] + c["start"]) > 64 * 8 * 128 * 8192:
                continue
            if c["op"] == "write":
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


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, inside [E_MIN, E_MAX]."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 9 + (m > 0.875).int(), torch.full_like(x, E_MIN)).clamp(E_MIN, E_MAX)


def _power(e):
    return torch.ldexp(torch.ones((), dtype=torch.float32, device=e.device), e)


def _codes(x, scale):
    """x / scale rounded to e4m3, as codes; what is not finite becomes NaN."""
    y = (x / scale).clamp(-TOP, TOP).to(F8).view(torch.uint8)
    return torch.where(torch.isfinite(x), y, torch.full_like(y, 0x7F))


def _values(codes):
    return codes.view(F8).float()


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev).manual_seed(seed)
    host = random.Random(seed)
    L, B, H, d, P, dt = case.get("L", 1), case["B"], case["H"], case["d"], case["page"], _dtype(case)
    start, count = _extent(case)
    used = [-(-(a + n) // P) if n or case["op"] == "write" else 0 for a, n in zip(start, count)]
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
    k = torch.zeros((L, n_pages, H, P, d), dtype=torch.uint8, device=dev)
    v = torch.zeros((L, n_pages, H, d, P), dtype=torch.uint8, device=dev)
    ks = torch.zeros((L, n_pages, H), dtype=torch.float32, device=dev)
    vs = torch.zeros((L, n_pages, H), dtype=torch.float32, device=dev)
    chan_k = torch.exp(0.5 * drawn(L, 1, H, 1, d))
    chan_v = torch.exp(0.5 * drawn(L, 1, H, 1, d))
    if case["op"] != "write" or case["start"]:
        for l in range(L):
            x = drawn(n_pages, H, P, d) * chan_k[l]
            ks[l] = _power(_exponent(x.abs().amax((-1, -2))))
            k[l] = _codes(x, ks[l][..., None, None])
            x = drawn(n_pages, H, P, d) * chan_v[l]
            vs[l] = _power(_exponent(x.abs().amax((-1, -2))))
            v[l] = _codes(x, vs[l][..., None, None]).transpose(-1, -2)
    s.update(k=k.view(F8), v=v.view(F8), k_scale=ks, v_scale=vs)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    if case["op"] == "attend":
        s["q"] = (1.5 * drawn(B, case["n_q"], H * case["G"], d)).to(dt)
        s["lens"] = ints(count)
    else:
        s["start"], s["n"] = ints(start), case["n"]
        s["count"] = ints(count) if case["ragged"] and case["n"] > 1 else None
    if case["op"] == "write":
        if case["layout"] == "tokens":   # the two parts of one projection's output
            both = drawn(L, B, case["n"], 2 * H, d)
            both = (both * torch.cat([chan_k, chan_v], 2).transpose(2, 3)).to(dt)
            s["new_k"], s["new_v"] = both[:, :, :, :H].transpose(2, 3), both[:, :, :, H:].transpose(2, 3)
        else:
            s["new_k"] = (drawn(L, B, H, case["n"], d) * chan_k).to(dt)
            s["new_v"] = (drawn(L, B, H, case["n"], d) * chan_v).to(dt)
        # the touched pages, known on the host where the lengths are: (sequence, its page), in order
        touched = [(b, j) for b in range(B) if count[b] for j in range(start[b] // P, (start[b] + count[b] - 1) // P + 1)]
        s["touched"] = torch.tensor(touched, dtype=torch.int64, device=dev).reshape(-1, 2).t().contiguous()
    if own:
        ctx = _context()
        s["cache"] = _held["kvmap"].Q8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] == "attend":
            ctx.q8_reserve(s["cache"], B, case["n_q"], H * case["G"], case["len"])
    return s


# ---- the plain forms -------------------------------------------------------------------

def _write_half(codes, scales, new, ids, first, start, count):
    """codes [L][n_pages][H][page][d] (a view), scales [L][n_pages][H]; new [L][B][H][n][d]; the touched pages'
    ids, their first positions, and their sequences' start and count ([touched] each)."""
    b, ids = ids
    P, n = codes.shape[3], new.shape[3]
    pos = first[:, None] + torch.arange(P, device=first.device)          # [touched][P]
    i = pos - start[:, None]
    enters = (i >= 0) & (i < count[:, None])
    held = pos < start[:, None]
    x = new[:, b[:, None], :, i.clamp(0, n - 1)].float()                 # [touched][P][L][H][d]
    x = x.permute(2, 0, 3, 1, 4)                                         # [L][touched][H][P][d]
    enters, held = enters[None, :, None, :, None], held[None, :, None, :, None]
    amax = torch.where(enters & torch.isfinite(x), x.abs(), 0.0).amax((-1, -2))
    scale = _power(_exponent(amax))
    before = torch.where(held.any(3)[..., 0], scales[:, ids], 0.0)
    scale = torch.maximum(scale, before)
    was = codes[:, ids]
    again = _codes(_values(was) * before[..., None, None], scale[..., None, None])
    codes[:, ids] = torch.where(enters, _codes(x, scale[..., None, None]), torch.where(held, again, was))
    scales[:, ids] = scale


def _write(s):
    b, j = s["touched"]
    P = s["k"].shape[3]
    ids = (b, s["pages"].long()[b, j])
    start = s["start"].long()[b]
    count = torch.full_like(start, s["n"]) if s["count"] is None else s["count"].long()[b]
    _write_half(s["k"].view(torch.uint8), s["k_scale"], s["new_k"], ids, j * P, start, count)
    _write_half(s["v"].view(torch.uint8).transpose(-1, -2), s["v_scale"], s["new_v"], ids, j * P, start, count)
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _gathered(codes, scales, pages):
    """[L][B][H][max_pages * page][d] in 32 bits of codes [L][n_pages][H][page][d] (a view)."""
    x = _values(codes.view(torch.uint8)[:, pages].contiguous()) * scales[:, pages][..., None, None]
    L, B, N, H, P, d = x.shape
    return x.permute(0, 1, 3, 2, 4, 5).reshape(L, B, H, N * P, d)


def _read(s):
    case, pages = s["case"], s["pages"].long().clamp(min=0)
    i = torch.arange(s["n"], device=pages.device)
    pos = s["start"].long()[:, None] + i
    inside = torch.ones_like(pos, dtype=torch.bool) if s["count"] is None else i < s["count"].long()[:, None]
    b = torch.arange(pos.shape[0], device=pages.device)[:, None]
    P = s["k"].shape[3]
    ids, off = pages[b, (pos // P).clamp(max=pages.shape[1] - 1)], pos % P      # [B][n]
    inside = inside[:, None, :, None]
    k = _values(s["k"].view(torch.uint8)[:, ids, :, off]) * s["k_scale"].permute(1, 0, 2)[ids][..., None]
    v = _values(s["v"].view(torch.uint8).transpose(-1, -2)[:, ids, :, off]) * s["v_scale"].permute(1, 0, 2)[ids][..., None]
    dt = _dtype(case)                                                           # [B][n][L][H][d] -> [L][B][H][n][d]
    return {"k": torch.where(inside, k.permute(2, 0, 3, 1, 4), 0.0).to(dt),
            "v": torch.where(inside, v.permute(2, 0, 3, 1, 4), 0.0).to(dt)}


def _attend(s):
    q, lens, pages = s["q"], s["lens"].long(), s["pages"].long().clamp(min=0)
    B, n, Hq, d = q.shape
    H = s["k"].shape[2]
    G = Hq // H
    k = _gathered(s["k"], s["k_scale"], pages)[0]
    v = _gathered(s["v"].transpose(-1, -2), s["v_scale"], pages)[0]
    t = torch.arange(k.shape[2], device=q.device)
    v = torch.where((t < lens[:, None])[:, None, :, None], v, 0.0)
    rows = q.float().view(B, n, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, d) * (1.0 / math.sqrt(d))
    x = torch.matmul(rows, k.transpose(-1, -2))
    at = lens[:, None] - n + torch.arange(n, device=q.device)
    hidden = (t > at[..., None]).repeat_interleave(G, 1)[:, None]                # [B][1][n * G][T]
    x.masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    lse = (m + torch.log(l)).view(B, H, n, G).permute(0, 2, 1, 3).reshape(B, n, Hq)
    o = o.view(B, H, n, G, d).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, d)
    return {"out": o.to(q.dtype), "lse": lse.contiguous()}


def run(s):
    if own:
        ctx, cache = _held["ctx"], s["cache"]
        if s["op"] == "write":
            ctx.q8_write(cache, s["new_k"], s["new_v"], s["pages"], s["start"], count=s["count"])
            return {"k": cache.k, "v": cache.v, "k_scale": cache.k_scale, "v_scale": cache.v_scale}
        if s["op"] == "read":
            k, v = ctx.q8_read(cache, s["pages"], s["start"], s["n"], count=s["count"], dtype=_dtype(s["case"]))
            return {"k": k, "v": v}
        out, lse = ctx.q8_attend(cache, s["q"], s["pages"], s["lens"], s["case"]["len"], lse=True)
        return {"out": out, "lse": lse}
    return {"write": _write, "read": _read, "attend": _attend}[s["op"]](s)


def work(case):
    start, count = _extent(case)
    B, H, d, P = case["B"], case["H"], case["d"], case["page"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attend":
        n, Hq = case["n_q"], case["H"] * case["G"]
        seen = sum(max(0, l - n + i + 1) for l in count for i in range(n))
        scales = sum(-(-l // P) for l in count)
        return {"bytes": 2 * sum(count) * H * d + 8 * scales * H + 2 * B * n * Hq * d * size + 4 * B * n * Hq,
                "flops": 4 * seen * Hq * d}
    L, tokens = case["L"], sum(count)
    touched = sum(-(-(a + n) // P) - a // P for a, n in zip(start, count) if n)
    moved = tokens if case["op"] == "write" else B * case["n"]   # rows past a sequence's count read back as zeros
    return {"bytes": 2 * L * H * d * (moved * size + tokens) + 8 * L * touched * H, "flops": 2 * L * H * d * tokens}


# ---- the definitions in 64 bits ----------------------------------------------------------

def _nearest(y):
    """The e4m3 value nearest to y (64 bits), ties to the even one; |y| <= 448."""
    m, x = torch.frexp(y.abs().clamp(min=2.0 ** -20))
    step = torch.exp2((x - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def _exact_write(case, s):
    P, (start, count), pages = case["page"], _extent(case), s["pages"].tolist()
    got = {}
    for name, dim_major in (("k", False), ("v", True)):
        codes = s[name].double()
        scales = s[name + "_scale"].double()
        new = s["new_" + name]
        rows = codes.transpose(-1, -2) if dim_major else codes
        for b in range(case["B"]):
            for j in range(start[b] // P, -(-(start[b] + count[b]) // P) if count[b] else 0):
                first, last = max(start[b], j * P), min(start[b] + count[b], (j + 1) * P)
                x = new[:, b, :, first - start[b]:last - start[b]].double()
                top = x.abs().amax((-1, -2))
                e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / TOP))
                e = torch.where(top > TOP * torch.exp2(e), e + 1, torch.where(top <= TOP * torch.exp2(e - 1), e - 1, e))
                scale = torch.exp2(torch.where(top > 0, e, float(E_MIN)).clamp(E_MIN, E_MAX))
                page, old = rows[:, pages[b][j]], first - j * P
                if old:
                    before = scales[:, pages[b][j]]
                    scale = torch.maximum(scale, before)
                    page[:, :, :old] = _nearest(page[:, :, :old] * (before / scale)[..., None, None])
                page[:, :, old:last - j * P] = _nearest((x / scale[..., None, None]).clamp(-TOP, TOP))
                scales[:, pages[b][j]] = scale
        got[name], got[name + "_scale"] = codes, scales
    return got


def _tokens(s, name, layer, ids, upto):
    """Tokens 0 .. upto of the pages `ids` of one layer, [H][upto][d] in 64 bits."""
    x = s[name][layer].view(torch.uint8)[ids].view(F8).double() * s[name + "_scale"][layer][ids].double()[..., None, None]
    x = x.transpose(-1, -2) if name == "v" else x
    return x.transpose(0, 1).flatten(1, 2)[:, :upto]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(case, s)
    (start, count), P, H, d = _extent(case), case["page"], case["H"], case["d"]
    ids = [s["pages"][b, :-(-(a + n) // P)].long() for b, (a, n) in enumerate(zip(start, count))]
    if case["op"] == "read":
        got = {n: torch.zeros((case["L"], case["B"], H, case["n"], d), dtype=torch.float64, device="cuda") for n in ("k", "v")}
        for name in got:
            for l in range(case["L"]):
                for b in range(case["B"]):
                    if count[b]:
                        got[name][l, b, :, :count[b]] = _tokens(s, name, l, ids[b], start[b] + count[b])[:, start[b]:]
        return got
    n, G = case["n_q"], case["G"]
    out = torch.zeros((case["B"], n, H * G, d), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], n, H * G), -math.inf, dtype=torch.float64, device="cuda")
    for b, upto in enumerate(count):
        a = max(0, n - upto)                  # rows before it see nothing
        if a == n:
            continue
        k, v = _tokens(s, "k", 0, ids[b], upto), _tokens(s, "v", 0, ids[b], upto)
        ahead = torch.arange(upto, device="cuda") > torch.arange(upto - n + a, upto, device="cuda")[:, None]
        for h in range(H * G):
            x = s["q"][b, a:, h].double() @ k[h // G].t() / math.sqrt(d)
            x = x.masked_fill(ahead, -math.inf)
            lse[b, a:, h] = torch.logsumexp(x, -1)
            out[b, a:, h] = torch.exp(x - lse[b, a:, h, None]) @ v[h // G]
    return {"out": out, "lse": lse}
