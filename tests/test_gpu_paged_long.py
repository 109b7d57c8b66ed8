"""Attention over the paged cache where its work is dealt out in every way: long sequences cut over many workgroups, items that
a workgroup takes whole, more items than workgroups, blocks of rows, hundreds of sequences.  Against the formula in float64 on
the device, to the tolerances of test_gpu_paged.py (a row's sums are spread over at least 4 waves, so T / 4 of them follow
one another, and the waves' and pieces' are few)."""

import numpy as np
import pytest

from test_gpu_paged import THETA, _attend_close, _dt, _f64, _ints, _table

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ctx():
    from cross_model_kv_amd import kvmap as K
    c = K.Context(0)
    yield c
    c.close()


def _turned(x, cs):
    h = x.shape[-1] // 2
    lo, hi, c, s = x[..., :h], x[..., h:], cs[..., 0], cs[..., 1]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def _reference(cache, q, pages, lens, rot):
    """out, lse, the weighted sum of |v| and the largest scale * sum |q k| of every row, in float64."""
    B, n, Hq, d = q.shape
    H, G = cache.H, Hq // cache.H
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(out)
    lse = torch.full((B, n, Hq), -np.inf, dtype=torch.float64, device="cuda")
    prod = torch.zeros_like(lse)
    for b, T in enumerate(lens):
        a = max(0, n - T)
        if a == n:
            continue
        ids = torch.tensor(pages[b][:-(-T // cache.page)], device="cuda")
        k = cache.k[0, ids].double().transpose(0, 1).flatten(1, 2)[:, :T]
        v = cache.v[0, ids].double().transpose(0, 1).flatten(1, 2)[:, :T]
        x = q[b, a:].double()
        pos = torch.arange(T - n + a, T, device="cuda")
        if rot is not None:
            x = _turned(x, rot[pos].double()[:, None])
        ahead = torch.arange(T, device="cuda") > pos[:, None, None]
        for h in range(H):
            rows = x[:, h * G:(h + 1) * G]
            y = (rows.reshape(-1, d) @ k[h].t()).view(n - a, G, T) * d ** -0.5
            y = y.masked_fill(ahead, -np.inf)
            z = torch.logsumexp(y, -1, keepdim=True)
            w = torch.exp(y - z).view(-1, T)
            lse[b, a:, h * G:(h + 1) * G] = z[..., 0]
            out[b, a:, h * G:(h + 1) * G] = (w @ v[h]).view(n - a, G, d)
            size[b, a:, h * G:(h + 1) * G] = (w @ v[h].abs()).view(n - a, G, d)
            prod[b, a:, h * G:(h + 1) * G] = (rows.abs().reshape(-1, d) @ k[h].abs().t()).amax(-1).view(n - a, G) * d ** -0.5
    return [t.cpu().numpy() for t in (out, lse, size, prod)]


def _spread(top, B):
    return [top - int(top * ((b * 0.618) % 1.0)) for b in range(B)]


CASES = [
    # what it reaches: B, n_q, H, G, lens, d, page, dtype, rope
    ("one sequence", 1, 1, 8, 8, [32768], 128, 64, "bf16", False),
    ("one sequence, turned", 1, 1, 8, 8, [32700], 128, 64, "bf16", True),
    ("pieces of many items", 70, 1, 4, 4, _spread(3000, 70), 128, 32, "bf16", False),
    ("more items than workgroups", 70, 1, 16, 2, _spread(2600, 69) + [0], 64, 16, "bf16", True),
    ("more items than workgroups, fp32", 66, 1, 16, 3, _spread(2500, 66), 128, 64, "f32", True),
    ("row blocks, more items than pieces", 40, 16, 8, 8, _spread(2100, 38) + [3, 0], 128, 64, "bf16", True),
    ("row blocks, cut", 3, 8, 2, 12, [5000, 17, 9000], 64, 32, "f32", True),
    ("row blocks, cut, bf16", 3, 8, 2, 12, [5000, 7, 9000], 128, 128, "bf16", False),
    ("whole items", 130, 1, 2, 5, _spread(1024, 129) + [0], 128, 64, "bf16", False),
    ("whole items, turned", 130, 1, 2, 5, _spread(1000, 129) + [1], 64, 16, "bf16", True),
    ("whole items, row blocks", 40, 16, 8, 8, _spread(1500, 39) + [0], 128, 64, "bf16", False),
    ("drafts", 16, 4, 4, 5, _spread(5003, 15) + [0], 64, 16, "bf16", True),
    ("drafts, fp32", 16, 4, 4, 5, _spread(5003, 15) + [2], 128, 16, "f32", True),
    ("drafts of 32 rows", 8, 4, 4, 8, _spread(6000, 8), 128, 64, "bf16", True),
    ("one long among many", 200, 1, 2, 4, [0] * 99 + [20000] + [i % 3 for i in range(100)], 128, 64, "bf16", True),
    ("one long among many, fp32", 130, 1, 2, 4, [1] * 129 + [12345], 64, 128, "f32", False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: c[0].replace(" ", "-"))
def test_attend(ctx, case):
    from cross_model_kv_amd import kvmap as K
    name, B, n_q, H, G, lens, d, page, dtype, rope = case
    gen = torch.Generator(device="cuda").manual_seed(len(name))
    rng = np.random.default_rng(len(name))
    need = [-(-l // page) for l in lens]
    n_pages = sum(need) + 1
    pages = _table(rng, n_pages, need, max(need) + 1)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(_dt(dtype))
    cache = K.PagedCache(rand(1, n_pages, H, page, d), rand(1, n_pages, H, page, d))
    q = (1.5 * rand(B, n_q, H * G, d).float()).to(_dt(dtype))
    rot = ctx.rope_table(max(lens), d, theta=THETA) if rope else None
    print(f"[paged long] {name}", flush=True)
    tab, ln = _ints(pages), _ints(lens)
    out, lse = ctx.paged_attend(cache, q, tab, ln, max(lens), rope=rot, lse=True)
    again, lse2 = ctx.paged_attend(cache, q, tab, ln, max(lens), rope=rot, lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    ref = _reference(cache, q, pages, lens, rot)
    assert _attend_close(_f64(out), _f64(lse), ref, dtype, d, [max(lens) // 4 + 64], rope, name).all()
