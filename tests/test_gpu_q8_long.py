"""Attention over the 8-bit cache where every workgroup has many steps of work, on the GPU against the definition in 64 bits: loops that
go round many times, pieces that end inside an item and go on into the next one, a maximum that moves all the way.

Bounds as in test_gpu_q8.py, with the sums as they are made: a wave adds T / 16 products at most to an output, and up to 1,024 pieces
are joined, each rounded to 2^-24 of what there is; the sum of a row's weights is held in 64 bits up to the join.  A weight has
8 bits at least (bf16 calls) or 24.  Besides, the whole output: the rounding of bf16 is 2^-9 of a value in the mean square at most, 2^-8
leaves as much for everything else, and a tile of 64 tokens that was left out or counted twice would show in both bounds."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def K():
    from cross_model_kv_amd import kvmap as K
    return K


@pytest.fixture(scope="module")
def ctx(K):
    c = K.Context(0)
    yield c
    c.close()


def _cache(K, gen, lens, H, page, d, rise):
    """Random codes and scales in pages anywhere in the pool; with `rise`, dim 0 of the keys grows along every sequence."""
    F8 = torch.float8_e4m3fn
    used = [-(-t // page) for t in lens]
    n_pages, max_pages = sum(used) + 1, max(max(used), 1)
    ids = torch.randperm(n_pages, generator=gen, device="cuda").int()
    pages = torch.full((len(lens), max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, u in enumerate(used):
        pages[b, :u] = ids[at:at + u]
        at += u
    k = 16 * torch.randn((1, n_pages, H, page, d), generator=gen, device="cuda")
    power = lambda lo, hi: 2.0 ** torch.randint(lo, hi, (1, n_pages, H), generator=gen, device="cuda").float()
    ks = power(-5, -3)
    if rise:
        for b, (t, u) in enumerate(zip(lens, used)):
            if u:
                level = torch.linspace(-rise, rise, u * page, device="cuda").view(u, 1, page)
                k[0, pages[b, :u].long(), :, :, 0] = level / ks[0, pages[b, :u].long()][..., None]
    v = 16 * torch.randn((1, n_pages, H, d, page), generator=gen, device="cuda")
    return K.Q8Cache(k.clamp(-448, 448).to(F8), v.to(F8), ks, power(-6, -2)), pages


def _reference(c, q, pages, lens, scale):
    """out, lse, and per row and dim sum w |v|, per row the largest scale sum |q k| seen: [B][n][Hq](d), 64 bits."""
    B, n, Hq, d = q.shape
    H, P = c.H, c.page
    G = Hq // H
    f64 = dict(dtype=torch.float64, device="cuda")
    out, absv = torch.zeros((B, n, Hq, d), **f64), torch.zeros((B, n, Hq, d), **f64)
    lse, abss = torch.full((B, n, Hq), -np.inf, **f64), torch.zeros((B, n, Hq), **f64)
    for b in range(B):
        T = lens[b]
        if not T:
            continue
        ids = pages[b, :-(-T // P)].long()
        k = (c.k[0, ids].double() * c.k_scale[0, ids].double()[..., None, None]).transpose(0, 1).reshape(H, -1, d)[:, :T]
        v = c.v[0, ids].transpose(-1, -2).double() * c.v_scale[0, ids].double()[..., None, None]
        v = v.transpose(0, 1).reshape(H, -1, d)[:, :T]
        rows = q[b].double().view(n, H, G, d).permute(1, 2, 0, 3).reshape(H, G * n, d)
        ahead = (torch.arange(T, device="cuda") > torch.arange(T - n, T, device="cuda")[:, None]).repeat(G, 1)
        for h in range(H):
            y = (scale * (rows[h] @ k[h].t().contiguous())).masked_fill(ahead, -np.inf)
            l = torch.logsumexp(y, -1)
            w = torch.exp(y - torch.where(torch.isinf(l), 0.0, l)[:, None])
            back = lambda x: x.view(G, n, *x.shape[1:]).transpose(0, 1)
            at = (b, slice(None), slice(h * G, (h + 1) * G))
            out[at], absv[at], lse[at] = back(w @ v[h]), back(w @ v[h].abs()), back(l)
            abss[at] = back((scale * (rows[h].abs() @ k[h].t().abs().contiguous())).masked_fill(ahead, 0.0).amax(-1))
    return out, lse, absv, abss


def _check(ctx, c, q, pages, lens, dtype, where):
    T, d = max(lens), q.shape[-1]
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = ctx.q8_attend(c, q, pages, length, T, lse=True)
    again, lse2 = ctx.q8_attend(c, q, pages, length, T, lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2), where
    ro, rl, absv, abss = _reference(c, q, pages, lens, d ** -0.5)
    empty = torch.isinf(rl)
    assert (out[empty] == 0).all() and (lse[empty] == -np.inf).all(), where
    u, w, whole = (2.0 ** -8, 2.0 ** -8, 2.0 ** -8) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -24, None)
    rl = torch.where(empty, 0.0, rl)
    delta = (d + 4) * 2.0 ** -24 * abss + 8 * 2.0 ** -24 * (1 + rl.abs())
    err, lerr = (out.double() - ro).abs(), (torch.where(empty, 0.0, lse).double() - rl).abs()
    worst = float((err / (u * ro.abs() + (w + 2 * delta[..., None] + (T / 16 + 1024) * 2.0 ** -24) * absv + 1e-300)).max())
    lworst = float((lerr / (delta + 1024 * 2.0 ** -24 + 2.0 ** -24 * rl.abs())).max())
    norm = float(err.norm() / ro.norm())
    print(f"[q8 long] {where}: out err/bound {worst:.3f}, of its size {norm:.2e}, lse err/bound {lworst:.3f}", flush=True)
    assert bool(torch.isfinite(out).all()) and worst <= 1.0 and lworst <= 1.0, where
    assert whole is None or norm <= whole, where


def _lens(rng, B, top):
    x = [top] + [int(t) for t in rng.integers(1, top + 1, B - 1)]
    if B > 3:
        x[B // 2] = 0
    return x


def _queries(gen, B, n_q, Hq, d, dtype, rise):
    q = 1.5 * torch.randn((B, n_q, Hq, d), generator=gen, device="cuda")
    if rise:
        q[..., 0] = 8.0
    return q.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


DECODES = [
    # B, n_q, H, G, d, page, longest, dtype, workgroups a CU, of them at work
    (1, 1, 2, 8, 128, 64, 200001, "bf16", 3, 2),
    (96, 1, 16, 4, 64, 16, 900, "bf16", 3, 2),
    (98, 1, 16, 4, 128, 16, 900, "bf16", 3, 3),
    (24, 4, 8, 5, 128, 32, 3000, "bf16", 2, 2),
    (12, 1, 8, 3, 128, 64, 8192, "f32", 2, 2),
    (8, 3, 8, 8, 64, 128, 4096, "f32", 1, 1),
]


@pytest.mark.parametrize("rise", [0.0, 5.0])
@pytest.mark.parametrize("B,n_q,H,G,d,page,top,dtype,per_cu,at_work", DECODES)
def test_many_steps_a_workgroup(ctx, K, B, n_q, H, G, d, page, top, dtype, per_cu, at_work, rise):
    """Up to 32 rows of a KV head (q8_attend.hip): steps of 256 tokens, three at least for each workgroup."""
    rng = np.random.default_rng([2026, 881, B, n_q, H])
    lens = _lens(rng, B, top)
    assert n_q * G <= 32
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    steps = H * sum(max(1, -(-t // 256)) for t in lens)
    assert steps > 2 * per_cu * cus, "a workgroup has less to do than this test is for"
    if per_cu == 3 and cus == 256:   # the third workgroup of a CU goes where the pieces' whole steps fit better without it
        share, share2 = -(-steps // (3 * cus)), -(-steps // (2 * cus))
        assert at_work == (2 if 2 * share2 < 3 * share + share // 8 else 3)
    gen = torch.Generator(device="cuda").manual_seed(881)
    c, pages = _cache(K, gen, lens, H, page, d, rise)
    q = _queries(gen, B, n_q, H * G, d, dtype, rise)
    _check(ctx, c, q, pages, lens, dtype, f"B {B} n_q {n_q} H {H} G {G} d {d} page {page} top {top} rise {rise} {dtype}")


PROMPTS = [
    # B, n_q, H, G, d, page, longest, dtype, rows of a workgroup, workgroups a CU
    (2, 300, 16, 4, 128, 64, 9000, "bf16", 256, 1),
    (3, 700, 8, 1, 128, 16, 7000, "bf16", 256, 1),
    (16, 8, 8, 8, 128, 64, 6000, "bf16", 128, 2),
    (8, 100, 8, 2, 64, 32, 5000, "bf16", 128, 2),
    (8, 60, 8, 2, 128, 128, 4000, "f32", 128, 1),
    (8, 40, 8, 4, 64, 64, 6000, "f32", 128, 2),
]


@pytest.mark.parametrize("rise", [0.0, 5.0])
@pytest.mark.parametrize("B,n_q,H,G,d,page,top,dtype,rows,per_cu", PROMPTS)
def test_many_tiles_a_workgroup(ctx, K, B, n_q, H, G, d, page, top, dtype, rows, per_cu, rise):
    """More rows (q8_prompt.hip): tiles of 64 tokens, eight at least for each workgroup, so that each buffer of keys and values is
    read three times and more."""
    rng = np.random.default_rng([2026, 882, B, n_q, H])
    lens = _lens(rng, B, top)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    R = n_q * G
    assert R > 32 and rows == (256 if dtype == "bf16" and d == 128 and R > 128 else 128)
    blocks = -(-R // rows)
    if dtype == "bf16" and d == 128 and rows == 128:   # where two workgroups share a CU
        assert B * H * blocks * (-(-top // 64) + 5) >= 16 * cus
    tiles = 0
    for t in lens:
        for rb in range(blocks):
            last = (min((rb + 1) * rows, R) - 1) // G
            tiles += H * max(1, -(-(t - n_q + last + 1) // 64))
    assert tiles > 7 * per_cu * cus, "a workgroup has less to do than this test is for"
    gen = torch.Generator(device="cuda").manual_seed(882)
    c, pages = _cache(K, gen, lens, H, page, d, rise)
    q = _queries(gen, B, n_q, H * G, d, dtype, rise)
    _check(ctx, c, q, pages, lens, dtype, f"B {B} n_q {n_q} H {H} G {G} d {d} page {page} top {top} rise {rise} {dtype}")
