"""The paged cache's calls at the ends of their sizes: a call of 2^27 tokens, tens of thousands of sequences, a group of thousands of
query heads, and tokens of one call that enter the same row."""

import numpy as np
import pytest

from test_gpu_paged import _attend_close, _bits, _dt, _f64, _ints
from test_gpu_paged_long import _reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ctx():
    from cross_model_kv_amd import kvmap as K
    c = K.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("dtype,d", [("f32", 128), ("bf16", 64)])
def test_append_of_the_most_tokens(ctx, dtype, d):
    """n = 2^27 rows (one row, repeated), of which 5 and the last 3 that the page table reaches count."""
    n = 1 << 27
    cache = ctx.paged_cache(1, 3, 1, 16, d, _dt(dtype))
    row = torch.randn((1, 1, 1, 1, d), device="cuda").to(_dt(dtype))
    many = row.expand(1, 1, 1, n, d)
    print(f"[paged sizes] append {dtype}", flush=True)
    ctx.paged_append(cache, many, many, _ints([[2, 0]]), _ints([7]), count=_ints([5]))
    torch.cuda.synchronize()
    assert ctx.paged_dropped() == 0
    want = torch.zeros_like(cache.k)
    want[0, 2, 0, 7:12] = row[0, 0, 0]
    assert torch.equal(cache.k, want) and torch.equal(cache.v, want)
    ctx.paged_append(cache, many, many, _ints([[2, 1]]), _ints([29]))
    torch.cuda.synchronize()
    assert ctx.paged_dropped() == n - 3
    want[0, 1, 0, 13:16] = row[0, 0, 0]
    assert torch.equal(cache.k, want) and torch.equal(cache.v, want)


@pytest.mark.parametrize("max_len", [16, 4000], ids=["own", "pieces"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_the_most_sequences(ctx, dtype, max_len):
    """65,535 sequences, most of them empty, by whole items and by pieces of thousands of them."""
    from cross_model_kv_amd import kvmap as K
    B, G, d, page = 65535, 2, 64, 16
    rng = np.random.default_rng(1)
    full = np.sort(rng.choice(B, 300, replace=False))
    lens = np.zeros(B, int)
    lens[full] = rng.integers(1, 17, 300)
    gen = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(_dt(dtype))
    cache = K.PagedCache(rand(1, 301, 1, page, d), rand(1, 301, 1, page, d))
    slots = -(-max_len // page)
    pages = np.full((B, slots), -1)
    pages[full, 0] = rng.permutation(301)[:300]
    q = rand(B, 1, G, d)
    tab = torch.from_numpy(pages.astype(np.int32)).cuda()
    print(f"[paged sizes] sequences {dtype} {max_len}", flush=True)
    out, lse = ctx.paged_attend(cache, q, tab, _ints(lens), max_len, lse=True)
    torch.cuda.synchronize()
    empty = torch.ones(B, dtype=torch.bool, device="cuda")
    empty[torch.from_numpy(full).cuda()] = False
    assert not bool(out[empty].any()) and bool((lse[empty] == -np.inf).all())
    at = torch.from_numpy(full).cuda()
    ref = _reference(cache, q[at], pages[full].tolist(), lens[full].tolist(), None)
    _attend_close(_f64(out[at]), _f64(lse[at]), ref, dtype, d, [16], False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_the_largest_groups(ctx, dtype):
    """65,536 query heads of one KV head, four drafted tokens: 262,144 rows in blocks of 32."""
    from cross_model_kv_amd import kvmap as K
    G, n_q, d, page, T = 65536, 4, 64, 16, 37
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(_dt(dtype))
    cache = K.PagedCache(rand(1, 4, 1, page, d), rand(1, 4, 1, page, d))
    q, pages = rand(1, n_q, G, d), [[2, 0, 3]]
    rot = ctx.rope_table(T, d, theta=1.0e4)
    print(f"[paged sizes] groups {dtype}", flush=True)
    out, lse = ctx.paged_attend(cache, q, _ints(pages), _ints([T]), T, rope=rot, lse=True)
    torch.cuda.synchronize()
    ref = _reference(cache, q, pages, [T], rot)
    _attend_close(_f64(out), _f64(lse), ref, dtype, d, [T], True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_that_enter_the_same_row(ctx, dtype):
    """Two sequences that share a page: every element of the row is one of the two tokens', and nothing else changes."""
    H, d, page, n = 3, 128, 16, 16
    cache = ctx.paged_cache(1, 2, H, page, d, _dt(dtype))
    k = torch.randn((2, H, n, d), device="cuda").to(_dt(dtype))
    ctx.paged_append(cache, k, -k, _ints([[1], [1]]), _ints([0, 0]), count=_ints([16, 5]))
    torch.cuda.synchronize()
    for got, new in ((cache.k, k), (cache.v, -k)):
        got, new = _bits(got), _bits(new)
        assert not got[0, 0].any() and np.array_equal(got[0, 1, :, 5:], new[0, :, 5:])
        assert ((got[0, 1, :, :5] == new[0, :, :5]) | (got[0, 1, :, :5] == new[1, :, :5])).all()
