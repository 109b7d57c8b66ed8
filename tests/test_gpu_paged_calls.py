"""Calls of the paged cache in the model's own type beside its kernels' numbers: together with the mapping, what the binding and
the device refuse, graphs side by side, and the same page twice."""

import ctypes

import numpy as np
import pytest

from oracle import paged_oracle as O
from test_gpu_paged import _attend_close, _bits, _dev, _f64, _ints, _turned_close

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


def _rand(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def test_from_a_source_models_pages_to_the_targets_decode_steps(K, ctx):
    """The whole way: a source model's tokens are appended to its cache with its rotation, read back, mapped, the mapped cache is
    appended to the target model's pages, and decoded on with the target's rotation."""
    L, H, d, page, T, k = 4, 2, 64, 16, 90, 2
    src, tgt = ctx.paged_cache(L, 8, H, page, d), ctx.paged_cache(L, 8, H, page, d)
    rs, rt = ctx.rope_table(128, d, theta=1e4), ctx.rope_table(128, d, theta=1e6)
    pages, zero = _ints([[5, 2, 7, 0, 1, 3, 6]]), _ints([0])
    raw = _rand(1, 2, L, 1, H, T, d)
    ctx.paged_append(src, raw[0], raw[1], pages, zero, rope=rs)
    held_k, held_v = ctx.paged_read(src, pages, zero, T)
    # read stripped, the keys are what was appended, but for two roundings
    back, _ = ctx.paged_read(src, pages, zero, T, rope=rs)
    assert float((back.float() - raw[0].float()).abs().max()) <= 2 * 2.0 ** -8 * 1.5 * float(raw[0].float().abs().max())
    n, f = H * d, k * H * d
    sel = [[0, 1], [1, 2], [2, 3], [0, 3]]
    mk, mv = ctx.apply(held_k[:, 0].contiguous(), held_v[:, 0].contiguous(), sel, _rand(2, L, n, f, scale=f ** -0.5), _rand(3, L, n),
                       _rand(4, L, n, f, scale=f ** -0.5), _rand(5, L, n), 1e4, 1e6)
    ctx.paged_append(tgt, mk.unsqueeze(1), mv.unsqueeze(1), pages, zero)
    new, q = _rand(6, 2, L, 1, H, 1, d), _rand(7, L, 1, 1, 4 * H, d)
    for l in range(L):
        ctx.paged_append(tgt, new[0, l], new[1, l], pages, _ints([T]), layer=l, rope=rt)
        out, lse = ctx.paged_attend(tgt, q[l], pages, _ints([T + 1]), 112, layer=l, rope=rt, lse=True)
        torch.cuda.synchronize()
        kk = np.concatenate([_f64(mk[l]), O.turn(_f64(new[0, l, 0]), _f64(rt)[T])], 1)
        vv = np.concatenate([_f64(mv[l]), _f64(new[1, l, 0])], 1)
        flat = dict(k=kk.transpose(1, 0, 2)[None, :, :, None], v=vv.transpose(1, 0, 2)[None, :, :, None])  # pages of one token
        ref = O.attend(flat, _f64(q[l]), [list(range(T + 1))], [T + 1], d ** -0.5, rot=_f64(rt))
        # the appended key's rounding moves its score by half a step of at most scale * sum |q k|
        r_out, r_lse, size, prod = ref
        near = 2.0 ** -8 * prod
        assert (abs(_f64(lse) - r_lse) <= near + 1e-5 * (1 + abs(r_lse))).all()
        assert (abs(_f64(out) - r_out) <= 2.0 ** -8 * abs(r_out) + (2 * near[..., None] + 1e-4) * size).all()
    assert ctx.paged_dropped() == 0


def test_moving_a_cache_to_other_positions(K, ctx):
    """Tokens read back stripped and appended at other positions are what appending them there gives, but for one more rounding."""
    H, d, page, T = 3, 128, 32, 70
    a, b = ctx.paged_cache(1, 4, H, page, d, torch.float32), ctx.paged_cache(1, 8, H, page, d, torch.float32)
    rot = ctx.rope_table(300, d, theta=1e5)
    raw = _rand(11, 2, 1, H, T, d, dtype=torch.float32)
    ctx.paged_append(a, raw[0], raw[1], _ints([[2, 0, 3]]), _ints([0]), rope=rot)
    k, v = ctx.paged_read(a, _ints([[2, 0, 3]]), _ints([0]), T, rope=rot)
    there = _ints([[-1, -1, -1, -1, 6, 1, 4]])
    ctx.paged_append(b, k, v, there, _ints([140]), rope=rot)
    got, gv = ctx.paged_read(b, there, _ints([140]), T)
    torch.cuda.synchronize()
    r64 = _f64(rot)
    ref = np.stack([O.turn(_f64(raw[0, 0, :, i]), r64[140 + i]) for i in range(T)], 1)
    assert np.array_equal(_f64(gv[0, 0]), _f64(raw[1, 0]))
    # three turns of fp32 (6 roundings of elements at most sqrt 2 times the pair's larger one) and the tables' own, 2^-24 each
    top = np.maximum(abs(_f64(raw[0, 0])), abs(np.roll(_f64(raw[0, 0]), d // 2, -1)))
    assert (abs(_f64(got[0, 0]) - ref) <= 16 * 2.0 ** -24 * 2 * top).all()


def test_what_the_binding_refuses(K, ctx):
    c = ctx.paged_cache(2, 4, 2, 16, 64)
    pages, start = _ints([[0, 1], [2, 3]]), _ints([0, 0])
    rows = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    rot = ctx.rope_table(32, 64, theta=1e4)
    raises = lambda e, f, *a, **kw: pytest.raises(e, f, *a, **kw)
    raises(TypeError, ctx.paged_append, c, rows.float(), rows.float(), pages, start)          # not the cache's dtype
    raises(TypeError, ctx.paged_append, c, rows, rows.float(), pages, start)
    raises(ValueError, ctx.paged_append, c, rows[..., :32], rows[..., :32], pages, start)     # another head dim
    raises(ValueError, ctx.paged_append, c, rows[:1], rows[:1], pages, start)                 # another batch
    raises(ValueError, ctx.paged_append, c, rows.cpu(), rows.cpu(), pages, start)
    raises(ValueError, ctx.paged_append, c, rows.transpose(-1, -2).contiguous().transpose(-1, -2), rows, pages, start)
    raises(ValueError, ctx.paged_append, c, rows, rows, pages.long(), start)
    raises(ValueError, ctx.paged_append, c, rows, rows, pages, start[:1])
    raises(ValueError, ctx.paged_append, c, rows, rows, pages, start, rope=rot[:, :16])
    raises(ValueError, ctx.paged_append, c, rows, rows, pages, start, rope=rot.double())
    raises(K.KvmapError, ctx.paged_append, c, rows, rows, pages, start, layer=2)
    raises(K.KvmapError, ctx.paged_read, c, pages, start, 3, layer=1, n_layers=2)
    raises(K.KvmapError, ctx.paged_read, c, pages, start, 3, layer=0, n_layers=1, out_k=c.k[:1, :2, :, :3], out_v=rows[None])
    raises(TypeError, ctx.paged_attend, c, q.float(), pages, start, 20)
    raises(ValueError, ctx.paged_attend, c, q[..., :32], pages, start, 20)
    raises(ValueError, ctx.paged_attend, c, q, pages, start, 20, out=q.float())
    raises(ValueError, ctx.paged_attend, c, q, pages, start, 20, lse=torch.zeros((2, 4), device="cuda"))
    raises(K.KvmapError, ctx.paged_attend, c, q, pages, start, 33)                             # past the page table
    raises(K.KvmapError, ctx.paged_attend, c, q, pages, start, 20, rope=rot[:19])              # past the rotations
    raises(K.KvmapError, ctx.paged_attend, c, q[:, :, :3].contiguous(), pages, start, 20)      # heads that do not divide
    raises(K.KvmapError, ctx.paged_attend, c, q, pages, start, 20, out=q)
    raises(K.KvmapError, ctx.paged_attend, c, q.expand(2, 17, 4, 64), pages, start, 20)
    raises(K.KvmapError, ctx.rope_table, 0, 64, theta=1e4)
    raises(K.KvmapError, ctx.rope_table, 8, 96, theta=1e4)
    raises(K.KvmapError, ctx.rope_table, 8, 64, theta=-1.0)
    raises(K.KvmapError, ctx.rope_table, 8, 64, theta=1e4, style=K.ROPE_INTERLEAVED)
    raises(ValueError, ctx.rope_table, 8, 64, theta=1e4, out=rot)
    assert not bool(c.k.any()) and not bool(c.v.any()) and ctx.paged_dropped() == 0


def test_a_capture_without_scratch_is_refused(K):
    """The first call that cuts allocates; inside a capture it is refused, and taken once the scratch is there."""
    fresh = K.Context(0)
    c = fresh.paged_cache(1, 10, 1, 64, 64)
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    pages, lens, out = _ints([list(range(10))]), _ints([600]), torch.empty_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q += 0
        with pytest.raises(K.KvmapError):
            fresh.paged_attend(c, q, pages, lens, 640, out=out)
    fresh.paged_reserve(c, 1, 1, 1, 640)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fresh.paged_attend(c, q, pages, lens, 640, out=out)
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert not bool(out.any())
    fresh.close()


def test_two_graphs_of_two_contexts(K):
    """Graphs of different contexts replayed side by side on two streams, over and over: each has its own scratch."""
    B, H, G, d, page, T = 2, 2, 4, 64, 32, 3000
    n = -(-T // page)
    made = []
    for i in range(2):
        c = K.Context(0)
        cache = K.PagedCache(_rand(20 + i, 1, B * n, H, page, d), _rand(30 + i, 1, B * n, H, page, d))
        pages = torch.arange(B * n, dtype=torch.int32, device="cuda").view(B, n).flip(1).contiguous()
        q, lens = _rand(40 + i, B, 1, H * G, d), _ints([T, 1700])
        rot = c.rope_table(T, d, theta=1e4)
        want = c.paged_attend(cache, q, pages, lens, T, rope=rot)
        out = torch.empty_like(q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                c.paged_attend(cache, q, pages, lens, T, rope=rot, out=out)
        made.append((c, cache, pages, q, lens, rot, want, out, g, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for m in made:
            m[7].zero_()
        torch.cuda.synchronize()
        for m in made:
            with torch.cuda.stream(m[9]):
                m[8].replay()
        torch.cuda.synchronize()
        for m in made:
            assert torch.equal(m[6], m[7])
    for m in made:
        m[0].close()


def test_a_page_in_several_slots_and_sequences(K, ctx):
    """Sequences that share a prompt's pages, and a page listed twice in one: attention and reads take tables as they are."""
    H, G, d, page = 2, 3, 128, 16
    k, k64 = _dev(np.random.default_rng(1).standard_normal((1, 5, H, page, d)), "bf16")
    v, v64 = _dev(np.random.default_rng(2).standard_normal((1, 5, H, page, d)), "bf16")
    cache, o = K.PagedCache(k, v), dict(k=k64, v=v64)
    pages, lens = [[0, 1, 2, 2, 2], [0, 1, 3, 0, 0], [4, 4, 4, 4, 4]], [75, 40, 80]
    q, q64 = _dev(np.random.default_rng(3).standard_normal((3, 2, H * G, d)), "bf16")
    rot = ctx.rope_table(80, d, theta=1e4)
    out, lse = ctx.paged_attend(cache, q, _ints(pages), _ints(lens), 80, rope=rot, lse=True)
    gk, gv = ctx.paged_read(cache, _ints(pages), _ints([0, 0, 0]), 40)
    torch.cuda.synchronize()
    _attend_close(_f64(out), _f64(lse), O.attend(o, q64, pages, lens, d ** -0.5, rot=_f64(rot)), "bf16", d, lens, True)
    rk, rv, _ = O.read(o, pages, [0, 0, 0], 40)
    assert np.array_equal(_f64(gk), rk) and np.array_equal(_f64(gv), rv)


def test_strided_rows_around_what_is_written(K, ctx):
    """Rows with gaps, repeated inputs (a stride of 0), values that are the keys; outputs leave what lies between them alone."""
    B, H, n, d, page = 2, 2, 21, 64, 16
    cache = ctx.paged_cache(1, 4, H, page, d, torch.float32)
    pages, start = _ints([[3, 0], [1, 2]]), _ints([0, 5])
    one = _rand(5, 1, H, n, d, dtype=torch.float32)
    rot = ctx.rope_table(32, d, theta=1e3)
    both = one.expand(B, H, n, d)
    ctx.paged_append(cache, both, both, pages, start, rope=rot)
    wide = torch.full((1, B, n + 2, H, d + 4), 7.0, device="cuda")
    view = lambda t: t[:, :, 1:-1, :, :d].transpose(2, 3)
    also = wide.clone()
    gk, gv = ctx.paged_read(cache, pages, start, n, rope=rot, out_k=view(wide), out_v=view(also))
    torch.cuda.synchronize()
    for b in range(B):
        assert torch.equal(gv[0, b], one[0])
        size = O.turn_size(_f64(one[0]), np.stack([_f64(rot)[i + (0, 5)[b]] for i in range(n)])) * 2
        # turned there and back: two roundings each way of elements no larger than the pair's sum
        assert (abs(_f64(gk[0, b]) - _f64(one[0])) <= 6 * 2.0 ** -24 * size + 2.0 ** -24 * abs(_f64(one[0]))).all()
    for t in (wide, also):
        t[:, :, 1:-1, :, :d] = 7.0
        assert bool((t == 7.0).all())


def test_a_table_of_ones_own(K, ctx):
    """A caller's table (angles that do not run evenly, cosines and sines scaled) is taken as it is."""
    H, d, page, n = 1, 64, 16, 16
    cache = ctx.paged_cache(1, 1, H, page, d)
    g = np.random.default_rng(9)
    a = g.uniform(0, 6.28, (n, d // 2))
    table = torch.from_numpy((1.3 * np.stack([np.cos(a), np.sin(a)], -1)).astype(np.float32)).cuda()
    k, k64 = _dev(g.standard_normal((1, H, n, d)), "bf16")
    ctx.paged_append(cache, k, k, _ints([[0]]), _ints([0]), rope=table)
    torch.cuda.synchronize()
    t64 = _f64(table)
    _turned_close(_f64(cache.k[0, 0]), O.turn(k64[0], t64), O.turn_size(k64[0], t64), "bf16", "keys")


def test_status_codes_of_the_c_calls(K, ctx):
    L = K.lib()
    c = ctx.paged_cache(1, 2, 1, 16, 64)
    n = ctypes.c_uint32(77)
    assert L.kvmap_paged_dropped(ctx._h, ctypes.byref(n), None) == K.OK and n.value == 0
    assert L.kvmap_paged_reserve(ctx._h, c.ref, 1, 1, 1, 32) == K.OK
    assert L.kvmap_paged_reserve(ctx._h, c.ref, 1, 1, 1, -1) == K.ERR_SHAPE
    r = K.Rope(1e4, -1, 0, None)
    assert L.kvmap_rope_table(ctx._h, ctypes.byref(r), 8, 64, c.c.k, None) == K.ERR_INVALID_ARGUMENT
    r = K.Rope(1e4, 0, 0, None)
    assert L.kvmap_rope_table(ctx._h, ctypes.byref(r), 8, 64, None, None) == K.ERR_INVALID_ARGUMENT
    assert L.kvmap_rope_table(ctx._h, ctypes.byref(r), 1 << 40, 64, c.c.k, None) == K.ERR_SHAPE
