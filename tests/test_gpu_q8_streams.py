"""Calls on a stream that is not the current one, on the GPU: what they allocate is not memory that the current stream may still use."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ctx():
    from cross_model_kv_amd import kvmap as K
    c = K.Context(0)
    yield c
    c.close()


def test_outputs_belong_to_the_calls_stream(ctx):
    """A tensor freed on the current stream is what the next allocation there gets, while its last kernel may still be waiting to run;
    a call on another stream must not write there."""
    B, H, G, d, page, n = 2, 2, 4, 128, 64, 33
    c = ctx.q8_cache(1, 4, H, page, d)
    pages = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    start, lens = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.randn((B, 1, H * G, d), device="cuda").bfloat16()
    k = torch.randn((B, H, n, d), device="cuda").bfloat16()
    ctx.q8_write(c, k, k, pages, start)
    want, want_lse = ctx.q8_attend(c, q, pages, lens, n, lse=True)
    want_k, want_v = ctx.q8_read(c, pages, start, n)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def freed(*like):
        held = [torch.empty_like(x) for x in like for _ in range(4)]
        return {x.untyped_storage().data_ptr() for x in held}

    gone = freed(want, want_lse, want_k)
    out, lse = ctx.q8_attend(c, q, pages, lens, n, lse=True, stream=side)
    got_k, got_v = ctx.q8_read(c, pages, start, n, stream=side)
    side.synchronize()
    assert not gone & {x.untyped_storage().data_ptr() for x in (out, lse, got_k, got_v)}
    for got, ref in ((out, want), (lse, want_lse), (got_k, want_k), (got_v, want_v)):
        assert torch.equal(got, ref)
