"""What the binding of the paged caches' calls asks of tensors, on the CPU: stand-ins that say where they lie, and calls that must
not get as far as the library."""

import types

import pytest

from cross_model_kv_amd import kvmap as K

torch = pytest.importorskip("torch")


class Tensor:
    """A contiguous device tensor's outside."""

    def __init__(self, *shape, dtype=torch.bfloat16, device=0):
        self.shape, self.dtype, self.is_cuda, self.index = torch.Size(shape), dtype, device >= 0, device
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 40

    def dim(self):
        return len(self.shape)

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()


class Refused(Exception):
    pass


@pytest.fixture
def ctx(monkeypatch):
    """A context of device 0 without a device; a call that passes the binding's checks raises Refused."""
    K._torch()
    c = object.__new__(K.Context)
    c.device, c._h = 0, None
    c._seqs, c._rows, c._rot = K.Q8SeqsC(), (K.Q8RowsC(), K.Q8RowsC()), K.RotationC()
    c._seqs_ref = c._rows_ref = None
    c._rows_ref, c._rot_ref = (None, None), "rot"
    def reached(*a):
        raise Refused
    names = ("kvmap_paged_append", "kvmap_paged_read", "kvmap_paged_attend", "kvmap_q8_write", "kvmap_q8_read", "kvmap_q8_attend",
             "kvmap_rope_table")
    monkeypatch.setattr(K, "lib", lambda: types.SimpleNamespace(**{n: reached for n in names}))
    monkeypatch.setattr(K, "_stream_of", lambda *a: 0)
    monkeypatch.setattr(K, "_stream_handle", lambda *a: 0)
    return c


def _ints(*shape, device=0):
    return Tensor(*shape, dtype=torch.int32, device=device)


def _cache(device=0):
    return types.SimpleNamespace(L=3, H=2, d=64, dtype=torch.bfloat16, index=device, ref=None, k=Tensor(3, 9, 2, 16, 64, device=device))


def _rows(ctx, kind, cache=None, k=None, v=None, **over):
    a = dict(pages=_ints(4, 5), start=_ints(4), count=_ints(4), rope=Tensor(80, 32, 2, dtype=torch.float32))
    a.update(over)
    if kind == "q8":
        a.pop("rope")
    call = ctx.paged_append if kind == "paged" else ctx.q8_write
    call(cache or _cache(), k or Tensor(2, 4, 2, 7, 64), v or Tensor(2, 4, 2, 7, 64), a.pop("pages"), a.pop("start"), **a)


@pytest.mark.parametrize("kind", ["paged", "q8"])
def test_rows_lie_on_the_contexts_device(ctx, kind):
    with pytest.raises(Refused):
        _rows(ctx, kind)
    for where in (1, -1):                                # another card, the host
        far = dict(cache=_cache(where), k=Tensor(2, 4, 2, 7, 64, device=where), v=Tensor(2, 4, 2, 7, 64, device=where),
                   pages=_ints(4, 5, device=where), start=_ints(4, device=where), count=_ints(4, device=where))
        if kind == "paged":
            far["rope"] = Tensor(80, 32, 2, dtype=torch.float32, device=where)
        for name, t in far.items():
            with pytest.raises(ValueError):
                _rows(ctx, kind, **{name: t})


@pytest.mark.parametrize("kind", ["paged", "q8"])
def test_attention_lies_on_the_contexts_device(ctx, kind):
    q = lambda device=0: Tensor(4, 1, 6, 64, device=device)
    lse = lambda device=0: Tensor(4, 1, 6, dtype=torch.float32, device=device)

    def call(cache=None, query=None, pages=None, lens=None, **over):
        a = dict(out=q(), lse=lse(), rope=Tensor(80, 32, 2, dtype=torch.float32))
        a.update(over)
        if kind == "q8":
            a.pop("rope")
        (ctx.paged_attend if kind == "paged" else ctx.q8_attend)(cache or _cache(), query or q(), pages or _ints(4, 5), lens or _ints(4), 80, **a)

    with pytest.raises(Refused):
        call()
    for where in (1, -1):
        far = dict(cache=_cache(where), query=q(where), pages=_ints(4, 5, device=where), lens=_ints(4, device=where), out=q(where),
                   lse=lse(where))
        if kind == "paged":
            far["rope"] = Tensor(80, 32, 2, dtype=torch.float32, device=where)
        for name, t in far.items():
            with pytest.raises(ValueError):
                call(**{name: t})


def test_tables_lie_on_the_contexts_device(ctx):
    with pytest.raises(Refused):
        ctx.rope_table(80, 64, theta=1e4, out=Tensor(80, 32, 2, dtype=torch.float32))
    for where in (1, -1):
        with pytest.raises(ValueError):
            ctx.rope_table(80, 64, theta=1e4, out=Tensor(80, 32, 2, dtype=torch.float32, device=where))


@pytest.mark.parametrize("kind", ["paged", "q8"])
def test_a_reads_layers(ctx, kind):
    """n_layers and the rows that are given have to agree; either says how many."""
    read = ctx.paged_read if kind == "paged" else ctx.q8_read
    rows = lambda L: Tensor(L, 4, 2, 7, 64)

    def call(**a):
        read(_cache(), _ints(4, 5), _ints(4), 7, **a)

    with pytest.raises(Refused):
        call(out_k=rows(2), out_v=rows(2), n_layers=2)
    with pytest.raises(Refused):
        call(out_k=rows(2), out_v=rows(2))
    for bad in (dict(n_layers=1, out_k=rows(2), out_v=rows(2)), dict(n_layers=2, out_k=rows(1), out_v=rows(1)),
                dict(n_layers=1, out_k=rows(2), out_v=rows(1)), dict(n_layers=2, out_k=rows(2), out_v=rows(1))):
        with pytest.raises(ValueError):
            call(**bad)
