"""The paged cache in the model's own type on the CPU: what its calls refuse before any device work, the tensors that the
binding takes, and the kernels' registers."""

import ctypes
import os
import re
import subprocess

import pytest

from cross_model_kv_amd import kvmap as K

A = 1 << 40          # addresses that are never read
STEP = 1 << 34


def _cache(**over):
    f = dict(L=3, n_pages=10, H_kv=2, page=64, head_dim=128, dtype=K.BF16, k=A, v=A + STEP)
    f.update(over)
    return K.PagedCacheC(**f)


def _seqs(**over):
    f = dict(B=4, max_pages=5, pages=A + 4 * STEP, start=A + 5 * STEP, count=A + 6 * STEP)
    f.update(over)
    return K.Q8SeqsC(**f)


def _rows(base, L=2, B=4, H=2, n=7, d=128, **over):
    f = dict(base=base, layer_stride=B * H * n * d, seq_stride=H * n * d, head_stride=n * d, token_stride=d)
    f.update(over)
    return K.Q8RowsC(**f)


def _rot(**over):
    f = dict(table=A + 9 * STEP, n_pos=400)
    f.update(over)
    return K.RotationC(**f)


def _rows_call(**over):
    a = dict(cache=_cache(), layer0=1, n_layers=2, seqs=_seqs(), n=7, k=_rows(A + 7 * STEP), v=_rows(A + 8 * STEP), rot=_rot(),
             output=False)
    a.update(over)
    return K.validate_paged_rows(**a)


@pytest.mark.parametrize("output", [False, True])
def test_good_rows_are_taken(output):
    assert _rows_call(output=output) == K.OK
    assert _rows_call(output=output, cache=_cache(dtype=K.F32), rot=None) == K.OK
    assert _rows_call(output=output, seqs=_seqs(count=None)) == K.OK
    # the key and value parts of one projection's output [layers][B][n][2 H][d]
    s = dict(layer_stride=4 * 7 * 4 * 128, seq_stride=7 * 4 * 128, head_stride=128, token_stride=4 * 128)
    assert _rows_call(output=output, k=_rows(A + 7 * STEP, **s), v=_rows(A + 7 * STEP + 2 * 128 * 2, **s)) == K.OK


ROWS_REFUSED = [
    (dict(cache=None), K.ERR_INVALID_ARGUMENT),
    (dict(cache=_cache(k=None)), K.ERR_INVALID_ARGUMENT),
    (dict(cache=_cache(v=A + STEP + 8)), K.ERR_INVALID_ARGUMENT),
    (dict(cache=_cache(v=A + 64)), K.ERR_INVALID_ARGUMENT),                  # overlaps k
    (dict(cache=_cache(dtype=2)), K.ERR_UNSUPPORTED),
    (dict(cache=_cache(dtype=-1)), K.ERR_UNSUPPORTED),
    (dict(cache=_cache(L=0)), K.ERR_SHAPE),
    (dict(cache=_cache(n_pages=0)), K.ERR_SHAPE),
    (dict(cache=_cache(H_kv=-1)), K.ERR_SHAPE),
    (dict(cache=_cache(L=1 << 30, n_pages=1 << 30)), K.ERR_SHAPE),
    (dict(cache=_cache(page=48)), K.ERR_UNSUPPORTED),
    (dict(cache=_cache(page=256)), K.ERR_UNSUPPORTED),
    (dict(cache=_cache(head_dim=96)), K.ERR_UNSUPPORTED),
    (dict(layer0=2), K.ERR_SHAPE),
    (dict(layer0=-1), K.ERR_SHAPE),
    (dict(n_layers=0), K.ERR_SHAPE),
    (dict(layer0=0x7FFFFFFF), K.ERR_SHAPE),
    (dict(seqs=None), K.ERR_INVALID_ARGUMENT),
    (dict(seqs=_seqs(B=0)), K.ERR_SHAPE),
    (dict(seqs=_seqs(max_pages=0)), K.ERR_SHAPE),
    (dict(seqs=_seqs(max_pages=1 << 26)), K.ERR_SHAPE),
    (dict(seqs=_seqs(pages=None)), K.ERR_INVALID_ARGUMENT),
    (dict(seqs=_seqs(pages=A + 4 * STEP + 1)), K.ERR_INVALID_ARGUMENT),
    (dict(seqs=_seqs(start=None)), K.ERR_INVALID_ARGUMENT),
    (dict(seqs=_seqs(start=A + 5 * STEP + 2)), K.ERR_INVALID_ARGUMENT),
    (dict(n=0), K.ERR_SHAPE),
    (dict(n=(1 << 27) + 1), K.ERR_SHAPE),
    (dict(n=1 << 20, seqs=_seqs(B=1 << 20)), K.ERR_SHAPE),                   # too many tokens for one launch
    (dict(k=None), K.ERR_INVALID_ARGUMENT),
    (dict(v=_rows(None)), K.ERR_INVALID_ARGUMENT),
    (dict(k=_rows(A + 7 * STEP + 4)), K.ERR_INVALID_ARGUMENT),
    (dict(k=_rows(A + 7 * STEP, token_stride=129)), K.ERR_INVALID_ARGUMENT),
    (dict(k=_rows(A + 7 * STEP, head_stride=-128)), K.ERR_INVALID_ARGUMENT),
    (dict(k=_rows(A + 7 * STEP, seq_stride=1 << 60)), K.ERR_INVALID_ARGUMENT),
    (dict(k=_rows(A)), K.ERR_INVALID_ARGUMENT),                              # the new rows inside the cache
    (dict(seqs=_seqs(pages=A + 4096)), K.ERR_INVALID_ARGUMENT),              # the table inside the cache
    (dict(rot=_rot(table=None)), K.ERR_INVALID_ARGUMENT),
    (dict(rot=_rot(table=A + 9 * STEP + 8)), K.ERR_INVALID_ARGUMENT),
    (dict(rot=_rot(table=A + STEP - 4096)), K.ERR_INVALID_ARGUMENT),         # the rotations reach into the cache
    (dict(rot=_rot(n_pos=0)), K.ERR_SHAPE),
    (dict(rot=_rot(n_pos=1 << 60)), K.ERR_SHAPE),
]


@pytest.mark.parametrize("over,status", ROWS_REFUSED)
def test_refused_rows(over, status):
    assert _rows_call(**over) == status
    assert K.last_error()


@pytest.mark.parametrize("over", [
    dict(k=_rows(A + 7 * STEP, token_stride=0)),
    dict(k=_rows(A + 7 * STEP, head_stride=128, token_stride=128)),
    dict(v=_rows(A + 7 * STEP)),
    dict(v=_rows(A + 7 * STEP + 128)),
    dict(v=_rows(A + 7 * STEP + 4096, token_stride=256, head_stride=7 * 256, seq_stride=14 * 256, layer_stride=56 * 256)),
    dict(seqs=_seqs(start=A + 7 * STEP)),
    dict(rot=_rot(table=A + 8 * STEP + 64)),
])
def test_outputs_that_overlap_are_refused(over):
    assert _rows_call(output=True, **over) == K.ERR_INVALID_ARGUMENT


def test_inputs_may_repeat_rows():
    assert _rows_call(k=_rows(A + 7 * STEP, seq_stride=0)) == K.OK
    assert _rows_call(v=_rows(A + 7 * STEP)) == K.OK                          # values that are the keys


def _attend(**over):
    B, n, Hq, d = 4, 3, 6, 128
    q = dict(layer_stride=0, seq_stride=n * Hq * d, head_stride=d, token_stride=Hq * d)
    a = dict(cache=_cache(), layer=2, B=B, n_q=n, H_q=Hq, q=_rows(A + 4 * STEP, **q), pages=A + 5 * STEP, max_pages=5,
             lens=A + 6 * STEP, max_len=320, scale=0.1, out=_rows(A + 7 * STEP, **q), rot=_rot(), lse=A + 8 * STEP)
    a.update(over)
    return K.validate_paged_attend(**a)


def test_good_attend_is_taken():
    assert _attend() == K.OK
    assert _attend(lse=None, cache=_cache(dtype=K.F32), max_len=0, rot=None) == K.OK
    assert _attend(rot=_rot(n_pos=320)) == K.OK
    assert _attend(n_q=16, q=_rows(A + 4 * STEP, seq_stride=16 * 6 * 128, head_stride=128, token_stride=6 * 128),
                   out=_rows(A + 7 * STEP, seq_stride=16 * 6 * 128, head_stride=128, token_stride=6 * 128)) == K.OK


ATTEND_REFUSED = [
    (dict(cache=None), K.ERR_INVALID_ARGUMENT),
    (dict(layer=3), K.ERR_SHAPE),
    (dict(layer=-1), K.ERR_SHAPE),
    (dict(B=0), K.ERR_SHAPE),
    (dict(n_q=0), K.ERR_SHAPE),
    (dict(n_q=17), K.ERR_UNSUPPORTED),
    (dict(H_q=5), K.ERR_SHAPE),
    (dict(H_q=0), K.ERR_SHAPE),
    (dict(H_q=1 << 17), K.ERR_SHAPE),
    (dict(B=1 << 15), K.ERR_SHAPE),
    (dict(max_len=321), K.ERR_SHAPE),
    (dict(max_len=-1), K.ERR_SHAPE),
    (dict(max_len=1 << 30, max_pages=1 << 24), K.ERR_SHAPE),
    (dict(max_pages=0), K.ERR_SHAPE),
    (dict(pages=None), K.ERR_INVALID_ARGUMENT),
    (dict(lens=None), K.ERR_INVALID_ARGUMENT),
    (dict(scale=0.0), K.ERR_INVALID_ARGUMENT),
    (dict(scale=float("nan")), K.ERR_INVALID_ARGUMENT),
    (dict(scale=float("inf")), K.ERR_INVALID_ARGUMENT),
    (dict(scale=1e300), K.ERR_INVALID_ARGUMENT),
    (dict(rot=_rot(n_pos=319)), K.ERR_SHAPE),                                # shorter than max_len
    (dict(rot=_rot(table=None)), K.ERR_INVALID_ARGUMENT),
    (dict(rot=_rot(table=A + 7 * STEP + 64)), K.ERR_INVALID_ARGUMENT),       # out over the rotations
    (dict(q=None), K.ERR_INVALID_ARGUMENT),
    (dict(out=None), K.ERR_INVALID_ARGUMENT),
    (dict(lse=A + 8 * STEP + 2), K.ERR_INVALID_ARGUMENT),
    (dict(lse=A + 7 * STEP), K.ERR_INVALID_ARGUMENT),                        # lse over out
    (dict(lse=A + 4 * STEP), K.ERR_INVALID_ARGUMENT),                        # lse over q
    (dict(pages=A + 7 * STEP), K.ERR_INVALID_ARGUMENT),                      # out over the table
    (dict(out=_rows(A + 7 * STEP, seq_stride=0, head_stride=128, token_stride=6 * 128)), K.ERR_INVALID_ARGUMENT),
    (dict(out=_rows(A, seq_stride=3 * 6 * 128, head_stride=128, token_stride=6 * 128)), K.ERR_INVALID_ARGUMENT),
]


@pytest.mark.parametrize("over,status", ATTEND_REFUSED)
def test_refused_attend(over, status):
    assert _attend(**over) == status
    assert K.last_error()


def test_calls_without_a_context_are_refused():
    L, c, s, k, r = K.lib(), _cache(), _seqs(), _rows(A + 7 * STEP), K.Rope(1e4, 0, 0, None)
    n = ctypes.c_uint32()
    ref = ctypes.byref
    for name in ("kvmap_paged_append", "kvmap_paged_read"):
        assert getattr(L, name)(None, ref(c), 0, 1, ref(s), 7, ref(k), ref(k), None, None) == K.ERR_INVALID_ARGUMENT
    assert L.kvmap_rope_table(None, ref(r), 7, 128, A, None) == K.ERR_INVALID_ARGUMENT
    assert L.kvmap_paged_dropped(None, ref(n), None) == K.ERR_INVALID_ARGUMENT
    assert L.kvmap_paged_reserve(None, ref(c), 1, 1, 2, 10) == K.ERR_INVALID_ARGUMENT
    assert L.kvmap_paged_reserve(None, ref(c), 0, 1, 2, 10) == K.ERR_SHAPE
    assert L.kvmap_paged_reserve(None, ref(c), 1, 17, 2, 10) == K.ERR_UNSUPPORTED
    assert L.kvmap_paged_attend(None, ref(c), 0, 1, 1, 2, ref(k), None, 1, None, 1, 1.0, None, ref(k), None, None) == K.ERR_INVALID_ARGUMENT


def test_cache_tensors_are_checked():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 3, 4, 16, 64)
    with pytest.raises(ValueError):
        K.PagedCache(x[0], x[0])
    with pytest.raises(ValueError):
        K.PagedCache(x, x.transpose(-1, -2))
    with pytest.raises(TypeError):
        K.PagedCache(x, x.bfloat16())
    with pytest.raises(TypeError):
        K.PagedCache(x.half(), x.half())
    with pytest.raises(ValueError):
        K.PagedCache(x, x)                                                   # not on the device


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="no ROCm toolchain")
@pytest.mark.parametrize("name,kernels", [("paged_attend", 16), ("paged_rows", 16)])
def test_no_kernel_spills(tmp_path, name, kernels):
    """Every instance keeps its state in registers: a spill would cost its speed, and spills of parts of matrix operands have
    given wrong sums."""
    from cross_model_kv_amd import build
    asm = str(tmp_path / (name + ".s"))
    r = subprocess.run(["/opt/rocm/bin/hipcc", *build.HIP_FLAGS, "-S", "--offload-device-only",
                        os.path.join(build.CSRC, name + ".hip"), "-o", asm], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    src = open(asm).read()
    names = re.findall(r"\.name: +(_ZN5kvmap\S+)", src)
    assert len(names) >= kernels
    for field in ("private_segment_fixed_size", "vgpr_spill_count"):
        sizes = [int(x) for x in re.findall(rf"\.{field}: +(\d+)", src)]
        assert len(sizes) == len(names) and not any(sizes), dict(zip(names, sizes))
