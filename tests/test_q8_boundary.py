"""The 8-bit cache's calls on the CPU: what they refuse before any device work, and the page resolution
that the kernels use, under the sanitizers."""

import os
import shutil
import subprocess

import pytest

from cross_model_kv_amd import kvmap as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 40          # addresses that are never read
STEP = 1 << 34


def _cache(**over):
    f = dict(L=3, n_pages=10, H_kv=2, page=64, head_dim=128, k=A, v=A + STEP, k_scale=A + 2 * STEP, v_scale=A + 3 * STEP)
    f.update(over)
    return K.Q8CacheC(**f)


def _seqs(**over):
    f = dict(B=4, max_pages=5, pages=A + 4 * STEP, start=A + 5 * STEP, count=A + 6 * STEP)
    f.update(over)
    return K.Q8SeqsC(**f)


def _rows(base, L=2, B=4, H=2, n=7, d=128, **over):
    f = dict(base=base, layer_stride=B * H * n * d, seq_stride=H * n * d, head_stride=n * d, token_stride=d)
    f.update(over)
    return K.Q8RowsC(**f)


def _rows_call(**over):
    a = dict(cache=_cache(), layer0=1, n_layers=2, seqs=_seqs(), n=7, dtype=K.BF16, k=_rows(A + 7 * STEP),
             v=_rows(A + 8 * STEP), output=False)
    a.update(over)
    return K.validate_q8_rows(**a)


@pytest.mark.parametrize("output", [False, True])
def test_good_rows_are_taken(output):
    assert _rows_call(output=output) == K.OK
    assert _rows_call(output=output, dtype=K.F32) == K.OK
    assert _rows_call(output=output, seqs=_seqs(count=None)) == K.OK
    # the key and value parts of one projection's output [layers][B][n][2 H][d]
    s = dict(layer_stride=4 * 7 * 4 * 128, seq_stride=7 * 4 * 128, head_stride=128, token_stride=4 * 128)
    assert _rows_call(output=output, k=_rows(A + 7 * STEP, **s), v=_rows(A + 7 * STEP + 2 * 128 * 2, **s)) == K.OK


ROWS_REFUSED = [
    (dict(cache=None), K.ERR_INVALID_ARGUMENT),
    (dict(cache=_cache(k=None)), K.ERR_INVALID_ARGUMENT),
    (dict(cache=_cache(v=A + STEP + 8)), K.ERR_INVALID_ARGUMENT),
    (dict(cache=_cache(v=A + 64)), K.ERR_INVALID_ARGUMENT),                  # overlaps k
    (dict(cache=_cache(L=0)), K.ERR_SHAPE),
    (dict(cache=_cache(n_pages=0)), K.ERR_SHAPE),
    (dict(cache=_cache(H_kv=-1)), K.ERR_SHAPE),
    (dict(cache=_cache(L=1 << 30, n_pages=1 << 30)), K.ERR_SHAPE),
    (dict(cache=_cache(page=48)), K.ERR_UNSUPPORTED),
    (dict(cache=_cache(head_dim=96)), K.ERR_UNSUPPORTED),
    (dict(layer0=2), K.ERR_SHAPE),
    (dict(layer0=-1), K.ERR_SHAPE),
    (dict(n_layers=0), K.ERR_SHAPE),
    (dict(layer0=0x7FFFFFFF), K.ERR_SHAPE),
    (dict(dtype=2), K.ERR_UNSUPPORTED),
    (dict(seqs=None), K.ERR_INVALID_ARGUMENT),
    (dict(seqs=_seqs(B=0)), K.ERR_SHAPE),
    (dict(seqs=_seqs(max_pages=0)), K.ERR_SHAPE),
    (dict(seqs=_seqs(max_pages=1 << 26)), K.ERR_SHAPE),
    (dict(seqs=_seqs(pages=None)), K.ERR_INVALID_ARGUMENT),
    (dict(seqs=_seqs(start=None)), K.ERR_INVALID_ARGUMENT),
    (dict(seqs=_seqs(start=A + 5 * STEP + 2)), K.ERR_INVALID_ARGUMENT),
    (dict(n=0), K.ERR_SHAPE),
    (dict(n=(1 << 30) + 1), K.ERR_SHAPE),
    (dict(n=1 << 30, seqs=_seqs(B=1 << 14)), K.ERR_SHAPE),                   # too many pages for one launch
    (dict(k=None), K.ERR_INVALID_ARGUMENT),
    (dict(v=_rows(None)), K.ERR_INVALID_ARGUMENT),
    (dict(k=_rows(A + 7 * STEP + 4)), K.ERR_INVALID_ARGUMENT),
    (dict(k=_rows(A + 7 * STEP, token_stride=129)), K.ERR_INVALID_ARGUMENT),
    (dict(k=_rows(A + 7 * STEP, head_stride=-128)), K.ERR_INVALID_ARGUMENT),
    (dict(k=_rows(A + 7 * STEP, seq_stride=1 << 60)), K.ERR_INVALID_ARGUMENT),
    (dict(k=_rows(A)), K.ERR_INVALID_ARGUMENT),                              # the new rows inside the cache
    (dict(seqs=_seqs(pages=A + 4096)), K.ERR_INVALID_ARGUMENT),              # the table inside the cache
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
    dict(seqs=_seqs(start=A + 7 * STEP)),
])
def test_outputs_that_overlap_are_refused(over):
    assert _rows_call(output=True, **over) == K.ERR_INVALID_ARGUMENT


def test_inputs_may_repeat_rows():
    assert _rows_call(k=_rows(A + 7 * STEP, seq_stride=0)) == K.OK


def _attend(**over):
    B, n, Hq, d = 4, 3, 6, 128
    q = dict(layer_stride=0, seq_stride=n * Hq * d, head_stride=d, token_stride=Hq * d)
    a = dict(cache=_cache(), layer=2, B=B, n_q=n, H_q=Hq, dtype=K.BF16, q=_rows(A + 4 * STEP, **q), pages=A + 5 * STEP,
             max_pages=5, lens=A + 6 * STEP, max_len=320, scale=0.1, out=_rows(A + 7 * STEP, **q), lse=A + 8 * STEP)
    a.update(over)
    return K.validate_q8_attend(**a)


def test_good_attend_is_taken():
    assert _attend() == K.OK
    assert _attend(lse=None, dtype=K.F32, max_len=0) == K.OK


ATTEND_REFUSED = [
    (dict(cache=None), K.ERR_INVALID_ARGUMENT),
    (dict(layer=3), K.ERR_SHAPE),
    (dict(layer=-1), K.ERR_SHAPE),
    (dict(B=0), K.ERR_SHAPE),
    (dict(n_q=0), K.ERR_SHAPE),
    (dict(H_q=5), K.ERR_SHAPE),
    (dict(H_q=0), K.ERR_SHAPE),
    (dict(B=1 << 15), K.ERR_SHAPE),
    (dict(n_q=1 << 30), K.ERR_SHAPE),
    (dict(max_len=321), K.ERR_SHAPE),
    (dict(max_len=-1), K.ERR_SHAPE),
    (dict(max_pages=0), K.ERR_SHAPE),
    (dict(dtype=7), K.ERR_UNSUPPORTED),
    (dict(pages=None), K.ERR_INVALID_ARGUMENT),
    (dict(lens=None), K.ERR_INVALID_ARGUMENT),
    (dict(scale=0.0), K.ERR_INVALID_ARGUMENT),
    (dict(scale=float("nan")), K.ERR_INVALID_ARGUMENT),
    (dict(scale=float("inf")), K.ERR_INVALID_ARGUMENT),
    (dict(scale=1e300), K.ERR_INVALID_ARGUMENT),
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
    import ctypes
    L, c, s, k = K.lib(), _cache(), _seqs(), _rows(A + 7 * STEP)
    n = ctypes.c_uint32()
    ref = ctypes.byref
    for name in ("kvmap_q8_write", "kvmap_q8_read"):
        assert getattr(L, name)(None, ref(c), 0, 1, ref(s), 7, 0, ref(k), ref(k), None) == K.ERR_INVALID_ARGUMENT
    assert L.kvmap_q8_dropped(None, ref(n), None) == K.ERR_INVALID_ARGUMENT
    assert L.kvmap_q8_reserve(None, ref(c), 1, 1, 2, 10) == K.ERR_INVALID_ARGUMENT
    assert L.kvmap_q8_reserve(None, ref(c), 0, 1, 2, 10) == K.ERR_SHAPE
    assert L.kvmap_q8_attend(None, ref(c), 0, 1, 1, 2, 0, ref(k), None, 1, None, 1, 1.0, ref(k), None, None) == K.ERR_INVALID_ARGUMENT


def test_cache_tensors_are_checked():
    torch = pytest.importorskip("torch")
    f8 = lambda *s: torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError):
        K.Q8Cache(f8(2, 3, 4, 16, 64), f8(2, 3, 4, 16, 64), sc, sc)         # v must be dim-major
    with pytest.raises(TypeError):
        K.Q8Cache(f8(2, 3, 4, 16, 64).view(torch.uint8), f8(2, 3, 4, 64, 16), sc, sc)
    with pytest.raises(ValueError):
        K.Q8Cache(f8(2, 3, 4, 16, 64), f8(2, 3, 4, 64, 16), sc, sc[:1])
    with pytest.raises(ValueError):
        K.Q8Cache(f8(2, 3, 4, 16, 64), f8(2, 3, 4, 64, 16), sc, sc)         # not on the device


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_page_resolution_under_sanitizers(tmp_path):
    exe = str(tmp_path / "q8_span_checks")
    r = subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=address", "-fsanitize=undefined",
                        "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "sanitize", "q8_span_checks.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0 and " 0 failure(s)" in r.stdout, (r.stdout + r.stderr)[-3000:]


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="no ROCm toolchain")
def test_no_attention_kernel_spills(tmp_path):
    """Every instance keeps its state in registers: a spill would cost its speed, and spills of parts of matrix
    operands have given wrong sums."""
    from cross_model_kv_amd import build
    asm = str(tmp_path / "q8_attend.s")
    r = subprocess.run(["/opt/rocm/bin/hipcc", *build.HIP_FLAGS, "-S", "--offload-device-only",
                        os.path.join(build.CSRC, "q8_attend.hip"), "-o", asm], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    import re
    src = open(asm).read()
    names = re.findall(r"\.name: +(_ZN5kvmap\S+)", src)
    assert len(names) >= 6
    for field in ("private_segment_fixed_size", "vgpr_spill_count"):
        sizes = [int(x) for x in re.findall(rf"\.{field}: +(\d+)", src)]
        assert len(sizes) == len(names) and not any(sizes), dict(zip(names, sizes))
