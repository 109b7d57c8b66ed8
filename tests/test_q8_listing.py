"""The prompt kernel's listing: its key products are written out, so the compiler does not keep the distances that a
matrix product asks for; the source has to, and this reads whether it did."""

import os
import re
import subprocess

import pytest

pytestmark = pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="no ROCm toolchain")

AFTER_PRODUCT = 13   # instructions between a product of 8 passes and a vector instruction that touches its result
AFTER_VECTOR = 2     # between a vector instruction and a product that reads its result


def _listing(tmp_path, name):
    from cross_model_kv_amd import build
    asm = str(tmp_path / (name + ".s"))
    r = subprocess.run(["/opt/rocm/bin/hipcc", *build.HIP_FLAGS, "-S", "--offload-device-only",
                        os.path.join(build.CSRC, name + ".hip"), "-o", asm], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return open(asm).read()


def _regs(text):
    out = {(m[1], i) for m in re.finditer(r"\b([va])\[(\d+):(\d+)\]", text) for i in range(int(m[2]), int(m[3]) + 1)}
    return out | {(m[1], int(m[2])) for m in re.finditer(r"\b([va])(\d+)\b", text)}


def _instructions(body):
    """(text, written out) of a function's instructions, in the listing's order."""
    asm = False
    for line in body.split("\n"):
        t = line.strip()
        if "ASMSTART" in t or "ASMEND" in t:
            asm = "ASMSTART" in t
        elif t and not t.startswith((";", ".")) and not t.endswith(":"):
            yield t.split(";")[0].strip(), asm


def _close(instructions):
    """What stands too near to a written-out product, and how many of those there are."""
    found, products = [], 0
    results, vectors = [], []                    # (registers, instructions left, text)
    for t, asm in instructions:
        op = t.split()[0]
        args = re.split(r",\s*", t[len(op):].strip())
        used = _regs(t)
        if "mfma" in op:
            dst, reads = _regs(args[0]), _regs(",".join(args[1:3]))
            same = _regs(args[3]) | dst
            found += [(src, t) for r, _, src in results if r & reads or (r & same and r != dst)]
            if asm:
                found += [(src, t) for r, _, src in vectors if r & (reads | _regs(args[3]))]
        else:
            found += [(src, t) for r, _, src in results if r & used]
        n = int(args[0]) + 1 if op == "s_nop" else 1
        results = [(r, left - n, src) for r, left, src in results if left > n]
        vectors = [(r, left - n, src) for r, left, src in vectors if left > n]
        if "mfma" in op and asm:
            products += 1
            results = [x for x in results if x[0] != dst] + [(dst, AFTER_PRODUCT, t)]
        elif op.startswith("v_") and "mfma" not in op and not op.startswith("v_cmp"):
            vectors.append((_regs(args[0]), AFTER_VECTOR, t))
    return found, products


def test_written_out_products_keep_their_distances(tmp_path):
    src = _listing(tmp_path, "q8_prompt")
    kernels = re.findall(r"^(_ZN5kvmap\S*q8_prompt_kernel\S*):(.*?)\.Lfunc_end", src, re.M | re.S)
    assert len(kernels) >= 4
    for name, body in kernels:
        found, products = _close(_instructions(body))
        assert products >= 12, name
        assert not found, (name, found[:5])


def test_the_check_sees_what_is_too_near():
    product = [("v_mfma_f32_32x32x16_bf16 v[0:15], v[16:19], a[0:3], v[0:15]", True)]
    assert _close(product + [("v_add_f32_e32 v20, v3, v21", False)])[0]
    assert _close(product + [("s_nop 11", False), ("v_add_f32_e32 v20, v3, v21", False)])[0]
    assert not _close(product + [("s_nop 12", False), ("v_add_f32_e32 v20, v3, v21", False)])[0]
    assert not _close(product * 2)[0]
    assert _close(product + [("v_mfma_f32_32x32x16_f16 a[4:19], v[0:3], v[30:33], a[4:19]", False)])[0]
    assert _close([("v_accvgpr_write_b32 a2, v7", False)] + product)[0]
    assert _close([("v_accvgpr_write_b32 a2, v7", False), ("s_nop 0", False)] + product)[0]
    assert not _close([("v_accvgpr_write_b32 a2, v7", False), ("s_nop 1", False)] + product)[0]


@pytest.mark.parametrize("name", ["q8_prompt", "q8_join"])
def test_no_kernel_spills(tmp_path, name):
    src = _listing(tmp_path, name)
    names = re.findall(r"\.name: +(_ZN5kvmap\S+)", src)
    assert len(names) >= 4
    for field in ("private_segment_fixed_size", "vgpr_spill_count"):
        sizes = [int(x) for x in re.findall(rf"\.{field}: +(\d+)", src)]
        assert len(sizes) == len(names) and not any(sizes), dict(zip(names, sizes))
