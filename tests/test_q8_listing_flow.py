"""The prompt kernel's listing along its control flow: the distances that its written-out matrix products need hold on every path,
over branches and the loops' back edges, not only in the order in which the listing has the instructions."""

import os
import re

import pytest

from test_q8_listing import AFTER_PRODUCT, AFTER_VECTOR, _listing, _regs

pytestmark = pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="no ROCm toolchain")


def _blocks(body):
    """{label: ([(text, written out)], successors)} of a function; the first label is None."""
    blocks, label, asm, order = {None: []}, None, False, [None]
    for line in body.split("\n"):
        t = line.strip()
        m = re.match(r"(\.L\w+):", t)
        if m:
            label = m[1]
            blocks[label] = []
            order.append(label)
        elif "ASMSTART" in t or "ASMEND" in t:
            asm = "ASMSTART" in t
        elif t and not t.startswith((";", ".")) and not t.endswith(":"):
            blocks[label].append((t.split(";")[0].strip(), asm))
    flow = {}
    for i, b in enumerate(order):
        after, falls = [], True
        for t, _ in blocks[b]:
            m = re.match(r"s_(c?)branch\S* (\.L\w+)", t)
            if m:
                after.append(m[2])
                falls = bool(m[1])
            assert not t.startswith(("s_setpc", "s_swappc", "s_call")), t     # (a path that is not followed here)
            falls = falls and not t.startswith("s_endpgm")
        if falls and i + 1 < len(order):
            after.append(order[i + 1])
        flow[b] = (blocks[b], after)
    return flow


def _walk(instructions, results, vectors, found):
    """Steps over a block.  results, vectors: {(registers, text): instructions that have still to pass}."""
    for t, asm in instructions:
        op = t.split()[0]
        args = re.split(r",\s*", t[len(op):].strip())
        if "mfma" in op:
            dst, reads, acc = _regs(args[0]), _regs(",".join(args[1:3])), _regs(args[3])
            found.update((src, t) for (r, src) in results if r & reads or (r & (acc | dst) and r != dst))
            # (the compiler keeps its own products from its own vector instructions)
            found.update((src, t) for (r, src, own) in vectors if (asm or own) and r & (reads | acc))
        else:
            found.update((src, t) for (r, src) in results if r & _regs(t))
        n = int(args[0]) + 1 if op == "s_nop" else 1
        results = {k: left - n for k, left in results.items() if left > n}
        vectors = {k: left - n for k, left in vectors.items() if left > n}
        if "mfma" in op and asm:
            results = {k: left for k, left in results.items() if k[0] != dst}
            results[frozenset(dst), t] = AFTER_PRODUCT
        elif op.startswith("v_") and "mfma" not in op and not op.startswith("v_cmp"):
            vectors[frozenset(_regs(args[0])), t, asm] = AFTER_VECTOR
    return results, vectors


def _too_near(body):
    flow = _blocks(body)
    entry = {b: ({}, {}) for b in flow}
    todo, found = list(flow), set()
    while todo:
        b = todo.pop()
        out = _walk(flow[b][0], *entry[b], found)
        for succ in flow[b][1]:
            grown = False
            for mine, theirs in zip(entry[succ], out):
                for k, left in theirs.items():
                    if mine.get(k, 0) < left:
                        mine[k] = left
                        grown = True
            if grown and succ not in todo:
                todo.append(succ)
    return found


def test_written_out_products_keep_their_distances_on_every_path(tmp_path):
    src = _listing(tmp_path, "q8_prompt")
    kernels = re.findall(r"^(_ZN5kvmap\S*q8_prompt_kernel\S*):(.*?)\.Lfunc_end", src, re.M | re.S)
    assert len(kernels) >= 4
    for name, body in kernels:
        assert sum("mfma" in t and asm for block, _ in _blocks(body).values() for t, asm in block) >= 12, name
        found = _too_near(body)
        assert not found, (name, sorted(found)[:5])


PRODUCT = "\t;ASMSTART\n\tv_mfma_f32_32x32x16_bf16 v[0:15], v[16:19], a[0:3], 0\n\t;ASMEND\n"


def test_a_back_edge_and_a_branch_are_followed():
    use = "\tv_add_f32_e32 v20, v3, v21\n"
    wait = "\ts_nop 15\n"
    assert _too_near(".LBB0_1:\n" + use + wait + PRODUCT + "\ts_cbranch_scc1 .LBB0_1\n\ts_endpgm\n")
    assert not _too_near(".LBB0_1:\n" + use + PRODUCT + wait + "\ts_cbranch_scc1 .LBB0_1\n\ts_endpgm\n")
    assert _too_near(PRODUCT + "\ts_branch .LBB0_2\n.LBB0_1:\n" + wait + "\ts_endpgm\n.LBB0_2:\n" + use + "\ts_branch .LBB0_1\n")
    assert not _too_near(PRODUCT + "\ts_branch .LBB0_2\n.LBB0_1:\n" + use + "\ts_endpgm\n.LBB0_2:\n" + wait + "\ts_branch .LBB0_1\n")
