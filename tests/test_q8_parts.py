"""What 24 bits of queries and weights in fp32 calls are worth, on the CPU: the bound on the whole answer that tests/test_gpu_q8_f32.py
holds the kernels to is one that two bf16 parts of queries, of weights, or of both do not meet."""

import numpy as np

from oracle import q8_oracle as Q
from q8_f32_cases import CASES, WHOLE, case, whole
from test_gpu_q8_rows import reference


def _parts(x, n):
    """x as a sum of n bf16 parts."""
    left, total = np.asarray(x, np.float32), np.zeros(np.shape(x))
    for _ in range(n):
        u = left.view(np.uint32).astype(np.uint64)
        part = ((u + 0x7FFF + (u >> 16 & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
        total += part
        left = (left - part).astype(np.float32)
    return total


def _answer(o, q, table, lens, scale, q_parts, w_parts):
    """reference() with queries and weights cut."""
    B, n, Hq, d = q.shape
    H = o["k"].shape[2]
    G = Hq // H
    out = np.zeros(q.shape)
    q = _parts(q, q_parts)
    for b in range(B):
        T = lens[b]
        if not T:
            continue
        ahead = np.arange(T) > (T - n + np.arange(n))[:, None]
        for h in range(H):
            k, v = Q.tokens(o, "k", 0, h, table[b], T), Q.tokens(o, "v", 0, h, table[b], T)
            y = np.where(ahead, -np.inf, scale * (q[b, :, h * G:(h + 1) * G].transpose(1, 0, 2) @ k.T))
            m = y.max(-1, keepdims=True)
            p = np.exp(y - np.where(np.isneginf(m), 0.0, m))
            s = p.sum(-1, keepdims=True)
            out[b, :, h * G:(h + 1) * G] = (_parts(p, w_parts) @ v / np.where(s > 0, s, 1.0)).transpose(1, 0, 2)
    return out


def test_two_parts_are_told_from_three():
    """Queries in two parts fail the bound in every case, weights in two in nearly all (a row of a few tokens takes little harm)."""
    few = [c for c in CASES if sum(c[0]) * c[1] * c[2] * c[3] < 400000]
    err = {}
    for c in few:
        o, table, q = case(*c)
        ref = reference(o, q, table, c[0], 0, c[4] ** -0.5)[0]
        for parts in ((3, 3), (2, 3), (3, 2), (2, 2)):
            err.setdefault(parts, []).append(whole(_answer(o, q, table, c[0], c[4] ** -0.5, *parts), ref))
    assert len(few) >= 8 and max(err[3, 3]) < WHOLE / 4
    assert min(err[2, 3]) > WHOLE and min(err[2, 2]) > WHOLE, err
    assert sum(e > WHOLE for e in err[3, 2]) >= len(few) - 1, err
