"""The paged cache in the model's own type in float64 numpy: appends, reads and attention, token by token.

Test infrastructure: shares no code with the library.  A cache is a dict of arrays k, v [L][n_pages][H][page][d]; a table of
rotations is [n_pos][d / 2][2] (cosine, sine).
"""

import numpy as np


def table(n_pos, d, theta=None, inv_freq=None, pos0=0):
    """Cosines and sines in float64 of the angles position times frequency, rounded once each."""
    f = theta ** (-2.0 * np.arange(d // 2) / d) if inv_freq is None else np.asarray(inv_freq, np.float64)
    a = np.arange(pos0, pos0 + n_pos, dtype=np.float64)[:, None] * f
    return np.stack([np.cos(a), np.sin(a)], -1)


def turn(x, cs, sign=1.0):
    """Rows x [..., d] turned by the angles of cs [..., d/2, 2]."""
    h = x.shape[-1] // 2
    z = (x[..., :h] + 1j * x[..., h:]) * (cs[..., 0] + 1j * sign * cs[..., 1])
    return np.concatenate([z.real, z.imag], -1)


def turn_size(x, cs):
    """What the two products of a turned element add up to, signs aside."""
    h = x.shape[-1] // 2
    lo, hi, c, s = abs(x[..., :h]), abs(x[..., h:]), abs(cs[..., 0]), abs(cs[..., 1])
    return np.concatenate([lo * c + hi * s, hi * c + lo * s], -1)


def _where(c, pages, b, pos, n_pos):
    """(page, row) of a position, or None where it is out of range."""
    P, n_pages = c["k"].shape[3], c["k"].shape[1]
    if pos < 0 or pos // P >= len(pages[b]) or (n_pos is not None and pos >= n_pos):
        return None
    page = pages[b][pos // P]
    return (page, pos % P) if 0 <= page < n_pages else None


def places(c, pages, start, count, n, n_pos=None):
    """For every (b, i): (page, row), None (out of range) or "past" (beyond the sequence's count)."""
    out = {}
    for b in range(len(pages)):
        cnt = n if count is None else count[b]
        bad = start[b] < 0 or not 0 <= cnt <= n
        for i in range(n):
            out[b, i] = None if bad else "past" if i >= cnt else _where(c, pages, b, start[b] + i, n_pos)
    return out


def append(c, k, v, pages, start, count=None, layer=0, rot=None):
    """k, v [layers][B][H][n][d] float64; returns the tokens left out, and the size of every written key element (for
    tolerances; as c["k"], zero where nothing was written)."""
    L, B, H, n, d = k.shape
    size = np.zeros_like(c["k"])
    dropped = 0
    for (b, i), at in places(c, pages, start, count, n, None if rot is None else len(rot)).items():
        if at == "past":
            continue
        if at is None:
            dropped += 1
            continue
        page, row = at
        for l in range(L):
            x = k[l, b, :, i]
            if rot is not None:
                size[layer + l, page, :, row] = turn_size(x, rot[start[b] + i])
                x = turn(x, rot[start[b] + i])
            c["k"][layer + l, page, :, row] = x
            c["v"][layer + l, page, :, row] = v[l, b, :, i]
    return dropped, size


def read(c, pages, start, n, count=None, layer=0, n_layers=None, rot=None):
    L = c["k"].shape[0] - layer if n_layers is None else n_layers
    H, d = c["k"].shape[2], c["k"].shape[4]
    k = np.zeros((L, len(pages), H, n, d))
    v, size = np.zeros_like(k), np.zeros_like(k)
    for (b, i), at in places(c, pages, start, count, n, None if rot is None else len(rot)).items():
        if at == "past":
            continue
        if at is None:
            k[:, b, :, i] = v[:, b, :, i] = np.nan
            continue
        page, row = at
        x = c["k"][layer:layer + L, page, :, row]
        if rot is not None:
            size[:, b, :, i] = turn_size(x, rot[start[b] + i])
            x = turn(x, rot[start[b] + i], -1.0)
        k[:, b, :, i] = x
        v[:, b, :, i] = c["v"][layer:layer + L, page, :, row]
    return k, v, size


def attend(c, q, pages, lens, scale, layer=0, rot=None):
    """q [B][n_q][H_q][d].  Returns out, lse and, for tolerances, per row: the softmax-weighted sum of |v|, and the largest
    scale * sum |q k| that it sees."""
    B, n, Hq, d = q.shape
    H, P = c["k"].shape[2], c["k"].shape[3]
    G = Hq // H
    out, size = np.zeros((B, n, Hq, d)), np.zeros((B, n, Hq, d))
    lse, prod = np.full((B, n, Hq), -np.inf), np.zeros((B, n, Hq))
    for b in range(B):
        for i in range(n):
            pos = lens[b] - n + i
            if pos < 0:
                continue
            at = [_where(c, pages, b, t, None) for t in range(pos + 1)]
            lost = np.array([a is None for a in at])
            pg = np.array([0 if a is None else a[0] for a in at])
            rw = np.array([0 if a is None else a[1] for a in at])
            for hq in range(Hq):
                h = hq // G
                x = q[b, i, hq] if rot is None else turn(q[b, i, hq], rot[pos])
                K, V = c["k"][layer, pg, h, rw], c["v"][layer, pg, h, rw]
                with np.errstate(invalid="ignore", over="ignore"):
                    y = scale * (K @ x)
                    y[lost] = np.nan
                    m = np.max(y)
                    m = 0.0 if m == -np.inf else m
                    w = np.exp(y - m)
                    s = w.sum()
                    lse[b, i, hq] = m + np.log(s) if s != 0 else -np.inf
                    if s == 0:
                        continue
                    w = w / s
                    out[b, i, hq] = (w[:, None] * V).sum(0)
                    size[b, i, hq] = (w[:, None] * abs(V)).sum(0)
                    prod[b, i, hq] = scale * (abs(K) @ abs(x)).max()
    return out, lse, size, prod
