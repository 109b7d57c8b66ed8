"""The 8-bit paged cache in float64 numpy: codes, scales, writes, reads and attention, token by token.

Test infrastructure: shares no code with the library.  A cache is a dict of arrays
  k [L][n_pages][H][page][d] and v [L][n_pages][H][d][page] uint8 codes, ks, vs [L][n_pages][H] float64.
"""

import numpy as np

E_MIN, E_MAX = -110, 119
NAN_CODE = 0x7F


def _table():
    """Value of every code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return out


VALUE = _table()
_GRID = VALUE[:127]                              # 0 .. 448, ascending with the code
_MID = (_GRID[1:] + _GRID[:-1]) / 2


def e4m3_code(y):
    """Codes of y rounded to the nearest value, ties to the even code, saturating at 448; NaN for non-finite y."""
    y = np.asarray(y, np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(y), y, 0.0)), 448.0)
    lo = np.searchsorted(_MID, a, side="left")   # first code whose upper midpoint is >= a
    tie = (lo < 126) & (a == _MID[np.minimum(lo, 125)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.uint8)
    code = code | np.where(np.signbit(y), 0x80, 0).astype(np.uint8)
    return np.where(np.isfinite(y), code, NAN_CODE).astype(np.uint8)


def scale_for(amax):
    e = E_MIN
    while e < E_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def new_cache(L, n_pages, H, page, d):
    return dict(k=np.zeros((L, n_pages, H, page, d), np.uint8), v=np.zeros((L, n_pages, H, d, page), np.uint8),
                ks=np.zeros((L, n_pages, H)), vs=np.zeros((L, n_pages, H)))


def _page(c, which, l, pid, h):
    """A view [page][d] of one page's codes."""
    x = c[which][l, pid, h]
    return x.T if which == "v" else x


def write(c, k, v, pages, start, count, layer=0):
    """k, v [layers][B][H][n][d] float64; returns the pages left out."""
    L, B, H, n, d = k.shape
    P, n_pages = c["k"].shape[3], c["k"].shape[1]
    dropped = 0
    for l in range(L):
        for which, new in (("k", k), ("v", v)):
            scales = c["ks" if which == "k" else "vs"]
            for b in range(B):
                if start[b] < 0 or count[b] < 0 or count[b] > n:
                    dropped += H
                    continue
                first, end = int(start[b]), int(start[b]) + int(count[b])
                for j in range(first // P, -(-end // P) if end > first else 0):
                    pid = pages[b][j] if j < len(pages[b]) else -1
                    if not 0 <= pid < n_pages:
                        dropped += H
                        continue
                    lo, hi = max(first - j * P, 0), min(end - j * P, P)
                    for h in range(H):
                        rows = _page(c, which, layer + l, pid, h)
                        x = new[l, b, h, j * P + lo - first:j * P + hi - first]
                        fin = np.abs(x[np.isfinite(x)])
                        s = scale_for(fin.max() if fin.size else 0.0)
                        if lo:
                            was = scales[layer + l, pid, h]
                            if was > s:
                                s = was
                            elif was < s:
                                rows[:lo] = e4m3_code(VALUE[rows[:lo]] * was / s)
                        rows[lo:hi] = e4m3_code(x / s)
                        scales[layer + l, pid, h] = s
    return dropped


def tokens(c, which, layer, h, pages, n):
    """Values [n][d] of a sequence's first n tokens; NaN where the page is out of range."""
    P, d = c["k"].shape[3], c["k"].shape[4]
    out = np.empty((n, d))
    for j in range(-(-n // P)):
        m = min(P, n - j * P)
        pid = pages[j]
        if 0 <= pid < c["k"].shape[1]:
            out[j * P:j * P + m] = VALUE[_page(c, which, layer, pid, h)[:m]] * c["ks" if which == "k" else "vs"][layer, pid, h]
        else:
            out[j * P:j * P + m] = np.nan
    return out


def read(c, pages, start, n, count, layer=0, n_layers=1):
    B, H, d = len(pages), c["k"].shape[2], c["k"].shape[4]
    out = {w: np.zeros((n_layers, B, H, n, d)) for w in "kv"}
    for w in "kv":
        for l in range(n_layers):
            for b in range(B):
                for h in range(H):
                    x = tokens(c, w, layer + l, h, pages[b], start[b] + count[b])
                    out[w][l, b, h, :count[b]] = x[start[b]:]
    return out["k"], out["v"]


def attend(c, q, pages, lens, layer, scale):
    """q [B][n_q][H_q][d] float64 -> out, lse, and what bounds on their errors are made of, per row:
    absv = sum w |v| (per dim), abss = the largest scale * sum |q_e k_e| of a visible token, and
    wv = the largest w * v_scale of a visible token."""
    B, n, Hq, d = q.shape
    H, P = c["k"].shape[2], c["k"].shape[3]
    G = Hq // H
    out, absv = np.zeros((B, n, Hq, d)), np.zeros((B, n, Hq, d))
    lse, abss, wv = np.full((B, n, Hq), -np.inf), np.zeros((B, n, Hq)), np.zeros((B, n, Hq))
    for b in range(B):
        T = int(lens[b])
        if T == 0:
            continue
        sv = np.array([c["vs"][layer, p] if 0 <= p < c["vs"].shape[1] else np.full(H, np.nan)
                       for p in pages[b][:-(-T // P)]]).repeat(P, axis=0)[:T]
        for h in range(H):
            k, v = tokens(c, "k", layer, h, pages[b], T), tokens(c, "v", layer, h, pages[b], T)
            for i in range(n):
                end = T - n + i + 1
                if end <= 0:
                    continue
                for g in range(G):
                    r = b, i, h * G + g
                    y = scale * (k[:end] @ q[r])
                    m = y.max()
                    p = np.exp(y - m)
                    w = p / p.sum()
                    out[r] = w @ v[:end]
                    lse[r] = m + np.log(p.sum())
                    absv[r] = w @ np.abs(v[:end])
                    abss[r] = scale * (np.abs(k[:end]) @ np.abs(q[r])).max()
                    wv[r] = (w * sv[:end, h]).max()
    return out, lse, dict(absv=absv, abss=abss, wv=wv)
