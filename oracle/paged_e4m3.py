"""Plain fp64 definitions of the paged cache in 8 bits and of reading a few of
its pages: e4m3 codes with a scale per page and kv head, the append that
quantises, key bounds by columns, the selection of pages by score, and the
attention over selected pages.

TEST INFRASTRUCTURE ONLY, like the rest of this package: nothing is blocked,
fused or reordered, and nothing is shared with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from . import paged


def _code_values():
    v = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if c & 127 == 127 else -x if c & 128 else x
    return v


VALUES = _code_values()                 # of every code; 0x7f and 0xff are NaN
_POSITIVE = VALUES[:127]                # ascending, 0 .. 448


def encode(x):
    """Codes of the nearest e4m3 values, ties to the even code; beyond 448 to
    448; what is not finite to NaN."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.minimum(np.abs(x), 448.0), 0.0)
    up = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo, hi = _POSITIVE[up - 1], _POSITIVE[up]
    down = (a - lo < hi - a) | ((a - lo == hi - a) & ((up - 1) % 2 == 0))
    code = np.where(down, up - 1, up).astype(np.uint8)
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(np.isfinite(x), code, 127).astype(np.uint8)


def pow2_at_least(x, top):
    """The smallest power of two s >= 2^-100 with x <= top * s; 0 for x = 0."""
    if x == 0:
        return 0.0
    e = -100
    while x > top * 2.0 ** e:
        e += 1
    return 2.0 ** e


def quantise(x, pow2=True):
    """Codes and scales [P, Hkv] of pages x [P, Hkv, ps, d]."""
    amax = np.abs(x).max((2, 3))
    if pow2:
        s = np.array([[pow2_at_least(v, 448.0) for v in row] for row in amax])
    else:
        s = (amax / 448.0).astype(np.float32).astype(np.float64) * (1 + 2.0 ** -20)
        s = s.astype(np.float32).astype(np.float64)
    safe = np.where(s > 0, s, 1.0)
    return encode(x / safe[..., None, None]), s


def decode(codes, scales):
    return VALUES[codes] * np.asarray(scales, np.float64)[..., None, None]


def append(codes, scales, x, table, lengths, offsets, positions_below=None):
    """New (codes, scales) of pools [P, Hkv, ps, d] after the rows x [T, Hkv, d]
    of packed new tokens; tokens at positions from positions_below on are left
    out."""
    codes, scales = codes.copy(), np.asarray(scales, np.float64).copy()
    ps = codes.shape[2]
    for b in range(len(lengths)):
        q0, q1, n = int(offsets[b]), int(offsets[b + 1]), int(lengths[b])
        first = n - (q1 - q0)
        stop = n if positions_below is None else min(n, positions_below)
        col = first // ps
        while q1 > q0 and col * ps < stop:
            a, z = max(first, col * ps), min(stop, (col + 1) * ps)
            if a < z:
                page, older = table[b][col], a - col * ps
                for g in range(codes.shape[1]):
                    rows = x[q0 + a - first:q0 + z - first, g]
                    old = scales[page, g] if older else 0.0
                    fin = np.abs(rows[np.isfinite(rows)])
                    s = max(old, pow2_at_least(fin.max() if fin.size else 0.0, 448.0))
                    if older and s > old:
                        codes[page, g, :older] = encode(VALUES[codes[page, g, :older]] * (old / s))
                    codes[page, g, older:older + z - a] = encode(rows / s if s else 0 * rows)
                    scales[page, g] = s
            col += 1
    return codes, scales


def bounds(keys, table, lengths, offsets, out, out_scale, key_scale=None):
    """New (bounds, bound_scale) after the newest tokens: keys [P, Hkv, ps, d]
    are the pages' values, or with key_scale their codes' values."""
    out, out_scale = out.copy(), np.asarray(out_scale, np.float64).copy()
    ps = keys.shape[2]
    for b in range(len(lengths)):
        n = int(lengths[b])
        new = int(offsets[b + 1]) - int(offsets[b])
        for col in range((n - new) // ps, n // ps) if new else ():
            page = table[b][col]
            for g in range(keys.shape[1]):
                lo, hi = keys[page, g].min(0), keys[page, g].max(0)
                s = pow2_at_least(max(np.abs(lo).max(), np.abs(hi).max()), 127.0)
                out[page, g, 0] = np.floor(lo / (s or 1.0))
                out[page, g, 1] = np.ceil(hi / (s or 1.0))
                out_scale[page, g] = s if key_scale is None else s * key_scale[page, g]
    return out, out_scale


def select(Q, page_size, table, lengths, offsets, bnds, bound_scale, n_select):
    """(selected [T, Hkv, n_select], lengths [T]) of packed queries Q [T, H, d]."""
    T, H, d = Q.shape
    Hkv = bnds.shape[1]
    G = H // Hkv
    sel = np.full((T, Hkv, n_select), -1, np.int32)
    rows = np.zeros(T, np.int32)
    for b in range(len(lengths)):
        q0, q1, n = int(offsets[b]), int(offsets[b + 1]), int(lengths[b])
        for t in range(q0, q1):
            pos = n - (q1 - q0) + t - q0
            newest = pos // page_size
            count = min(newest + 1, n_select)
            rows[t] = (count - 1) * page_size + pos % page_size + 1
            for g in range(Hkv):
                score = np.full(newest, -np.inf)
                for h in range(g * G, (g + 1) * G):
                    q = np.where(np.isfinite(Q[t, h]), Q[t, h], 0.0)
                    s = pow2_at_least(np.abs(q).max(), 127.0)
                    qi = np.rint(q / (s or 1.0))
                    for c in range(newest):
                        lo, hi = bnds[table[b][c], g].astype(np.float64)
                        # max(qi lo, qi hi) column by column, for lo <= hi
                        v = (np.maximum(qi, 0) @ hi + np.minimum(qi, 0) @ lo) * s
                        v *= bound_scale[table[b][c], g]
                        score[c] = max(score[c], v)
                best = sorted(range(newest), key=lambda c: (-score[c], c))[:count - 1]
                for i, c in enumerate(sorted(best) + [newest]):
                    sel[t, g, i] = table[b][c]
    return sel, rows


def sdpa_selected(Q, K, V, selected, lengths, scale=0.0):
    """(O, A) of tokens over their own pages per kv head, as paged.sdpa_paged's."""
    T, H, d = Q.shape
    Hkv = K.shape[1]
    G = H // Hkv
    O, A = np.zeros((T, H, d)), np.zeros((T, H, d))
    for t in range(T):
        if lengths[t] == 0:
            continue
        for g in range(Hkv):
            o, a = paged.sdpa_paged(Q[t:t + 1, g * G:(g + 1) * G], K[:, g:g + 1], V[:, g:g + 1],
                                    selected[t, g][None], [lengths[t]], [0, 1], scale=scale)
            O[t, g * G:(g + 1) * G], A[t, g * G:(g + 1) * G] = o[0], a[0]
    return O, A
