"""Plain fp64 definitions of the paged cache's operators, in numpy: attention
of packed new tokens over pages, the query/key norm and rotation with its
gradient, and the forking and compacting of pages.

TEST INFRASTRUCTURE ONLY, like the rest of this package: nothing is blocked,
fused or reordered, and nothing is shared with the CUDA library.
"""
from __future__ import annotations

import numpy as np

INTERLEAVED, HALF = 0, 1


def gather(pages, table_row, length):
    """Rows [Hkv, length, d] that a sequence holds in pages [P, Hkv, ps, d]."""
    ps = pages.shape[2]
    rows = [pages[table_row[j // ps], :, j % ps] for j in range(length)]
    return np.stack(rows, axis=1) if rows else np.zeros((pages.shape[1], 0, pages.shape[3]))


def sdpa_paged(Q, K_pages, V_pages, table, lengths, offsets, causal=True, scale=0.0):
    """(O, A) [T, H, d]: the attention of packed queries, and sum_j w_j |v_j|
    per output, which bounds what rounding the weights can do to it.  Rows of
    no sequence are zero."""
    Q = np.asarray(Q, np.float64)
    T, H, d = Q.shape
    G = H // K_pages.shape[1]
    scale = scale or 1.0 / np.sqrt(d)
    O, A = np.zeros((T, H, d)), np.zeros((T, H, d))
    for b in range(len(lengths)):
        q0, q1, n = int(offsets[b]), int(offsets[b + 1]), int(lengths[b])
        if q1 == q0:
            continue
        K = gather(np.asarray(K_pages, np.float64), table[b], n)
        V = gather(np.asarray(V_pages, np.float64), table[b], n)
        for i in range(q1 - q0):
            seen = n - (q1 - q0) + i + 1 if causal else n
            for h in range(H):
                s = scale * (K[h // G, :seen] @ Q[q0 + i, h])
                w = np.exp(s - s.max())
                w /= w.sum()
                O[q0 + i, h] = w @ V[h // G, :seen]
                A[q0 + i, h] = w @ np.abs(V[h // G, :seen])
    return O, A


def _pairs(r, pairing):
    i = np.arange(r // 2)
    return (i, i + r // 2) if pairing == HALF else (2 * i, 2 * i + 1)


def qk_norm_rope(x, gamma, pe, pairing, eps):
    """x [..., d] at table rows pe [..., r] -> the normed, rotated rows."""
    x, pe = np.asarray(x, np.float64), np.asarray(pe, np.float64)
    z = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(gamma, np.float64)
    a, b = _pairs(pe.shape[-1], pairing)
    sn, cs = pe[..., 0::2], pe[..., 1::2]
    y = z.copy()
    y[..., a] = z[..., a] * cs - z[..., b] * sn
    y[..., b] = z[..., b] * cs + z[..., a] * sn
    return y


def qk_norm_rope_backward(x, gamma, pe, dy, pairing, eps):
    """(dx, dgamma) and the sums of magnitudes that bound their rounding."""
    x, pe, dy = (np.asarray(v, np.float64) for v in (x, pe, dy))
    gamma = np.asarray(gamma, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xh = x * rstd
    a, b = _pairs(pe.shape[-1], pairing)
    sn, cs = pe[..., 0::2], pe[..., 1::2]
    dz, mag = dy.copy(), np.abs(dy)
    dz[..., a] = dy[..., a] * cs + dy[..., b] * sn
    dz[..., b] = dy[..., b] * cs - dy[..., a] * sn
    mag[..., a] = np.abs(dy[..., a] * cs) + np.abs(dy[..., b] * sn)
    mag[..., b] = np.abs(dy[..., b] * cs) + np.abs(dy[..., a] * sn)
    u = dz * gamma
    dx = rstd * (u - xh * np.mean(u * xh, -1, keepdims=True))
    mu = mag * np.abs(gamma)
    dx_mag = rstd * (mu + np.abs(xh) * np.mean(mu * np.abs(xh), -1, keepdims=True))
    lead = tuple(range(x.ndim - 1))
    return dx, (dz * xh).sum(lead), dx_mag, (mag * np.abs(xh)).sum(lead)


def fork(K, V, table, lengths, parents, children, fresh):
    """New (K, V, table, lengths) of pools [layers, P, Hkv, ps, d]."""
    K, V, table, lengths = K.copy(), V.copy(), table.copy(), lengths.copy()
    ps = K.shape[3]
    for p, c, f in zip(parents, children, fresh):
        full, rem = divmod(int(lengths[p]), ps)
        table[c, :full] = table[p, :full]
        if rem:
            src = table[p, full]
            K[:, f, :, :rem] = K[:, src, :, :rem]
            V[:, f, :, :rem] = V[:, src, :, :rem]
            table[c, full] = f
        lengths[c] = lengths[p]
    return K, V, table, lengths


def compact(K, V, table, lengths, K_out, V_out, table_out):
    """New (K_out, V_out, table_out) and the number of held pages."""
    K_out, V_out, table_out = K_out.copy(), V_out.copy(), table_out.copy()
    ps = K.shape[3]
    held = [-(-int(n) // ps) for n in lengths]
    live = sorted({int(p) for b, m in enumerate(held) for p in table[b, :m]})
    for r, p in enumerate(live):
        K_out[:, r], V_out[:, r] = K[:, p], V[:, p]
    for b, m in enumerate(held):
        for j in range(m):
            table_out[b, j] = live.index(int(table[b, j]))
    return K_out, V_out, table_out, len(live)
