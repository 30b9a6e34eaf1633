"""Pins of oracle/paged.py (CPU): against the contiguous oracle, torch float64
autograd, finite differences and the properties the formulas fix."""
import numpy as np
import pytest
import torch

import oracle
from oracle import paged
from tests.paged_util import make_pages


@pytest.mark.parametrize("causal", [True, False])
def test_paged_attention_is_decode_over_the_gathered_cache(causal):
    rng = np.random.default_rng(3)
    H = Hkv = 2
    lens, new, ps, d = [37, 5, 64], [4, 5, 1], 16, 8
    K, V, table, offs, _ = make_pages(rng, lens, new, Hkv, ps, d)
    Q = rng.standard_normal((offs[-1], H, d))
    O, A = paged.sdpa_paged(Q, K, V, table, lens, offs, causal)
    for b, (n, m) in enumerate(zip(lens, new)):
        k, v = (paged.gather(x, table[b], n)[None] for x in (K, V))
        q = Q[offs[b]:offs[b + 1]].transpose(1, 0, 2)[None]
        mask = oracle.MASK_CAUSAL_BOTTOM_RIGHT if causal else 0
        ref = oracle.sdpa(q, k, v, mask_kind=mask)
        np.testing.assert_allclose(O[offs[b]:offs[b + 1]].transpose(1, 0, 2), ref[0], atol=1e-13)
    assert np.all(A >= np.abs(O) - 1e-13)


def test_shared_heads_equal_repeated_heads():
    rng = np.random.default_rng(4)
    lens, new, ps, d, Hkv, G = [20, 9], [2, 3], 16, 8, 2, 3
    K, V, table, offs, _ = make_pages(rng, lens, new, Hkv, ps, d)
    Q = rng.standard_normal((offs[-1], Hkv * G, d))
    O, _ = paged.sdpa_paged(Q, K, V, table, lens, offs)
    O2, _ = paged.sdpa_paged(Q, np.repeat(K, G, 1), np.repeat(V, G, 1), table, lens, offs)
    np.testing.assert_array_equal(O, O2)


def _table(n, r):
    return oracle.sinusoidal_pe(n, r)


@pytest.mark.parametrize("pairing", [paged.INTERLEAVED, paged.HALF])
@pytest.mark.parametrize("d,r", [(8, 8), (10, 6), (64, 32)])
def test_norm_rope_gradient(pairing, d, r):
    """The formula's gradient equals torch float64 autograd of the forward
    written with torch operations, and central differences of it."""
    rng = np.random.default_rng(5)
    x, dy = rng.standard_normal((2, 5, 3, d))
    gamma, pe, eps = 1 + 0.3 * rng.standard_normal(d), _table(5, r)[:, None], 1e-3
    y = paged.qk_norm_rope(x, gamma, pe, pairing, eps)
    xt, gt = (torch.tensor(v, requires_grad=True) for v in (x, gamma))
    z = xt * torch.rsqrt((xt * xt).mean(-1, keepdim=True) + eps) * gt
    sn, cs = (torch.tensor(np.ascontiguousarray(pe[..., k::2])) for k in (0, 1))
    a, b = (z[..., :r // 2], z[..., r // 2:r]) if pairing else (z[..., 0:r:2], z[..., 1:r:2])
    u, v = a * cs - b * sn, b * cs + a * sn
    rot = torch.cat((u, v), -1) if pairing else torch.stack((u, v), -1).flatten(-2)
    yt = torch.cat((rot, z[..., r:]), -1)
    np.testing.assert_allclose(y, yt.detach().numpy(), atol=1e-14)
    gx, gg = torch.autograd.grad(yt, (xt, gt), torch.tensor(dy))
    dx, dg, dx_mag, dg_mag = paged.qk_norm_rope_backward(x, gamma, pe, dy, pairing, eps)
    np.testing.assert_allclose(dx, gx.numpy(), atol=1e-13)
    np.testing.assert_allclose(dg, gg.numpy(), atol=1e-13)
    assert np.all(dx_mag >= np.abs(dx) - 1e-13) and np.all(dg_mag >= np.abs(dg) - 1e-13)
    step = 1e-6
    for idx in [(0, 0, 0), (4, 2, d - 1), (2, 1, r - 1)]:
        e = np.zeros_like(x)
        e[idx] = step
        f = [np.sum(paged.qk_norm_rope(x + k * e, gamma, pe, pairing, eps) * dy) for k in (1, -1)]
        assert abs((f[0] - f[1]) / (2 * step) - dx[idx]) < 1e-8


@pytest.mark.parametrize("pairing", [paged.INTERLEAVED, paged.HALF])
def test_rotation_keeps_norms_and_depends_on_the_shift_only(pairing):
    rng = np.random.default_rng(6)
    d, eps = 16, 1e-6
    q, k = rng.standard_normal((2, d))
    pe = _table(200, d)
    rot = lambda x, p: paged.qk_norm_rope(x, np.ones(d), pe[p], pairing, eps)
    assert abs(np.linalg.norm(rot(q, 150)) - np.linalg.norm(rot(q, 0))) < 1e-12
    dots = [rot(q, p + 7) @ rot(k, p) for p in (0, 1, 90, 190)]
    assert np.ptp(dots) < 1e-11


def test_fork_then_attention_matches_the_parent():
    rng = np.random.default_rng(7)
    lens, ps, d, Hkv = [37, 32], 16, 8, 2
    K, V, table, _, free = make_pages(rng, lens, [1, 1], Hkv, ps, d, spare=4)
    table = np.concatenate((table, np.full((2, table.shape[1]), -1, np.int32)))
    lens = np.array(lens + [0, 0], np.int32)
    K2, V2, t2, l2 = paged.fork(K[None], V[None], table, lens, [0, 1], [3, 2], free[:2])
    assert list(l2) == [37, 32, 32, 37] and t2[2, 1] == table[1, 1] and t2[3, 2] == free[0]
    for p, c in ((0, 3), (1, 2)):
        np.testing.assert_array_equal(paged.gather(K2[0], t2[c], l2[c]),
                                      paged.gather(K[:], table[p], lens[p]))


def test_compaction_keeps_every_sequence():
    rng = np.random.default_rng(8)
    lens, ps, d, Hkv = [37, 0, 64, 3], 16, 8, 2
    K, V, table, _, _ = make_pages(rng, lens, [0] * 4, Hkv, ps, d, spare=9)
    table[3, 0] = table[0, 0]
    Ko, Vo = np.zeros((1, 9, Hkv, ps, d)), np.zeros((1, 9, Hkv, ps, d))
    Ko, Vo, to, n = paged.compact(K[None], V[None], table, lens, Ko, Vo, np.full_like(table, -1))
    assert n == 7 and to[3, 0] == to[0, 0]
    for b in range(4):
        np.testing.assert_array_equal(paged.gather(Vo[0], to[b], lens[b]),
                                      paged.gather(V, table[b], lens[b]))
