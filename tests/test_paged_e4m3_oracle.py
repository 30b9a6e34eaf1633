"""The 8-bit cache's oracle against torch's e4m3, closed forms and brute force."""
import numpy as np
import torch

import oracle.paged as paged
import oracle.paged_e4m3 as ref


def test_codes_are_torch_s():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, ref.VALUES, equal_nan=True)
    x = np.concatenate((np.random.default_rng(1).standard_normal(20000) * 2.0 ** np.arange(-12, 8).repeat(1000),
                        ref.VALUES[:127], (ref.VALUES[:126] + ref.VALUES[1:127]) / 2))
    x = np.clip(np.concatenate((x, -x)), -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(x), want)
    assert np.array_equal(ref.encode([1e9, -1e9, np.nan, np.inf]) & 127, [126, 126, 127, 127])


def test_powers_of_two():
    for top in (448.0, 127.0):
        for x in (1e-45, 1e-30, 0.3, top / 2, top, np.nextafter(top, 999), 1e6, 3e38):
            s = ref.pow2_at_least(x, top)
            assert x <= top * s and (s == 2.0 ** -100 or x > top * s / 2)
    assert ref.pow2_at_least(0.0, 448.0) == 0.0


def test_growing_by_powers_of_two_is_exact_but_for_small_codes():
    for k in (1, 3, 6):
        v = ref.VALUES[:127]
        moved = ref.VALUES[ref.encode(v * 2.0 ** -k)] * 2.0 ** k
        normal = v * 2.0 ** -k >= 2.0 ** -6
        assert np.array_equal(moved[normal], v[normal])
        assert np.all(np.abs(moved - v) <= 2.0 ** (k - 10))


def test_append_in_steps_holds_what_was_appended():
    """Rows of growing size, one, a few or many at a time: every stored row is
    within half a step of its own (and, once the scale has passed it by, of
    the scale's smallest step) however the append was cut."""
    rng = np.random.default_rng(2)
    ps, d, n = 16, 32, 45
    x = rng.standard_normal((n, 2, d)) * 2.0 ** rng.integers(-4, 5, (n, 2, 1))
    table = np.array([[3, 0, 2]])
    for cut in ([45], [1] * 45, [7, 20, 18], [16, 16, 13]):
        codes, scales = np.zeros((4, 2, ps, d), np.uint8), np.full((4, 2), 7.0)
        at = 0
        for k in cut:
            codes, scales = ref.append(codes, scales, x[at:at + k], table, [at + k], [0, k])
            at += k
        got = paged.gather(ref.decode(codes, scales), table[0], n).transpose(1, 0, 2)
        step = np.maximum(2.0 ** -4 * np.abs(x), paged.gather(
            np.broadcast_to(scales[..., None, None], codes.shape), table[0], n).transpose(1, 0, 2)
            * 2.0 ** -10 * 2)     # a code that moves twice is off by two of the smallest half steps
        assert np.all(np.abs(got - x) <= step)


def test_bounds_hold_the_keys_and_scores_bound_the_products():
    rng = np.random.default_rng(3)
    ps, d, P = 16, 64, 9
    K = rng.standard_normal((P, 2, ps, d))
    table = np.array([[5, 1, 7, 0, 2]])
    b, s = np.zeros((P, 2, 2, d), np.int8), np.zeros((P, 2))
    b, s = ref.bounds(K, table, [5 * ps - 3], [0, 5 * ps - 3], b, s)
    assert np.all(s[2] == 0) and np.all(s[table[0, :4]] > 0)    # the last page is not full
    for p in table[0, :4]:
        lo, hi = b[p, :, 0] * s[p, :, None], b[p, :, 1] * s[p, :, None]
        assert np.all(lo[:, None] <= K[p]) and np.all(K[p] <= hi[:, None])
    q = rng.integers(-127, 128, (1, 4, d)).astype(np.float64)    # rounds to itself
    sel, rows = ref.select(q, ps, table, [5 * ps - 3], [0, 1], b, s, 3)
    assert rows[0] == 3 * ps - 3
    for g in range(2):
        top = [max(np.maximum(q[0, h] * b[p, g, 0], q[0, h] * b[p, g, 1]).sum() * s[p, g]
                   for h in (2 * g, 2 * g + 1)) for p in table[0, :4]]
        assert all(top[c] >= (K[p, g] @ q[0, 2 * g:2 * g + 2].T).max() for c, p in enumerate(table[0, :4]))
        best = sorted(np.argsort(top)[-2:])
        assert sel[0, g].tolist() == [*table[0][best], table[0, 4]]


def test_select_with_few_pages_takes_all_and_ties_go_to_the_first():
    b, s = np.ones((6, 1, 2, 64), np.int8), np.ones((6, 1))
    table = np.array([[4, 2, 0, 5, 1]])
    q = np.ones((1, 1, 64))
    sel, rows = ref.select(q, 16, table, [70], [0, 1], b, s, 8)
    assert sel[0, 0].tolist() == [4, 2, 0, 5, 1, -1, -1, -1] and rows[0] == 70
    sel, rows = ref.select(q, 16, table, [70], [0, 1], b, s, 3)
    assert sel[0, 0].tolist() == [4, 2, 1] and rows[0] == 38
    sel, rows = ref.select(q, 16, table, [64], [0, 1], b, s, 1)
    assert sel[0, 0].tolist() == [5] and rows[0] == 16


def test_all_pages_selected_is_the_whole_attention():
    rng = np.random.default_rng(4)
    K, V = rng.standard_normal((2, 5, 2, 16, 32))
    Q = rng.standard_normal((2, 4, 32))
    table = np.array([[3, 1, 4], [0, 2, -1]])
    O, A = paged.sdpa_paged(Q, K, V, table, [40, 20], [0, 1, 2])
    got = ref.sdpa_selected(Q, K, V, np.repeat(table[:, None], 2, 1), [40, 20])
    assert np.allclose(got[0], O, atol=1e-14) and np.allclose(got[1], A, atol=1e-14)
