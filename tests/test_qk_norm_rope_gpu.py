"""qk_norm_rope, its backward and its paged form on the GPU against
oracle/paged.py.

Tolerances, from the arithmetic in fp32 (half step 2^-24): the mean of d <= 256
squares carries at most 8 + 5 roundings along any path, half of which reaches
rstd, rsqrt adds two steps, x * rstd * gamma and the rotation five more: under
2^-19 of |z_a cos| + |z_b sin|, which is at most sqrt(2) times the pair's
length.  Backwards the same for the terms of dx, with the mean of u * xh: under
2^-18 of their magnitudes' sum.  dgamma sums N rows: at most (N + 32) half
steps of the sum of magnitudes.  Outputs round once: 2^-8 (bf16), 2^-24."""
import numpy as np
import pytest
import torch

import oracle.paged as ref
import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from transformer_head_scaled_03_gb300.inputs import round_to_bf16
from tests.gpu_util import to_np
from tests.paged_util import dev, i32, make_pages

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


def draws(rng, shape, dtype, scale=1.0):
    x = rng.standard_normal(shape, dtype=np.float32) * np.float32(scale)
    return round_to_bf16(x) if dtype == BF else x


def within(got, want, mag, rel, dtype, what):
    bound = rel * mag + HALF_STEP[dtype] * np.abs(want) + 1e-35
    worst = float(np.max(np.abs(to_np(got) - want) / bound)) if want.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


def pair_mag(y, r, pairing):
    """|z_a cos| + |z_b sin| <= sqrt(2) |(y_a, y_b)|: a rotation keeps lengths."""
    m = np.abs(y)
    a, b = ref._pairs(r, pairing)
    m[..., a] = m[..., b] = np.sqrt(2) * np.hypot(y[..., a], y[..., b])
    return m


CASES = [
    # dtype, B, L, H, Hkv, d, r, pairing, dq dtype, dk dtype
    (BF, 2, 33, 4, 4, 64, 64, mha.ROPE_INTERLEAVED, F32, BF),
    (BF, 1, 1, 1, 1, 128, 128, mha.ROPE_HALF, F32, BF),
    (BF, 3, 17, 7, 1, 128, 64, mha.ROPE_HALF, BF, F32),
    (BF, 2, 50, 3, 3, 64, 16, mha.ROPE_INTERLEAVED, F32, F32),
    (F32, 1, 128, 8, 8, 64, 64, mha.ROPE_HALF, F32, F32),
    (F32, 2, 9, 5, 2, 128, 32, mha.ROPE_INTERLEAVED, F32, F32),
    (F32, 2, 7, 2, 1, 96, 96, mha.ROPE_HALF, F32, F32),         # any head size
    (BF, 2, 7, 3, 2, 80, 20, mha.ROPE_INTERLEAVED, BF, BF),
    (BF, 1, 5, 2, 2, 64, 24, mha.ROPE_HALF, F32, BF),           # rope_dim not a multiple of 16
    (F32, 1, 3, 1, 1, 2, 2, mha.ROPE_HALF, F32, F32),
    (BF, 1, 4, 2, 1, 256, 250, mha.ROPE_HALF, F32, BF),
    (F32, 1, 6, 2, 0, 64, 64, mha.ROPE_HALF, F32, F32),         # queries alone
    (BF, 1, 700, 16, 2, 128, 128, mha.ROPE_INTERLEAVED, F32, BF),
]


@pytest.mark.parametrize("c", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("given", [False, True])
def test_forward_and_gradient(c, given):
    dt, B, L, H, Hkv, d, r, pairing, dqt, dkt = c
    rng = np.random.default_rng(CASES.index(c))
    off = 0 if given else 5
    n_pos = L + 40
    pos = rng.integers(0, n_pos, (B, L)) if given else off + np.tile(np.arange(L), (B, 1))
    pe = mha.sinusoidal_pe(n_pos, r)
    pe_rows = to_np(pe)[pos][:, :, None]
    positions = i32(pos) if given else None
    # q and k as slices of one projection's output
    wide = dev(draws(rng, (B, L, (H + Hkv) * d + 16), dt, 3.0), dt)
    heads = [wide[..., :H * d].view(B, L, H, d), wide[..., H * d:(H + Hkv) * d].view(B, L, Hkv, d)]
    if d % 8:
        heads = [h.contiguous() for h in heads]
    gammas = [draws(rng, (d,), dt) for _ in range(2)]
    dys = [draws(rng, (B, h, L, d), t) for h, t in ((H, dqt), (Hkv, dkt))]
    kw = dict(pos_offset=off, positions=positions, pairing=pairing, eps=EPS)
    ys = mha.qk_norm_rope(*heads, *(dev(g, dt) for g in gammas), pe, **kw)
    grads = mha.qk_norm_rope_backward(*heads, *(dev(g, dt) for g in gammas), pe,
                                      dev(dys[0], dqt), dev(dys[1], dkt), **kw)
    assert mha.mha_check() == mha.MHA_OK
    for w, h in enumerate((H, Hkv)):
        if h == 0:
            continue
        x = to_np(heads[w])
        y = ref.qk_norm_rope(x, gammas[w], pe_rows, pairing, EPS)
        within(ys[w], y.transpose(0, 2, 1, 3), pair_mag(y, r, pairing).transpose(0, 2, 1, 3),
               2.0 ** -19, dt, "y")
        dx, dg, dx_mag, dg_mag = ref.qk_norm_rope_backward(
            x, gammas[w], pe_rows, dys[w].transpose(0, 2, 1, 3), pairing, EPS)
        within(grads[w], dx, dx_mag, 2.0 ** -18, dt, "dx")
        within(grads[2 + w], dg, dg_mag, (B * L * h + 32) * 2.0 ** -24, F32, "dgamma")
    again = mha.qk_norm_rope_backward(*heads, *(dev(g, dt) for g in gammas), pe,
                                      dev(dys[0], dqt), dev(dys[1], dkt), **kw)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_gradient_agrees_with_differences():
    """Central differences of the library's own fp32 forward.  With |y| < 16
    and steps of 2^-6 the forward's rounding (2^-19 |y| per output, d outputs
    of the row) moves a quotient by less than 2^6 * 2^-19 * 16 * 64 = 0.125;
    in truth by a tenth of it; the third derivative's share is 2^-12 / 6 of
    values of order rstd^3."""
    rng = np.random.default_rng(50)
    d = 64
    x = rng.standard_normal((1, 1, 1, d), dtype=np.float32)
    dy = rng.standard_normal((1, 1, 1, d), dtype=np.float32)
    g = dev(draws(rng, (d,), F32))
    pe = mha.sinusoidal_pe(9, d)
    f = lambda v: float((mha.qk_norm_rope(dev(v), dev(v), g, g, pe, pos_offset=8)[0].double()
                         * dev(dy).double()).sum())
    dx = to_np(mha.qk_norm_rope_backward(dev(x), dev(x), g, g, pe, dev(dy), dev(dy),
                                         pos_offset=8)[0])
    h = np.float32(2.0 ** -6)
    for c in (0, 1, 31, 32, 63):
        e = np.zeros_like(x)
        e[..., c] = h
        assert abs((f(x + e) - f(x - e)) / (2 * float(h)) - dx[0, 0, 0, c]) < 0.125


def test_strided_gradients_and_given_outputs():
    """dQ and dK into slices of one gradient tensor; what lies between stays."""
    rng = np.random.default_rng(51)
    B, L, H, Hkv, d = 2, 11, 4, 2, 64
    wide = dev(draws(rng, (B, L, (H + 2 * Hkv) * d), BF), BF)
    q, k = wide[..., :H * d].view(B, L, H, d), wide[..., H * d:(H + Hkv) * d].view(B, L, Hkv, d)
    g = dev(draws(rng, (d,), BF), BF)
    pe = mha.sinusoidal_pe(L, d)
    dys = [dev(draws(rng, (B, h, L, d), F32)) for h in (H, Hkv)]
    want = mha.qk_norm_rope_backward(q, k, g, g, pe, *dys)
    dwide = torch.full_like(wide, 7.0)
    out = (dwide[..., :H * d].view(B, L, H, d), dwide[..., H * d:(H + Hkv) * d].view(B, L, Hkv, d))
    mha.qk_norm_rope_backward(q, k, g, g, pe, *dys, out=out)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert torch.all(dwide[..., (H + Hkv) * d:] == 7.0)
    ys = mha.qk_norm_rope(q, k, g, g, pe)
    given = tuple(torch.empty_like(y) for y in ys)
    mha.qk_norm_rope(q, k, g, g, pe, out=given)
    assert all(torch.equal(a, b) for a, b in zip(ys, given))


@pytest.mark.parametrize("d,r", [(64, 64), (96, 32)])
def test_bad_positions_are_reported(d, r):
    rng = np.random.default_rng(52)
    B, L, H = 1, 6, 3
    x = dev(draws(rng, (B, L, H, d), F32))
    g = dev(draws(rng, (d,), F32))
    pe = mha.sinusoidal_pe(10, r)
    dy = dev(draws(rng, (B, H, L, d), F32))
    pos = i32([[0, 9, 10, -1, 2 ** 31 - 1, 3]])
    fine = i32([[0, 9, 0, 0, 0, 3]])
    good = [0, 1, 5]
    yq, yk = mha.qk_norm_rope(x, x, g, g, pe, positions=pos)
    assert mha.mha_check() == mha.MHA_ERR_DEVICE
    dq, dk, dgq, dgk = mha.qk_norm_rope_backward(x, x, g, g, pe, dy, dy, positions=pos)
    assert mha.mha_check() == mha.MHA_ERR_DEVICE
    bad = [2, 3, 4]
    assert torch.all(yq[:, :, bad] == 0) and torch.all(dq[:, bad] == 0)
    wq, _ = mha.qk_norm_rope(x, x, g, g, pe, positions=fine)
    masked = dy.clone()
    masked[:, :, bad] = 0
    wdq, _, wdgq, _ = mha.qk_norm_rope_backward(x, x, g, g, pe, masked, masked, positions=fine)
    assert mha.mha_check() == mha.MHA_OK
    assert torch.equal(yq[:, :, good], wq[:, :, good]) and torch.equal(dq[:, good], wdq[:, good])
    assert torch.equal(dgq, wdgq) and torch.equal(dgk, dgq) and torch.equal(yk, yq)


def test_no_rows_give_zero_gamma_gradients():
    x = torch.empty((0, 4, 2, 64), dtype=BF, device="cuda")
    g = torch.ones(64, dtype=BF, device="cuda")
    pe = mha.sinusoidal_pe(4, 64)
    dy = torch.empty((0, 2, 4, 64), dtype=BF, device="cuda")
    *_, dgq, dgk = mha.qk_norm_rope_backward(x, x, g, g, pe, dy, dy)
    assert torch.all(dgq == 0) and torch.all(dgk == 0) and mha.mha_check() == mha.MHA_OK


def test_nan_stays_in_its_row():
    rng = np.random.default_rng(53)
    x = draws(rng, (1, 5, 3, 64), F32)
    g = dev(draws(rng, (64,), F32))
    pe = mha.sinusoidal_pe(5, 64)
    clean = mha.qk_norm_rope(dev(x), dev(x), g, g, pe)[0]
    x[0, 2, 1, 7], x[0, 4, 2, 0] = np.nan, np.inf
    y = mha.qk_norm_rope(dev(x), dev(x), g, g, pe)[0]
    same = torch.ones((1, 3, 5), dtype=torch.bool, device="cuda")
    same[0, 1, 2] = same[0, 2, 4] = False
    assert torch.equal(y[same], clean[same]) and torch.all(torch.isnan(y[0, 1, 2]))


def test_step_captured_while_an_eager_one_lives():
    """Forward and backward in a graph on another stream, replayed on new
    inputs, give the eager call's bits."""
    rng = np.random.default_rng(54)
    B, L, H, d = 2, 40, 4, 64
    x = dev(draws(rng, (B, L, H, d), BF), BF)
    g, pe = dev(draws(rng, (d,), BF), BF), mha.sinusoidal_pe(L, d)
    dy = dev(draws(rng, (B, H, L, d), F32))
    eager = mha.qk_norm_rope(x, x, g, g, pe)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        y = mha.qk_norm_rope(x, x, g, g, pe)
        gr = mha.qk_norm_rope_backward(x, x, g, g, pe, dy, dy)
    for k in range(2):
        x.copy_(dev(draws(rng, (B, L, H, d), BF), BF))
        graph.replay()
        want = mha.qk_norm_rope_backward(x, x, g, g, pe, dy, dy)
        wy = mha.qk_norm_rope(x, x, g, g, pe)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(gr, want))
        assert all(torch.equal(a, b) for a, b in zip(y, wy))
    assert eager[0].shape == y[0].shape and mha.mha_check() == mha.MHA_OK


# --------------------------------------------------------------------- paged form

def paged_case(seed, lens, new, H, Hkv, ps, d, r, spare=3, extra=0):
    rng = np.random.default_rng(seed)
    K, V, table, offs, _ = make_pages(rng, lens, new, Hkv, ps, d, bf16=True, spare=spare)
    T = int(offs[-1]) + extra
    rows = [draws(rng, (T, h, d), BF, 2.0) for h in (H, Hkv, Hkv)]
    gammas = [draws(rng, (d,), BF) for _ in range(2)]
    return K, V, table, np.asarray(lens, np.int32), offs, rows, gammas


PAGED = [
    # lens, new, H, Hkv, page, d, r, pairing
    ([1], [1], 1, 1, 16, 64, 64, mha.ROPE_HALF),
    ([37, 16, 90], [1, 1, 1], 8, 2, 16, 128, 128, mha.ROPE_HALF),
    ([37, 0, 90, 5], [20, 0, 33, 5], 5, 1, 32, 64, 32, mha.ROPE_INTERLEAVED),
    ([300], [300], 4, 4, 128, 128, 64, mha.ROPE_INTERLEAVED),
    ([3] * 70, [1, 2] * 35, 3, 3, 16, 64, 64, mha.ROPE_HALF),
    ([513, 600], [2, 200], 32, 8, 256, 128, 128, mha.ROPE_HALF),
]


@pytest.mark.parametrize("c", PAGED, ids=[str(i) for i in range(len(PAGED))])
def test_paged_parity(c):
    lens, new, H, Hkv, ps, d, r, pairing = c
    K, V, table, lens, offs, (q, k, v), gammas = paged_case(60 + PAGED.index(c), lens, new, H, Hkv,
                                                            ps, d, r, extra=3)
    kp, vp = dev(K, BF), dev(V, BF)
    pe = mha.sinusoidal_pe(int(lens.max()), r)
    T = int(offs[-1])
    wide = torch.cat([dev(x, BF).flatten(1) for x in (q, k, v)], 1)
    parts = [x.view(T + 3, -1, d) for x in wide.split([H * d, Hkv * d, Hkv * d], 1)]
    out = torch.full((T + 3, H, d), 7.0, dtype=BF, device="cuda")
    mha.qk_norm_rope_paged(*parts, *(dev(g, BF) for g in gammas), pe, kp, vp, i32(table), i32(lens),
                           i32(offs), pairing=pairing, eps=EPS, out=out)
    assert mha.mha_check() == mha.MHA_OK
    seq = np.repeat(np.arange(len(lens)), np.diff(offs))
    pos = (lens - np.diff(offs))[seq] + np.arange(T) - offs[seq]
    rows = to_np(pe)[pos][:, None]
    y = ref.qk_norm_rope(q[:T], gammas[0], rows, pairing, EPS)
    within(out[:T], y, pair_mag(y, r, pairing), 2.0 ** -19, BF, "q")
    assert torch.all(out[T:] == 7.0)
    y = ref.qk_norm_rope(k[:T], gammas[1], rows, pairing, EPS)
    page, row = table[seq, pos // ps], pos % ps
    within(kp[page, :, row], y, pair_mag(y, r, pairing), 2.0 ** -19, BF, "k")
    assert np.array_equal(to_np(vp[page, :, row]), v[:T])
    touched = np.zeros(K.shape[:1] + K.shape[2:3], bool)
    touched[page, row] = True
    assert np.array_equal(to_np(kp).transpose(0, 2, 1, 3)[~touched], K.transpose(0, 2, 1, 3)[~touched])
    assert np.array_equal(to_np(vp).transpose(0, 2, 1, 3)[~touched], V.transpose(0, 2, 1, 3)[~touched])


@pytest.mark.parametrize("new", [1, 9])
def test_paged_bad_entries_touch_nothing(new):
    K, V, table, lens, offs, parts, gammas = paged_case(80, [40, 50, 30], [new] * 3, 4, 2, 16, 64, 64)
    parts = [dev(x, BF) for x in parts]
    g = [dev(x, BF) for x in gammas]
    pe = mha.sinusoidal_pe(64, 64)
    rows = lambda b: slice(int(offs[b]), int(offs[b + 1]))

    def call(table=table, lens=lens, offs=offs, pe=pe):
        kp, vp = dev(K, BF), dev(V, BF)
        out = torch.full((int(parts[0].shape[0]), 4, 64), 7.0, dtype=BF, device="cuda")
        mha.qk_norm_rope_paged(*parts, *g, pe, kp, vp, i32(table), i32(lens), i32(offs), out=out)
        return out, kp, vp, mha.mha_check()

    fine, kf, vf, st = call()
    assert st == mha.MHA_OK
    pages1 = torch.from_numpy(table[1][table[1] >= 0].astype(np.int64)).cuda()

    def only_1_missing(res):
        out, kp, vp, st = res
        assert st == mha.MHA_ERR_DEVICE and mha.mha_check() == mha.MHA_OK
        assert torch.all(out[rows(1)] == 0)
        for b in (0, 2):
            assert torch.equal(out[rows(b)], fine[rows(b)])
        wk, wv = kf.clone(), vf.clone()
        wk[pages1], wv[pages1] = dev(K, BF)[pages1], dev(V, BF)[pages1]
        assert torch.equal(kp, wk) and torch.equal(vp, wv)

    for n in (new - 1, table.shape[1] * 16 + 1, -3, 2 ** 31 - 1):
        only_1_missing(call(lens=[lens[0], n, lens[2]]))
    for page in (-1, K.shape[0], 2 ** 31 - 1):
        t = table.copy()
        t[1] = page
        only_1_missing(call(table=t))
    only_1_missing(call(pe=mha.sinusoidal_pe(41, 64)))      # the table ends before position 41
    T = int(offs[-1])
    out, kp, vp, st = call(offs=[0, offs[1], offs[2], T + 4])
    assert st == mha.MHA_ERR_DEVICE and torch.all(out[rows(2)] == 7.0)
    assert torch.equal(out[rows(0)], fine[rows(0)])


def test_paged_empty():
    K, V, table, lens, offs, parts, gammas = paged_case(90, [5], [1], 2, 1, 16, 64, 64)
    pe = mha.sinusoidal_pe(5, 64)
    args = lambda T, o: [*(dev(x[:T], BF) for x in parts), *(dev(g, BF) for g in gammas), pe,
                         dev(K, BF), dev(V, BF), i32(table), i32(lens), i32(o)]
    assert mha.qk_norm_rope_paged(*args(0, [0, 0])).shape == (0, 2, 64)
    a = args(1, [0, 0])
    mha.qk_norm_rope_paged(*a)
    assert mha.mha_check() == mha.MHA_OK and torch.equal(a[6], dev(K, BF))


@pytest.mark.parametrize("lead", [1, 9, 40])
@pytest.mark.parametrize("new", [[1, 1, 1], [0, 5, 12]])
def test_paged_tokens_ahead_of_the_first_sequence(lead, new):
    """q_offsets[0] > 0 is allowed: the tokens ahead of it belong to no
    sequence and are passed over, like those behind the last one."""
    K, V, table, lens, offs, parts, gammas = paged_case(95, [40, 50, 30], new, 4, 2, 16, 64, 64,
                                                        extra=lead + 3)
    g, pe = [dev(x, BF) for x in gammas], mha.sinusoidal_pe(64, 64)
    T = int(offs[-1])

    def call(first):
        kp, vp = dev(K, BF), dev(V, BF)
        rows = [dev(np.roll(x, first, 0), BF) for x in parts]
        out = torch.full(rows[0].shape, 7.0, dtype=BF, device="cuda")
        mha.qk_norm_rope_paged(*rows, *g, pe, kp, vp, i32(table), i32(lens), i32(offs + first),
                               out=out)
        assert mha.mha_check() == mha.MHA_OK
        assert torch.all(out[:first] == 7.0) and torch.all(out[first + T:] == 7.0)
        return out[first:first + T], kp, vp

    for a, b in zip(call(0), call(lead)):
        assert torch.equal(a, b)


def test_paged_offsets_that_do_not_ascend_are_reported():
    K, V, table, lens, offs, parts, gammas = paged_case(96, [40, 50, 30], [4, 4, 4], 4, 2, 16, 64, 64)
    g, pe = [dev(x, BF) for x in gammas], mha.sinusoidal_pe(64, 64)
    for o in ([-1, 4, 8, 12], [6, 4, 8, 12], [0, 4, 8, 13], [0, 9, 12, 2], [0, 9, 1, 2]):
        mha.qk_norm_rope_paged(*(dev(x, BF) for x in parts), *g, pe, dev(K, BF), dev(V, BF),
                               i32(table), i32(lens), i32(o))
        assert mha.mha_check() == mha.MHA_ERR_DEVICE, o


@pytest.mark.parametrize("value", [np.inf, np.nan])
@pytest.mark.parametrize("dt,d,r", [(BF, 64, 64), (F32, 64, 32), (F32, 128, 128), (F32, 96, 32)])
@pytest.mark.parametrize("pairing", [mha.ROPE_INTERLEAVED, mha.ROPE_HALF])
def test_bad_positions_give_zeros_whatever_gamma_holds(value, dt, d, r, pairing):
    rng = np.random.default_rng(55)
    B, L, H, Hkv = 1, 7, 3, 2
    q, k = (dev(draws(rng, (B, L, h, d), dt), dt) for h in (H, Hkv))
    gammas = draws(rng, (d,), dt), draws(rng, (d,), dt)
    for x in gammas:
        x[[0, d // 2, d - 1]] = value
    g = [dev(x, dt) for x in gammas]
    pe = mha.sinusoidal_pe(10, r)
    dys = [dev(draws(rng, (B, h, L, d), F32)) for h in (H, Hkv)]
    pos, bad = i32([[0, 10, 9, -1, 3, 2 ** 31 - 1, 4]]), [1, 3, 5]
    ys = mha.qk_norm_rope(q, k, *g, pe, positions=pos, pairing=pairing)
    assert mha.mha_check() == mha.MHA_ERR_DEVICE
    grads = mha.qk_norm_rope_backward(q, k, *g, pe, *dys, positions=pos, pairing=pairing)
    assert mha.mha_check() == mha.MHA_ERR_DEVICE
    for y, dx in zip(ys, grads):
        assert torch.all(y[:, :, bad] == 0) and torch.all(dx[:, bad] == 0)
        assert not torch.all(torch.isfinite(y)) and not torch.all(torch.isfinite(dx))
    # dgamma takes no gamma: the other rows' sums, finite
    assert all(torch.all(torch.isfinite(x)) for x in grads[2:])


@pytest.mark.parametrize("value", [np.inf, np.nan])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pairing", [mha.ROPE_INTERLEAVED, mha.ROPE_HALF])
def test_paged_bad_entries_give_zeros_whatever_gamma_holds(value, d, pairing):
    K, V, table, lens, offs, parts, gammas = paged_case(97, [40, 50, 30], [4, 4, 4], 4, 2, 16, d, d)
    for x in gammas:
        x[[0, d // 2, d - 1]] = value
    lens[0], table[1] = 3, K.shape[0]           # a length below its new tokens, pages out of range
    kp, vp = dev(K, BF), dev(V, BF)
    out = torch.full(parts[0].shape, 7.0, dtype=BF, device="cuda")
    mha.qk_norm_rope_paged(*(dev(x, BF) for x in parts), *(dev(x, BF) for x in gammas),
                           mha.sinusoidal_pe(64, d), kp, vp, i32(table), i32(lens), i32(offs),
                           pairing=pairing, out=out)
    assert mha.mha_check() == mha.MHA_ERR_DEVICE
    assert torch.all(out[:8] == 0) and not torch.all(torch.isfinite(out[8:]))
    others = [p for p in range(K.shape[0]) if p not in table[2]]
    assert torch.equal(kp[others], dev(K, BF)[others]) and torch.equal(vp[others], dev(V, BF)[others])


@pytest.mark.parametrize("d", [64, 96])
def test_no_heads_give_zero_gamma_gradients(d):
    """H = Hkv = 0: dgamma is overwritten all the same, with a sum of nothing."""
    x = torch.empty((2, 5, 0, d), dtype=BF, device="cuda")
    dy = torch.empty((2, 0, 5, d), dtype=F32, device="cuda")
    g, pe = torch.ones(d, dtype=BF, device="cuda"), mha.sinusoidal_pe(5, d)
    for _ in range(3):
        # the pieces that the allocator hands out next are not zeros
        junk = [torch.full((n,), 7.0, device="cuda") for n in (2 * d,) * 8]
        del junk
        dq, dk, dgq, dgk = mha.qk_norm_rope_backward(x, x, g, g, pe, dy, dy)
        assert dq.shape == dk.shape == (2, 5, 0, d)
        assert torch.all(dgq == 0) and torch.all(dgk == 0) and mha.mha_check() == mha.MHA_OK
