"""kv_pages_bounds, kv_pages_select and sdpa_paged_selected on the GPU against
the oracle: bounds and choices are whole numbers and powers of two, so those
comparisons are exact; the attention's tolerances are the paged attention's."""
import numpy as np
import pytest
import torch

import oracle.paged as paged
import oracle.paged_e4m3 as ref
import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from transformer_head_scaled_03_gb300.inputs import round_to_bf16
from tests.e4m3_util import attention_bound, codes_of, dev8, f32, make_pages8
from tests.gpu_util import to_np
from tests.paged_util import dev, i32, make_pages

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


def i8(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int8)).cuda()


# ------------------------------------------------------------------------ bounds

def bounds_case(seed, lens, new, Hkv, ps, d, e8, layers=None):
    rng = np.random.default_rng(seed)
    if e8:
        kc, ks, vc, vs, table, offs, _ = make_pages8(rng, lens, new, Hkv, ps, d, pow2=seed % 2 == 0,
                                                     layers=layers)
        keys, pools = ref.VALUES[kc], (dev8(kc), dev8(vc))
        sc = dict(K_scale=f32(ks), V_scale=f32(vs))
    else:
        K, V, table, offs, _ = make_pages(rng, lens, new, Hkv, ps, d, bf16=True, layers=layers)
        K = round_to_bf16((K * 2.0 ** rng.integers(-20, 20, (*K.shape[:-2], 1, 1))).astype(np.float32))
        ks, keys, pools, sc = None, K.astype(np.float64), (dev(K, BF), dev(V, BF)), {}
    shape = (*keys.shape[:-2], 2, d)
    b = rng.integers(-128, 128, shape).astype(np.int8)
    s = rng.random(shape[:-2]).astype(np.float32)
    return keys, ks, pools, sc, table, np.asarray(lens, np.int32), offs, b, s


BOUNDS = [
    ([16], [1], 1, 16, 64), ([16], [16], 1, 16, 64), ([15, 17], [15, 2], 2, 16, 128),
    ([48, 0, 100, 33], [1, 0, 70, 1], 3, 16, 64), ([300, 129, 64], [300, 65, 1], 2, 64, 128),
    ([513, 256], [400, 256], 8, 256, 64), ([700] + [32] * 80, [650] + [1] * 80, 1, 32, 128),
]


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("c", BOUNDS, ids=[str(i) for i in range(len(BOUNDS))])
def test_bounds(c, e8):
    keys, ks, pools, sc, table, lens, offs, b, s = bounds_case(500 + BOUNDS.index(c), *c, e8)
    want, ws = ref.bounds(keys, table, lens, offs, b, s, None if ks is None else np.float32(ks))
    gb, gs = i8(b), f32(s)
    mha.kv_pages_bounds(*pools, i32(table), i32(lens), i32(offs), gb, gs, int(offs[-1]), **sc)
    assert mha.mha_check() == mha.MHA_OK
    assert np.array_equal(gb.cpu().numpy(), want)
    assert np.array_equal(to_np(gs), ws.astype(np.float32))


@pytest.mark.parametrize("e8", [False, True])
def test_bounds_of_zeros_edges_and_one_layer(e8):
    """A page of zeros, of one sign, of a largest element that is 127 steps, or
    just more; in the middle layer."""
    keys, ks, pools, sc, table, lens, offs, b, s = bounds_case(520, [80], [80], 2, 16, 64, e8, layers=3)
    v = keys[1]
    p = table[0]
    v[p[0]], v[p[1]], v[p[2]] = 0, np.abs(v[p[1]]), -np.abs(v[p[2]])
    if not e8:
        v[p[3]] = np.clip(v[p[3]], -1, 1)
        v[p[3], 0, 3, 5], v[p[3], 1, 3, 5] = 127 * 2.0 ** 7, -(127 + 1) * 2.0 ** 7
        pools[0].copy_(dev(keys, BF))
    else:
        codes = np.stack([ref.encode(x) for x in keys])
        pools[0].view(torch.uint8).copy_(dev(codes))
    want, ws = ref.bounds(v, table, lens, offs, b[1], s[1], None if ks is None else np.float32(ks[1]))
    gb, gs = i8(b), f32(s)
    mha.kv_pages_bounds(*pools, i32(table), i32(lens), i32(offs), gb, gs, 80, layer=1, **sc)
    assert mha.mha_check() == mha.MHA_OK
    assert np.array_equal(gb[1].cpu().numpy(), want) and np.array_equal(to_np(gs[1]), ws.astype(np.float32))
    for y in (0, 2):
        assert np.array_equal(gb[y].cpu().numpy(), b[y]) and np.array_equal(to_np(gs[y]), s[y])


def test_bounds_report_bad_entries_and_leave_them():
    c = ([64, 48, 80], [64, 48, 80], 2, 16, 64)
    keys, ks, pools, sc, table, lens, offs, b, s = bounds_case(530, *c, False)
    want, ws = ref.bounds(keys, table, lens, offs, b, s)

    def call(untouched, table=table, lens=lens, offs=offs):
        gb, gs = i8(b), f32(s)
        mha.kv_pages_bounds(*pools, i32(table), i32(lens), i32(offs), gb, gs, 192)
        assert mha.mha_check() == mha.MHA_ERR_DEVICE
        wb, w2 = want.copy(), ws.copy()
        for p in untouched:
            wb[p], w2[p] = b[p], s[p]
        assert np.array_equal(gb.cpu().numpy(), wb) and np.array_equal(to_np(gs), w2.astype(np.float32))

    for n in (47, -1, 81, 2 ** 31 - 1):
        call(table[1, :3], lens=[64, n, 80])
    for page in (-1, keys.shape[0], 2 ** 31 - 1):
        t = table.copy()
        t[1, 1] = page
        call(table[1, 1:2], table=t)
    call(table[2, :5], offs=[0, 64, 112, 193])


# ------------------------------------------------------------------------ select

def select_case(seed, lens, new, H, Hkv, ps, d, spread=0, cols=None):
    rng = np.random.default_rng(seed)
    held = [-(-n // ps) for n in lens]
    P = sum(held) + 3
    perm = rng.permutation(P).astype(np.int32)
    table = np.full((len(lens), cols or max(1, max(held))), -1, np.int32)
    at = 0
    for i, m in enumerate(held):
        table[i, :m] = perm[at:at + m]
        at += m
    mid, reach = rng.integers(-60, 61, (P, Hkv, d)), rng.integers(0, 68, (P, Hkv, d))
    b = np.stack((mid - reach, mid + reach), 2).astype(np.int8)
    s = 2.0 ** rng.integers(-6 - spread, -4 + spread, (P, Hkv))
    offs = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    Q = round_to_bf16(rng.standard_normal((offs[-1], H, d), dtype=np.float32)
                      * np.float32(2.0) ** rng.integers(-spread, spread + 1, (offs[-1], H, 1)))
    return Q, ps, table, np.asarray(lens, np.int32), offs, b, s


def run_select(x, n, Q=None, **kw):
    Qx, ps, table, lens, offs, b, s = x
    Q = Qx if Q is None else Q
    P, Hkv, _, d = b.shape
    pool = torch.zeros((P, Hkv, ps, d), dtype=BF, device="cuda")
    sel, rows = mha.kv_pages_select(dev(Q, BF), pool, pool, i32(table), i32(lens), i32(offs), i8(b), f32(s),
                                    n, **kw)
    return sel, rows


SELECTS = [
    # lens, new, H, Hkv, page, d, n_select
    ([1], [1], 1, 1, 16, 64, 1), ([700], [1], 8, 8, 16, 64, 8), ([700], [1], 8, 2, 16, 128, 1),
    ([700, 0, 64, 65, 48], [1, 0, 1, 1, 1], 8, 2, 16, 128, 5), ([520, 100], [3, 40], 6, 2, 32, 64, 4),
    ([2000], [2], 14, 2, 16, 128, 100), ([300], [1], 128, 1, 16, 64, 7), ([300, 600], [2, 1], 33, 3, 16, 128, 9),
    ([9000], [1], 2, 1, 16, 64, 300), ([1000, 260], [1, 1], 4, 4, 256, 64, 2), ([100], [1], 4, 2, 16, 64, 50),
    ([16 * 40] * 40, [1] * 40, 2, 1, 16, 64, 6),
    ([50000, 33], [1, 1], 2, 1, 16, 64, 40), ([16 * 9000 + 5], [1], 1, 1, 16, 64, 3000),    # thousands of pages
]


@pytest.mark.parametrize("c", SELECTS, ids=[str(i) for i in range(len(SELECTS))])
def test_select(c):
    *shape, n = c
    x = select_case(540 + SELECTS.index(c), *shape, spread=SELECTS.index(c) % 3)
    want, rows = ref.select(x[0], *x[1:], n)
    sel, got = run_select(x, n)
    assert mha.mha_check() == mha.MHA_OK
    assert np.array_equal(got.cpu().numpy(), rows) and np.array_equal(sel.cpu().numpy(), want)


def test_equal_scores_go_to_the_first_pages():
    x = select_case(560, [3000], [1], 4, 2, 16, 64)
    b = x[5]
    for few in (1, 3):       # one value, or three values, in all pages
        b[:] = np.random.default_rng(few).integers(-9, 10, (few, 1, 2, 64)).repeat(-(-len(b) // few), 0)[:len(b)]
        x[6][:] = 0.25
        for n in (1, 2, 60, 187, 188, 189):
            want, rows = ref.select(x[0], *x[1:], n)
            sel, got = run_select(x, n)
            assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(got.cpu().numpy(), rows)
    x[6][:] = 0.0            # no score at all
    want, _ = ref.select(x[0], *x[1:], 20)
    assert np.array_equal(run_select(x, 20)[0].cpu().numpy(), want)


@pytest.mark.parametrize("pages", [700, 9000])
def test_one_score_far_from_the_rest(pages):
    """An outlier, infinite scores, and more equal scores than are compared with
    one another: the search by bits."""
    x = select_case(570, [16 * pages + 3], [1], 1, 1, 16, 64)
    Q, ps, table, lens, offs, b, s = x
    first = s.copy()
    for far in (2.0 ** 100, 3e38, np.inf):
        s[:] = first
        s[table[0, 17], 0] = far
        s[table[0, 400], 0] = far / 4
        for n in (1, 2, 3, 300, pages - 5):
            with np.errstate(invalid="ignore"):
                want, rows = ref.select(Q, *x[1:], n)
            sel, got = run_select(x, n)
            assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(got.cpu().numpy(), rows)
    b[table[0, 5:]] = b[table[0, 5]]        # and nearly all equal beside it
    s[:] = 0.5
    s[table[0, 3], 0] = 2.0 ** 90
    for n in (1, 2, 5, 600, pages - 2):
        want, rows = ref.select(Q, *x[1:], n)
        assert np.array_equal(run_select(x, n)[0].cpu().numpy(), want)
    assert mha.mha_check() == mha.MHA_OK


def test_queries_of_zeros_any_size_and_not_finite():
    x = select_case(561, [900], [6], 2, 1, 16, 64)
    Q = x[0]
    Q[0] = 0
    Q[1] *= np.float32(2.0 ** -90)
    Q[2] = round_to_bf16(Q[2] * np.float32(2.0 ** 100))
    Q[3, 0, 5], Q[3, 1, 9], Q[4, 0, :] = np.nan, np.inf, -np.inf
    want, rows = ref.select(Q, *x[1:], 7)
    sel, got = run_select(x, 7)
    assert mha.mha_check() == mha.MHA_OK
    assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(got.cpu().numpy(), rows)


def test_products_beyond_fp32_are_no_bad_pages():
    """The largest queries: products in fp32 as documented, so infinities, which
    times a page's scale of 0 are NaN and count least."""
    x = select_case(562, [900], [3], 2, 1, 16, 64)
    Q, ps, table, lens, offs, b, s = x
    Q[:] = round_to_bf16(np.sign(Q) * np.float32(2.0 ** 126) * (1 + np.abs(Q) / 8))
    s[table[0, 3:50:5]] = 0
    n = 12
    sel, got = run_select(x, n)
    assert mha.mha_check() == mha.MHA_OK
    assert got.tolist() == [(n - 1) * ps + p % ps + 1 for p in (897, 898, 899)]
    f = np.float32
    with np.errstate(over="ignore", invalid="ignore"):
        for t in range(3):
            newest = (897 + t) // ps
            page = table[0, :newest]
            best = np.full(newest, -np.inf, f)
            for h in range(2):
                step = ref.pow2_at_least(np.abs(Q[t, h]).max(), 127.0)
                qi = np.rint(Q[t, h] / step)
                v = np.maximum(qi, 0) @ b[page, 0, 1].T.astype(float) \
                    + np.minimum(qi, 0) @ b[page, 0, 0].T.astype(float)
                best = np.maximum(best, f(v) * f(step))
            score = best * s[page, 0].astype(f)
            key = np.where(np.isnan(score), -np.inf, score)
            order = sorted(range(newest), key=lambda c: (bool(np.isnan(score[c])), -key[c], c))[:n - 1]
            assert np.isnan(score).any() and np.isinf(score).any()
            assert sel[t, 0].tolist() == [table[0, c] for c in sorted(order)] + [table[0, newest]]


def test_what_lies_behind_the_newest_page_is_never_used():
    """Bounds and scales of spare, partly filled and later pages, and entries
    behind the last page, may hold anything."""
    x = select_case(562, [500, 47], [3, 1], 4, 2, 16, 64, cols=40)
    want, rows = ref.select(x[0], *x[1:], 6)
    Q, ps, table, lens, offs, b, s = x
    full = {int(p) for i, n in enumerate(lens) for p in table[i, :n // ps]}
    rest = [p for p in range(len(b)) if p not in full]
    b[rest], s[rest] = 127, np.nan
    table[table < 0] = 2 ** 31 - 1
    want[want < 0] = -1
    sel, got = run_select(x, 6)
    assert mha.mha_check() == mha.MHA_OK
    assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(got.cpu().numpy(), rows)


def test_select_reports_bad_entries():
    x = select_case(563, [500, 400, 300], [2, 2, 2], 4, 2, 16, 64)
    Q, ps, table, lens, offs, b, s = x
    want, rows = ref.select(Q, *x[1:], 6)

    def call(bad, none=(), **kw):
        y = list(x)
        for k, v in kw.items():
            y[dict(table=2, lens=3, offs=4)[k]] = np.asarray(v, np.int32)
        sel, got = run_select(y, 6)
        assert mha.mha_check() == mha.MHA_ERR_DEVICE
        sel, got = sel.cpu().numpy(), got.cpu().numpy()
        for t in range(6):
            if t in bad or t in none:
                assert np.all(sel[t] == -1) and got[t] == (-1 if t in bad else 0)
            else:
                assert np.array_equal(sel[t], want[t]) and got[t] == rows[t]

    for n in (1, -1, table.shape[1] * 16 + 1):
        call((2, 3), lens=[500, n, 300])
    for col in (0, 20, 24):            # the first page, one in the middle, the newest
        t = table.copy()
        t[1, col] = len(b) if col else -1
        call((2, 3), table=t)
    call((4, 5), offs=[0, 2, 4, 7])
    short = select_case(564, [40, 30], [1, 1], 2, 1, 16, 64)
    short[2][0, 1] = -5                # every page there is, one of them bad
    sel, got = run_select(short, 9)
    assert mha.mha_check() == mha.MHA_ERR_DEVICE
    assert got.tolist() == [-1, 30] and torch.all(sel[0] == -1) and torch.all(sel[1, 0, 2:] == -1)


def test_tokens_of_no_sequence():
    x = select_case(565, [100, 90], [2, 3], 2, 1, 16, 64)
    Q, ps, table, lens, offs, b, s = x
    pad = np.concatenate((Q[:1], Q, Q[:2]))
    want, rows = ref.select(pad, ps, table, lens, offs + 1, b, s, 3)
    sel, got = run_select((pad, ps, table, lens, offs + 1, b, s), 3)
    assert mha.mha_check() == mha.MHA_OK
    assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(got.cpu().numpy(), rows)
    assert rows[0] == 0 and rows[-1] == 0
    # and with no sequences at all
    none = (pad, ps, table[:0], lens[:0], np.zeros(1, np.int32), b, s)
    sel, got = run_select(none, 3)
    assert mha.mha_check() == mha.MHA_OK and torch.all(sel == -1) and torch.all(got == 0)


def test_select_into_given_tensors_on_streams_and_layers():
    x = select_case(566, [600, 333], [1, 2], 8, 2, 16, 128)
    Q, ps, table, lens, offs, b, s = x
    want, rows = ref.select(Q, *x[1:], 9)
    wide = torch.randn((3, 10 * 128), device="cuda").to(BF)
    q = wide[:, 128:9 * 128].view(3, 8, 128)
    q.copy_(dev(Q, BF))
    P = len(b)
    pool = torch.zeros((2, P, 2, ps, 128), dtype=BF, device="cuda")
    b2 = np.stack((np.random.default_rng(1).integers(-9, 9, b.shape).astype(np.int8), b))
    s2 = np.stack((s * 3, s))
    out = (torch.zeros((3, 2, 9), dtype=torch.int32, device="cuda"),
           torch.zeros(3, dtype=torch.int32, device="cuda"))
    need = mha.lib().kv_pages_select_workspace_bytes(3, 2, table.shape[1])
    for ws in (None, torch.empty(need, dtype=torch.uint8, device="cuda")):
        for stream in (None, torch.cuda.Stream()):
            out[0].zero_()
            out[1].zero_()
            torch.cuda.synchronize()
            got = mha.kv_pages_select(q, pool, pool, i32(table), i32(lens), i32(offs), i8(b2), f32(s2), 9,
                                      layer=1, out=out, workspace=ws, stream=stream)
            torch.cuda.synchronize()
            assert mha.mha_check() == mha.MHA_OK and got is out
            assert np.array_equal(out[0].cpu().numpy(), want) and np.array_equal(out[1].cpu().numpy(), rows)


# ------------------------------------------------------------- selected attention

def selected_case(seed, T, H, Hkv, ps, d, n, lens, e8, pow2=True):
    """Tokens over n pages of their own per kv head, the first lens[t] rows."""
    rng = np.random.default_rng(seed)
    P = 40 if n < 30 else n + 10
    Q = round_to_bf16(rng.standard_normal((T, H, d), dtype=np.float32))
    sel = np.full((T, Hkv, n), -1, np.int32)
    for t in range(T):
        for g in range(Hkv):
            m = -(-lens[t] // ps)
            sel[t, g, :m] = rng.permutation(P)[:m]
    if e8:
        kc, ks, vc, vs, *_ = make_pages8(rng, [P * ps], [1], Hkv, ps, d, pow2, spare=0)
        K, V = ref.decode(kc, ks), ref.decode(vc, vs)
        pools, sc = (dev8(kc), dev8(vc)), dict(K_scale=f32(ks), V_scale=f32(vs))
    else:
        K, V, *_ = make_pages(rng, [P * ps], [1], Hkv, ps, d, bf16=True, spare=0)
        vs, pools, sc = np.ones((P, Hkv)), (dev(K, BF), dev(V, BF)), {}
    return Q, K, V, vs, sel, np.asarray(lens, np.int32), pools, sc


def check_selected(got, x, e8, scale=0.0):
    Q, K, V, vs, sel, lens, _, _ = x
    O, A = ref.sdpa_selected(Q, K, V, sel, lens, scale)
    if e8:
        b = attention_bound(O, A, Q, K, vs.max(), lens.max(), scale or Q.shape[-1] ** -0.5, got.dtype == BF)
    else:
        b = (2.0 ** -8 + 2.0 ** -10) * A + 1e-30 + (2.0 ** -8 * np.abs(O) if got.dtype == BF else 0)
    used = lens > 0
    got = to_np(got)
    assert np.all(np.isfinite(got[used]))
    worst = np.max(np.abs(got - O)[used] / b[used]) if used.any() else 0.0
    assert worst <= 1.0, f"{worst:.3f} of the bound"


SELECTED = [
    # T, H, Hkv, page, d, n, lens, splits, out dtype
    (1, 2, 2, 16, 64, 4, [50], 0, BF), (1, 1, 1, 16, 64, 1, [1], 0, F32), (3, 8, 2, 16, 128, 9, [144, 1, 130], 0, F32),
    (4, 8, 8, 64, 128, 5, [300, 0, 64, 129], 3, BF), (2, 16, 1, 32, 128, 20, [640, 333], 16, F32),
    (3, 33, 1, 16, 64, 20, [320, 17, 200], 0, F32), (2, 128, 1, 64, 128, 6, [384, 100], 2, BF),
    (2, 24, 1, 256, 64, 4, [1000, 257], 0, F32), (300, 4, 2, 16, 64, 6, [i % 97 for i in range(300)], 0, BF),
    (300, 40, 2, 16, 128, 3, [i % 48 for i in range(300)], 0, F32), (1, 4, 1, 16, 128, 500, [7999], 0, F32),
]


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("c", SELECTED, ids=[str(i) for i in range(len(SELECTED))])
def test_selected(c, e8):
    T, H, Hkv, ps, d, n, lens, splits, odt = c
    x = selected_case(570 + SELECTED.index(c), T, H, Hkv, ps, d, n, lens, e8, SELECTED.index(c) % 2 == 0)
    Q, _, _, _, sel, rows, pools, sc = x
    out = torch.full(Q.shape, 7.0, dtype=odt, device="cuda")
    mha.sdpa_paged_selected(dev(Q, BF), *pools, i32(sel), i32(rows), out_dtype=odt, num_splits=splits, out=out,
                            **sc)
    assert mha.mha_check() == mha.MHA_OK
    check_selected(out, x, e8)
    assert torch.all(out[torch.from_numpy(rows == 0)] == 7.0)


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("H", [4, 40])
def test_selected_reports_bad_entries(e8, H):
    x = selected_case(590, 3, H, 2, 16, 64, 6, [90, 80, 70], e8)
    Q, K, V, vs, sel, rows, pools, sc = x

    def call(sel=sel, rows=rows):
        out = torch.full(Q.shape, 7.0, dtype=F32, device="cuda")
        mha.sdpa_paged_selected(dev(Q, BF), *pools, i32(sel), i32(rows), out_dtype=F32, out=out, **sc)
        assert mha.mha_check() == mha.MHA_ERR_DEVICE
        assert torch.all(out[1] == 0) if sel is x[4] else True
        return out

    for n in (-1, 97, 2 ** 31 - 1, -2 ** 31):
        check_selected(call(rows=[90, n, 70])[[0, 2]], tuple(
            v[[0, 2]] if i in (0, 4, 5) else v for i, v in enumerate(x)), e8)
    for page in (-1, K.shape[0], 2 ** 31 - 1, -2 ** 31):
        s = sel.copy()
        s[1, 1, 2] = page
        out = call(sel=s)
        G = H // 2
        assert torch.all(out[1, G:] == 0)
        y = list(x)
        y[0], y[4], y[5] = x[0][[0, 2]], x[4][[0, 2]], x[5][[0, 2]]
        check_selected(out[[0, 2]], tuple(y), e8)


@pytest.mark.parametrize("e8", [False, True])
def test_no_tokens(e8):
    x = selected_case(591, 1, 4, 2, 16, 64, 6, [90], e8)
    Q, _, _, _, sel, rows, pools, sc = x
    out = mha.sdpa_paged_selected(dev(Q[:0], BF), *pools, i32(sel[:0]), i32(rows[:0]), **sc)
    assert out.shape == (0, 4, 64) and mha.mha_check() == mha.MHA_OK


# ------------------------------------------------------------------ all together

@pytest.mark.parametrize("e8,H,Hkv,d,ps", [(True, 8, 2, 128, 16), (False, 8, 2, 64, 16), (True, 6, 1, 64, 32),
                                           (False, 20, 1, 128, 32)])
def test_serving_steps_over_selected_pages(e8, H, Hkv, d, ps):
    """Prompts appended in chunks, bounds kept after each, then decoding steps
    that select pages and attend to them, in two layers, one captured step
    replayed: each step's selection is the oracle's from the cache's own keys,
    its attention the oracle's over the cache's own rows, and with as many pages
    as there are it is sdpa_paged's."""
    rng = np.random.default_rng(600 + H)
    B, layers, cols, n_sel = 3, 2, 30, 5
    P = B * cols + 3
    shape = (layers, P, Hkv, ps, d)
    if e8:
        kp, vp = (torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                  for _ in range(2))
        sc = dict(K_scale=torch.full(shape[:3], 9.0, device="cuda"),
                  V_scale=torch.full(shape[:3], 9.0, device="cuda"))
    else:
        kp, vp = (torch.full(shape, float("nan"), dtype=BF, device="cuda") for _ in range(2))
        sc = {}
    bnd = torch.zeros((layers, P, Hkv, 2, d), dtype=torch.int8, device="cuda")
    bs = torch.zeros((layers, P, Hkv), device="cuda")
    table = i32(rng.permutation(P)[:B * cols].reshape(B, cols))
    lens = i32([0] * B)
    g1, g2 = (dev(round_to_bf16(1 + 0.1 * rng.standard_normal(d, dtype=np.float32)), BF) for _ in range(2))
    pe = mha.sinusoidal_pe(cols * ps, d)

    def rows(new):
        T = sum(new)
        return [torch.from_numpy(rng.standard_normal((T, h, d), dtype=np.float32)).to(BF).cuda()
                for h in (H, Hkv, Hkv)]

    def step(q, k, v, offs, n, sel=n_sel):
        outs = []
        for y in range(layers):
            qo = mha.qk_norm_rope_paged(q, k, v, g1, g2, pe, kp, vp, table, lens, offs, layer=y, **sc)
            mha.kv_pages_bounds(kp, vp, table, lens, offs, bnd, bs, q.shape[0], layer=y, **sc)
            chosen = mha.kv_pages_select(qo, kp, vp, table, lens, offs, bnd, bs, sel, layer=y, **sc)
            O = mha.sdpa_paged_selected(qo, kp, vp, *chosen, layer=y, **sc)
            outs.append((qo, *chosen, O))
        return outs

    def check(outs, offs, sel=n_sel):
        assert mha.mha_check() == mha.MHA_OK
        T = outs[0][0].shape[0]
        tb, ln = table.cpu().numpy(), lens.cpu().numpy()
        for y, (qo, chosen, count, O) in enumerate(outs):
            if e8:
                kc, ks = codes_of(kp[y]), to_np(sc["K_scale"][y])
                keys, K = ref.VALUES[kc], ref.decode(kc, ks)
                V, vs = ref.decode(codes_of(vp[y]), to_np(sc["V_scale"][y])), to_np(sc["V_scale"][y])
            else:
                keys = K = to_np(kp[y])
                V, ks, vs = to_np(vp[y]), None, np.ones((P, Hkv))
            # bounds of every full page, from the keys that lie there
            wb, ws = ref.bounds(keys, tb, ln, np.concatenate(([0], np.cumsum(ln))),
                                np.zeros(bnd.shape[1:], np.int8), np.zeros((P, Hkv)), ks)
            assert np.array_equal(bnd[y].cpu().numpy(), wb) and np.array_equal(to_np(bs[y]), ws)
            want, rows_seen = ref.select(to_np(qo), ps, tb, ln, offs, wb, ws, sel)
            assert np.array_equal(chosen.cpu().numpy(), want)
            assert np.array_equal(count.cpu().numpy(), rows_seen)
            held = [p for b in range(B) for p in tb[b, :-(-int(ln[b]) // ps)]]
            K, V = (np.where(np.isfinite(a), a, 0.0) for a in (K, V))
            check_selected(O, (to_np(qo), K, V, vs[held], want, rows_seen, None, None), e8)

    for new in ([70, 33, 1], [100, 0, 40], [1, 1, 1], [16, 2, 0]):
        lens += i32(new)
        offs = np.concatenate(([0], np.cumsum(new)))
        check(step(*rows(new), i32(offs), new), offs)
    # every page: the same attention as over the whole cache
    q, k, v = rows([1, 1, 1])
    offs = i32([0, 1, 2, 3])
    lens += 1
    outs = step(q, k, v, offs, None, sel=cols)
    check(outs, [0, 1, 2, 3], sel=cols)
    for y, (qo, _, _, O) in enumerate(outs):
        whole = mha.sdpa_paged(qo, kp, vp, table, lens, offs, max_new=1, layer=y, **sc)
        assert float((whole.float() - O.float()).abs().max()) <= 2.0 ** -6
    # compaction moves pages, scales with them; their bounds are made anew
    shape2 = (layers, P + 5, Hkv, ps, d)
    k2, v2 = (torch.zeros(shape2, dtype=torch.uint8 if e8 else BF, device="cuda").view(kp.dtype)
              for _ in range(2))
    t2 = torch.full_like(table, -1)
    sc2 = {k: torch.full(shape2[:3], 9.0, device="cuda") for k in sc}
    live = mha.kv_pages_compact(kp, vp, table, lens, k2, v2, t2, **sc, **{k + "_out": v for k, v in sc2.items()})
    assert int(live) == sum(-(-int(n) // ps) for n in lens)
    # what lies behind the held rows stays what it was at first: NaN
    k2.view(torch.uint8)[:, int(live):] = 0xff
    v2.view(torch.uint8)[:, int(live):] = 0xff
    spare = iter(range(int(live), P + 5))
    for b in range(B):
        for j in range(-(-int(lens[b]) // ps), cols):
            t2[b, j] = next(spare, -1)
    kp, vp, table, sc, P = k2, v2, t2, sc2, P + 5
    bnd, bs = torch.zeros((layers, P, Hkv, 2, d), dtype=torch.int8, device="cuda"), torch.zeros(
        (layers, P, Hkv), device="cuda")
    whole = i32(np.concatenate(([0], np.cumsum(lens.cpu().numpy()))))
    for y in range(layers):
        mha.kv_pages_bounds(kp, vp, table, lens, whole, bnd, bs, int(whole[-1]), layer=y, **sc)
    lens += 1
    check(step(q, k, v, offs, None), [0, 1, 2, 3])
    # a captured step follows the lengths
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        lens += 1
        kept = step(q, k, v, offs, None)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        check(kept, [0, 1, 2, 3])
