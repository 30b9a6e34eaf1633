"""Scales of 0, and far from one another, in a cache in 8 bits, on the GPU
against the oracle.

How far an attention may be off, row by row: its weights by 2^-8 of themselves
(two e4m3 parts; fp16 less), scores, exponentials and sums by 2^-10 as for the
bf16 cache, a score by 2^-17 max|q| max_j sum_c |k_jc| scale for the parts of q;
and for every key, since a weight meets the codes times its value scale, by the
smallest half step of that product's parts, 2^-23 of the row's largest product
of weight and scale (fp16: 2^-31), times a code, at most 448."""
import numpy as np
import pytest
import torch

import oracle.paged as paged
import oracle.paged_e4m3 as ref
import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from transformer_head_scaled_03_gb300.inputs import round_to_bf16
from tests.gpu_util import to_np
from tests.paged_util import i32
from tests.test_sdpa_paged_e4m3_gpu import Case

pytestmark = pytest.mark.gpu

F32 = torch.float32
TILES = [(20, 64, 16, 1), (20, 128, 64, 1), (300, 64, 16, 1), (300, 64, 64, 3), (300, 128, 32, 1),
         (300, 128, 16, 1), (20, 64, 32, 5), (20, 128, 16, 7), (300, 128, 64, 4)]


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


def expected(x, smallest, scale=0.0):
    """(O, bound) of a Case with one sequence, causal, output in fp32."""
    T, H, d = x.Q.shape
    n, G = int(x.lens[0]), H // x.kc.shape[1]
    scale = scale or d ** -0.5
    K, V = (paged.gather(ref.decode(c, s), x.table[0], n) for c, s in ((x.kc, x.ks), (x.vc, x.vs)))
    vs = np.repeat(x.vs[x.table[0]], x.kc.shape[2], 0)[:n].T.astype(np.float64)
    O, b = np.zeros((T, H, d)), np.zeros((T, H, d))
    for t in range(T):
        seen = n - T + t + 1
        for h in range(H):
            g, q = h // G, x.Q[t, h].astype(np.float64)
            s = scale * (K[g, :seen] @ q)
            w = np.exp(s - s.max())
            w /= w.sum()
            O[t, h] = w @ V[g, :seen]
            parts = 2 * 2.0 ** -17 * np.abs(q).max() * np.abs(K[g, :seen]).sum(-1).max() * scale
            b[t, h] = (2.0 ** -8 + 2.0 ** -10 + parts) * (w @ np.abs(V[g, :seen])) \
                + seen * smallest * 448 * (w * vs[g, :seen]).max() + 2.0 ** -149
    return O, b


def check(got, want, what):
    O, b = want
    got = to_np(got)
    assert np.all(np.isfinite(got)), what
    worst = float(np.max(np.abs(got - O) / b))
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"


@pytest.mark.parametrize("new,d,ps,splits", TILES)
@pytest.mark.parametrize("shrink", [2.0 ** -28, 2.0 ** -110])
def test_a_first_page_of_zeros(new, d, ps, splits, shrink):
    """The first page's scale is 0, and a later one's; the others' are small."""
    x = Case(900, [400], [new], 4, 2, ps, d)
    x.vs *= shrink
    x.vs[x.table[0, 0]] = 0
    x.vs[x.table[0, 5]] = 0
    check(x.run(out_dtype=F32, max_new=new, num_splits=splits), expected(x, 2.0 ** -31), f"{new} {d}")


@pytest.mark.parametrize("new,d,ps,splits", TILES)
def test_large_values_of_little_weight_and_a_page_of_zeros(new, d, ps, splits):
    """The first page's values are 2^34 times the others', and its keys such that
    they hardly count; a later page's scale is 0."""
    x = Case(901, [400], [new], 4, 2, ps, d)
    x.Q[...] = round_to_bf16(np.abs(x.Q) / 2 + 0.5)
    first = x.table[0, 0]
    x.kc[first], x.ks[first] = ref.encode(-448.0), 2.0 ** -7
    x.vs[first] *= 2.0 ** 34
    x.vs[x.table[0, 5]] = 0
    scale = 8.0 / d
    check(x.run(out_dtype=F32, max_new=new, num_splits=splits, scale=scale),
          expected(x, 2.0 ** -31, scale), f"{new} {d}")


@pytest.mark.parametrize("new,d,ps,splits", TILES)
def test_zeros_under_a_scale_of_zero_keep_their_weight(new, d, ps, splits):
    """Half the pages' scale is 0, some of the others' 2^90 times the rest: the
    softmax's sum counts the keys of scale 0 like any others, and so it does
    where a split meets nothing else."""
    x = Case(902, [400], [new], 4, 2, ps, d)
    pages = x.table[0, :-(-400 // ps)]
    x.vs[pages[::2]] = 0
    x.vs[pages[1::4]] *= 2.0 ** 90
    check(x.run(out_dtype=F32, max_new=new, num_splits=splits), expected(x, 2.0 ** -31), f"{new} {d}")
    x.vs[pages[len(pages) // 3:]] = 0
    check(x.run(out_dtype=F32, max_new=new, num_splits=splits), expected(x, 2.0 ** -31), f"{new} {d}, a third")
    x.vs[pages] = 0
    assert torch.all(x.run(out_dtype=F32, max_new=new, num_splits=splits) == 0)


@pytest.mark.parametrize("new,d,ps,splits", TILES)
@pytest.mark.parametrize("faint", [False, True])
def test_zeros_first_and_large_values_late(new, d, ps, splits, faint):
    """Two key tiles of scale 0, then values 2^90 apart; or one whose values are
    the smaller ones under keys that hardly count, and then the larger ones."""
    x = Case(903, [700], [new], 4, 2, ps, d)
    x.Q[...] = round_to_bf16(np.abs(x.Q) / 2 + 0.5)
    pages = x.table[0, :-(-700 // ps)]
    zeros, small = pages[:256 // ps], pages[256 // ps:384 // ps] if faint else pages[256 // ps::2]
    x.vs[pages] *= 2.0 ** 45
    x.vs[small] *= 2.0 ** -90
    x.vs[zeros] = 0
    if faint:
        x.kc[small], x.ks[small] = ref.encode(-448.0), 2.0 ** -6
    scale = 8.0 / d
    check(x.run(out_dtype=F32, max_new=new, num_splits=splits, scale=scale),
          expected(x, 2.0 ** -31, scale), f"{new} {d}")


FEW = [(1, 64, 16, 1), (1, 128, 64, 1), (2, 128, 16, 4), (4, 64, 32, 3), (8, 128, 16, 1), (3, 64, 64, 7)]


@pytest.mark.parametrize("new,d,ps,splits", FEW)
@pytest.mark.parametrize("seed", range(3))
def test_few_rows_hold_weights_against_their_own_products(new, d, ps, splits, seed):
    """Values 2^34 times the others' under keys that hardly count, in the first
    page, the last full one, or a page that only the newest token sees."""
    n = 400 if seed < 2 else 384 - ps + 1
    x = Case(910 + seed, [n], [new], 4, 2, ps, d)
    x.Q[...] = round_to_bf16(np.abs(x.Q) / 2 + 0.5)
    pages = x.table[0, :-(-n // ps)]
    far = [pages[0], pages[-2], pages[-1]][seed]
    if seed < 2:
        x.kc[far], x.ks[far] = ref.encode(-448.0), 2.0 ** -7
    x.vs[far] *= 2.0 ** 34
    x.vs[pages[3]] = 0
    scale = 8.0 / d
    check(x.run(out_dtype=F32, max_new=new, num_splits=splits, scale=scale),
          expected(x, 2.0 ** -23, scale), f"{new} {d}")


@pytest.mark.parametrize("new,d,ps,splits", FEW)
@pytest.mark.parametrize("faint", [None, False, True])
def test_few_rows_count_zeros_like_any_keys(new, d, ps, splits, faint):
    """Half the pages of scale 0; or the first two key tiles, then values 2^90
    apart, the smaller ones under keys that hardly count or not."""
    x = Case(913, [700], [new], 4, 2, ps, d)
    x.Q[...] = round_to_bf16(np.abs(x.Q) / 2 + 0.5)
    pages = x.table[0, :-(-700 // ps)]
    if faint is None:
        x.vs[pages[1::4]] *= 2.0 ** 90
        x.vs[pages[::2]] = 0
    else:
        small = pages[256 // ps:384 // ps] if faint else pages[256 // ps::2]
        x.vs[pages] *= 2.0 ** 45
        x.vs[small] *= 2.0 ** -90
        x.vs[pages[:256 // ps]] = 0
        if faint:
            x.kc[small], x.ks[small] = ref.encode(-448.0), 2.0 ** -6
    scale = 8.0 / d
    check(x.run(out_dtype=F32, max_new=new, num_splits=splits, scale=scale),
          expected(x, 2.0 ** -23, scale), f"{new} {d}")
    x.vs[:] = 0
    assert torch.all(x.run(out_dtype=F32, max_new=new, num_splits=splits) == 0)


@pytest.mark.parametrize("new,d,ps,splits", FEW + TILES)
def test_values_that_are_not_finite_beside_zeros_show(new, d, ps, splits):
    """A page of zeros but for an infinity, which the append stores as NaN under a
    scale of 0: its column is NaN in whatever sees it, and no other is."""
    x = Case(920, [400], [new], 4, 2, ps, d)
    held = [x.table[0, 0], x.table[0, 2]]
    rows = torch.zeros((3 * ps, 2, d), dtype=torch.bfloat16, device="cuda")
    ones, pe = torch.ones(d, dtype=torch.bfloat16, device="cuda"), mha.sinusoidal_pe(3 * ps, d)
    rows[ps:2 * ps] = 1.0
    outs = []
    for bad in (0.0, float("inf")):
        rows[2 * ps + 3, 1, 7] = bad
        Q, K, V, table, lens, offs = x.args()
        sc = x.scales()
        mha.qk_norm_rope_paged(rows.repeat(1, 2, 1), rows, rows, ones, ones, pe, K, V, table,
                               i32([3 * ps]), i32([0, 3 * ps]), **sc)
        assert torch.all(sc["V_scale"][held] == 0)
        # the values of the append beside the keys of before
        K, sc["K_scale"] = x.args()[1], x.scales()["K_scale"]
        outs.append(to_np(mha.sdpa_paged(Q, K, V, table, lens, offs, max_new=new, num_splits=splits,
                                         out_dtype=F32, **sc)))
        assert mha.mha_check() == mha.MHA_OK
    clean, got = outs
    assert np.all(np.isfinite(clean))
    first = max(0, 2 * ps + 3 - (400 - new))           # the first token that sees the key
    assert first < new and np.all(np.isnan(got[first:, 2:, 7]))
    got[:, 2:, 7] = clean[:, 2:, 7]
    assert np.array_equal(got, clean)
