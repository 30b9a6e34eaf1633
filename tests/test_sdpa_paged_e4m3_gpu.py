"""sdpa_paged over a cache in 8 bits, on the GPU, against the oracle's
attention over the decoded rows (tolerance: e4m3_util.attention_bound)."""
import numpy as np
import pytest
import torch

import oracle.paged as paged
import oracle.paged_e4m3 as ref
import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from transformer_head_scaled_03_gb300.inputs import round_to_bf16
from tests.e4m3_util import attention_bound, dev8, f32, make_pages8
from tests.gpu_util import to_np
from tests.paged_util import dev, i32
from tests.test_sdpa_paged_gpu import CASES

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


class Case:
    def __init__(self, seed, lens, new, H, Hkv, ps, d, q_scale=1.0, pow2=True, **kw):
        rng = np.random.default_rng(seed)
        self.kc, self.ks, self.vc, self.vs, self.table, self.offs, self.free = make_pages8(
            rng, lens, new, Hkv, ps, d, pow2, **kw)
        self.Q = round_to_bf16(rng.standard_normal((self.offs[-1], H, d), dtype=np.float32)
                               * np.float32(q_scale))
        self.lens = np.asarray(lens, np.int32)

    def args(self, Q=None, table=None, lens=None, offs=None):
        pick = lambda x, y: y if x is None else x
        return (dev(pick(Q, self.Q), BF), dev8(self.kc), dev8(self.vc), i32(pick(table, self.table)),
                i32(pick(lens, self.lens)), i32(pick(offs, self.offs)))

    def scales(self):
        return dict(K_scale=f32(self.ks), V_scale=f32(self.vs))

    def run(self, **kw):
        O = mha.sdpa_paged(*self.args(), **self.scales(), **kw)
        assert mha.mha_check() == mha.MHA_OK
        return O

    def want(self, causal=True, scale=0.0, layer=None):
        at = (lambda x: x) if layer is None else (lambda x: x[layer])
        K, V = ref.decode(at(self.kc), at(self.ks)), ref.decode(at(self.vc), at(self.vs))
        O, A = paged.sdpa_paged(self.Q, K, V, self.table, self.lens, self.offs, causal, scale)
        held = [p for row in self.table for p in row if p >= 0]
        bound = lambda dtype: attention_bound(
            O, A, self.Q, K[held], at(self.vs)[held].max(), self.lens.max(),
            scale or self.Q.shape[-1] ** -0.5, dtype == BF)
        return O, bound


def check(got, want, what="", rows=slice(None)):
    O, bound = want
    b = bound(got.dtype)[rows]
    got = to_np(got)[rows]
    assert np.all(np.isfinite(got)), what
    worst = float(np.max(np.abs(got - O[rows]) / b)) if b.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


@pytest.mark.parametrize("c", CASES, ids=[str(i) for i in range(len(CASES))])
def test_parity(c):
    lens, new, H, Hkv, ps, d, causal, splits, odt = c
    x = Case(270 + CASES.index(c), lens, new, H, Hkv, ps, d, pow2=CASES.index(c) % 3 != 2)
    want = x.want(causal)
    check(x.run(causal=causal, num_splits=splits, out_dtype=odt), want, str(c))
    # the tight bound on new tokens picks the same answer as the loose one
    check(x.run(causal=causal, num_splits=splits, out_dtype=odt, max_new=max(new)), want, f"{c} max_new")


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_every_split_count_merges_to_one_softmax(new, d):
    x = Case(320, [1900], [new], 8, 4, 64, d, q_scale=4.0)
    want = x.want()
    for splits in range(1, 17):
        check(x.run(num_splits=splits, out_dtype=F32, max_new=new), want, f"{splits} splits")


@pytest.mark.parametrize("new", [1, 30, 300])
def test_scales_of_very_different_sizes(new):
    """Values of one page a million times another's, a page of zeros under a
    scale of 0, and scales far below 1 throughout: the softmax's sum counts
    every key alike."""
    for shrink in (1.0, 2.0 ** -90):
        x = Case(330, [400], [new], 4, 2, 32, 64)
        x.vs[x.table[0, 2]] *= 2.0 ** 20
        x.vs[x.table[0, 5]] = 0
        x.ks[x.table[0, 7]] = 0
        x.vs *= shrink
        check(x.run(out_dtype=F32, max_new=new), x.want(), f"{new} {shrink}")
    x.vs[:] = 0
    assert torch.all(x.run(out_dtype=F32, max_new=new) == 0)


@pytest.mark.parametrize("new,H,Hkv,d", [(1, 4, 2, 64), (1, 4, 2, 128), (30, 4, 2, 64),
                                         (30, 2, 2, 128), (64, 128, 8, 64), (64, 128, 8, 128)])
def test_what_lies_behind_the_length_is_never_used(new, H, Hkv, d):
    """NaN codes in the rows behind the last one and in spare pages, NaN and
    infinite scales of spare pages: the same bits as with zeros there."""
    for ps, lens in ((16, [137, 65]), (64, [70, 129]), (256, [200, 300])):
        x = Case(340, lens, [new, new], H, Hkv, ps, d, cols=9)
        held = np.zeros(x.kc.shape[0], bool)
        outs = []
        for code, scale, entry in ((0, 1.0, -1), (0x7f, np.nan, 2 ** 31 - 1), (0xfe, np.inf, -2 ** 31)):
            for b, n in enumerate(lens):
                m = -(-n // ps)
                held[x.table[b, :m]] = True
                x.table[b, m:] = entry
                if n % ps:
                    for pool in (x.kc, x.vc):
                        pool[x.table[b, m - 1], :, n % ps:] = code
            for pool, s in ((x.kc, x.ks), (x.vc, x.vs)):
                pool[~held] = code
                s[~held] = scale
            outs.append(to_np(x.run(max_new=new)))
            assert np.all(np.isfinite(outs[0]))
        assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_strides_layers_scale_and_out(new, d):
    lens, H, Hkv, ps = [100, 45], 6, 2, 32
    x = Case(350, lens, [new, new], H, Hkv, ps, d, layers=3)
    T, P = x.offs[-1], x.kc.shape[1]
    wide = torch.randn((T + 5, (H + 4) * d), device="cuda").to(BF)
    q = wide[:, d:(H + 1) * d].view(T + 5, H, d)
    q[:T].copy_(dev(x.Q, BF))
    both = torch.empty((P, 3, 2, Hkv, ps, d), dtype=torch.uint8, device="cuda")
    kp, vp = (both[:, :, i].transpose(0, 1) for i in (0, 1))
    kp.copy_(torch.from_numpy(x.kc).cuda())
    vp.copy_(torch.from_numpy(x.vc).cuda())
    E8 = torch.float8_e4m3fn
    out = torch.full((T + 5, H, d), 7.0, dtype=F32, device="cuda")
    mha.sdpa_paged(q, kp.view(E8), vp.view(E8), i32(x.table), i32(x.lens), i32(x.offs), max_new=new,
                   scale=0.3, layer=1, out_dtype=F32, out=out, **x.scales())
    assert mha.mha_check() == mha.MHA_OK
    check(out[:T], x.want(scale=0.3, layer=1))
    assert torch.all(out[T:] == 7.0)


@pytest.mark.parametrize("new", [1, 25])
def test_bad_tables_lengths_and_offsets_are_reported(new):
    x = Case(360, [90, 80, 70], [new] * 3, 4, 2, 16, 64)
    want = x.want()
    T, offs, full = int(x.offs[-1]), x.offs, x.table.shape[1] * 16
    rows = lambda b: slice(offs[b], offs[b + 1])

    def call(max_new=new, **kw):
        out = torch.full(x.Q.shape, 7.0, dtype=F32, device="cuda")
        mha.sdpa_paged(*x.args(**kw), max_new=max_new, out_dtype=F32, out=out, **x.scales())
        assert mha.mha_check() == mha.MHA_ERR_DEVICE
        assert mha.mha_check() == mha.MHA_OK
        return out

    for n in (0, new - 1, full + 1, -5, 2 ** 31 - 1):
        got = call(lens=[x.lens[0], n, x.lens[2]])
        assert torch.all(got[rows(1)] == 0)
        for b in (0, 2):
            check(got, want, rows=rows(b))
    for page in (-1, x.kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = x.table.copy()
        t[1, 2] = page
        got = call(table=t)
        assert torch.all(got[rows(1)] == 0)
        for b in (0, 2):
            check(got, want, rows=rows(b))
    if new > 1:
        assert torch.all(call(max_new=new - 1) == 7.0)
    got = call(offs=[offs[0], offs[1], offs[2], T + 1])
    check(got, want, rows=rows(0))
    assert torch.all(got[rows(2)] == 7.0)
    call(offs=[0, T + 9, offs[2], T], max_new=T)
    call(offs=[-4, offs[1], offs[2], T], max_new=T)


@pytest.mark.parametrize("new,splits", [(1, 1), (1, 5), (40, 1), (40, 4), (200, 1), (200, 3)])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_queries_that_are_not_finite_stay_in_their_rows(new, splits, bad):
    x = Case(365, [300, 260], [new, new], 4, 2, 16, 64)
    want = to_np(x.run(num_splits=splits, max_new=new))
    x.Q[new // 2, 1, 5] = bad
    got = to_np(x.run(num_splits=splits, max_new=new))
    assert np.all(np.isnan(got[new // 2, 1]))
    got[new // 2, 1] = want[new // 2, 1]
    assert np.array_equal(got, want)


@pytest.mark.parametrize("new", [1, 20, 150])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -120, 2.0 ** 60])
def test_queries_of_any_size(new, size):
    """Rows of zeros, and rows far from 1 under a scale that brings the scores
    back: a row's parts are taken against its own largest element."""
    x = Case(366, [300], [new], 4, 2, 16, 64, q_scale=size)
    scale = 0.125 if size == 0 else 0.125 / size
    check(x.run(out_dtype=F32, scale=scale, max_new=new), x.want(scale=scale))


@pytest.mark.parametrize("new", [1, 9, 130])
def test_rows_with_elements_of_very_different_sizes(new):
    x = Case(367, [300], [new], 4, 2, 16, 128)
    x.Q[...] = round_to_bf16(x.Q * np.float32(2.0) ** np.random.default_rng(1).integers(-12, 1, x.Q.shape))
    check(x.run(out_dtype=F32, max_new=new, scale=1.0), x.want(scale=1.0))


@pytest.mark.parametrize("new,G,d", [(1, 2, 64), (1, 7, 64), (2, 16, 64), (2, 2, 128), (1, 8, 128),
                                     (1, 16, 128), (3, 16, 128)])
def test_more_sequences_than_are_ranked(new, G, d):
    rng = np.random.default_rng(368)
    lens = rng.integers(new, 60, 300)
    news = np.where(np.arange(300) % 7, new, 0)
    x = Case(369, list(lens), list(news), G, 1, 16, d)
    want = x.want()
    for splits in (1, 2):
        check(x.run(num_splits=splits, max_new=new, out_dtype=F32), want)


def test_no_tokens_and_no_sequences():
    x = Case(370, [20], [1], 4, 2, 16, 64)
    O = mha.sdpa_paged(*x.args(Q=x.Q[:0], offs=[0, 0]), **x.scales())
    assert O.shape == (0, 4, 64) and O.dtype == BF
    out = torch.full((1, 4, 64), 7.0, dtype=BF, device="cuda")
    mha.sdpa_paged(*x.args(offs=[0, 0]), out=out, **x.scales())
    assert mha.mha_check() == mha.MHA_OK and torch.all(out == 7.0)


@pytest.mark.parametrize("new", [1, 70])
def test_captured_and_replayed_beside_another(new):
    graphs = []
    for x in (Case(371, [200, 333], [new, new], 8, 2, 32, 128), Case(372, [150], [new], 4, 4, 16, 64)):
        args, sc = list(x.args()), x.scales()
        out = mha.sdpa_paged(*args, max_new=new, **sc)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            mha.sdpa_paged(*args, max_new=new, out=out, **sc)
        graphs.append((g, s, args, sc, out))
    for shift in (0, 3):
        want = []
        for g, s, args, sc, out in graphs:
            args[4] -= shift
            want.append(mha.sdpa_paged(*args, max_new=new, **sc))
            out.zero_()
        torch.cuda.synchronize()
        for g, s, *_ in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, (*_, out) in zip(want, graphs):
            assert torch.equal(w, out)
    assert mha.mha_check() == mha.MHA_OK


@pytest.mark.parametrize("new", [1, 33])
def test_equal_calls_give_equal_bits_on_any_stream(new):
    x = Case(373, [900, 412, 77], [new] * 3, 12, 4, 64, 64)
    args, sc = x.args(), x.scales()
    first = mha.sdpa_paged(*args, max_new=new, **sc)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        assert torch.equal(first, mha.sdpa_paged(*args, max_new=new, **sc))
        with torch.cuda.stream(s):
            other = mha.sdpa_paged(*args, max_new=new, **sc)
        given = mha.sdpa_paged(*args, max_new=new, stream=s, **sc)
        s.synchronize()
        assert torch.equal(first, other) and torch.equal(first, given)


@pytest.mark.parametrize("new", [1, 40])
def test_pages_past_2_31_elements(new):
    """A pool of 2.3 GB whose held pages lie at its end."""
    ps, Hkv, d = 128, 8, 128
    P = 2 ** 31 // (Hkv * ps * d) + 2100
    x = Case(374, [300], [new], 8, Hkv, ps, d)
    n = x.kc.shape[0]
    pools, at = [], np.arange(P - n, P)
    for codes in (x.kc, x.vc):
        pool = torch.zeros((P, Hkv, ps, d), dtype=torch.uint8, device="cuda")
        pool[P - n:] = torch.from_numpy(codes).cuda()
        pools.append(pool.view(torch.float8_e4m3fn))
    sc = {}
    for k, v in x.scales().items():
        sc[k] = torch.zeros((P, Hkv), device="cuda")
        sc[k][P - n:] = v
    table = np.where(x.table >= 0, at[x.table], -1)
    a = x.args(table=table)
    O = mha.sdpa_paged(a[0], *pools, *a[3:], max_new=new, out_dtype=F32, **sc)
    assert mha.mha_check() == mha.MHA_OK
    check(O, x.want())
