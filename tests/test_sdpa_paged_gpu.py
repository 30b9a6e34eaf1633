"""sdpa_paged on the GPU against oracle/paged.py.

Tolerance, from the arithmetic (bf16's half step is 2^-8 of the value): the
weights are rounded to bf16 before they meet V, so an output moves by at most
2^-8 A with A = sum_j w_j |v_j|; scores and exponentials in fp32 move the
weights by less than 2^-10 of themselves (|s| < 2^7 times 2^-24 times the 64
or 128 terms of a product, plus 2^-22 of the exponential), and so do the sums;
a bf16 output rounds by 2^-8 |o| once more.
    |err| <= (2^-8 + 2^-10) A (+ 2^-8 |o| for a bf16 output) + 1e-30"""
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


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


def check(got, O, A, dtype, what=""):
    bound = (2.0 ** -8 + 2.0 ** -10) * A + 1e-30
    if dtype == BF:
        bound = bound + 2.0 ** -8 * np.abs(O)
    assert np.all(np.isfinite(got)), what
    worst = float(np.max(np.abs(got - O) / bound)) if O.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"
    return worst


def case(seed, lens, new, H, Hkv, ps, d, q_scale=1.0, **kw):
    rng = np.random.default_rng(seed)
    K, V, table, offs, free = make_pages(rng, lens, new, Hkv, ps, d, bf16=True, **kw)
    Q = round_to_bf16(rng.standard_normal((offs[-1], H, d), dtype=np.float32) * np.float32(q_scale))
    return Q, K, V, table, np.asarray(lens, np.int32), offs


def run(Q, K, V, table, lens, offs, **kw):
    O = mha.sdpa_paged(dev(Q, BF), dev(K, BF), dev(V, BF), i32(table), i32(lens), i32(offs), **kw)
    assert mha.mha_check() == mha.MHA_OK
    return to_np(O)


CASES = [
    # lens, new, H, Hkv, page, d, causal, splits, out dtype
    ([37], [1], 2, 2, 16, 64, True, 0, BF),                     # one token
    ([1], [1], 4, 1, 16, 64, True, 0, F32),                     # the first token of all
    ([128, 129, 127], [1, 1, 1], 8, 2, 16, 128, True, 0, F32),  # tile edges
    ([300, 17, 513], [2, 3, 1], 6, 3, 32, 64, True, 3, BF),     # a few tokens each
    ([700, 64, 5, 2000], [1, 1, 1, 1], 16, 1, 64, 128, True, 16, BF),   # one shared head
    ([40, 0, 41], [1, 0, 1], 4, 4, 16, 64, True, 2, BF),        # an idle, empty sequence
    ([50, 60], [50, 60], 2, 2, 16, 64, True, 0, BF),            # whole prompts
    ([300, 129, 2], [300, 128, 2], 6, 2, 32, 128, True, 0, F32),
    ([1000, 400], [33, 257], 10, 2, 128, 64, True, 0, BF),      # chunks over a longer cache
    ([777], [500], 7, 1, 256, 128, True, 0, F32),               # seven heads to one, large pages
    ([513, 100, 900], [130, 1, 1], 8, 8, 64, 128, True, 0, BF),  # mixed chunk and single tokens
    ([600], [20], 4, 1, 16, 128, True, 8, F32),                 # a chunk whose keys are split
    ([90, 600], [40, 17], 12, 4, 32, 64, False, 0, F32),        # every key visible
    ([3, 256], [5, 1], 4, 2, 16, 128, False, 0, F32),           # more queries than keys
    ([260], [3], 128, 1, 64, 64, True, 0, BF),                  # 128 heads to one
    ([500, 30], [9, 4], 33, 1, 16, 64, True, 0, F32),           # an odd group
    # enough blocks for two query tiles per CTA, the last ones with one or none
    ([400, 0, 333], [350, 0, 300], 64, 8, 64, 128, True, 0, BF),
    ([411, 333], [340, 301], 64, 8, 16, 64, True, 0, F32),
    ([270, 333], [340, 300], 48, 8, 128, 64, False, 0, BF),
    ([500], [481], 56, 8, 256, 128, True, 0, F32),
]


@pytest.mark.parametrize("c", CASES, ids=[str(i) for i in range(len(CASES))])
def test_parity(c):
    lens, new, H, Hkv, ps, d, causal, splits, odt = c
    x = case(70 + CASES.index(c), lens, new, H, Hkv, ps, d)
    O, A = ref.sdpa_paged(*x, causal=causal)
    got = run(*x, causal=causal, num_splits=splits, out_dtype=odt)
    check(got, O, A, odt, str(c))
    # the tight bound on new tokens picks the same answer as the loose one
    tight = run(*x, causal=causal, num_splits=splits, out_dtype=odt, max_new=max(new))
    check(tight, O, A, odt, f"{c} max_new")


@pytest.mark.parametrize("new", [1, 40])
def test_every_split_count_merges_to_one_softmax(new):
    """Peaked rows (scores of std 4) whose maximum lies in another split per
    head."""
    x = case(120, [1900], [new], 8, 4, 64, 128, q_scale=4.0)
    O, A = ref.sdpa_paged(*x)
    for splits in range(1, 17):
        check(run(*x, num_splits=splits, out_dtype=F32, max_new=new), O, A, F32, f"{splits} splits")


@pytest.mark.parametrize("new,H,Hkv,d", [(1, 4, 2, 64), (1, 4, 2, 128), (30, 4, 2, 64),
                                         (30, 2, 2, 128), (64, 128, 8, 64), (64, 128, 8, 128)])
def test_what_lies_behind_the_length_is_never_used(new, H, Hkv, d):
    """NaN and infinities in the rows behind the last one, in spare pages and
    behind table entries: the same bits as with zeros there."""
    for ps, lens in ((16, [137, 65]), (64, [70, 129]), (256, [200, 300])):
        Q, K, V, table, lens, offs = case(130, lens, [new, new], H, Hkv, ps, d, cols=9)
        outs = []
        for fill in (0.0, np.nan, np.inf):
            k, v = K.copy(), V.copy()
            held = np.zeros(K.shape[0], bool)
            for b, n in enumerate(lens):
                m = -(-n // ps)
                held[table[b, :m]] = True
                if n % ps:
                    k[table[b, m - 1], :, n % ps:] = fill
                    v[table[b, m - 1], :, n % ps:] = fill
            k[~held], v[~held] = fill, fill
            t = table.copy()
            t[table < 0] = -1 if fill == 0.0 else 2 ** 31 - 1
            outs.append(run(Q, k, v, t, lens, offs, max_new=new))
        assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


@pytest.mark.parametrize("new", [1, 20])
def test_strides_layers_scale_and_out(new):
    """Q as a slice of a wider projection, pools as layers of one array whose
    pages interleave K, V and layers, an explicit scale, a given output whose
    rows of no sequence stay as they were."""
    lens, H, Hkv, ps, d = [100, 45], 6, 2, 32, 64
    Q, K, V, table, lens, offs = case(140, lens, [new, new], H, Hkv, ps, d, layers=3)
    T = offs[-1]
    wide = torch.randn((T + 5, (H + 4) * d), device="cuda").to(BF)
    q = wide[:, d:(H + 1) * d].view(T + 5, H, d)
    q[:T].copy_(dev(Q, BF))
    P = K.shape[1]
    both = torch.empty((P, 3, 2, Hkv, ps, d), dtype=BF, device="cuda")
    kp, vp = (both[:, :, i].transpose(0, 1) for i in (0, 1))
    kp.copy_(dev(K, BF))
    vp.copy_(dev(V, BF))
    out = torch.full((T + 5, H, d), 7.0, dtype=F32, device="cuda")
    mha.sdpa_paged(q, kp, vp, i32(table), i32(lens), i32(offs), max_new=new, scale=0.3, layer=1,
                   out_dtype=F32, out=out)
    assert mha.mha_check() == mha.MHA_OK
    O, A = ref.sdpa_paged(Q, K[1], V[1], table, lens, offs, scale=0.3)
    check(to_np(out[:T]), O, A, F32)
    assert torch.all(out[T:] == 7.0)


@pytest.mark.parametrize("new", [1, 25])
def test_bad_tables_lengths_and_offsets_are_reported(new):
    """Checked on the device; the other sequences keep their results."""
    x = case(150, [90, 80, 70], [new] * 3, 4, 2, 16, 64)
    Q, K, V, table, lens, offs = x
    O, A = ref.sdpa_paged(*x)
    full = table.shape[1] * 16
    rows = lambda b: slice(offs[b], offs[b + 1])
    dq, dk, dv = dev(Q, BF), dev(K, BF), dev(V, BF)

    def call(table=table, lens=lens, offs=offs, max_new=new):
        out = torch.full(Q.shape, 7.0, dtype=F32, device="cuda")
        mha.sdpa_paged(dq, dk, dv, i32(table), i32(lens), i32(offs), max_new=max_new,
                       out_dtype=F32, out=out)
        assert mha.mha_check() == mha.MHA_ERR_DEVICE
        assert mha.mha_check() == mha.MHA_OK
        return to_np(out)

    for n in (0, new - 1, full + 1, -5, 2 ** 31 - 1):
        got = call(lens=[lens[0], n, lens[2]])
        assert np.all(got[rows(1)] == 0)
        for b in (0, 2):
            check(got[rows(b)], O[rows(b)], A[rows(b)], F32)
    for page in (-1, K.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.copy()
        t[1, 2] = page
        got = call(table=t)
        assert np.all(got[rows(1)] == 0)
        for b in (0, 2):
            check(got[rows(b)], O[rows(b)], A[rows(b)], F32)
    T = int(offs[-1])
    if new > 1:
        got = call(max_new=new - 1)                       # more new tokens than announced
        assert np.all(got == 7.0)
    got = call(offs=[offs[0], offs[1], offs[2], T + 1])   # past the packed tokens
    check(got[rows(0)], O[rows(0)], A[rows(0)], F32)
    assert np.all(got[rows(2)] == 7.0)
    call(offs=[0, T + 9, offs[2], T], max_new=T)          # descending
    call(offs=[-4, offs[1], offs[2], T], max_new=T)


@pytest.mark.parametrize("new,splits", [(1, 1), (1, 5), (40, 1), (40, 4), (200, 1), (200, 3)])
def test_nan_queries_give_nan_and_stay_in_their_rows(new, splits):
    x = case(155, [300, 260], [new, new], 4, 2, 16, 64)
    want = run(*x, num_splits=splits, max_new=new)
    Q = x[0].copy()
    Q[new // 2, 1, 5] = np.nan
    got = mha.sdpa_paged(dev(Q, BF), *(dev(v, BF) for v in x[1:3]), *(i32(v) for v in x[3:]),
                         num_splits=splits, max_new=new)
    assert mha.mha_check() == mha.MHA_OK
    got = got.float().cpu().numpy()
    assert np.all(np.isnan(got[new // 2, 1]))
    got[new // 2, 1] = want[new // 2, 1]
    assert np.array_equal(got, want)


@pytest.mark.parametrize("new,G,d", [(1, 2, 64), (1, 7, 64), (2, 16, 64), (2, 2, 128), (1, 8, 128),
                                     (1, 16, 128), (3, 16, 128)])
def test_more_sequences_than_are_ranked(new, G, d):
    """300 sequences, one in seven of them idle: more than a CTA ranks and than
    SMs, in both kernels and every number of query slots."""
    rng = np.random.default_rng(156)
    lens = rng.integers(new, 60, 300)
    news = np.where(np.arange(300) % 7, new, 0)
    x = case(157, list(lens), list(news), G, 1, 16, d)
    O, A = ref.sdpa_paged(*x)
    for splits in (1, 2):
        check(run(*x, num_splits=splits, max_new=new, out_dtype=F32), O, A, F32)


def test_no_tokens_and_no_sequences():
    Q, K, V, table, lens, offs = case(160, [20], [1], 4, 2, 16, 64)
    O = mha.sdpa_paged(dev(Q[:0], BF), dev(K, BF), dev(V, BF), i32(table), i32(lens), i32([0, 0]))
    assert O.shape == (0, 4, 64)
    out = torch.full((1, 4, 64), 7.0, dtype=BF, device="cuda")
    mha.sdpa_paged(dev(Q, BF), dev(K, BF), dev(V, BF), i32(table), i32(lens), i32([0, 0]), out=out)
    assert mha.mha_check() == mha.MHA_OK and torch.all(out == 7.0)


@pytest.mark.parametrize("new", [1, 70])
def test_captured_and_replayed_beside_another(new):
    """Two graphs on two streams, replayed at once and again after the lengths
    moved on: the bits of eager calls on the same state."""
    a = case(170, [200, 333], [new, new], 8, 2, 32, 128)
    b = case(171, [150], [new], 4, 4, 16, 64)
    graphs = []
    for x in (a, b):
        Q, K, V, table, lens, offs = x
        args = [dev(Q, BF), dev(K, BF), dev(V, BF), i32(table), i32(lens), i32(offs)]
        out = mha.sdpa_paged(*args, max_new=new)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            mha.sdpa_paged(*args, max_new=new, out=out)
        graphs.append((g, s, args, out))
    for shift in (0, 3):
        want = []
        for g, s, args, out in graphs:
            args[4] -= shift
            want.append(mha.sdpa_paged(*args, max_new=new))
            out.zero_()
        torch.cuda.synchronize()
        for g, s, args, out in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, (g, s, args, out) in zip(want, graphs):
            assert torch.equal(w, out)
    assert mha.mha_check() == mha.MHA_OK


@pytest.mark.parametrize("new", [1, 33])
def test_equal_calls_give_equal_bits_on_any_stream(new):
    x = case(180, [900, 412, 77], [new] * 3, 12, 4, 64, 64)
    args = [dev(x[0], BF), dev(x[1], BF), dev(x[2], BF), *(i32(v) for v in x[3:])]
    first = mha.sdpa_paged(*args, max_new=new)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [mha.sdpa_paged(*args, max_new=new, stream=s) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)


def test_rows_beyond_32_bit_offsets():
    """Pages past 2^31 elements of the pool (a 4.3 GB pool of zeros whose last
    pages hold the sequence)."""
    Hkv, ps, d, lens, new = 8, 128, 128, [300], [2]
    Q, K, V, table, lens, offs = case(190, lens, new, 16, Hkv, ps, d, spare=0)
    P = (1 << 31) // (Hkv * ps * d) + 8
    kp = torch.zeros((P, Hkv, ps, d), dtype=BF, device="cuda")
    kp[-3:] = dev(K, BF)
    vp = torch.zeros_like(kp)
    vp[-3:] = dev(V, BF)
    O, A = ref.sdpa_paged(Q, K, V, table, lens, offs)
    for m in (2, 64):
        got = mha.sdpa_paged(dev(Q, BF), kp, vp, i32(table + P - 3), i32(lens), i32(offs),
                             max_new=m, out_dtype=F32)
        assert mha.mha_check() == mha.MHA_OK
        check(to_np(got), O, A, F32)


@pytest.mark.parametrize("lead", [1, 40])
@pytest.mark.parametrize("new", [[1, 1, 1], [0, 5, 33]])
def test_tokens_ahead_of_the_first_sequence_are_passed_over(lead, new):
    """q_offsets[0] > 0: the same bits as without them, their rows untouched."""
    Q, K, V, table, lens, offs = case(195, [90, 80, 70], new, 4, 2, 16, 64)
    args = [dev(K, BF), dev(V, BF), i32(table), i32(lens)]
    want = mha.sdpa_paged(dev(Q, BF), *args, i32(offs), max_new=max(new))
    wide = dev(np.concatenate((np.full((lead, *Q.shape[1:]), np.nan, np.float32), Q)), BF)
    out = torch.full(wide.shape, 7.0, dtype=BF, device="cuda")
    mha.sdpa_paged(wide, *args, i32(offs + lead), max_new=max(new), out=out)
    assert mha.mha_check() == mha.MHA_OK
    assert torch.all(out[:lead] == 7.0) and torch.equal(out[lead:], want)


def test_a_batch_without_sequences():
    """B = 0 through every paged call: the tokens are nobody's, no page is held."""
    Hkv, ps, d = 2, 16, 64
    kp = torch.randn((5, Hkv, ps, d), device="cuda").to(BF)
    vp = torch.randn((5, Hkv, ps, d), device="cuda").to(BF)
    keep = kp.clone(), vp.clone()
    table = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    g, pe = torch.ones(d, dtype=BF, device="cuda"), mha.sinusoidal_pe(8, d)
    for T in (0, 3):
        q, k = (torch.randn((T, h, d), device="cuda").to(BF) for h in (4, Hkv))
        for call in (lambda out: mha.qk_norm_rope_paged(q, k, k, g, g, pe, kp, vp, table, none,
                                                        i32([0]), out=out),
                     lambda out: mha.sdpa_paged(q, kp, vp, table, none, i32([0]), out=out)):
            out = torch.full_like(q, 7.0)
            assert call(out) is out and torch.all(out == 7.0)
    mha.kv_pages_fork(kp, vp, table, none, none, none, none)
    dst = torch.full_like(kp, 3.0), torch.full_like(vp, 5.0)
    n = mha.kv_pages_compact(kp, vp, table, none, *dst, torch.empty_like(table))
    assert mha.mha_check() == mha.MHA_OK and n.tolist() == [0]
    assert torch.all(dst[0] == 3.0) and torch.all(dst[1] == 5.0)
    assert torch.equal(kp, keep[0]) and torch.equal(vp, keep[1])
