"""qk_norm_rope_paged, kv_pages_fork and kv_pages_compact on a cache in 8 bits,
on the GPU, against the oracle.

Values, scales and older rows are exact.  A key is normed and rotated in fp32,
off by at most 2^-18 of the sum of its terms' magnitudes (64 or 128 squares
summed in chains of 16 and a tree, a reciprocal root, three products and two
sums: fewer than 2^6 roundings of 2^-24), and stored in e4m3, half a step of
2^-4 of it or of 2^-10 of the scale."""
import numpy as np
import pytest
import torch

import oracle.paged as paged
import oracle.paged_e4m3 as ref
import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from transformer_head_scaled_03_gb300.inputs import round_to_bf16
from tests.e4m3_util import codes_of, dev8, f32, make_pages8
from tests.gpu_util import to_np
from tests.paged_util import dev, i32

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


class Append:
    def __init__(self, seed, lens, new, H, Hkv, ps, d, r, pairing, layers=None, size=None, pow2=True):
        rng = np.random.default_rng(seed)
        self.kc, self.ks, self.vc, self.vs, self.table, self.offs, _ = make_pages8(
            rng, lens, new, Hkv, ps, d, pow2, layers=layers)
        T = int(self.offs[-1])
        normal = lambda *s: rng.standard_normal(s, dtype=np.float32)
        self.q, self.k = round_to_bf16(normal(T, H, d)), round_to_bf16(normal(T, Hkv, d))
        v = normal(T, Hkv, d)
        if size is not None:
            v = v * size(rng, T)[:, None, None]
        self.v = round_to_bf16(v.astype(np.float32))
        self.gq, self.gk = (round_to_bf16(1 + 0.2 * normal(d)) for _ in range(2))
        self.lens, self.r, self.pairing, self.ps = np.asarray(lens, np.int32), r, pairing, ps
        self.pe = mha.sinusoidal_pe(max(max(lens), 1), r)
        self.pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)]).astype(int)

    def state(self):
        return [dev8(self.kc), dev8(self.vc), f32(self.ks), f32(self.vs)]

    def run(self, state, rows=slice(None), lens=None, offs=None, **kw):
        out = mha.qk_norm_rope_paged(
            dev(self.q[rows], BF), dev(self.k[rows], BF), dev(self.v[rows], BF), dev(self.gq, BF),
            dev(self.gk, BF), self.pe, state[0], state[1], i32(self.table),
            i32(self.lens if lens is None else lens), i32(self.offs if offs is None else offs),
            pairing=self.pairing, K_scale=state[2], V_scale=state[3], **kw)
        return out

    def keys(self):
        pe = to_np(self.pe)[self.pos][:, None]
        y = paged.qk_norm_rope(self.k, self.gk, pe, self.pairing, 1e-6)
        # a rotated element's two terms are at most the row's largest element each
        z = np.abs(self.k) / np.sqrt(np.mean(self.k.astype(np.float64) ** 2, -1, keepdims=True) + 1e-6) \
            * np.abs(self.gk)
        return y, 2 * z.max(-1, keepdims=True)

    def queries(self):
        return paged.qk_norm_rope(self.q, self.gq, to_np(self.pe)[self.pos][:, None], self.pairing, 1e-6)

    def check(self, state, layer=None):
        """The state after one call with everything, from the first state."""
        at = (lambda x: x) if layer is None else (lambda x: x[layer])
        kc, vc, ks, vs = codes_of(state[0]), codes_of(state[1]), to_np(state[2]), to_np(state[3])
        if layer is not None:       # the other layers are untouched
            for other in set(range(len(kc))) - {layer}:
                for g, w in ((kc, self.kc), (vc, self.vc), (ks, self.ks), (vs, self.vs)):
                    assert np.array_equal(g[other], w[other])
        wv, wvs = ref.append(at(self.vc), at(self.vs), self.v, self.table, self.lens, self.offs)
        assert np.array_equal(at(vc), wv) and np.array_equal(at(vs), wvs)
        y, mag = self.keys()
        wk, wks = ref.append(at(self.kc), at(self.ks), y, self.table, self.lens, self.offs)
        assert np.array_equal(at(ks), wks)
        new = np.zeros(wk.shape, bool)
        page = np.concatenate([self.table[b][self.pos[self.offs[b]:self.offs[b + 1]] // self.ps]
                               for b in range(len(self.lens))])
        new[page, :, self.pos % self.ps] = True
        assert np.array_equal(at(kc)[~new], wk[~new])
        got = ref.decode(at(kc), at(ks))[page, :, self.pos % self.ps]
        s = wks[page][..., None]
        half = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s)
        assert np.all(np.abs(got - y) <= half + 2.0 ** -18 * mag * (1 + 2.0 ** -4))


CASES = [
    # lens, new, H, Hkv, page, d, rope_dim, pairing
    ([1], [1], 1, 1, 16, 64, 64, mha.ROPE_HALF),
    ([37, 100], [1, 1], 4, 2, 16, 64, 32, mha.ROPE_INTERLEAVED),
    ([48, 33, 16], [1, 1, 1], 8, 8, 16, 128, 128, mha.ROPE_HALF),      # a page's first row, its last
    ([40, 0, 77], [3, 0, 20], 6, 3, 32, 128, 64, mha.ROPE_INTERLEAVED),
    ([300, 129], [300, 64], 4, 2, 64, 128, 128, mha.ROPE_HALF),
    ([513], [400], 2, 1, 256, 128, 128, mha.ROPE_INTERLEAVED),         # rows computed twice
    ([700], [650], 3, 3, 256, 64, 16, mha.ROPE_HALF),
    ([260, 5, 31], [250, 5, 1], 4, 4, 128, 64, 64, mha.ROPE_INTERLEAVED),
    ([16 * 70] + [9] * 50, [16 * 60] + [1] * 50, 2, 1, 16, 64, 64, mha.ROPE_HALF),
    ([160] + [9] * 99, [150] + [1] * 99, 2, 1, 16, 128, 64, mha.ROPE_HALF),   # a warp to a unit
    ([600] + [9] * 199, [500] + [0] * 150 + [1] * 49, 2, 2, 256, 128, 64, mha.ROPE_HALF),
]


@pytest.mark.parametrize("c", CASES, ids=[str(i) for i in range(len(CASES))])
def test_append(c):
    x = Append(400 + CASES.index(c), *c, pow2=CASES.index(c) % 2 == 0)
    state = x.state()
    q = x.run(state)
    assert mha.mha_check() == mha.MHA_OK
    x.check(state)
    y = x.queries()
    assert np.all(np.abs(to_np(q) - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -16 * np.abs(y).max(-1, keepdims=True))


def test_one_layer_of_many_and_given_out():
    x = Append(420, [70, 40], [30, 2], 4, 2, 32, 64, 64, mha.ROPE_HALF, layers=3)
    state = x.state()
    out = torch.full((32, 4, 64), 7.0, dtype=BF, device="cuda")
    assert x.run(state, layer=1, out=out) is out
    assert mha.mha_check() == mha.MHA_OK
    x.check(state, layer=1)


@pytest.mark.parametrize("cut", [[45], [1] * 45, [7, 20, 18], [16, 16, 13]])
def test_steps_of_any_size_store_the_same_values(cut):
    """Values whose size grows from row to row, one, a few or all at a time:
    the oracle's state after every step."""
    x = Append(421, [45], [45], 2, 2, 16, 64, 64, mha.ROPE_HALF,
               size=lambda rng, T: 2.0 ** np.linspace(-6, 6, T))
    state = x.state()
    vc, vs = x.vc, x.vs
    at = 0
    for k in cut:
        vc, vs = ref.append(vc, vs, x.v[at:at + k], x.table, [at + k], [0, k])
        x.run(state, slice(at, at + k), lens=[at + k], offs=[0, k])
        at += k
        assert np.array_equal(codes_of(state[1]), vc) and np.array_equal(to_np(state[3]), vs)
    assert mha.mha_check() == mha.MHA_OK


def test_zeros_tiny_and_not_finite_values():
    x = Append(422, [64], [64], 2, 2, 16, 64, 64, mha.ROPE_HALF)
    x.v[:16] = 0
    x.v[16:32] = round_to_bf16(x.v[16:32] * np.float32(2.0 ** -110))
    x.v[40, 0, 3], x.v[41, 1, 4], x.v[50] = np.nan, -np.inf, np.inf
    state = x.state()
    x.run(state)
    assert mha.mha_check() == mha.MHA_OK
    wv, wvs = ref.append(x.vc, x.vs, x.v, x.table, x.lens, x.offs)
    got, vs = codes_of(state[1]), to_np(state[3])
    assert np.array_equal(vs, wvs) and np.all(vs[x.table[0, 0]] == 0)
    assert np.all(np.isfinite(vs)) and np.all(vs[x.table[0, 1]] == 2.0 ** -100)
    assert np.array_equal(ref.VALUES[got], ref.VALUES[wv], equal_nan=True)


def test_zeros_behind_rows_of_the_smallest_scales():
    """A scale below the smallest normal number has no inverse in fp32: the page
    keeps it, and the new rows are zeros all the same."""
    x = Append(423, [9, 20], [1, 3], 2, 2, 16, 64, 64, mha.ROPE_HALF)
    x.v[:] = 0
    x.vs[:] = np.float32(1e-40)
    state = x.state()
    x.run(state)
    assert mha.mha_check() == mha.MHA_OK
    wv, wvs = ref.append(x.vc, x.vs, x.v, x.table, x.lens, x.offs)
    assert np.array_equal(to_np(state[3]), wvs.astype(np.float32))
    assert np.array_equal(ref.VALUES[codes_of(state[1])], ref.VALUES[wv], equal_nan=True)


@pytest.mark.parametrize("new", [1, 30])
def test_bad_entries_touch_nothing(new):
    """A bad page or length, a position behind the table, bad offsets: those
    tokens' queries are zeros (or untouched), their pages and scales as they
    were; the other sequences are served."""
    x = Append(423, [90, 80, 70], [new] * 3, 4, 2, 16, 64, 64, mha.ROPE_HALF)
    good = x.state()
    x.run(good)
    assert mha.mha_check() == mha.MHA_OK

    def call(table=None, untouched=(1,), **kw):
        keep, x.table = x.table, x.table if table is None else table
        state = x.state()
        out = torch.full((3 * new, 4, 64), 7.0, dtype=BF, device="cuda")
        x.run(state, out=out, **kw)
        x.table = keep
        assert mha.mha_check() == mha.MHA_ERR_DEVICE
        for b in range(3):
            held = keep[b, :-(-int(x.lens[b]) // 16)]
            for got, first, after in zip(state, x.state(), good):
                bits = lambda t: t.view(torch.uint8)[torch.from_numpy(held).long().cuda()]
                assert torch.equal(bits(got), bits(first if b in untouched else after))
        return out

    full = x.table.shape[1] * 16
    for n in (new - 1, full + 1, -5, 2 ** 31 - 1):
        out = call(lens=[90, n, 70])
        assert torch.all(out[new:2 * new] == 0)
    for page in (-1, x.kc.shape[0], 2 ** 31 - 1):
        t = x.table.copy()
        t[1, -(-80 // 16) - 1] = page
        if new == 1:
            out = call(table=t)
            assert torch.all(out[new:2 * new] == 0)
    call(offs=[0, new, 2 * new, 3 * new + 1], untouched=(2,))
    keep, x.pe = x.pe, x.pe[:80]
    if new == 1:
        out = call(untouched=(0,))
        assert torch.all(out[:1] == 0)
    x.pe = x.pe[:75]
    state = x.state()
    x.run(state)
    assert mha.mha_check() == mha.MHA_ERR_DEVICE
    x.pe = keep
    wv, wvs = ref.append(x.vc, x.vs, x.v, x.table, x.lens, x.offs, positions_below=75)
    assert np.array_equal(codes_of(state[1]), wv) and np.array_equal(to_np(state[3]), wvs)


def test_rows_in_a_wider_projection_and_streams():
    x = Append(424, [70, 40], [30, 12], 4, 2, 32, 64, 64, mha.ROPE_HALF)
    T = 42
    wide = torch.cat([dev(a, BF).view(T, -1) for a in (x.q, x.k, x.v)], 1)
    q, k, v = wide[:, :256].view(T, 4, 64), wide[:, 256:384].view(T, 2, 64), wide[:, 384:].view(T, 2, 64)
    s = torch.cuda.Stream()
    outs = []
    for stream in (None, s):
        state = x.state()
        s.wait_stream(torch.cuda.current_stream())
        outs.append(mha.qk_norm_rope_paged(q, k, v, dev(x.gq, BF), dev(x.gk, BF), x.pe, state[0], state[1],
                                           i32(x.table), i32(x.lens), i32(x.offs), pairing=x.pairing,
                                           K_scale=state[2], V_scale=state[3], stream=stream))
        torch.cuda.synchronize()
        assert mha.mha_check() == mha.MHA_OK
        x.check(state)
    assert torch.equal(*outs)


@pytest.mark.parametrize("new", [1, 30])
def test_captured_append_follows_the_lengths(new):
    x = Append(425, [90, 80], [new] * 2, 4, 2, 16, 128, 64, mha.ROPE_HALF)
    state, eager = x.state(), x.state()
    lens = i32(x.lens - new)
    args = [dev(a, BF) for a in (x.q, x.k, x.v, x.gq, x.gk)] + [x.pe]
    tail = lambda st, n: (st[0], st[1], i32(x.table), n, i32(x.offs))
    kw = lambda st: dict(pairing=x.pairing, K_scale=st[2], V_scale=st[3])
    t = tail(state, lens)
    mha.qk_norm_rope_paged(*args, *t, **kw(state))
    g = torch.cuda.CUDAGraph()
    out = torch.empty((2 * new, 4, 128), dtype=BF, device="cuda")
    with torch.cuda.graph(g):
        mha.qk_norm_rope_paged(*args, *t, out=out, **kw(state))
    mha.qk_norm_rope_paged(*args, *tail(eager, i32(x.lens - new)), **kw(eager))
    lens += new
    g.replay()
    want = mha.qk_norm_rope_paged(*args, *tail(eager, i32(x.lens)), **kw(eager))
    assert mha.mha_check() == mha.MHA_OK and torch.equal(out, want)
    for a, b in zip(state, eager):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("layers,Hkv,ps,d", [(1, 1, 16, 16), (3, 2, 16, 64), (2, 3, 128, 128)])
def test_fork_and_compact(layers, Hkv, ps, d):
    """Codes and scales move together; what they leave alone stays."""
    rng = np.random.default_rng(430)
    lens = [2 * ps + 5, 0, ps, ps - 1]
    kc, ks, vc, vs, table, _, free = make_pages8(rng, lens, [0] * 4, Hkv, ps, d, layers=layers, spare=6)
    parents, children = [3, 0, 2, 0], [4, 5, 6, 7]
    table = np.concatenate((table, np.full((4, table.shape[1]), -1, np.int32)))
    lens = np.concatenate((lens, np.full(4, 99))).astype(np.int32)
    fresh = free[:4]
    K, V, wt, wl = paged.fork(kc, vc, table, lens, parents, children, fresh)
    wks, wvs = ks.copy(), vs.copy()
    for p, f in zip(parents, fresh):
        if lens[p] % ps:
            wks[:, f], wvs[:, f] = ks[:, table[p, lens[p] // ps]], vs[:, table[p, lens[p] // ps]]
    a = [dev8(kc), dev8(vc), i32(table), i32(lens)]
    sc = dict(K_scale=f32(ks), V_scale=f32(vs))
    mha.kv_pages_fork(*a, i32(parents), i32(children), i32(fresh), **sc)
    assert mha.mha_check() == mha.MHA_OK
    for got, want in zip((codes_of(a[0]), codes_of(a[1]), to_np(a[2]), to_np(a[3]), to_np(sc["K_scale"]),
                          to_np(sc["V_scale"])), (K, V, wt, wl, wks, wvs)):
        assert np.array_equal(got, want)
    wl[5] = 0                                        # one sample ends
    a[3] = i32(wl)
    shape = (layers, 13, Hkv, ps, d)
    ko, vo = np.full(shape, 3, np.uint8), np.full(shape, 5, np.uint8)
    to = np.full((8, table.shape[1]), -9, np.int32)
    so = np.full((layers, 13, Hkv), 2.5)
    wk, wv, wto, n = paged.compact(K, V, wt, wl, ko, vo, to)
    live = sorted({int(p) for b, m in enumerate(-(-wl // ps)) for p in wt[b, :m]})
    wko, wvo = so.copy(), so.copy()
    wko[:, :n], wvo[:, :n] = wks[:, live], wvs[:, live]
    out = [dev8(ko), dev8(vo), i32(to)]
    sco = dict(K_scale_out=f32(so), V_scale_out=f32(so))
    count = mha.kv_pages_compact(*a, *out, **sc, **sco)
    assert mha.mha_check() == mha.MHA_OK and int(count) == n
    for got, want in zip((codes_of(out[0]), codes_of(out[1]), to_np(out[2]), to_np(sco["K_scale_out"]),
                          to_np(sco["V_scale_out"])), (wk, wv, wto, wko, wvo)):
        assert np.array_equal(got, want)


def test_pages_past_2_31_elements():
    ps, Hkv, d = 128, 8, 128
    P = 2 ** 31 // (Hkv * ps * d) + 2100
    x = Append(431, [300], [200], 2, Hkv, ps, d, 128, mha.ROPE_HALF)
    n = x.kc.shape[0]
    state = [torch.zeros((P, Hkv, ps, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    state += [torch.zeros((P, Hkv), device="cuda") for _ in range(2)]
    for big, small in zip(state, x.state()):
        big[P - n:] = small.view(big.dtype) if big.dtype is torch.uint8 else small
    keep = x.table
    x.table = np.where(keep >= 0, keep + P - n, -1).astype(np.int32)
    E8 = torch.float8_e4m3fn
    x.run([state[0].view(E8), state[1].view(E8), state[2], state[3]])
    assert mha.mha_check() == mha.MHA_OK
    x.table = keep
    for pool in state:
        assert not pool[:P - n].any()
    x.check([p[P - n:].view(E8) if p.dtype is torch.uint8 else p[P - n:] for p in state])
