"""kv_pages_fork and kv_pages_compact on the GPU against oracle/paged.py:
copies and tables, so every comparison is exact."""
import numpy as np
import pytest
import torch

import oracle.paged as ref
import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from tests.gpu_util import to_np
from tests.paged_util import dev, i32, make_pages

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


def forks(seed, lens, kids, layers, Hkv, ps, d, spare=2):
    """A cache with room for `kids` children behind the parents' rows."""
    rng = np.random.default_rng(seed)
    K, V, table, _, free = make_pages(rng, lens, [0] * len(lens), Hkv, ps, d, bf16=True,
                                      spare=kids + spare, layers=layers)
    table = np.concatenate((table, np.full((kids, table.shape[1]), -1, np.int32)))
    lengths = np.concatenate((lens, np.full(kids, 99))).astype(np.int32)
    return K, V, table, lengths, free, rng


FORKS = [
    # lens, children of which parents, layers, Hkv, page, d, dtype
    ([37], [0], 1, 1, 16, 64, BF),
    ([37, 0, 32, 5], [3, 0, 0, 2, 1, 0], 3, 2, 16, 64, BF),
    ([300, 129], [0, 1, 1], 2, 3, 128, 128, BF),
    ([70, 64], [1, 0], 2, 1, 64, 96, F32),
    ([255], [0] * 40, 1, 8, 256, 128, BF),
    ([33] * 9, list(range(9)) * 60, 1, 1, 32, 64, BF),     # more pairs than threads of a block
]


@pytest.mark.parametrize("c", FORKS, ids=[str(i) for i in range(len(FORKS))])
def test_fork(c):
    lens, parents, layers, Hkv, ps, d, dt = c
    K, V, table, lengths, free, rng = forks(FORKS.index(c), lens, len(parents), layers, Hkv, ps, d)
    children = len(lens) + rng.permutation(len(parents))
    fresh = free[:len(parents)]
    want = ref.fork(K, V, table, lengths, parents, children, fresh)
    got = [dev(K, dt), dev(V, dt), i32(table), i32(lengths)]
    for _ in range(2):      # a second, equal call changes nothing more
        mha.kv_pages_fork(*got, i32(parents), i32(children), i32(fresh))
        assert mha.mha_check() == mha.MHA_OK
        for g, w in zip(got, want):
            assert np.array_equal(to_np(g), w)


def test_fork_refuses_bad_pairs_alone():
    """Every bad pair changes nothing and is reported; the good one beside it
    is carried out."""
    K, V, table, lengths, free, _ = forks(20, [37, 20, 16], 4, 2, 2, 16, 64)
    P = K.shape[1]
    good = (0, 3, free[0])
    # sequence 6 stands with a bad length, sequence 5 with a bad last page
    lengths[6], lengths[5], table[5, 1] = table.shape[1] * 16 + 1, 20, P
    bad = [
        [(-1, 4, free[1])], [(7, 4, free[1])], [(1, -1, free[1])], [(1, 7, free[1])],
        [(1, 1, free[1])],                                   # its own child
        [(1, 0, free[1])],                                   # the child is a parent
        [(1, 4, free[1]), (2, 4, free[2])],                  # one child of two
        [(1, 4, -1)], [(1, 4, P)],                           # no such page
        [(1, 4, free[0])],                                   # the good pair's page: neither
        [(6, 4, free[1])], [(5, 4, free[1])],
    ]
    for pairs in bad:
        rows = [good, *pairs]
        shared_page = any(p[2] == free[0] for p in pairs)
        child_is_parent = any(p[1] == 0 for p in pairs)
        par, chi, fr = ([p[i] for p in rows] for i in range(3))
        want = (K, V, table, lengths) if shared_page else ref.fork(
            K, V, table, lengths, par[:1], chi[:1], fr[:1])
        got = [dev(K, BF), dev(V, BF), i32(table), i32(lengths)]
        mha.kv_pages_fork(*got, i32(par), i32(chi), i32(fr))
        assert mha.mha_check() == mha.MHA_ERR_DEVICE
        for g, w in zip(got, want):
            assert np.array_equal(to_np(g), w), (pairs, child_is_parent)
    # a full last page needs no fresh one: any value will do, twice too
    got = [dev(K, BF), dev(V, BF), i32(table), i32(lengths)]
    mha.kv_pages_fork(*got, i32([2, 2]), i32([3, 4]), i32([-7, -7]))
    assert mha.mha_check() == mha.MHA_OK
    assert got[3].tolist()[3:5] == [16, 16] and torch.equal(got[0], dev(K, BF))


COMPACTS = [
    # lens, spare, layers, Hkv, page, d, dtype, room beyond the held pages
    ([37, 0, 32, 5], 9, 1, 2, 16, 64, BF, 0),
    ([300, 1, 129], 1, 3, 1, 128, 128, BF, 4),
    ([70] * 20, 300, 2, 2, 32, 96, F32, 0),
    ([0, 0], 40, 1, 1, 16, 64, BF, 1),
    ([1], 0, 1, 1, 16, 64, BF, 0),
    ([16 * 90, 7], 2500, 1, 1, 16, 64, BF, 3),              # more words than threads of a warp
]


@pytest.mark.parametrize("c", COMPACTS, ids=[str(i) for i in range(len(COMPACTS))])
def test_compact(c):
    lens, spare, layers, Hkv, ps, d, dt, room = c
    rng = np.random.default_rng(40 + COMPACTS.index(c))
    K, V, table, _, _ = make_pages(rng, lens, [0] * len(lens), Hkv, ps, d, spare=spare, bf16=True,
                                   layers=layers)
    if len(lens) > 2 and lens[0] > ps and lens[2] > ps:
        table[2, :1] = table[0, :1]         # shared, as forks leave them
    table[table < 0] = 2 ** 31 - 1          # never read
    lens = np.asarray(lens, np.int32)
    n = len({int(p) for b, m in enumerate(-(-lens // ps)) for p in table[b, :m]})
    shape = (layers, max(1, n) + room, Hkv, ps, d)
    Ko, Vo = np.full(shape, 3.0, np.float32), np.full(shape, 5.0, np.float32)
    to = np.full((len(lens), table.shape[1] + 2), -9, np.int32)
    wk, wv, wt, count = ref.compact(K, V, table, lens, Ko, Vo, to)
    assert count == n
    dst = [dev(Ko, dt), dev(Vo, dt), i32(to)]
    got = mha.kv_pages_compact(dev(K, dt), dev(V, dt), i32(table), i32(lens), *dst)
    assert mha.mha_check() == mha.MHA_OK and got.tolist() == [n]
    for g, w in zip(dst, (wk, wv, wt)):
        assert np.array_equal(to_np(g), w)


def test_compact_between_strided_pools():
    """Layers and K/V interleaved page by page on one side, dense on the other."""
    rng = np.random.default_rng(60)
    lens, layers, Hkv, ps, d = [100, 30, 64], 3, 2, 32, 64
    K, V, table, _, _ = make_pages(rng, lens, [0] * 3, Hkv, ps, d, spare=5, bf16=True, layers=layers)
    P = K.shape[1]
    both = torch.zeros((P, layers, 2, Hkv, ps, d), dtype=BF, device="cuda")
    kp, vp = (both[:, :, i].transpose(0, 1) for i in (0, 1))
    kp.copy_(dev(K, BF))
    vp.copy_(dev(V, BF))
    zero = np.zeros((layers, 9, Hkv, ps, d), np.float32)
    want = ref.compact(K, V, table, np.asarray(lens), zero, zero, table)
    dst = [dev(zero, BF), dev(zero, BF), i32(table)]
    mha.kv_pages_compact(kp, vp, i32(table), i32(lens), *dst)
    assert mha.mha_check() == mha.MHA_OK
    for g, w in zip(dst, want):
        assert np.array_equal(to_np(g), w)


def test_compact_reports_what_it_cannot_place():
    rng = np.random.default_rng(61)
    lens, Hkv, ps, d = np.array([40, 33, 20], np.int32), 1, 16, 64
    K, V, table, _, _ = make_pages(rng, lens, [0] * 3, Hkv, ps, d, spare=4, bf16=True, layers=1)
    P = K.shape[1]
    zero = np.zeros((1, 8, Hkv, ps, d), np.float32)
    blank = np.full_like(table, -9)

    def call(table=table, lens=lens, room=8):
        dst = [dev(zero[:, :room], BF), dev(zero[:, :room], BF), i32(blank)]
        n = mha.kv_pages_compact(dev(K, BF), dev(V, BF), i32(table), i32(lens), *dst)
        assert mha.mha_check() == mha.MHA_ERR_DEVICE and mha.mha_check() == mha.MHA_OK
        return [to_np(x) for x in dst], int(n)

    for n in (-1, table.shape[1] * ps + 1, 2 ** 31 - 1):     # a bad length counts as empty
        (k, v, t), count = call(lens=np.array([40, n, 20], np.int32))
        want = ref.compact(K, V, table, [40, 0, 20], zero, zero, blank)
        assert count == want[3] and all(np.array_equal(a, b) for a, b in zip((k, v, t), want))
    for page in (-1, P, 2 ** 31 - 1):
        bad = table.copy()
        bad[1, 1] = page
        (k, v, t), count = call(table=bad)
        held = sorted({int(p) for b, m in enumerate((3, 3, 2)) for p in table[b, :m]}
                      - {int(table[1, 1])})
        assert count == 7 and t[1, 1] == -1
        for b, m in enumerate((3, 3, 2)):
            for j in range(m):
                if (b, j) != (1, 1):
                    assert t[b, j] == held.index(table[b, j])
                    assert np.array_equal(k[0, int(t[b, j])], K[0, table[b, j]])
    # a pool too small for the held pages
    (k, v, t), count = call(room=5)
    held = sorted(int(p) for b, m in enumerate((3, 3, 2)) for p in table[b, :m])
    assert count == 8 and np.array_equal(k[0], K[0, held[:5]])
    for b, m in enumerate((3, 3, 2)):
        for j in range(m):
            r = held.index(table[b, j])
            assert t[b, j] == (r if r < 5 else -1)


def test_captured_compaction_follows_the_lengths():
    """One graph, replayed after a sequence ended: the counts of eager calls."""
    rng = np.random.default_rng(62)
    lens = [100, 60, 200]
    K, V, table, _, _ = make_pages(rng, lens, [0] * 3, 2, 16, 64, spare=5, bf16=True, layers=1)
    src = [dev(K, BF), dev(V, BF), i32(table), i32(lens)]
    dst = [torch.zeros_like(src[0]), torch.zeros_like(src[1]), torch.full_like(src[2], -1)]
    mha.kv_pages_compact(*src, *dst)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        n = mha.kv_pages_compact(*src, *dst)
    for end in (None, 1, 0):
        if end is not None:
            src[3][end] = 0
        for x in dst:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = ref.compact(K, V, table, src[3].tolist(), *(np.zeros_like(to_np(x)) for x in dst))
        assert int(n) == want[3]
        for a, w in zip(dst, want):
            assert np.array_equal(to_np(a), w)
    assert mha.mha_check() == mha.MHA_OK


def test_pages_beyond_32_bit_offsets():
    """Append, fork and compaction over 4.3 GB pools whose sequence lies past
    2^31 elements: what a pool of the last pages alone gives."""
    rng = np.random.default_rng(70)
    Hkv, ps, d, last = 8, 128, 128, 6
    P = (1 << 31) // (Hkv * ps * d) + 8
    T, H = 9, 8
    draw = lambda *shape: dev(rng.standard_normal(shape, dtype=np.float32), BF)
    q, k, v, g = draw(T, H, d), draw(T, Hkv, d), draw(T, Hkv, d), draw(d)
    K, V = draw(last, Hkv, ps, d), draw(last, Hkv, ps, d)
    pe = mha.sinusoidal_pe(400, d)
    table = np.array([[4, 1, 3, 2], [-1] * 4], np.int32)     # page 5 and page 0 are free

    def steps(kp, vp, first):
        t = i32(np.where(table < 0, -1, table + first))
        lens, one = i32([300 + T, 0]), lambda x: i32([x])
        out = mha.qk_norm_rope_paged(q, k, v, g, g, pe, kp, vp, t, lens, i32([0, T, T]))
        mha.kv_pages_fork(kp, vp, t, lens, one(0), one(1), one(first + 5))
        dst = [torch.zeros((5, Hkv, ps, d), dtype=BF, device="cuda") for _ in range(2)]
        to = torch.full_like(t, -1)
        n = mha.kv_pages_compact(kp, vp, t, lens, *dst, to)
        assert mha.mha_check() == mha.MHA_OK
        return [out, kp[first:first + last], vp[first:first + last], lens, *dst, to, n]

    want = steps(K.clone(), V.clone(), 0)
    assert want[-1].tolist() == [4]
    first = P - last
    big = [torch.zeros((P, Hkv, ps, d), dtype=BF, device="cuda") for _ in range(2)]
    big[0][first:], big[1][first:] = K, V
    for a, b in zip(want, steps(*big, first)):
        assert torch.equal(a, b)
    assert not torch.any(big[0][:first]) and not torch.any(big[1][:first])
