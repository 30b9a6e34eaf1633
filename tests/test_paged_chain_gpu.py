"""The paged cache's operators together, as a server runs them: prompts are
normed, rotated and appended in chunks, attended to, forked into samples that
decode on, and compacted into another pool and decoded further, all on one
stream; against the same steps in fp64 over contiguous sequences.

Tolerance: keys and queries are stored in bf16, and the fp64 side stores them
so too, rounding its own fp64 values; where the two round a value to different
neighbours (it lay within the fp32 arithmetic's error of a tie), scores and
outputs move by a bf16 step of one component.  The attention's own bound is
(2^-8 + 2^-10) A + 2^-8 |o|; one component of a row of 64 moving by a step
(2^-7 of it) moves a score by at most 2^-7 |q_c k_c| / 8 <= 2^-7 * 16 / 8 =
2^-6 for components up to 4, so each weight by 2^-6 of itself: 2 * 2^-6 A is
added for it."""
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

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


@pytest.mark.parametrize("H,Hkv,d,ps,pairing", [(4, 2, 64, 16, mha.ROPE_HALF),
                                                (6, 1, 128, 32, mha.ROPE_INTERLEAVED)])
def test_serving_steps(H, Hkv, d, ps, pairing):
    rng = np.random.default_rng(H)
    B, cols, P, layers = 5, 12, 64, 2
    kp = torch.full((layers, P, Hkv, ps, d), float("nan"), dtype=BF, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    free = list(rng.permutation(P))
    table = np.full((B, cols), -1, np.int32)
    lens = np.zeros(B, np.int32)
    gq, gk = (round_to_bf16(1 + 0.1 * rng.standard_normal(d, dtype=np.float32)) for _ in range(2))
    pe = mha.sinusoidal_pe(cols * ps, d)
    pe_np = to_np(pe)
    keys = [[np.zeros((0, Hkv, d)) for _ in range(B)] for _ in range(layers)]
    vals = [[np.zeros((0, Hkv, d)) for _ in range(B)] for _ in range(layers)]
    state = dict(kp=kp, vp=vp, table=i32(table), lens=i32(lens))

    def step(new):
        """new[b] more tokens for sequence b, through both layers."""
        nonlocal table
        before = lens.copy()
        for b, n in enumerate(new):
            while (table[b] >= 0).sum() * ps < lens[b] + n:
                table[b, (table[b] >= 0).sum()] = free.pop()
            lens[b] += n
        state["table"].copy_(i32(table))
        state["lens"].copy_(i32(lens))
        offs = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        T = int(offs[-1])
        for y in range(layers):
            q, k, v = (round_to_bf16(rng.standard_normal((T, h, d), dtype=np.float32))
                       for h in (H, Hkv, Hkv))
            qo = mha.qk_norm_rope_paged(*(dev(x, BF) for x in (q, k, v)), dev(gq, BF), dev(gk, BF),
                                        pe, state["kp"], state["vp"], state["table"],
                                        state["lens"], i32(offs), pairing=pairing, layer=y)
            O = mha.sdpa_paged(qo, state["kp"], state["vp"], state["table"], state["lens"],
                               i32(offs), max_new=max(new), layer=y)
            got = to_np(O)
            for b, n in enumerate(new):
                if n == 0:
                    continue
                rows = slice(offs[b], offs[b + 1])
                at = pe_np[before[b]:before[b] + n][:, None]
                kr = round_to_bf16(ref.qk_norm_rope(k[rows], gk, at, pairing, 1e-6).astype(np.float32))
                qr = round_to_bf16(ref.qk_norm_rope(q[rows], gq, at, pairing, 1e-6).astype(np.float32))
                keys[y][b] = np.concatenate((keys[y][b], kr))
                vals[y][b] = np.concatenate((vals[y][b], v[rows]))
                one = lambda x: x.transpose(1, 0, 2)[None]
                m = len(keys[y][b])
                page = -(-m // ps) * ps
                pad = lambda x: np.concatenate((x, np.zeros((page - m, Hkv, d)))).reshape(
                    -1, ps, Hkv, d).transpose(0, 2, 1, 3)
                w, A = ref.sdpa_paged(qr, pad(keys[y][b]), pad(vals[y][b]),
                                      np.arange(page // ps)[None], [m], [0, n])
                bound = (2.0 ** -5 + 2.0 ** -8 + 2.0 ** -10) * A + 2.0 ** -8 * np.abs(w)
                assert np.all(np.abs(got[rows] - w) <= bound), (b, y)

    step([40, 7, 0, 0, 0])            # two prompts
    step([33, 0, 0, 0, 0])            # the longer one's second chunk
    step([1, 1, 0, 0, 0])             # one token each
    # sequences 2 and 3 continue 0, sequence 4 continues 1
    fresh = [free.pop() for _ in range(3)]
    mha.kv_pages_fork(state["kp"], state["vp"], state["table"], state["lens"], i32([0, 0, 1]),
                      i32([2, 3, 4]), i32(fresh))
    table, lens[:] = state["table"].cpu().numpy().copy(), state["lens"].cpu().numpy()
    assert list(lens) == [74, 8, 74, 74, 8]
    for c, p in ((2, 0), (3, 0), (4, 1)):
        for y in range(layers):
            keys[y][c], vals[y][c] = keys[y][p].copy(), vals[y][p].copy()
    step([1, 1, 1, 1, 1])             # the samples part ways
    step([2, 0, 1, 3, 1])
    # sequences 1 and 3 end; the rest moves into a smaller pool
    lens[[1, 3]] = 0
    table[[1, 3]] = -1
    state["lens"].copy_(i32(lens))
    state["table"].copy_(i32(table))
    for y in range(layers):
        for b in (1, 3):
            keys[y][b] = keys[y][b][:0]
            vals[y][b] = vals[y][b][:0]
    small = dict(kp=torch.full((layers, 30, Hkv, ps, d), float("nan"), dtype=BF, device="cuda"),
                 table=torch.full((B, cols), -1, dtype=torch.int32, device="cuda"),
                 lens=state["lens"])
    small["vp"] = torch.full_like(small["kp"], float("nan"))
    n = mha.kv_pages_compact(state["kp"], state["vp"], state["table"], state["lens"], small["kp"],
                             small["vp"], small["table"])
    live = int(n)
    assert live == len({int(p) for b in range(B) for p in table[b, :-(-lens[b] // ps)]})
    state.update(small)
    table = state["table"].cpu().numpy().copy()
    free[:] = list(range(29, live - 1, -1))
    step([1, 20, 1, 0, 1])            # decoding goes on, a new prompt in the freed place
    assert mha.mha_check() == mha.MHA_OK


def test_training_step_through_the_attention():
    """qk_norm_rope -> sdpa_forward_lse -> sdpa_backward -> qk_norm_rope's
    backward: finite, zero where nothing is learned from (a value's rows do
    not reach dK through one visible key), and the gradient of a scale of x is
    zero: the norm divides it out.  <x, dx> per row is rstd eps-small; in
    arithmetic, dx rounds to bf16, so |<x, dx>| <= 2^-8 sum |x dx| + 2^-17 of
    the terms' magnitudes, bounded by the same sum with a margin of 2."""
    rng = np.random.default_rng(9)
    B, L, H, d = 2, 200, 4, 64
    q, k = (dev(round_to_bf16(rng.standard_normal((B, L, H, d), dtype=np.float32)), BF)
            for _ in range(2))
    v, dO = (dev(round_to_bf16(rng.standard_normal((B, H, L, d), dtype=np.float32)), BF)
             for _ in range(2))
    g = dev(round_to_bf16(1 + 0.1 * rng.standard_normal(d, dtype=np.float32)), BF)
    pe = mha.sinusoidal_pe(L, d)
    Q, K = mha.qk_norm_rope(q, k, g, g, pe)
    O, lse = mha.sdpa_forward_lse(Q, K, v, mask_kind=mha.MASK_CAUSAL)
    dQ, dK, dV = mha.sdpa_backward(Q, K, v, O, dO, lse, mask_kind=mha.MASK_CAUSAL)
    dq, dk, dgq, dgk = mha.qk_norm_rope_backward(q, k, g, g, pe, dQ, dK)
    assert mha.mha_check() == mha.MHA_OK
    for x, dx in ((q, dq), (k, dk)):
        a, b = to_np(x), to_np(dx)
        assert np.all(np.isfinite(b))
        assert np.all(np.abs((a * b).sum(-1)) <= 2 * 2.0 ** -8 * np.abs(a * b).sum(-1) + 1e-5)
    # dgamma against the fp64 formula on the same dQ, dK
    rows = to_np(pe)[None, :, None]
    for x, dy, got in ((q, dQ, dgq), (k, dK, dgk)):
        _, dg, _, mag = ref.qk_norm_rope_backward(to_np(x), to_np(g), rows,
                                                  to_np(dy).transpose(0, 2, 1, 3), 0, 1e-6)
        assert np.all(np.abs(to_np(got) - dg) <= (B * L * H + 32) * 2.0 ** -24 * mag + 1e-35)


def side_stream_calls(rng):
    """(name, call(stream), tensors that it updates in place) for every paged
    and norm call on state of its own."""
    H, Hkv, d, ps, lens = 4, 2, 64, 16, [70, 41, 0, 0]
    K, V, table, offs, free = make_pages(rng, lens, [3, 2, 0, 0], Hkv, ps, d, bf16=True, spare=4)
    state = lambda: [dev(K, BF), dev(V, BF), i32(table), i32(lens)]
    T = int(offs[-1])
    draw = lambda *shape, dt=BF: dev(rng.standard_normal(shape, dtype=np.float32), dt)
    q, k, v = draw(T, H, d), draw(T, Hkv, d), draw(T, Hkv, d)
    x, y = draw(2, 300, H, d), draw(2, 300, Hkv, d)
    dx, dy = draw(2, H, 300, d, dt=torch.float32), draw(2, Hkv, 300, d)
    g, pe = draw(d), mha.sinusoidal_pe(300, d)
    o, pair = i32(offs), [i32([0, 1]), i32([2, 3]), i32(free[:2])]
    a, f, c, p = state(), state(), state(), state()
    dst = [torch.zeros_like(c[0]), torch.zeros_like(c[1]), torch.full_like(c[2], -1)]
    return [
        ("qk_norm_rope", lambda s: mha.qk_norm_rope(x, y, g, g, pe, stream=s), []),
        ("qk_norm_rope_backward",
         lambda s: mha.qk_norm_rope_backward(x, y, g, g, pe, dx, dy, stream=s), []),
        ("qk_norm_rope_paged",
         lambda s: [mha.qk_norm_rope_paged(q, k, v, g, g, pe, *a, o, stream=s)], a[:2]),
        ("sdpa_paged", lambda s: [mha.sdpa_paged(q, *p, o, max_new=3, stream=s)], []),
        ("kv_pages_fork", lambda s: mha.kv_pages_fork(*f, *pair, stream=s) or [], f),
        ("kv_pages_compact", lambda s: [mha.kv_pages_compact(*c, *dst, stream=s)], dst),
    ]


@pytest.mark.parametrize("which", range(6))
def test_calls_on_a_side_stream(which):
    """The bits of the current stream's calls; and while a call still waits on
    the side stream, what the current stream allocates and writes meanwhile
    lies on none of the call's outputs or workspace."""
    name, call, touched = side_stream_calls(np.random.default_rng(300))[which]
    want = [t.clone() for t in (*call(None), *touched)]
    torch.cuda.synchronize()
    name, call, touched = side_stream_calls(np.random.default_rng(300))[which]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)       # about 10 ms
    got = list(call(s))
    over = [torch.full((n,), -7.0, device="cuda") for n in (4, 64, 1024, 1 << 16, 1 << 18, 1 << 19)
            for _ in range(4)]
    torch.cuda.synchronize()
    assert mha.mha_check() == mha.MHA_OK, name
    assert all(torch.equal(a, b) for a, b in zip(want, [*got, *touched])), name
    assert all(torch.all(t == -7.0) for t in over)
    # outputs given up while the call waits: their memory is not handed out before it has run
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    gone = call(s)
    sizes = [(t.shape, t.dtype) for t in gone]
    del gone
    over = [torch.full(shape, -7, dtype=dt, device="cuda") for shape, dt in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.all(t == -7) for t in over), name
    mha.mha_check()                         # a second fork of the same pairs is another's matter


def test_paged_calls_refuse_streams_of_another_device():
    """On the host, before anything is launched."""
    for name, call, _ in side_stream_calls(np.random.default_rng(301)):
        class Elsewhere:
            device_index, cuda_stream = 1 + torch.cuda.current_device(), 0
        with pytest.raises(ValueError, match="current device"):
            call(Elsewhere())
