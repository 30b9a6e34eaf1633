"""The calls on pages in 8 bits and on selected pages, on streams of their own:
the bits of the current stream's calls, no memory handed out too early, streams
of another device refused, two calls at once."""
import numpy as np
import pytest
import torch

import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from tests.e4m3_util import dev8, f32, make_pages8
from tests.paged_util import dev, i32

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


def side_stream_calls(rng):
    """(name, call(stream), tensors that it updates in place) for every call on
    state of its own."""
    H, Hkv, d, ps, lens = 4, 2, 64, 16, [170, 141, 0, 0]
    kc, ks, vc, vs, table, offs, free = make_pages8(rng, lens, [23, 20, 0, 0], Hkv, ps, d, spare=4)
    P, T = kc.shape[0], int(offs[-1])
    state = lambda: [dev8(kc), dev8(vc), i32(table), i32(lens)]
    scales = lambda: dict(K_scale=f32(ks), V_scale=f32(vs))
    draw = lambda *shape: dev(rng.standard_normal(shape, dtype=np.float32), BF)
    q, k, v, g, pe = draw(T, H, d), draw(T, Hkv, d), draw(T, Hkv, d), draw(d), mha.sinusoidal_pe(300, d)
    o, one, pair = i32(offs), i32([0, 1, 2, 2, 2]), [i32([0, 1]), i32([2, 3]), i32(free[:2])]
    b = torch.from_numpy(np.sort(rng.integers(-99, 99, (P, Hkv, 2, d)), 2).astype(np.int8)).cuda()
    bs = f32(rng.random((P, Hkv)) + 0.5)
    b2, bs2 = torch.zeros_like(b), torch.zeros_like(bs)
    a, f, c, p = state(), state(), state(), state()
    sa, sf, sc, sp = scales(), scales(), scales(), scales()
    raw = lambda ts: [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in ts]
    dst = [torch.zeros_like(c[0].view(torch.uint8)).view(c[0].dtype) for _ in range(2)]
    dst.append(torch.full_like(c[2], -1))
    so = dict(K_scale_out=torch.zeros_like(sc["K_scale"]), V_scale_out=torch.zeros_like(sc["V_scale"]))
    sel, rows = mha.kv_pages_select(q, *p, o, b, bs, 4, **sp)
    torch.cuda.synchronize()
    return [
        ("qk_norm_rope_paged", lambda s: [mha.qk_norm_rope_paged(q, k, v, g, g, pe, *a, o, stream=s, **sa)],
         raw([*a[:2], *sa.values()])),
        ("sdpa_paged rows", lambda s: [mha.sdpa_paged(q, *p, o, stream=s, **sp)], []),
        ("sdpa_paged few", lambda s: [mha.sdpa_paged(q[:2], *p, one, max_new=1, stream=s, **sp)], []),
        ("kv_pages_fork", lambda s: mha.kv_pages_fork(*f, *pair, stream=s, **sf) or [],
         raw([*f, *sf.values()])),
        ("kv_pages_compact", lambda s: [mha.kv_pages_compact(*c, *dst, stream=s, **sc, **so)],
         raw([*dst, *so.values()])),
        ("kv_pages_bounds", lambda s: mha.kv_pages_bounds(*p, o, b2, bs2, T, stream=s, **sp) or [], [b2, bs2]),
        ("kv_pages_select", lambda s: list(mha.kv_pages_select(q, *p, o, b, bs, 4, stream=s, **sp)), []),
        ("sdpa_paged_selected", lambda s: [mha.sdpa_paged_selected(q, *p[:2], sel, rows, stream=s, **sp)], []),
    ]


@pytest.mark.parametrize("which", range(8))
def test_calls_on_a_side_stream(which):
    name, call, touched = side_stream_calls(np.random.default_rng(700))[which]
    want = [t.clone() for t in (*call(None), *touched)]
    torch.cuda.synchronize()
    name, call, touched = side_stream_calls(np.random.default_rng(700))[which]
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


def test_calls_refuse_streams_of_another_device():
    for name, call, _ in side_stream_calls(np.random.default_rng(701)):
        class Elsewhere:
            device_index, cuda_stream = 1 + torch.cuda.current_device(), 0
        with pytest.raises(ValueError, match="current device"):
            call(Elsewhere())


def test_many_calls_at_once_on_several_streams():
    """Selections and attentions of four states, interleaved on four streams
    again and again: the bits of each alone."""
    states = [side_stream_calls(np.random.default_rng(710 + i)) for i in range(4)]
    calls = [{n: c for n, c, _ in s} for s in states]
    names = ("kv_pages_select", "sdpa_paged_selected", "sdpa_paged rows", "sdpa_paged few")
    want = [{n: [t.clone() for t in c[n](None)] for n in names} for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i, (c, s) in enumerate(zip(calls, streams)):
            got += [(i, n, c[n](s)) for n in names]
    torch.cuda.synchronize()
    assert mha.mha_check() == mha.MHA_OK
    for i, n, out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want[i][n])), n
