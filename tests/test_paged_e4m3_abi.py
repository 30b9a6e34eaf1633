"""Refusals of the 8-bit cache's and the selection's entry points, without a
GPU: the C ABI rejects bad arguments before touching CUDA (its pointers are
never dereferenced), and the binding rejects mismatched tensors."""
import pytest
import torch

import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from tests.test_paged_abi import BAD_PAGES, BR, INVALID, MIS, OK, P, P2, P3, UNSUPPORTED, cache
from tests.test_paged_abi import pages as any_pages

E8 = torch.float8_e4m3fn
WS = 1 << 20


@pytest.fixture(scope="module")
def lib():
    mha_build.build()
    return mha.lib()


def pages(**kw):
    return any_pages(**{"dtype": mha.MHA_E4M3, **kw})


SC = mha.KvScales(P, P2)


def attend(lib, Q=P3, ts=0, pg=None, sc=SC, layer=0, offs=P, O=P2, T=5, H=4, max_new=5, scale=0.0,
           mask=BR, odt=mha.MHA_BF16, splits=0):
    return lib.sdpa_paged_e4m3(Q, ts, pages() if pg is None else pg, sc, layer, offs, O, T, H, max_new,
                               scale, mask, odt, splits, None)


def append(lib, Q=P, ts=0, gamma=P, pe=P, rows=9, r=64, Qo=P2, pg=None, sc=SC, layer=0, offs=P, T=5,
           H=4, eps=1e-6, pairing=0):
    return lib.qk_norm_rope_paged_e4m3(Q, ts, P, 0, P, 0, gamma, gamma, pe, rows, r, pairing, Qo,
                                       pages() if pg is None else pg, sc, layer, offs, T, H, eps, None)


def bounds(lib, pg=None, sc=SC, layer=0, offs=P, T=5, b=P, s=P):
    return lib.kv_pages_bounds(pages() if pg is None else pg, sc, layer, offs, T, b, s, None)


def select(lib, Q=P, ts=0, pg=None, layer=0, offs=P, b=P, s=P, T=5, H=4, n=3, sel=P, lens=P, ws=P,
           size=WS):
    return lib.kv_pages_select(Q, ts, pages() if pg is None else pg, layer, offs, b, s, T, H, n, sel,
                               lens, ws, size, None)


def selected(lib, Q=P3, ts=0, pg=None, sc=SC, layer=0, sel=P, lens=P, n=3, O=P2, T=5, H=4, scale=0.0,
             odt=mha.MHA_BF16, splits=0):
    return lib.sdpa_paged_selected(Q, ts, pages() if pg is None else pg, sc, layer, sel, lens, n, O, T,
                                   H, scale, odt, splits, None)


def fork(lib, pg=None, sc=SC, n=2):
    return lib.kv_pages_fork_e4m3(pages() if pg is None else pg, sc, P, P, P, n, None)


def compact(lib, src=None, sc=SC, dst=None, dsc=mha.KvScales(P3, P3 + 64)):
    dst = pages(K=P3, V=P3 + 4096, page_table=P2) if dst is None else dst
    return lib.kv_pages_compact_e4m3(pages() if src is None else src, sc, dst, dsc, P, P, 4096, None)


CALLS = [attend, append, bounds, select, selected, fork]


@pytest.mark.parametrize("kw,code", BAD_PAGES + [(dict(d=8), UNSUPPORTED)])
def test_every_entry_point_checks_the_pages(lib, kw, code):
    for call in CALLS:
        assert call(lib, pg=pages(**kw)) == code, call.__name__
    assert compact(lib, src=pages(**kw)) == code
    if "kv_lengths" not in kw:
        assert compact(lib, dst=pages(**{"K": P3, "V": P3 + 4096, "page_table": P2, **kw})) in (
            code, INVALID)


def test_scales_go_with_the_type(lib):
    bf, f32 = any_pages(), any_pages(dtype=mha.MHA_F32)
    bad = (None, mha.KvScales(None, P), mha.KvScales(P, None), mha.KvScales(P + 2, P),
           mha.KvScales(P, P2 + 1))
    for call in (attend, append, bounds, selected, fork):
        for sc in bad:
            assert call(lib, sc=sc) == INVALID, call.__name__
        for pg in (bf, f32):          # scales for pages that are not in 8 bits
            assert call(lib, pg=pg) == INVALID, call.__name__
    for call in (bounds, selected):
        assert call(lib, pg=f32, sc=None) == UNSUPPORTED
    for call in (bounds, select, selected):
        assert call(lib, pg=None if call is select else bf, T=0, **({} if call is select else dict(sc=None))) == OK
    assert select(lib, pg=f32) == UNSUPPORTED
    for sc in bad:
        assert compact(lib, sc=sc) == INVALID and compact(lib, dsc=sc) == INVALID
    assert compact(lib, src=bf) == INVALID and compact(lib, dsc=SC) == INVALID     # shared memory
    # the calls without scales know no 8 bits
    assert lib.sdpa_paged(P3, 0, pages(), 0, P, P2, 5, 4, 5, 0.0, BR, 1, 0, None) == INVALID
    assert lib.kv_pages_fork(pages(), P, P, P, 2, None) == INVALID
    assert lib.kv_pages_compact(pages(), pages(K=P3, V=P3 + 4096, page_table=P2), P, P, 4096,
                                None) == INVALID
    assert lib.qk_norm_rope_paged(P, 0, P, 0, P, 0, P, P, P, 9, 64, 0, P2, pages(), 0, P, 5, 4, 1e-6,
                                  None) == INVALID
    # nor is 8 bits an output
    assert attend(lib, odt=mha.MHA_E4M3) == INVALID and selected(lib, odt=mha.MHA_E4M3) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), INVALID), (dict(Q=MIS), INVALID), (dict(O=None), INVALID), (dict(O=P3), INVALID),
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=5), INVALID), (dict(layer=1), INVALID),
    (dict(layer=-1), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(odt=7), INVALID), (dict(splits=17), INVALID), (dict(splits=-1), INVALID),
    (dict(ts=255), INVALID), (dict(ts=260), INVALID), (dict(H=258), UNSUPPORTED),
    (dict(pg=pages(d=32)), UNSUPPORTED), (dict(pg=pages(d=256)), UNSUPPORTED), (dict(T=0), OK),
])
def test_attention_rejects_before_launch(lib, kw, code):
    assert attend(lib, **kw) == code
    assert selected(lib, **kw) == code


def test_attention_rejects_its_own(lib):
    for kw in (dict(offs=None), dict(offs=0x10002), dict(max_new=0), dict(mask=1), dict(mask=6)):
        assert attend(lib, **kw) == INVALID
    for kw in (dict(sel=None), dict(lens=None), dict(sel=P + 1), dict(lens=P + 2), dict(n=0), dict(n=-1)):
        assert selected(lib, **kw) == INVALID
    assert selected(lib, n=(1 << 26) + 1) == UNSUPPORTED
    # its pages' tables are not used
    assert selected(lib, pg=pages(B=0, page_table=None, kv_lengths=None), T=0) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(Q=MIS), INVALID), (dict(ts=255), INVALID), (dict(gamma=MIS), INVALID), (dict(pe=None), INVALID),
    (dict(rows=0), INVALID), (dict(r=66), INVALID), (dict(r=8), UNSUPPORTED), (dict(Qo=P), INVALID),
    (dict(layer=1), INVALID), (dict(offs=None), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID),
    (dict(eps=0.0), INVALID), (dict(pairing=2), INVALID), (dict(pg=pages(d=32), r=32), UNSUPPORTED),
    (dict(T=0), OK), (dict(pg=pages(B=0, page_table=None, kv_lengths=None)), OK),
])
def test_append_rejects_before_launch(lib, kw, code):
    assert append(lib, **kw) == code


@pytest.mark.parametrize("call,kw,code", [
    (bounds, dict(T=-1), INVALID), (bounds, dict(layer=1), INVALID), (bounds, dict(offs=None), INVALID),
    (bounds, dict(offs=P + 2), INVALID), (bounds, dict(b=None), INVALID), (bounds, dict(b=MIS), INVALID),
    (bounds, dict(s=None), INVALID), (bounds, dict(s=P + 2), INVALID),
    (bounds, dict(pg=pages(d=32)), UNSUPPORTED), (bounds, dict(T=0), OK),
    (select, dict(Q=None), INVALID), (select, dict(Q=P + 1), INVALID), (select, dict(ts=255), INVALID),
    (select, dict(layer=-1), INVALID), (select, dict(offs=None), INVALID), (select, dict(b=MIS), INVALID),
    (select, dict(s=None), INVALID), (select, dict(T=-1), INVALID), (select, dict(H=5), INVALID),
    (select, dict(H=0), INVALID), (select, dict(n=0), INVALID), (select, dict(n=65537), UNSUPPORTED),
    (select, dict(sel=None), INVALID), (select, dict(lens=P + 2), INVALID), (select, dict(ws=None), INVALID),
    (select, dict(ws=MIS), INVALID), (select, dict(size=5 * 2 * 4 * 4 - 1), INVALID),
    (select, dict(H=258), UNSUPPORTED), (select, dict(pg=pages(d=32)), UNSUPPORTED),
    (select, dict(T=0), OK),
])
def test_bounds_and_select_reject_before_launch(lib, call, kw, code):
    assert call(lib, **kw) == code


def test_workspace_sizes(lib):
    assert lib.kv_pages_select_workspace_bytes(5, 2, 4) == 160
    assert lib.kv_pages_select_workspace_bytes(1 << 16, 128, 1 << 20) == 1 << 45
    for bad in ((-1, 2, 4), (5, 0, 4), (5, 2, 0)):
        assert lib.kv_pages_select_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------- binding

def refused(what):
    return pytest.raises(ValueError, match=what)


def test_binding_checks_scales():
    K, V, table, lens = cache(dtype=torch.uint8)
    K, V = K.view(E8), V.view(E8)
    bf = torch.bfloat16
    Q, offs = torch.zeros((3, 4, 64), dtype=bf), torch.arange(4, dtype=torch.int32)
    kv, g, pe = torch.zeros((3, 2, 64), dtype=bf), torch.ones(64, dtype=bf), torch.zeros((5, 64))
    sc = torch.ones((6, 2))
    one, sel = torch.ones(3, dtype=torch.int32), torch.zeros((3, 2, 2), dtype=torch.int32)
    b, bs = torch.zeros((6, 2, 2, 64), dtype=torch.int8), torch.zeros((6, 2))
    two = lens[:2]
    calls = [
        lambda K=K, V=V, **kw: mha.sdpa_paged(Q, K, V, table, lens, offs, **kw),
        lambda K=K, V=V, **kw: mha.qk_norm_rope_paged(Q, kv, kv, g, g, pe, K, V, table, lens, offs, **kw),
        lambda K=K, V=V, **kw: mha.kv_pages_fork(K, V, table, lens, two, two, two, **kw),
        lambda K=K, V=V, **kw: mha.kv_pages_bounds(K, V, table, lens, offs, b, bs, 3, **kw),
        lambda K=K, V=V, **kw: mha.sdpa_paged_selected(Q, K, V, sel, one, **kw),
    ]
    for call in calls:
        for kw in ({}, dict(K_scale=sc), dict(V_scale=sc)):
            with refused("need K_scale and V_scale"):
                call(**kw)
        for bad in (sc.double(), sc[:5], sc[None], sc.T.contiguous().T, sc[:1].expand(6, 2)):
            with refused("scale must be a contiguous"):
                call(K_scale=bad, V_scale=sc)
            with refused("scale must be a contiguous"):
                call(K_scale=sc, V_scale=bad)
        wide = K.view(torch.uint8).to(bf)
        with refused("for pages in 8 bits"):
            call(K=wide, V=wide.clone(), K_scale=sc, V_scale=sc)
        with refused("CUDA"):
            call(K_scale=sc, V_scale=sc)
        with pytest.raises(ValueError):
            call(V=V.view(torch.uint8), K_scale=sc, V_scale=sc)
    with pytest.raises(ValueError):
        mha.sdpa_paged(Q.float(), K, V, table, lens, offs, K_scale=sc, V_scale=sc)
    two_layers = K[None].expand(2, *K.shape).clone()
    with refused("scale must be a contiguous"):
        mha.sdpa_paged(Q, two_layers, two_layers.clone(), table, lens, offs, K_scale=sc, V_scale=sc)
    with refused("need K_scale"):
        mha.kv_pages_compact(K, V, table, lens, K.clone(), V.clone(), table.clone(), K_scale=sc, V_scale=sc)
    with refused("need K_scale"):
        mha.kv_pages_compact(K, V, table, lens, K.clone(), V.clone(), table.clone(), K_scale_out=sc,
                             V_scale_out=sc)


def test_binding_checks_bounds_and_selections():
    K, V, table, lens = cache()
    bf = torch.bfloat16
    Q, offs = torch.zeros((3, 4, 64), dtype=bf), torch.arange(4, dtype=torch.int32)
    b, bs = torch.zeros((6, 2, 2, 64), dtype=torch.int8), torch.zeros((6, 2))
    bnd = lambda offs=offs, b=b, bs=bs, T=3, **kw: mha.kv_pages_bounds(K, V, table, lens, offs, b, bs, T, **kw)
    sel = lambda Q=Q, offs=offs, b=b, bs=bs, n=2, **kw: mha.kv_pages_select(
        Q, K, V, table, lens, offs, b, bs, n, **kw)
    for call in (bnd, sel):
        for kw in (dict(offs=offs[:3]), dict(b=b.int()), dict(b=b[:, :, :1]), dict(b=b[:5]),
                   dict(b=b.transpose(2, 3).contiguous().transpose(2, 3)), dict(bs=bs.double()),
                   dict(bs=bs[:5]), dict(bs=bs.T.contiguous().T), dict(layer=2 ** 32)):
            with pytest.raises(ValueError):
                call(**kw)
        with refused("CUDA"):
            call()
    for kw in (dict(Q=Q.float()), dict(Q=Q[..., :32]), dict(n=0), dict(n=2 ** 32), dict(Q=Q[:1].expand_as(Q)),
               dict(workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 20))):
        with pytest.raises(ValueError):
            sel(**kw)
    with refused("T out of range"):
        bnd(T=2 ** 31)
    s, n = torch.zeros((3, 2, 2), dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    att = lambda Q=Q, s=s, n=n, **kw: mha.sdpa_paged_selected(Q, K, V, s, n, **kw)
    for kw in (dict(Q=Q.float()), dict(s=s[:2]), dict(s=s.long()), dict(s=s[:, :1]), dict(s=s[..., ::2]),
               dict(s=s[0]), dict(n=n[:2]), dict(n=n.long()), dict(layer=2 ** 31), dict(num_splits=2 ** 32),
               dict(Q=Q[:1].expand_as(Q))):
        with pytest.raises(ValueError):
            att(**kw)
    with refused("CUDA"):
        att()
