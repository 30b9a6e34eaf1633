"""Refusals of the paged cache's entry points, without a GPU: the C ABI
rejects bad arguments before touching CUDA (its pointers are never
dereferenced), and the binding rejects mismatched tensors."""
import ctypes

import pytest
import torch

import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build

OK, INVALID, UNSUPPORTED = mha.MHA_OK, mha.MHA_ERR_INVALID_ARG, mha.MHA_ERR_UNSUPPORTED
P, P2, P3, MIS = 0x10000, 0x20000, 0x30000, 0x10008   # never dereferenced
BR = mha.MASK_CAUSAL_BOTTOM_RIGHT


@pytest.fixture(scope="module")
def lib():
    mha_build.build()
    return mha.lib()


def pages(**kw):
    v = dict(K=P, V=P2, dtype=mha.MHA_BF16, num_pages=10, page_size=16, kv_heads=2, d=64, layers=1,
             page_stride=0, layer_stride=0, page_table=P, kv_lengths=P, B=3, table_cols=4)
    v.update(kw)
    return mha.KvPages(*[v[n] for n, _ in mha.KvPages._fields_])


BAD_PAGES = [
    (dict(K=None), INVALID), (dict(V=MIS), INVALID), (dict(page_table=None), INVALID),
    (dict(kv_lengths=0x10002), INVALID), (dict(page_table=0x10001), INVALID),
    (dict(dtype=5), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED), (dict(kv_heads=0), INVALID), (dict(d=0), INVALID),
    (dict(layers=0), INVALID), (dict(B=-1), INVALID), (dict(table_cols=0), INVALID),
    (dict(table_cols=1 << 27), UNSUPPORTED), (dict(page_stride=2047), INVALID),
    (dict(page_stride=2052), INVALID), (dict(layer_stride=-8), INVALID), (dict(d=4), UNSUPPORTED),
    (dict(layer_stride=64), INVALID),
]


def paged(lib, Q=P3, ts=0, pg=None, layer=0, offs=P, O=P2, T=5, H=4, max_new=5, scale=0.0, mask=BR,
          odt=mha.MHA_BF16, splits=0):
    return lib.sdpa_paged(Q, ts, pages() if pg is None else pg, layer, offs, O, T, H, max_new,
                          scale, mask, odt, splits, None)


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_every_entry_point_checks_the_pages(lib, kw, code):
    pg = pages(**kw)
    assert paged(lib, pg=pg) == code
    assert lib.kv_pages_fork(pg, P, P, P, 2, None) == code
    assert lib.kv_pages_compact(pg, pages(K=P3, V=P3 + 16), P, P, 4096, None) == code
    if "kv_lengths" not in kw:
        assert lib.kv_pages_compact(pages(), pages(**{"K": P3, "V": P3 + 4096, "page_table": P2,
                                                      **kw}), P, P, 4096, None) in (code, INVALID)
    assert lib.qk_norm_rope_paged(P, 0, P, 0, P, 0, P, P, P, 9, 64, 0, P2, pg, 0, P, 5, 4, 1e-6,
                                  None) == code


def test_null_pages(lib):
    assert lib.sdpa_paged(P, 0, None, 0, P, P2, 5, 4, 5, 0.0, BR, 1, 0, None) == INVALID
    assert lib.kv_pages_fork(None, P, P, P, 2, None) == INVALID
    assert lib.kv_pages_compact(pages(), None, P, P, 4096, None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), INVALID), (dict(Q=MIS), INVALID), (dict(O=None), INVALID), (dict(O=P3), INVALID),
    (dict(offs=None), INVALID), (dict(offs=0x10002), INVALID), (dict(T=-1), INVALID),
    (dict(H=0), INVALID), (dict(H=5), INVALID), (dict(max_new=0), INVALID), (dict(layer=1), INVALID),
    (dict(layer=-1), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(mask=1), INVALID), (dict(mask=2), INVALID),
    (dict(mask=6), INVALID), (dict(odt=7), INVALID), (dict(splits=17), INVALID),
    (dict(splits=-1), INVALID), (dict(ts=255), INVALID), (dict(ts=260), INVALID),
    (dict(H=258), UNSUPPORTED),
])
def test_sdpa_paged_rejects_before_launch(lib, kw, code):
    assert paged(lib, **kw) == code


@pytest.mark.parametrize("kw", [dict(d=32), dict(d=256), dict(dtype=mha.MHA_F32)])
def test_sdpa_paged_unsupported_caches(lib, kw):
    assert paged(lib, pg=pages(**kw), H=2) == UNSUPPORTED


def test_empty_calls_are_no_ops(lib):
    assert paged(lib, T=0, Q=None, O=None) == OK
    assert paged(lib, T=0, Q=None, O=None, max_new=0) == OK
    assert paged(lib, pg=pages(B=0), offs=None) == OK
    assert lib.kv_pages_fork(pages(), None, None, None, 0, None) == OK
    assert rope(lib, B=0, Q=None, K=None) == OK
    assert rope(lib, L=0) == OK
    assert rope(lib, H=0, Hkv=0) == OK


def rope(lib, Q=P, qts=0, K=P, kts=0, gq=P, gk=P, pe=P, rows=9, r=64, pairing=0, Qo=P2, Ko=P3, B=2,
         L=4, H=2, Hkv=1, d=64, off=0, pos=None, eps=1e-6, dt=mha.MHA_BF16):
    return lib.qk_norm_rope_forward(Q, qts, K, kts, gq, gk, pe, rows, r, pairing, Qo, Ko, B, L, H,
                                    Hkv, d, off, pos, eps, dt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), INVALID), (dict(K=MIS), INVALID), (dict(gq=None), INVALID),
    (dict(gk=0x10004), INVALID), (dict(pe=None), INVALID), (dict(pe=0x10008), INVALID),
    (dict(Qo=None), INVALID), (dict(Qo=P), INVALID), (dict(Ko=MIS), INVALID), (dict(B=-1), INVALID),
    (dict(L=10), INVALID), (dict(off=6), INVALID), (dict(off=-1), INVALID), (dict(r=0), INVALID),
    (dict(r=63), INVALID), (dict(r=66), INVALID), (dict(d=0), INVALID), (dict(d=300, r=64), UNSUPPORTED),
    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(pairing=2), INVALID), (dict(dt=3), INVALID), (dict(qts=127), INVALID),
    (dict(qts=132), INVALID), (dict(pos=0x10002), INVALID), (dict(rows=0), INVALID),
])
def test_qk_norm_rope_rejects_before_launch(lib, kw, code):
    assert rope(lib, **kw) == code


def rope_bwd(lib, Q=P, dQo=P2, dQ=P3, dts=0, dgq=P, H=2, Hkv=1, d=64, B=2, ws=P, nbytes=None,
             gdt=mha.MHA_F32):
    need = lib.qk_norm_rope_backward_workspace_bytes(d)
    return lib.qk_norm_rope_backward(Q, 0, P, 0, P, P, P, 9, 64, 0, dQo, P2, dQ, dts, P3, 0, dgq, P,
                                     B, 4, H, Hkv, d, 0, None, 1e-6, mha.MHA_BF16, gdt,
                                     mha.MHA_BF16, ws, need if nbytes is None else nbytes, None)


@pytest.mark.parametrize("kw", [
    dict(Q=None), dict(dQo=None), dict(dQ=None), dict(dQ=P), dict(dQ=P2), dict(dts=100),
    dict(dgq=None), dict(dgq=0x10004), dict(ws=None), dict(ws=MIS), dict(nbytes=64), dict(gdt=9),
    dict(B=0, dgq=None),
])
def test_qk_norm_rope_backward_rejects_before_launch(lib, kw):
    assert rope_bwd(lib, **kw) == INVALID


def test_workspace_queries(lib):
    assert lib.qk_norm_rope_backward_workspace_bytes(64) > 0
    assert lib.qk_norm_rope_backward_workspace_bytes(0) == 0
    assert lib.qk_norm_rope_backward_workspace_bytes(257) == 0
    assert lib.kv_pages_compact_workspace_bytes(33) >= 16
    assert lib.kv_pages_compact_workspace_bytes(0) == 0
    assert lib.kv_pages_compact_workspace_bytes((1 << 20) + 1) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), INVALID), (dict(K=MIS), INVALID), (dict(V=None), INVALID), (dict(r=24), UNSUPPORTED),
    (dict(Qo=P), INVALID), (dict(offs=None), INVALID), (dict(layer=1), INVALID), (dict(H=0), INVALID),
    (dict(T=-1), INVALID), (dict(vts=120), INVALID), (dict(vts=132), INVALID), (dict(gk=None), INVALID),
])
def test_qk_norm_rope_paged_rejects_before_launch(lib, kw, code):
    v = dict(Q=P, K=P, V=P, vts=0, gk=P, r=64, Qo=P2, layer=0, offs=P, T=5, H=4)
    v.update(kw)
    assert lib.qk_norm_rope_paged(v["Q"], 0, v["K"], 0, v["V"], v["vts"], P, v["gk"], P, 9, v["r"],
                                  0, v["Qo"], pages(), v["layer"], v["offs"], v["T"], v["H"], 1e-6,
                                  None) == code


def test_fork_and_compact_reject(lib):
    assert lib.kv_pages_fork(pages(), P, P, P, -1, None) == INVALID
    assert lib.kv_pages_fork(pages(), P, P, P, 4, None) == INVALID      # more pairs than sequences
    assert lib.kv_pages_fork(pages(), None, P, P, 2, None) == INVALID
    assert lib.kv_pages_fork(pages(), P, P, 0x10002, 2, None) == INVALID
    need = lib.kv_pages_compact_workspace_bytes(10)
    to = dict(K=P3, V=0x40000, page_table=P2)
    call = lambda src=None, dst=None, n=P, ws=P, nb=need: lib.kv_pages_compact(
        src or pages(), dst or pages(**to), n, ws, nb, None)
    for dst in (dict(d=128), dict(page_size=32), dict(kv_heads=1), dict(layers=2), dict(B=2),
                dict(table_cols=3), dict(dtype=mha.MHA_F32), dict(K=P), dict(V=P2), dict(V=P),
                dict(page_table=P)):
        assert call(dst=pages(**{**to, **dst})) == INVALID
    assert call(n=None) == INVALID and call(ws=None) == INVALID and call(nb=need - 1) == INVALID
    assert call(src=pages(num_pages=(1 << 20) + 1)) == UNSUPPORTED


# ------------------------------------------------------------------- binding

def cache(P=6, Hkv=2, ps=16, d=64, B=3, cols=4, dtype=torch.bfloat16):
    K = torch.zeros((P, Hkv, ps, d), dtype=dtype)
    return K, K.clone(), torch.zeros((B, cols), dtype=torch.int32), torch.ones(B, dtype=torch.int32)


def test_binding_checks_shapes_before_devices():
    K, V, table, lens = cache()
    Q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    offs = torch.arange(4, dtype=torch.int32)
    call = lambda Q=Q, K=K, V=V, t=table, n=lens, o=offs, **kw: mha.sdpa_paged(Q, K, V, t, n, o, **kw)
    for kw in (dict(Q=Q.float()), dict(Q=Q[..., :32]), dict(V=V[:, :1]), dict(V=V.float()),
               dict(K=K.transpose(1, 2)), dict(t=table.long()), dict(t=table[:, ::2]),
               dict(n=lens[:2]), dict(n=lens.long()), dict(o=offs[:3]), dict(o=offs.long()),
               dict(Q=Q.transpose(0, 1).contiguous().transpose(0, 1)), dict(t=table[0])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError, match="CUDA"):
        call()


def test_binding_checks_rows():
    x = torch.zeros((2, 5, 4, 64))
    g, pe = torch.ones(64), torch.zeros((5, 64))
    call = lambda Q=x, K=x, g=g, pe=pe, **kw: mha.qk_norm_rope(Q, K, g, g, pe, **kw)
    for kw in (dict(Q=x[..., ::2]), dict(Q=x[:, ::2]), dict(K=x.bfloat16()), dict(g=g[:32]),
               dict(g=g.bfloat16()), dict(pe=pe.double()), dict(pe=pe[:, :32]),
               dict(Q=x.transpose(1, 2)), dict(K=x.transpose(2, 3)),
               dict(positions=torch.zeros((2, 4), dtype=torch.int32)),
               dict(positions=torch.zeros((2, 5)))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(ValueError):
        mha.qk_norm_rope_backward(x, x, g, g, pe, x, x)       # [B, H, L, d] wanted
    K, V, table, lens = cache()
    with pytest.raises(ValueError):
        mha.kv_pages_fork(K, V, table, lens, lens[:2], lens[:2], lens[:1])
    with pytest.raises(ValueError, match="CUDA"):
        mha.kv_pages_compact(K, V, table, lens, K.clone(), V.clone(), table.clone())


def test_binding_refuses_broadcast_rows_and_pools():
    """expand() gives a stride of 0, which the C ABI reads as "dense": rows
    past the end of the storage.  Refused before any device is looked at."""
    K, V, table, lens = cache()
    bf = torch.bfloat16
    offs, g, pe = torch.arange(4, dtype=torch.int32), torch.ones(64, dtype=bf), torch.zeros((5, 64))
    q, kv = torch.zeros((3, 4, 64), dtype=bf), torch.zeros((3, 2, 64), dtype=bf)
    flat = lambda x: x[:1].expand_as(x)
    refused = lambda what: pytest.raises(ValueError, match=what)
    with refused("Q.*evenly spaced"):
        mha.sdpa_paged(flat(q), K, V, table, lens, offs)
    append = lambda q=q, k=kv, v=kv, K=K, V=V: mha.qk_norm_rope_paged(
        q, k, v, g, g, pe, K, V, table, lens, offs)
    for name, kw in (("Q", dict(q=flat(q))), ("K", dict(k=flat(kv))), ("V", dict(v=flat(kv)))):
        with refused(f"{name}.*evenly spaced"):
            append(**kw)
    # pools that are one page, or one layer, many times
    layered = lambda x: x[None].expand(3, *x.shape)
    two = lens[:2]
    for pool in (flat, layered):
        with refused("pages and layers"):
            mha.sdpa_paged(q, pool(K), pool(V), table, lens, offs)
        with refused("pages and layers"):
            append(K=pool(K), V=pool(V))
        with refused("pages and layers"):
            mha.kv_pages_fork(pool(K), pool(V), table, lens, two, two, two)
        with refused("pages and layers"):
            mha.kv_pages_compact(pool(K), pool(V), table, lens, K, V, table)
        with refused("pages and layers"):
            mha.kv_pages_compact(K, V, table, lens, pool(K), pool(V), table)
    # training rows: over the tokens of one item, over items of one token, over both
    for B, L in ((1, 5), (5, 1), (2, 5)):
        x = torch.zeros((1, 1, 4, 64)).expand(B, L, 4, 64)
        dense, dy, g = torch.zeros((B, L, 4, 64)), torch.zeros((B, 4, L, 64)), torch.ones(64)
        for pair in ((x, dense), (dense, x)):
            with refused("evenly spaced"):
                mha.qk_norm_rope(*pair, g, g, pe)
            with refused("evenly spaced"):
                mha.qk_norm_rope_backward(*pair, g, g, pe, dy, dy)


def test_binding_refuses_broadcast_gradient_outputs(monkeypatch):
    """The same for the given dQ and dK, which are looked at after the devices."""
    monkeypatch.setattr(mha._binding, "_launch_on", lambda *a: 0)
    x, dy, g = torch.zeros((1, 5, 4, 64)), torch.zeros((1, 4, 5, 64)), torch.ones(64)
    for out in ((x[:, :1].expand_as(x), x.clone()), (x.clone(), x[:, :1].expand_as(x))):
        with pytest.raises(ValueError, match="evenly spaced"):
            mha.qk_norm_rope_backward(x, x, g, g, torch.zeros((5, 64)), dy, dy, out=out)


def test_binding_refuses_scattered_workspaces():
    """A workspace's size is counted from its elements, so they must lie one
    after the other: one byte expanded to a million would pass for a megabyte."""
    x, dy, g = torch.zeros((1, 5, 4, 64)), torch.zeros((1, 4, 5, 64)), torch.ones(64)
    K, V, table, lens = cache()
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 22),
               torch.zeros(1 << 23, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            mha.qk_norm_rope_backward(x, x, g, g, torch.zeros((5, 64)), dy, dy, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            mha.kv_pages_compact(K, V, table, lens, K.clone(), V.clone(), table.clone(),
                                 workspace=ws)


def test_no_sequences_need_no_table(lib):
    """B = 0 as a binding passes it: an empty tensor's pointer is null."""
    none = dict(B=0, page_table=None, kv_lengths=None)
    assert paged(lib, pg=pages(**none), offs=None) == OK
    assert lib.kv_pages_fork(pages(**none), None, None, None, 0, None) == OK
    assert lib.qk_norm_rope_paged(P, 0, P, 0, P, 0, P, P, P, 9, 64, 0, P2, pages(**none), 0, P, 5, 4,
                                  1e-6, None) == OK
    # with sequences both are needed, the destination's table too
    assert paged(lib, pg=pages(kv_lengths=None)) == INVALID
    need = lib.kv_pages_compact_workspace_bytes(10)
    to = dict(K=P3, V=0x40000, page_table=None)
    assert lib.kv_pages_compact(pages(), pages(**to), P, P, need, None) == INVALID
    # and what else is checked still is
    assert paged(lib, pg=pages(**none, d=0)) == INVALID
    assert paged(lib, pg=pages(**none), max_new=-1) == INVALID
    assert lib.kv_pages_compact(pages(**none), pages(**{**none, **to}), None, P, need, None) == INVALID


def test_strides_of_size_one_do_not_count():
    """Pages of one head, rows first; one page; one layer: contiguous pages
    whatever torch says of the stride of a size of 1."""
    K, V, table, lens = cache(Hkv=1)
    Q, offs = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.arange(4, dtype=torch.int32)
    rows_first = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)
    one_page = lambda x: x[:1].as_strided((1, 1, 16, 64), (7, 5, 64, 1))
    one_layer = lambda x: x.as_strided((1, *x.shape), (3, *x.stride()))
    for a, b in ((rows_first(K), V), (K, rows_first(V)), (one_page(K), V[:1]),
                 (one_layer(K), V[None]), (one_page(K), one_page(V))):
        with pytest.raises(ValueError, match="CUDA"):
            mha.sdpa_paged(Q, a, b, table, lens, offs)
    got = mha._binding._kv_pages(one_page(K), V[:1], table, lens)
    assert (got.num_pages, got.layers, got.page_stride, got.layer_stride) == (1, 1, 0, 0)
    got = mha._binding._kv_pages(one_layer(rows_first(K)), V[None], table, lens)
    assert (got.num_pages, got.layers, got.page_stride, got.layer_stride) == (6, 1, 16 * 64, 0)
    # two heads' rows must follow each other, and K and V be alike, as before
    K, V, table, lens = cache(Hkv=2)
    for a, b in ((rows_first(K), rows_first(V)), (torch.cat((K, K))[::2], V)):
        with pytest.raises(ValueError, match="laid out alike"):
            mha.sdpa_paged(Q, a, b, table, lens, offs)


@pytest.mark.parametrize("wide", [2 ** 31, 2 ** 32, 2 ** 32 + 1, -2 ** 31 - 1])
def test_binding_refuses_integers_wider_than_c(wide):
    """ctypes would pass their low 32 bits: layer 2^32 would be layer 0."""
    K, V, table, lens = cache()
    bf = torch.bfloat16
    Q, offs = torch.zeros((3, 4, 64), dtype=bf), torch.arange(4, dtype=torch.int32)
    kv, g, pe = torch.zeros((3, 2, 64), dtype=bf), torch.ones(64, dtype=bf), torch.zeros((5, 64))
    x, dy = torch.zeros((1, 5, 4, 64), dtype=bf), torch.zeros((1, 4, 5, 64), dtype=bf)
    paged_call = lambda **kw: mha.sdpa_paged(Q, K, V, table, lens, offs, **kw)
    append = lambda **kw: mha.qk_norm_rope_paged(Q, kv, kv, g, g, pe, K, V, table, lens, offs, **kw)
    norm = lambda **kw: mha.qk_norm_rope(x, x, g, g, pe, **kw)
    grad = lambda **kw: mha.qk_norm_rope_backward(x, x, g, g, pe, dy, dy, **kw)
    for call, names in ((paged_call, ("layer", "num_splits")), (append, ("layer", "pairing")),
                        (norm, ("pos_offset", "pairing")), (grad, ("pos_offset", "pairing"))):
        for name in names:
            with pytest.raises(ValueError, match=f"{name} out of range"):
                call(**{name: wide})
    # a bound on new tokens may be as large as it likes, not as small
    with pytest.raises(ValueError, match="CUDA" if wide > 0 else "max_new out of range"):
        paged_call(max_new=wide)
