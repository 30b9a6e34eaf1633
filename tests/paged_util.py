"""Paged caches for the tests: shuffled pages, spare pages, tables whose
entries behind a sequence's last page are -1."""
from __future__ import annotations

import numpy as np
import torch


def make_pages(rng, lens, new, Hkv, ps, d, spare=3, bf16=False, cols=None, layers=None):
    """K, V [P, Hkv, ps, d] (or [layers, ...]) float arrays of normal values
    (rounded to bf16 when asked), the page table, the packed queries' offsets
    and the free pages."""
    from transformer_head_scaled_03_gb300.inputs import round_to_bf16
    held = [-(-n // ps) for n in lens]
    P = sum(held) + spare
    perm = rng.permutation(P).astype(np.int32)
    cols = cols or max(1, max(held, default=1))
    table = np.full((len(lens), cols), -1, np.int32)
    at = 0
    for b, m in enumerate(held):
        table[b, :m] = perm[at:at + m]
        at += m
    shape = (P, Hkv, ps, d) if layers is None else (layers, P, Hkv, ps, d)
    K, V = rng.standard_normal((2, *shape), dtype=np.float32 if bf16 else np.float64)
    if bf16:
        K, V = round_to_bf16(K), round_to_bf16(V)
    offs = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    return K, V, table, offs, perm[at:]


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(a):
    return dev(np.asarray(a, np.int32))
