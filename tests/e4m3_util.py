"""8-bit caches for the tests: shuffled pages of codes with their scales."""
from __future__ import annotations

import numpy as np
import torch

import oracle.paged_e4m3 as ref
from tests.paged_util import make_pages

E8 = torch.float8_e4m3fn


def make_pages8(rng, lens, new, Hkv, ps, d, pow2=True, **kw):
    """(K codes, K scales, V codes, V scales, table, offsets, free pages) of
    normal rows whose size differs by up to eight from page to page and head to
    head."""
    K, V, table, offs, free = make_pages(rng, lens, new, Hkv, ps, d, **kw)
    lead = K.shape[:-2]
    K, V = (x * 2.0 ** rng.uniform(-2, 1, (*lead, 1, 1)) for x in (K, V))
    if K.ndim == 4:
        (kc, ks), (vc, vs) = (ref.quantise(x, pow2) for x in (K, V))
    else:
        (kc, ks), (vc, vs) = ((np.stack(z) for z in zip(*(ref.quantise(y, pow2) for y in x)))
                              for x in (K, V))
    return kc, ks, vc, vs, table, offs, free


def dev8(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).cuda().view(E8)


def f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def attention_bound(O, A, Q, K, v_scale_max, keys, scale, bf16_out):
    """How far an attention over pages in 8 bits may be off, from the arithmetic.

    Weights: two e4m3 parts are off by (2^-4)^2 = 2^-8 of a weight (fp16, with
    more rows, by 2^-11); fp32 scores, exponentials and sums by 2^-10, as for the
    bf16 cache.  The parts' smallest half steps: 2^-10 / 2^5 against a largest
    weight of 2^8, so 2^-23 of the largest weight times scale for each key (fp16:
    2^-25 against 2^6 or more), times its code (at most 448); the weights' sum is
    at least 1 in the same units.
    Scores: two parts of q are off by 2^-18 of the row's largest element, so a
    score by 2^-18 max|q| max_j sum_c |k_jc| scale, and a weight by twice that."""
    q_max = np.abs(Q).max(-1)[..., None]
    k_sum = np.abs(K).sum(-1).max()
    b = (2.0 ** -8 + 2.0 ** -10 + 2 * 2.0 ** -18 * q_max * k_sum * scale) * A
    b = b + keys * 2.0 ** -23 * v_scale_max * 448 + 1e-30
    return b + 2.0 ** -8 * np.abs(O) if bf16_out else b
