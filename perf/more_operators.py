"""The operators of the 8-bit paged cache and of its sparse reading, as they are measured: attention over
pages of e4m3 codes with a scale per page and key/value head, the norm and rotation that appends to such
pages, and, for long caches, the bounds of a page's keys, the selection of pages by a score from those
bounds, and the attention over the selected pages.

``run`` holds each operator twice: in elementary torch operations (fp32), and as the library's calls.
``exact`` is the same definition in fp64, sequence by sequence.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
E4M3 = torch.float8_e4m3fn


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _hostgen(seed):
    g = torch.Generator()
    g.manual_seed(int(seed) + 7919)
    return g


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _pe_table(n_pos, r):
    """(sin, cos) pairs of pos / 10000^(2i/r), fp64 angles rounded to fp32."""
    pos = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None]
    inv = torch.pow(10000.0, -torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
    a = pos * inv
    return torch.stack((a.sin(), a.cos()), dim=-1).reshape(n_pos, r).float().contiguous()


# --------------------------------------------------------------------------------- cases

def _attn(name, B, H, Hkv, d, ps, lens, new):
    return dict(name=name, op="attn8", B=B, H=H, Hkv=Hkv, d=d, ps=ps, len_lo=lens[0], len_hi=lens[1],
                new_lo=new[0], new_hi=new[1])


def _append(name, B, H, Hkv, d, r, half, ps, lens, new):
    return dict(name=name, op="append8", B=B, H=H, Hkv=Hkv, d=d, r=r, half=half, ps=ps,
                len_lo=lens[0], len_hi=lens[1], new_lo=new[0], new_hi=new[1])


def _bounds(name, dtype, B, Hkv, d, ps, lens, new):
    return dict(name=name, op="bounds", dtype=dtype, B=B, Hkv=Hkv, d=d, ps=ps, len_lo=lens[0],
                len_hi=lens[1], new_lo=new[0], new_hi=new[1])


def _select(name, B, H, Hkv, d, ps, lens, new, n):
    return dict(name=name, op="select", B=B, H=H, Hkv=Hkv, d=d, ps=ps, len_lo=lens[0], len_hi=lens[1],
                new_lo=new[0], new_hi=new[1], n=n)


def _selected(name, dtype, B, H, Hkv, d, ps, lens, n):
    return dict(name=name, op="selected", dtype=dtype, B=B, H=H, Hkv=Hkv, d=d, ps=ps, len_lo=lens[0],
                len_hi=lens[1], new_lo=1, new_hi=1, n=n)


def listed():
    return [
        # one conversation, one new token, the base model's heads: latency of a step
        _attn("attn8_decode_one", 1, 8, 8, 64, 16, (700, 700), (1, 1)),
        # a server's batch of long conversations, one new token each, four query heads to a key head
        _attn("attn8_decode_batch", 16, 32, 8, 128, 64, (16384, 32768), (1, 1)),
        # chunks of prompts and single tokens in one batch, over caches of ragged length
        _attn("attn8_chunk_mixed", 6, 40, 8, 128, 32, (900, 8000), (1, 500)),
        # a long prompt taken in chunks of thousands of tokens: bound by the tensor cores
        _attn("attn8_prefill", 2, 32, 8, 128, 128, (8192, 8192), (4096, 4096)),
        # a decoding step of a few conversations: latency
        _append("append8_decode", 4, 32, 8, 128, 128, True, 16, (100, 4000), (1, 1)),
        # prompts of ragged length written to the pages
        _append("append8_prompt", 8, 32, 8, 128, 64, True, 64, (2000, 8192), (500, 2000)),
        # after a decoding step of a batch: a few of its pages have become full
        _bounds("bounds_step", "bf16", 48, 8, 128, 16, (500, 8000), (1, 1)),
        # after prompts were appended to an 8-bit cache
        _bounds("bounds_prompt", "e4m3", 16, 8, 128, 32, (2000, 8192), (1000, 8000)),
        # one long conversation: pages of a decoding step's query
        _select("select_one", 1, 32, 8, 128, 16, (32768, 32768), (1, 1), 64),
        # a batch of long conversations
        _select("select_batch", 16, 32, 8, 128, 32, (65536, 131072), (1, 1), 128),
        # the base model's heads over the selected pages of one conversation
        _selected("selected_one", "bf16", 1, 8, 8, 64, 16, (16384, 16384), 32),
        # a batch over its selected pages of an 8-bit cache
        _selected("selected_batch", "e4m3", 32, 32, 8, 128, 32, (16384, 32768), 128),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append", "bounds", "select", "select", "selected",
                     "selected"])
    d = rng.choice([64, 128])
    ps = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "e4m3"])
    while True:
        H = Hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        if op == "attn":
            B = _logint(rng, 1, 24)
            hi = _logint(rng, 8, 32768)
            lo = rng.randint(max(1, hi // 3), hi)
            kind = rng.choice(["one", "few", "chunk"])
            new = ((1, 1) if kind == "one" else (1, min(lo, rng.randint(2, 16))) if kind == "few"
                   else (1, min(lo, _logint(rng, 17, 4096))))
            c = _attn("", B, H, Hkv, d, ps, (lo, hi), new)
            if B * H * new[1] * hi * 4 > 4e9 or B * Hkv * hi * d > 4e8:
                continue
        elif op == "append":
            hi = _logint(rng, 2, 8192)
            lo = rng.randint(max(1, hi // 3), hi)
            new = (1, 1) if rng.random() < 0.4 else (1, min(lo, _logint(rng, 2, 2000)))
            c = _append("", _logint(rng, 1, 16), H, Hkv, d, rng.choice([d, d, d // 2]), rng.random() < 0.5,
                        ps, (lo, hi), new)
            if c["B"] * new[1] * (c["H"] + 2 * Hkv) * d > 6e7:
                continue
        elif op == "bounds":
            hi = _logint(rng, 20, 8192)
            lo = rng.randint(max(1, hi // 3), hi)
            new = (1, 1) if rng.random() < 0.4 else (1, _logint(rng, 2, lo))
            c = _bounds("", dtype, _logint(rng, 1, 24), Hkv, d, ps, (lo, hi), new)
        else:
            hi = _logint(rng, 40, 65536)
            lo = rng.randint(max(1, hi // 3), hi)
            B = _logint(rng, 1, 32)
            if op == "select":
                new = (1, 1) if rng.random() < 0.6 else (1, min(lo, rng.randint(2, 8)))
                c = _select("", B, H, Hkv, d, ps, (lo, hi), new, _logint(rng, 2, 256))
                if B * new[1] * H * hi // ps > 4e6:
                    continue
            else:
                c = _selected("", dtype, B, H, Hkv, d, ps, (lo, hi), _logint(rng, 2, 256))
                if B * Hkv * hi * d > 4e8 or B * Hkv * c["n"] * ps * d > 1.5e8:
                    continue
        del c["name"]
        return c


# -------------------------------------------------------------------------------- inputs

def _lengths(case, count, seed):
    """Held and new tokens of `count` sequences, on the host: the case fixes
    them (shapes go by their sums), the seed their order."""
    g = _hostgen(count)
    lens = torch.randint(case["len_lo"], case["len_hi"] + 1, (count,), generator=g)
    new = torch.randint(case["new_lo"], case["new_hi"] + 1, (count,), generator=g)
    order = torch.randperm(count, generator=_hostgen(seed))
    return lens[order], torch.minimum(new, lens)[order]


def _tables(lens, ps, spare, seed):
    """A page table whose pages lie in a shuffled pool with `spare` pages more
    than are held; entries behind a sequence's last page are -1."""
    held = (lens + ps - 1) // ps
    width = max(1, int(held.max()))
    n = int(held.sum())
    perm = torch.randperm(n + spare, generator=_hostgen(seed + 1)).to(torch.int32)
    table = torch.full((lens.numel(), width), -1, dtype=torch.int32)
    table[torch.arange(width)[None] < held[:, None]] = perm[:n]
    return table, n + spare


def _pow2_at_least(x, num, exp):
    """The smallest power of two s >= 2^-100 with x <= num * 2^exp * s, for
    0.5 <= num < 1; 0 where x is 0 (frexp splits exactly)."""
    m, e = torch.frexp(x)
    k = (e - exp + (m > num)).clamp(min=-100)
    return torch.where(x > 0, torch.ldexp(torch.ones_like(x), k), torch.zeros_like(x))


def _pool(g, P, Hkv, ps, d, dtype):
    """Rows of normal values; in 8 bits, codes and a scale per page and head
    whose magnitudes differ by up to four."""
    if dtype == "bf16":
        return _randn(g, (P, Hkv, ps, d), torch.bfloat16), None
    size = torch.exp2(torch.rand((P, Hkv, 1, 1), generator=g, device=DEV) * 2 - 1)
    x = torch.randn((P, Hkv, ps, d), generator=g, device=DEV).mul_(size)
    scale = _pow2_at_least(x.abs().amax((2, 3)), 0.875, 9)
    return x.div_(scale[:, :, None, None]).to(E4M3), scale


def prepare(case, seed):
    g = _gen(seed)
    op, d, Hkv, ps, B = case["op"], case["d"], case["Hkv"], case["ps"], case["B"]
    dtype = case.get("dtype", "e4m3")
    lens, new = _lengths(case, B, seed)
    table, P = _tables(lens, ps, 5, seed)
    T = int(new.sum())
    off = torch.zeros(B + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(new, 0)
    s = {"op": op, "d": d, "Hkv": Hkv, "ps": ps, "B": B, "T": T, "P": P, "H": case.get("H", Hkv),
         "max_new": int(new.max()), "table": table.to(DEV), "lens": lens.to(torch.int32).to(DEV),
         "off": off.to(DEV)}
    bf = torch.bfloat16
    if op != "select":
        s["kp"], s["ks"] = _pool(g, P, Hkv, ps, d, dtype)
        s["vp"], s["vs"] = (s["kp"], s["ks"]) if op == "bounds" else _pool(g, P, Hkv, ps, d, dtype)
    if op == "attn8":
        s["q"] = _randn(g, (T, s["H"], d), bf)
    elif op == "append8":
        s["qkv"] = _randn(g, (T, (s["H"] + 2 * Hkv) * d), bf)
        s["gq"] = (1 + 0.2 * _randn(g, (d,), torch.float32)).to(bf)
        s["gk"] = (1 + 0.2 * _randn(g, (d,), torch.float32)).to(bf)
        s["pe"] = _pe_table(case["len_hi"], case["r"])
        s.update(r=case["r"], half=case["half"])
    elif op == "bounds":
        # those of the pages that were full before
        reach = torch.randint(20, 97, (P, Hkv, 1, d), generator=g, device=DEV).to(torch.int8)
        s["bounds"] = torch.cat((-reach, reach), 2)
        s["bscale"] = torch.exp2(torch.randint(-6, -4, (P, Hkv), generator=g, device=DEV).float())
    elif op == "select":
        # the keys themselves are not read
        s["kp"] = s["vp"] = torch.zeros(P * Hkv * ps * d, dtype=torch.uint8, device=DEV).view(E4M3).view(
            P, Hkv, ps, d)
        s["ks"] = s["vs"] = torch.ones((P, Hkv), device=DEV)
        s["q"] = _randn(g, (T, s["H"], d), bf)
        mid = torch.randint(-30, 31, (P, Hkv, d), generator=g, device=DEV)
        reach = torch.randint(20, 97, (P, Hkv, d), generator=g, device=DEV)
        s["bounds"] = torch.stack((mid - reach, mid + reach), 2).to(torch.int8)
        s["bscale"] = torch.exp2(torch.randint(-6, -4, (P, Hkv), generator=g, device=DEV).float())
        s["n"] = case["n"]
    elif op == "selected":
        s["q"] = _randn(g, (T, s["H"], d), bf)
        # the newest page and others at random, by column, for every kv head
        n, held = case["n"], (s["lens"] + ps - 1) // ps
        width = s["table"].shape[1]
        col = torch.arange(width, device=DEV)
        luck = torch.rand((B, Hkv, width), generator=g, device=DEV)
        luck = torch.where((col == held[:, None] - 1)[:, None], 2.0, luck)
        luck = torch.where((col < held[:, None])[:, None], luck, -1.0)
        k = min(n, width)
        took, cols = luck.topk(k, -1)
        cols = torch.where(took >= 0, cols, width).sort(-1).values
        wide = torch.cat((s["table"], s["table"].new_full((B, 1), -1)), 1)
        pages = wide[:, None].expand(B, Hkv, width + 1).gather(2, cols)
        s["sel"] = torch.full((B, Hkv, n), -1, dtype=torch.int32, device=DEV)
        s["sel"][:, :, :k] = pages
        count = torch.minimum(held, torch.full_like(held, n))
        s["sel_lens"] = ((count - 1) * ps + (s["lens"] - 1) % ps + 1).to(torch.int32)
    return s


# ---------------------------------------------------------------------------- plain forms

def _rotate(z, sin, cos, r, half):
    """The rotation of z [..., d] by tables broadcast to [..., r/2]."""
    a, b = (z[..., :r // 2], z[..., r // 2:r]) if half else (z[..., 0:r:2], z[..., 1:r:2])
    x, y = a * cos - b * sin, b * cos + a * sin
    rot = torch.cat((x, y), -1) if half else torch.stack((x, y), -1).flatten(-2)
    return torch.cat((rot, z[..., r:]), -1)


def _norm_rope(x, gamma, sin, cos, r, half):
    x = x.float()
    xh = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _rotate(xh * gamma.float(), sin, cos, r, half)


def _split(s):
    H, Hkv, d, qkv = s["H"], s["Hkv"], s["d"], s["qkv"]
    return [x.view(s["T"], -1, d) for x in
            (qkv[:, :H * d], qkv[:, H * d:(H + Hkv) * d], qkv[:, (H + Hkv) * d:])]


def _token_places(s):
    """For every packed token: its sequence, its index there, its position."""
    t = torch.arange(s["T"], device=DEV, dtype=torch.int32)
    b = torch.searchsorted(s["off"][1:].contiguous(), t, right=True)
    i = t - s["off"][b]
    n = s["off"][1:] - s["off"][:-1]
    return b, i.long(), (s["lens"] - n)[b].long() + i


def _values(pool, scale, pages, heads=None):
    """The rows of pages in fp32: pool[pages] (or pool[pages, heads])."""
    at = pages if heads is None else (pages, heads)
    x = pool.view(torch.uint8)[at].view(E4M3).float() if pool.dtype is E4M3 else pool[at].float()
    return x if scale is None else x * scale[at][..., None, None]


def _softmax(S):
    P = torch.exp(S - S.amax(-1, keepdim=True))
    return P / P.sum(-1, keepdim=True)


def _plain_attn(s):
    B, H, Hkv, d, ps, n = s["B"], s["H"], s["Hkv"], s["d"], s["ps"], s["max_new"]
    G, table = H // Hkv, s["table"].clamp(min=0).long()
    L = table.shape[1] * ps
    K = _values(s["kp"], s["ks"], table).transpose(1, 2).reshape(B, Hkv, L, d)
    V = _values(s["vp"], s["vs"], table).transpose(1, 2).reshape(B, Hkv, L, d)
    i = torch.arange(n, device=DEV)
    tok = (s["off"][:-1, None] + i).clamp(max=s["T"] - 1).long()
    q = s["q"][tok].float().view(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    S = (q @ K.transpose(-1, -2)).view(B, Hkv, G, n, L) * (1 / math.sqrt(d))
    last = (s["lens"] - (s["off"][1:] - s["off"][:-1]))[:, None] + i
    last = torch.minimum(last, s["lens"][:, None] - 1)
    seen = torch.arange(L, device=DEV) <= last[..., None]
    w = _softmax(S.masked_fill(~seen[:, None, None], -math.inf))
    O = (w.view(B, Hkv, G * n, L) @ V).view(B, H, n, d)
    b, i, _ = _token_places(s)
    return O[b, :, i].to(torch.bfloat16)


def _plain_append(s):
    q, k, v = _split(s)
    r, half, ps, B, T = s["r"], s["half"], s["ps"], s["B"], s["T"]
    b, _, pos = _token_places(s)
    pe = s["pe"][pos]
    sin, cos = pe[:, 0::2][:, None], pe[:, 1::2][:, None]
    yq = _norm_rope(q, s["gq"], sin, cos, r, half).to(torch.bfloat16)
    yk = _norm_rope(k, s["gk"], sin, cos, r, half)
    n = s["off"][1:] - s["off"][:-1]
    first = (s["lens"] - n).long()
    # the pages that sequence b's new tokens touch: columns first // ps and on
    most = (s["max_new"] + ps - 2) // ps + 1
    col = (first // ps)[:, None] + torch.arange(most, device=DEV)
    touched = (col * ps < s["lens"][:, None]) & (n > 0)[:, None]
    page = s["table"].gather(1, col.clamp(max=s["table"].shape[1] - 1)).clamp(min=0).long()
    older = torch.where(touched, (first[:, None] - col * ps).clamp(min=0), 0).flatten()
    # a place behind the pool takes what does not count
    P = s["P"]
    page = torch.where(touched, page, P).flatten()
    at = s["table"][b, pos // ps].long()
    rows = torch.arange(ps, device=DEV)[:, None] < older[:, None, None, None]
    for pool, scale, x in ((s["kp"], s["ks"], yk), (s["vp"], s["vs"], v.float())):
        Hkv = scale.shape[1]
        amax = torch.zeros((P + 1, Hkv), device=DEV).scatter_reduce_(
            0, at[:, None].expand(T, Hkv), x.abs().amax(-1), "amax")
        old = torch.cat((scale, scale.new_zeros((1, Hkv))))
        base = torch.where(older[:, None] > 0, old[page], 0.0)
        new = torch.maximum(base, _pow2_at_least(amax[page], 0.875, 9))
        old[page] = new
        inside = page.clamp(max=P - 1)
        grow = (base / torch.where(new > 0, new, 1.0))[:, :, None, None]
        grown = (_values(pool, None, inside) * grow).to(E4M3).view(torch.uint8)
        kept = torch.where(rows, grown, pool.view(torch.uint8)[inside])
        # places that do not count write to a spare page, which no sequence holds
        spill = torch.cat((pool.view(torch.uint8), pool[:1].view(torch.uint8)))
        spill[page] = kept
        pool.view(torch.uint8).copy_(spill[:P])
        scale.copy_(old[:P])
        st = torch.where(scale > 0, scale, 1.0)[at]
        pool.view(torch.uint8)[at, :, pos % ps] = (x / st[..., None]).to(E4M3).view(torch.uint8)
    return [yq, s["kp"], s["vp"], s["ks"], s["vs"]]


def _plain_bounds(s):
    ps, P = s["ps"], s["P"]
    n = s["off"][1:] - s["off"][:-1]
    first = (s["lens"] - n).long() // ps
    most = (s["max_new"] + ps - 2) // ps + 1
    col = first[:, None] + torch.arange(most, device=DEV)
    full = ((col + 1) * ps <= s["lens"][:, None]) & (n > 0)[:, None]
    page = s["table"].gather(1, col.clamp(max=s["table"].shape[1] - 1)).clamp(min=0).long()
    x = _values(s["kp"], None, page.flatten())
    lo, hi = x.amin(2), x.amax(2)
    step = _pow2_at_least(torch.maximum(lo.abs(), hi.abs()).amax(-1), 127 / 128, 7)
    safe = torch.where(step > 0, step, 1.0)[..., None]
    b = torch.stack((torch.floor(lo / safe), torch.ceil(hi / safe)), 2).to(torch.int8)
    sc = step if s["ks"] is None else step * s["ks"][page.flatten()]
    at = torch.where(full, page, P).flatten()
    bounds = torch.cat((s["bounds"], s["bounds"][:1]))
    scale = torch.cat((s["bscale"], s["bscale"][:1]))
    bounds[at], scale[at] = b, sc
    s["bounds"].copy_(bounds[:P])
    s["bscale"].copy_(scale[:P])
    return [s["bounds"], s["bscale"]]


def _plain_select(s):
    H, Hkv, d, ps, T, n = s["H"], s["Hkv"], s["d"], s["ps"], s["T"], s["n"]
    G, width = H // Hkv, s["table"].shape[1]
    b, _, pos = _token_places(s)
    q = s["q"].float()
    step = _pow2_at_least(q.abs().amax(-1), 127 / 128, 7)
    qi = torch.round(q / torch.where(step > 0, step, 1.0)[..., None]).view(T, Hkv, G, d)
    table = s["table"].clamp(min=0).long()
    lo, hi = s["bounds"][table].float().permute(3, 0, 2, 4, 1)[:, b]     # [T, Hkv, d, width]
    # whole numbers below 2^24: any order of the sum gives the same
    S = qi.clamp(min=0) @ hi + qi.clamp(max=0) @ lo
    S = S * step.view(T, Hkv, G, 1) * s["bscale"][table].transpose(1, 2)[b][:, :, None]
    S = S.amax(2)
    newest = (pos // ps)[:, None, None]
    col = torch.arange(width, device=DEV)
    S = torch.where(col < newest, S, -math.inf)
    S = torch.where(col == newest, math.inf, S)
    k = min(n, width)
    order = torch.sort(S, dim=-1, descending=True, stable=True).indices[..., :k]
    order = torch.where(S.gather(-1, order) > -math.inf, order, width).sort(-1).values
    wide = torch.cat((s["table"], s["table"].new_full((s["B"], 1), -1)), 1)[b]
    sel = torch.full((T, Hkv, n), -1, dtype=torch.int32, device=DEV)
    sel[:, :, :k] = wide[:, None].expand(T, Hkv, width + 1).gather(2, order)
    count = (pos // ps + 1).clamp(max=n)
    return [sel, ((count - 1) * ps + pos % ps + 1).to(torch.int32)]


def _plain_selected(s):
    H, Hkv, d, ps, T = s["H"], s["Hkv"], s["d"], s["ps"], s["T"]
    sel, g = s["sel"].clamp(min=0).long(), torch.arange(Hkv, device=DEV)[None, :, None]
    L = sel.shape[2] * ps
    K = _values(s["kp"], s["ks"], sel, g).view(T, Hkv, L, d)
    V = _values(s["vp"], s["vs"], sel, g).view(T, Hkv, L, d)
    S = (s["q"].float().view(T, Hkv, H // Hkv, d) @ K.transpose(-1, -2)) * (1 / math.sqrt(d))
    seen = torch.arange(L, device=DEV) < s["sel_lens"][:, None]
    w = _softmax(S.masked_fill(~seen[:, None, None], -math.inf))
    return (w @ V).view(T, H, d).to(torch.bfloat16)


def _own(s):
    import transformer_head_scaled_03_gb300 as mha
    op = s["op"]
    if op == "attn8":
        return mha.sdpa_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["off"],
                              max_new=s["max_new"], K_scale=s["ks"], V_scale=s["vs"])
    if op == "append8":
        q, k, v = _split(s)
        pairing = mha.ROPE_HALF if s["half"] else mha.ROPE_INTERLEAVED
        yq = mha.qk_norm_rope_paged(q, k, v, s["gq"], s["gk"], s["pe"], s["kp"], s["vp"], s["table"],
                                    s["lens"], s["off"], pairing=pairing, eps=EPS, K_scale=s["ks"],
                                    V_scale=s["vs"])
        return [yq, s["kp"], s["vp"], s["ks"], s["vs"]]
    if op == "bounds":
        mha.kv_pages_bounds(s["kp"], s["vp"], s["table"], s["lens"], s["off"], s["bounds"], s["bscale"],
                            T=s["T"], K_scale=s["ks"], V_scale=s["vs"])
        return [s["bounds"], s["bscale"]]
    if op == "select":
        return list(mha.kv_pages_select(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["off"],
                                        s["bounds"], s["bscale"], s["n"], K_scale=s["ks"],
                                        V_scale=s["vs"]))
    return mha.sdpa_paged_selected(s["q"], s["kp"], s["vp"], s["sel"], s["sel_lens"], K_scale=s["ks"],
                                   V_scale=s["vs"])


def run(state):
    if own:
        return _own(state)
    return {"attn8": _plain_attn, "append8": _plain_append, "bounds": _plain_bounds,
            "select": _plain_select, "selected": _plain_selected}[state["op"]](state)


# ----------------------------------------------------------------------------- work, exact

def work(case):
    """Every input read once, every output written once; lengths at their mean."""
    op, d, Hkv, ps, B = case["op"], case["d"], case["Hkv"], case["ps"], case["B"]
    es = 2 if case.get("dtype") == "bf16" else 1
    mean = (case["len_lo"] + case["len_hi"]) / 2
    new = min(mean, (case["new_lo"] + case["new_hi"]) / 2)
    T, H = B * new, case.get("H", Hkv)
    if op == "attn8":
        return {"bytes": B * mean * Hkv * (d + 4 / ps) * 2 + 4 * T * H * d,
                "flops": 4 * d * H * T * (mean - new + (new + 1) / 2)}
    if op == "append8":
        return {"bytes": T * (4 * H + 6 * Hkv) * d + T * case["r"] * 4, "flops": 10 * T * (H + Hkv) * d}
    if op == "bounds":
        pages = T / ps
        return {"bytes": pages * Hkv * (ps * d * es + 2 * d + 4), "flops": 2 * pages * Hkv * ps * d}
    if op == "select":
        pages = math.ceil(mean / ps)
        return {"bytes": B * pages * Hkv * (2 * d + 4) + T * H * d * 2 + T * Hkv * case["n"] * 4,
                "flops": 4 * T * H * pages * d}
    rows = min(mean, case["n"] * ps)
    return {"bytes": T * Hkv * rows * (d * es + (4 / ps if es == 1 else 0)) * 2 + 4 * T * H * d,
            "flops": 4 * d * H * T * rows}


def _to_grid(x):
    """x rounded to the e4m3 values, ties to even, in fp64."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -9))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_rows(x, gamma, pe, r, half):
    """Norm and rotation of x [N, heads, d] at table rows pe [N, r], as pairs
    of columns turned by a 2 x 2 matrix each."""
    z = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * gamma
    m = torch.arange(r // 2, device=DEV)
    a, b = (m, m + r // 2) if half else (2 * m, 2 * m + 1)
    sn, cs = pe[:, None, 2 * m], pe[:, None, 2 * m + 1]
    y = z.clone()
    y[..., a] = z[..., a] * cs - z[..., b] * sn
    y[..., b] = z[..., b] * cs + z[..., a] * sn
    return y


def _rows_of(pool, scale, pages, g, length):
    x = _values(pool, None, pages, g).double()
    if scale is not None:
        x = x * scale[pages, g].double()[:, None, None]
    return x.reshape(-1, x.shape[-1])[:length]


def _exact_append(s):
    f = torch.float64
    q, k, v = _split(s)
    lens, off, ps = s["lens"].tolist(), s["off"].tolist(), s["ps"]
    first = [lens[b] - (off[b + 1] - off[b]) for b in range(s["B"])]
    pos = torch.cat([torch.arange(first[b], lens[b]) for b in range(s["B"])]).to(DEV)
    pe = s["pe"].to(f)[pos]
    yq = _exact_rows(q.to(f), s["gq"].to(f), pe, s["r"], s["half"])
    yk = _exact_rows(k.to(f), s["gk"].to(f), pe, s["r"], s["half"])
    out = [yq]
    scales = []
    table = s["table"].tolist()
    for pool, scale, x in ((s["kp"], s["ks"], yk), (s["vp"], s["vs"], v.to(f))):
        c, sc = pool.to(f), scale.to(f).clone()
        for b in range(s["B"]):
            if off[b + 1] == off[b]:
                continue
            for col in range(first[b] // ps, (lens[b] - 1) // ps + 1):
                r0, r1 = max(first[b], col * ps) - col * ps, min(lens[b], (col + 1) * ps) - col * ps
                t0 = off[b] + col * ps + r0 - first[b]
                rows = x[t0:t0 + r1 - r0].transpose(0, 1)
                need = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((1, 2)) / 448)).clamp(min=-100))
                page = table[b][col]
                base = sc[page] if r0 else torch.zeros_like(need)
                new = torch.maximum(base, need)
                if r0:
                    c[page, :, :r0] = _to_grid(c[page, :, :r0] * (base / new)[:, None, None])
                c[page, :, r0:r1] = _to_grid(rows / new[:, None, None])
                sc[page] = new
        out.append(c)
        scales.append(sc)
    return out + scales


def _exact_bounds(s):
    scale = s["bscale"].double()
    lens, off, ps, table = s["lens"].tolist(), s["off"].tolist(), s["ps"], s["table"].tolist()
    for b in range(s["B"]):
        first = lens[b] - (off[b + 1] - off[b])
        pages = table[b][first // ps:lens[b] // ps] if off[b + 1] > off[b] else []
        if pages:
            at = torch.tensor(pages, device=DEV)
            amax = _values(s["kp"], None, at).double().abs().amax((2, 3))
            scale[at] = torch.exp2(torch.ceil(torch.log2(amax / 127)).clamp(min=-100))
            if s["ks"] is not None:
                scale[at] *= s["ks"][at].double()
    return [None, scale]


def exact(case, seed):
    op = case["op"]
    if op == "select":
        return None   # whole numbers
    flops = work(case)["flops"]
    if flops > 2e12:
        return None
    s = prepare(case, seed)
    if op == "bounds":
        return _exact_bounds(s)
    if op == "append8":
        return _exact_append(s) if s["T"] <= 20000 else None
    f = torch.float64
    H, Hkv, d, ps = s["H"], s["Hkv"], s["d"], s["ps"]
    G = H // Hkv
    O = torch.zeros((s["T"], H, d), dtype=f, device=DEV)
    if op == "selected":
        lens, sel = s["sel_lens"].tolist(), s["sel"].long()
        for t in range(s["T"]):
            for g in range(Hkv):
                pages = sel[t, g, :-(-lens[t] // ps)]
                kk = _rows_of(s["kp"], s["ks"], pages, g, lens[t])
                vv = _rows_of(s["vp"], s["vs"], pages, g, lens[t])
                w = torch.softmax(s["q"][t, g * G:(g + 1) * G].to(f) @ kk.T / math.sqrt(d), -1)
                O[t, g * G:(g + 1) * G] = w @ vv
        return O
    lens, off, table = s["lens"].tolist(), s["off"].tolist(), s["table"].tolist()
    for b in range(s["B"]):
        n, length = off[b + 1] - off[b], lens[b]
        pages = torch.tensor(table[b][:-(-length // ps)], device=DEV)
        for g in range(Hkv):
            kk = _rows_of(s["kp"], s["ks"], pages, g, length)
            vv = _rows_of(s["vp"], s["vs"], pages, g, length)
            for i0 in range(0, n, 1024):
                i1 = min(n, i0 + 1024)
                qq = s["q"][off[b] + i0:off[b] + i1, g * G:(g + 1) * G].to(f)
                w = torch.einsum("igc,jc->igj", qq, kk) / math.sqrt(d)
                hidden = (torch.arange(length, device=DEV)[None]
                          > (length - n + torch.arange(i0, i1, device=DEV))[:, None])
                w = torch.softmax(w.masked_fill(hidden[:, None], -math.inf), -1)
                O[off[b] + i0:off[b] + i1, g * G:(g + 1) * G] = torch.einsum("igj,jc->igc", w, vv)
    return O
