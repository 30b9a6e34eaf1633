"""The paged key/value cache's operators, as they are measured: the attention that reads the pages, the
query/key norm and rotation that comes before it (with its gradient, and in the form that appends to the
pages), and the forking and compacting of pages.

``run`` holds each operator twice: in elementary torch operations (fp32), and as the library's calls.
``exact`` is the same definition in fp64, sequence by sequence.
"""
import math

import torch

own = False

DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _hostgen(seed):
    g = torch.Generator()
    g.manual_seed(int(seed) + 7919)
    return g


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


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
    return dict(name=name, op="sdpa_paged", dtype="bf16", B=B, H=H, Hkv=Hkv, d=d, ps=ps,
                len_lo=lens[0], len_hi=lens[1], new_lo=new[0], new_hi=new[1])


def _train(name, dtype, B, L, H, Hkv, d, r, half):
    return dict(name=name, op="qk_norm_rope", dtype=dtype, B=B, L=L, H=H, Hkv=Hkv, d=d, r=r, half=half)


def _append(name, B, H, Hkv, d, r, half, ps, lens, new):
    return dict(name=name, op="qk_norm_rope_paged", dtype="bf16", B=B, H=H, Hkv=Hkv, d=d, r=r,
                half=half, ps=ps, len_lo=lens[0], len_hi=lens[1], new_lo=new[0], new_hi=new[1])


def _fork(name, n, parents, layers, Hkv, d, ps, lens):
    return dict(name=name, op="kv_pages_fork", dtype="bf16", n=n, parents=parents, layers=layers,
                Hkv=Hkv, d=d, ps=ps, len_lo=lens[0], len_hi=lens[1])


def _compact(name, B, layers, Hkv, d, ps, lens, spare):
    return dict(name=name, op="kv_pages_compact", dtype="bf16", B=B, layers=layers, Hkv=Hkv, d=d,
                ps=ps, len_lo=lens[0], len_hi=lens[1], spare=spare)


def listed():
    return [
        # one conversation, one new token, the base model's heads: latency of a step
        _attn("attn_decode_one", 1, 8, 8, 64, 16, (700, 700), (1, 1)),
        # a server's batch of long conversations, one new token each, four query heads to a key head
        _attn("attn_decode_batch", 16, 32, 8, 128, 64, (16384, 32768), (1, 1)),
        # chunks of prompts and single tokens in one batch, over caches of ragged length
        _attn("attn_chunk_mixed", 6, 40, 8, 128, 32, (900, 8000), (1, 500)),
        # a long prompt taken in chunks of thousands of tokens: bound by the tensor cores
        _attn("attn_prefill", 2, 32, 8, 128, 128, (8192, 8192), (4096, 4096)),
        # a training step of the fp32 base shape
        _train("norm_train_base", "f32", 1, 128, 8, 8, 64, 64, True),
        # a training step of the decoder's causal shape
        _train("norm_train_causal", "bf16", 16, 2048, 16, 16, 64, 64, False),
        # a decoding step of a few conversations: latency
        _append("append_decode", 4, 32, 8, 128, 128, True, 16, (100, 4000), (1, 1)),
        # prompts of ragged length written to the pages
        _append("append_prompt", 8, 32, 8, 128, 64, True, 64, (2000, 8192), (500, 2000)),
        # two beams leave one parent each, one layer's pool
        _fork("fork_few", 2, 2, 1, 8, 64, 16, (40, 900)),
        # parallel samples of many prompts, the pools of eight layers
        _fork("fork_many", 96, 24, 8, 8, 128, 128, (300, 2000)),
        # a small pool after its conversations ended
        _compact("compact_small", 6, 1, 8, 64, 16, (0, 600), 64),
        # the pools of four layers, half of the pages free
        _compact("compact_large", 48, 4, 8, 128, 64, (0, 4096), 1600),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "train", "append", "fork", "compact"])
    d = rng.choice([64, 128])
    ps = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    while True:
        if op == "attn":
            B = _logint(rng, 1, 24)
            H = Hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
            hi = _logint(rng, 8, 32768)
            lo = rng.randint(max(1, hi // 3), hi)
            kind = rng.choice(["one", "few", "chunk"])
            new = ((1, 1) if kind == "one" else (1, min(lo, rng.randint(2, 16))) if kind == "few"
                   else (1, min(lo, _logint(rng, 17, 4096))))
            c = _attn("", B, H, Hkv, d, ps, (lo, hi), new)
            if B * H * new[1] * hi * 4 > 4e9 or B * Hkv * hi * d > 4e8:
                continue
        elif op == "train":
            r = rng.choice([d, d, d // 2])
            c = _train("", rng.choice(["bf16", "bf16", "f32"]), _logint(rng, 1, 16), _logint(rng, 1, 2048),
                       Hkv * rng.choice([1, 2, 3, 4]), Hkv, d, r, rng.random() < 0.5)
            if c["B"] * c["L"] * (c["H"] + c["Hkv"]) * d > 6e7:
                continue
        elif op == "append":
            hi = _logint(rng, 2, 8192)
            lo = rng.randint(max(1, hi // 3), hi)
            new = (1, 1) if rng.random() < 0.4 else (1, min(lo, _logint(rng, 2, 2000)))
            c = _append("", _logint(rng, 1, 16), Hkv * rng.choice([1, 3, 4, 8]), Hkv, d,
                        rng.choice([d, d, d // 2]), rng.random() < 0.5, ps, (lo, hi), new)
            if c["B"] * new[1] * (c["H"] + 2 * Hkv) * d > 6e7:
                continue
        elif op == "fork":
            parents = _logint(rng, 1, 24)
            hi = _logint(rng, 20, 2000)
            c = _fork("", _logint(rng, 1, 96), parents, rng.choice([1, 2, 3, 6, 8]), Hkv, d, ps,
                      (rng.randint(0, hi), hi))
        else:
            hi = _logint(rng, 20, 4096)
            c = _compact("", _logint(rng, 1, 48), rng.choice([1, 2, 3, 4]), Hkv, d, ps,
                         (rng.randint(0, hi // 2), hi), _logint(rng, 8, 1600))
        del c["name"]
        return c


# -------------------------------------------------------------------------------- inputs

def _lengths(case, count, seed):
    """Held and new tokens of `count` sequences, on the host: the case fixes
    them (shapes go by their sums), the seed their order."""
    g = _hostgen(count)
    lens = torch.randint(case["len_lo"], case["len_hi"] + 1, (count,), generator=g)
    new = torch.randint(case.get("new_lo", 0), case.get("new_hi", 0) + 1, (count,), generator=g)
    order = torch.randperm(count, generator=_hostgen(seed))
    return lens[order], torch.minimum(new, lens)[order]


def _tables(lens, ps, spare, seed):
    """A page table whose pages lie in a shuffled pool with `spare` pages more
    than are held; entries behind a sequence's last page are -1."""
    held = (lens + ps - 1) // ps
    width = max(1, int(held.max()))
    total = int(held.sum()) + spare
    perm = torch.randperm(max(1, total), generator=_hostgen(seed + 1)).to(torch.int32)
    table = torch.full((lens.numel(), width), -1, dtype=torch.int32)
    mask = torch.arange(width)[None] < held[:, None]
    n = int(held.sum())
    table[mask] = perm[:n]
    return table, max(1, total), perm[n:]


def prepare(case, seed):
    g, dt = _gen(seed), _dtype(case)
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    s = {"op": op, "d": d, "Hkv": Hkv}
    if op == "qk_norm_rope":
        B, L, H = case["B"], case["L"], case["H"]
        # the projection's output, queries and keys side by side
        s["qkv"] = _randn(g, (B, L, (H + Hkv) * d), dt)
        s["gq"] = (1 + 0.2 * _randn(g, (d,), torch.float32)).to(dt)
        s["gk"] = (1 + 0.2 * _randn(g, (d,), torch.float32)).to(dt)
        s["pe"] = _pe_table(L, case["r"])
        # what sdpa_backward returns: dQ in fp32, dK in the layer's type
        s["dq"] = _randn(g, (B, H, L, d), torch.float32)
        s["dk"] = _randn(g, (B, Hkv, L, d), dt)
        s.update(B=B, L=L, H=H, r=case["r"], half=case["half"])
        return s
    if op in ("sdpa_paged", "qk_norm_rope_paged"):
        B, H, ps = case["B"], case["H"], case["ps"]
        lens, new = _lengths(case, B, seed)
        table, P, _ = _tables(lens, ps, 5, seed)
        T = int(new.sum())
        s.update(B=B, H=H, ps=ps, T=T, max_new=int(new.max()))
        s["kp"] = _randn(g, (P, Hkv, ps, d), dt)
        s["vp"] = _randn(g, (P, Hkv, ps, d), dt)
        s["table"] = table.to(DEV)
        s["lens"] = lens.to(torch.int32).to(DEV)
        off = torch.zeros(B + 1, dtype=torch.int32)
        off[1:] = torch.cumsum(new, 0)
        s["off"] = off.to(DEV)
        if op == "sdpa_paged":
            s["q"] = _randn(g, (T, H, d), dt)
        else:
            s["qkv"] = _randn(g, (T, (H + 2 * Hkv) * d), dt)
            s["gq"] = (1 + 0.2 * _randn(g, (d,), torch.float32)).to(dt)
            s["gk"] = (1 + 0.2 * _randn(g, (d,), torch.float32)).to(dt)
            s["pe"] = _pe_table(case["len_hi"], case["r"])
            s.update(r=case["r"], half=case["half"])
        return s
    layers, ps = case["layers"], case["ps"]
    h = _hostgen(seed)
    if op == "kv_pages_fork":
        n, par = case["n"], case["parents"]
        lens, _ = _lengths(case, par, seed)
        table, P, free = _tables(lens, ps, n + 3, seed)
        rows = torch.full((par + n, table.shape[1]), -1, dtype=torch.int32)
        rows[:par] = table
        s["table"] = rows.to(DEV)
        s["lens"] = torch.cat((lens, torch.zeros(n, dtype=torch.int64))).to(torch.int32).to(DEV)
        s["parents"] = torch.randint(0, par, (n,), generator=h).to(torch.int32).to(DEV)
        s["children"] = (par + torch.randperm(n, generator=h)).to(torch.int32).to(DEV)
        s["fresh"] = free[:n].to(DEV)
        s["kp"] = _randn(g, (layers, P, Hkv, ps, d), dt)
        s["vp"] = _randn(g, (layers, P, Hkv, ps, d), dt)
    else:
        lens, _ = _lengths(case, case["B"], seed)
        table, P, _ = _tables(lens, ps, case["spare"], seed)
        if case["B"] > 1 and table.shape[1] > 0:
            # two conversations share their first page, as forks do
            both = (lens[0] > ps) & (lens[1] > ps)
            table[1, 0] = table[0, 0] if bool(both) else table[1, 0]
        live = int(((lens + ps - 1) // ps).sum())
        s["table"] = table.to(DEV)
        s["lens"] = lens.to(torch.int32).to(DEV)
        s["kp"] = _randn(g, (layers, P, Hkv, ps, d), dt)
        s["vp"] = _randn(g, (layers, P, Hkv, ps, d), dt)
        s["ko"] = torch.zeros((layers, max(1, live), Hkv, ps, d), dtype=dt, device=DEV)
        s["vo"] = torch.zeros((layers, max(1, live), Hkv, ps, d), dtype=dt, device=DEV)
        s["table_out"] = torch.full_like(s["table"], -1)
    s.update(ps=ps, layers=layers)
    return s


# ---------------------------------------------------------------------------- plain forms

def _rotate(z, sin, cos, r, half):
    """The rotation of z [..., d] by tables broadcast to [..., r/2]."""
    a, b = (z[..., :r // 2], z[..., r // 2:r]) if half else (z[..., 0:r:2], z[..., 1:r:2])
    x, y = a * cos - b * sin, b * cos + a * sin
    rot = torch.cat((x, y), -1) if half else torch.stack((x, y), -1).flatten(-2)
    return torch.cat((rot, z[..., r:]), -1)


def _norm(x, gamma, eps):
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * rstd, rstd


EPS = 1e-6


def _plain_norm_rope(x, gamma, sin, cos, r, half):
    xh, _ = _norm(x.float(), gamma, EPS)
    return _rotate(xh * gamma.float(), sin, cos, r, half)


def _plain_norm_rope_grad(x, gamma, dy, sin, cos, r, half):
    xh, rstd = _norm(x.float(), gamma, EPS)
    dz = _rotate(dy.float(), -sin, cos, r, half)
    dgamma = (dz * xh).flatten(0, -2).sum(0, dtype=torch.float64).float()
    u = dz * gamma.float()
    return rstd * (u - xh * (u * xh).mean(-1, keepdim=True)), dgamma


def _split(s):
    H, Hkv, d, qkv = s["H"], s["Hkv"], s["d"], s["qkv"]
    lead = qkv.shape[:-1]
    return [x.view(*lead, -1, d) for x in
            (qkv[..., :H * d], qkv[..., H * d:(H + Hkv) * d], qkv[..., (H + Hkv) * d:])]


def _plain_train(s):
    q, k, _ = _split(s)
    dt, r, half = q.dtype, s["r"], s["half"]
    sin, cos = s["pe"][:, 0::2][:, None], s["pe"][:, 1::2][:, None]
    yq = _plain_norm_rope(q, s["gq"], sin, cos, r, half).to(dt).transpose(1, 2).contiguous()
    yk = _plain_norm_rope(k, s["gk"], sin, cos, r, half).to(dt).transpose(1, 2).contiguous()
    dq, dgq = _plain_norm_rope_grad(q, s["gq"], s["dq"].transpose(1, 2), sin, cos, r, half)
    dk, dgk = _plain_norm_rope_grad(k, s["gk"], s["dk"].transpose(1, 2), sin, cos, r, half)
    return [yq, yk, dq.to(dt), dk.to(dt), dgq, dgk]


def _token_places(s):
    """For every packed token: its sequence, its index there, its position."""
    t = torch.arange(s["T"], device=DEV, dtype=torch.int32)
    b = torch.searchsorted(s["off"][1:].contiguous(), t, right=True)
    i = t - s["off"][b]
    n = s["off"][1:] - s["off"][:-1]
    return b, i.long(), (s["lens"] - n)[b].long() + i


def _plain_append(s):
    q, k, v = _split(s)
    dt, r, half, ps = q.dtype, s["r"], s["half"], s["ps"]
    b, _, pos = _token_places(s)
    pe = s["pe"][pos]
    sin, cos = pe[:, 0::2][:, None], pe[:, 1::2][:, None]
    yq = _plain_norm_rope(q, s["gq"], sin, cos, r, half).to(dt)
    yk = _plain_norm_rope(k, s["gk"], sin, cos, r, half).to(dt)
    page = s["table"][b, pos // ps].long()
    s["kp"][page, :, pos % ps] = yk
    s["vp"][page, :, pos % ps] = v
    return [yq, s["kp"], s["vp"]]


def _plain_attn(s):
    B, H, Hkv, d, ps, n = s["B"], s["H"], s["Hkv"], s["d"], s["ps"], s["max_new"]
    G, table = H // Hkv, s["table"].clamp(min=0).long()
    L = table.shape[1] * ps
    K = s["kp"][table].transpose(1, 2).reshape(B, Hkv, L, d).float()
    V = s["vp"][table].transpose(1, 2).reshape(B, Hkv, L, d).float()
    i = torch.arange(n, device=DEV)
    tok = (s["off"][:-1, None] + i).clamp(max=s["T"] - 1).long()
    q = s["q"][tok].float().view(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    S = (q @ K.transpose(-1, -2)).view(B, Hkv, G, n, L) * (1 / math.sqrt(d))
    last = (s["lens"] - (s["off"][1:] - s["off"][:-1]))[:, None] + i
    last = torch.minimum(last, s["lens"][:, None] - 1)
    seen = torch.arange(L, device=DEV) <= last[..., None]
    S = S.masked_fill(~seen[:, None, None], -math.inf)
    P = torch.exp(S - S.amax(-1, keepdim=True))
    P = P / P.sum(-1, keepdim=True)
    O = (P.view(B, Hkv, G * n, L) @ V).view(B, H, n, d)
    b, i, _ = _token_places(s)
    return O[b, :, i].to(s["q"].dtype)


def _plain_fork(s):
    ps, kp, vp, table, lens = s["ps"], s["kp"], s["vp"], s["table"], s["lens"]
    par, chi, fresh = s["parents"].long(), s["children"].long(), s["fresh"].long()
    n = lens[par].long()
    full, rem = (n // ps)[:, None], n % ps
    src = table[par].gather(1, full.clamp(max=table.shape[1] - 1))[:, 0].clamp(min=0).long()
    col = torch.arange(table.shape[1], device=DEV)[None]
    rows = torch.where(col < full, table[par], table[chi])
    rows = torch.where((col == full) & (rem > 0)[:, None], s["fresh"][:, None], rows)
    kept = (torch.arange(ps, device=DEV)[None] < rem[:, None])[None, :, None, :, None]
    kp[:, fresh] = torch.where(kept, kp[:, src], kp[:, fresh])
    vp[:, fresh] = torch.where(kept, vp[:, src], vp[:, fresh])
    table[chi] = rows
    lens[chi] = lens[par]
    return [kp, vp, table, lens]


def _plain_compact(s):
    ps, table, kp, vp = s["ps"], s["table"], s["kp"], s["vp"]
    P, Po = kp.shape[1], s["ko"].shape[1]
    held = torch.arange(table.shape[1], device=DEV)[None] * ps < s["lens"][:, None]
    pages = torch.where(held, table, P).long()
    live = torch.zeros(P + 1, dtype=torch.bool, device=DEV).index_fill(0, pages.flatten(), True)[:P]
    count = live.sum(dtype=torch.int32)
    order = torch.argsort(~live, stable=True)
    order = torch.cat((order, order.new_zeros(Po)))[:Po]
    take = (torch.arange(Po, device=DEV) < count)[None, :, None, None, None]
    s["ko"].copy_(torch.where(take, kp[:, order], s["ko"]))
    s["vo"].copy_(torch.where(take, vp[:, order], s["vo"]))
    rank = (torch.cumsum(live, 0) - 1).to(torch.int32)
    rank = torch.cat((rank, rank.new_zeros(1)))
    s["table_out"].copy_(torch.where(held, rank[pages], s["table_out"]))
    return [s["ko"], s["vo"], s["table_out"], count.view(1)]


def _own(s):
    import transformer_head_scaled_03_gb300 as mha
    op = s["op"]
    if op == "sdpa_paged":
        return mha.sdpa_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["off"],
                              max_new=s["max_new"])
    if op == "qk_norm_rope":
        q, k, _ = _split(s)
        pairing = mha.ROPE_HALF if s["half"] else mha.ROPE_INTERLEAVED
        yq, yk = mha.qk_norm_rope(q, k, s["gq"], s["gk"], s["pe"], pairing=pairing, eps=EPS)
        return [yq, yk, *mha.qk_norm_rope_backward(q, k, s["gq"], s["gk"], s["pe"], s["dq"], s["dk"],
                                                   pairing=pairing, eps=EPS)]
    if op == "qk_norm_rope_paged":
        q, k, v = _split(s)
        pairing = mha.ROPE_HALF if s["half"] else mha.ROPE_INTERLEAVED
        yq = mha.qk_norm_rope_paged(q, k, v, s["gq"], s["gk"], s["pe"], s["kp"], s["vp"], s["table"],
                                    s["lens"], s["off"], pairing=pairing, eps=EPS)
        return [yq, s["kp"], s["vp"]]
    if op == "kv_pages_fork":
        mha.kv_pages_fork(s["kp"], s["vp"], s["table"], s["lens"], s["parents"], s["children"],
                          s["fresh"])
        return [s["kp"], s["vp"], s["table"], s["lens"]]
    count = mha.kv_pages_compact(s["kp"], s["vp"], s["table"], s["lens"], s["ko"], s["vo"],
                                 s["table_out"])
    return [s["ko"], s["vo"], s["table_out"], count]


def run(state):
    if own:
        return _own(state)
    return {"sdpa_paged": _plain_attn, "qk_norm_rope": _plain_train,
            "qk_norm_rope_paged": _plain_append, "kv_pages_fork": _plain_fork,
            "kv_pages_compact": _plain_compact}[state["op"]](state)


# ----------------------------------------------------------------------------- work, exact

def work(case):
    """Every input read once, every output written once; lengths at their mean."""
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "qk_norm_rope":
        rows = case["B"] * case["L"]
        q, k = rows * case["H"] * d, rows * Hkv * d
        moved = (q + k) * 3 * es + q * 4 + k * es + case["L"] * case["r"] * 4 + 2 * d * (es + 4)
        return {"bytes": moved, "flops": 24 * (q + k)}
    mean = (case["len_lo"] + case["len_hi"]) / 2
    if op in ("sdpa_paged", "qk_norm_rope_paged"):
        new = min(mean, (case["new_lo"] + case["new_hi"]) / 2)
        T = case["B"] * new
        if op == "qk_norm_rope_paged":
            return {"bytes": 2 * T * (case["H"] + 2 * Hkv) * d * es + T * case["r"] * 4,
                    "flops": 10 * T * (case["H"] + Hkv) * d}
        return {"bytes": case["B"] * mean * Hkv * d * 2 * es + 2 * T * case["H"] * d * es,
                "flops": 4 * d * case["H"] * T * (mean - new + (new + 1) / 2)}
    if op == "kv_pages_fork":
        rem = min(case["ps"], max(1.0, mean)) / 2
        return {"bytes": case["n"] * case["layers"] * 2 * Hkv * rem * d * es * 2
                + case["n"] * mean / case["ps"] * 8, "flops": 0}
    pages = case["B"] * math.ceil(mean / case["ps"])
    return {"bytes": pages * case["layers"] * 2 * Hkv * case["ps"] * d * es * 2 + pages * 8, "flops": 0}


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


def exact(case, seed):
    op = case["op"]
    if op in ("kv_pages_fork", "kv_pages_compact"):
        return None   # nothing is computed: rows are copied
    s = prepare(case, seed)
    f = torch.float64
    H, Hkv, d = s["H"], s["Hkv"], s["d"]
    if op == "qk_norm_rope":
        q, k, _ = _split(s)
        out, grads, dgs = [], [], []
        for x, gamma, dy in ((q, s["gq"], s["dq"]), (k, s["gk"], s["dk"])):
            B, L, h, _ = x.shape
            xs = x.to(f).detach().clone().requires_grad_(True)
            gs = gamma.to(f).detach().clone().requires_grad_(True)
            pe = s["pe"].to(f).repeat(B, 1)
            y = _exact_rows(xs.reshape(B * L, h, d), gs, pe, s["r"], s["half"])
            y = y.view(B, L, h, d).transpose(1, 2)
            gx, gg = torch.autograd.grad(y, (xs, gs), dy.to(f))
            out.append(y.detach().contiguous())
            grads.append(gx)
            dgs.append(gg)
        return out + grads + dgs
    lens, off = s["lens"].tolist(), s["off"].tolist()
    ps, table = s["ps"], s["table"].tolist()
    if op == "qk_norm_rope_paged":
        q, k, v = _split(s)
        pos = torch.cat([torch.arange(lens[b] - (off[b + 1] - off[b]), lens[b]) for b in range(s["B"])])
        pe = s["pe"].to(f)[pos.to(DEV)]
        yq = _exact_rows(q.to(f), s["gq"].to(f), pe, s["r"], s["half"])
        yk = _exact_rows(k.to(f), s["gk"].to(f), pe, s["r"], s["half"])
        kp, vp = s["kp"].to(f), s["vp"].to(f)
        page = torch.tensor([table[b][p // ps] for b in range(s["B"])
                             for p in range(lens[b] - (off[b + 1] - off[b]), lens[b])], device=DEV)
        row = (pos % ps).to(DEV)
        kp[page, :, row] = yk
        vp[page, :, row] = v.to(f)
        return [yq, kp, vp]
    if work(case)["flops"] > 2e12:
        return None
    O = torch.zeros((s["T"], H, d), dtype=f, device=DEV)
    G = H // Hkv
    for b in range(s["B"]):
        n, length = off[b + 1] - off[b], lens[b]
        pages = torch.tensor(table[b][:-(-length // ps)], device=DEV)
        for g in range(Hkv):
            kk = s["kp"][pages, g].reshape(-1, d)[:length].to(f)
            vv = s["vp"][pages, g].reshape(-1, d)[:length].to(f)
            for i0 in range(0, n, 1024):
                i1 = min(n, i0 + 1024)
                qq = s["q"][off[b] + i0:off[b] + i1, g * G:(g + 1) * G].to(f)
                w = torch.einsum("igc,jc->igj", qq, kk) / math.sqrt(d)
                hidden = (torch.arange(length, device=DEV)[None]
                          > (length - n + torch.arange(i0, i1, device=DEV))[:, None])
                w = torch.softmax(w.masked_fill(hidden[:, None], -math.inf), -1)
                O[off[b] + i0:off[b] + i1, g * G:(g + 1) * G] = torch.einsum("igj,jc->igc", w, vv)
    return O
