"""The operators around the paged decode: per-head norms with the position
rotation, the append into the paged cache, and decode over a shared prefix.

Each case is one call a serving loop makes.  With ``own`` false the operators
are computed from elementary torch operations; with ``own`` true by the library.
"""
import math

import torch

own = False

FP8_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ---- the cases --------------------------------------------------------------


def listed():
    return [
        # a decode step of eight sequences: one launch's latency
        dict(name="norm_rope_step", op="norm_rope", T=8, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, far=4096),
        # a prefill chunk, normed heads, full rotation
        dict(name="norm_rope_prefill", op="norm_rope", T=16384, Hq=40, Hkv=8, D=128, rot=128, interleaved=False,
             far=32768),
        # a ragged chunk of long-context heads: a quarter of each row rotates, neighbours paired
        dict(name="norm_rope_partial", op="norm_rope", T=2001, Hq=16, Hkv=4, D=256, rot=64, interleaved=True,
             far=1000000),
        # a decode step: 64 sequences, queries normed and rotated in the same call
        dict(name="append_step", op="append", kv="bf16", B=64, T=64, Hq=40, Hkv=8, D=128, rot=128, interleaved=False,
             bs=16, ctx=8192, norm=True, pad=0),
        # a prefill chunk into an 8-bit cache
        dict(name="append_prefill_e4m3", op="append", kv="e4m3", B=4, T=8192, Hq=0, Hkv=8, D=128, rot=128,
             interleaved=False, bs=16, ctx=4096, norm=False, pad=0),
        # a padded chunk of a ragged batch, one KV head, with its queries
        dict(name="append_padded_mqa", op="append", kv="bf16", B=29, T=4099, Hq=32, Hkv=1, D=128, rot=64,
             interleaved=False, bs=32, ctx=2048, norm=False, pad=123),
        # a few requests behind one system prompt: latency
        dict(name="shared_few", op="shared", kv="bf16", B=6, Hq=32, Hkv=8, D=128, bs=16, prefix=1040, rest=48, empty=0),
        # a serving batch behind a long prompt
        dict(name="shared_serving", op="shared", kv="bf16", B=64, Hq=40, Hkv=8, D=128, bs=16, prefix=8192, rest=700,
             empty=0),
        # the same kind of batch on an 8-bit cache, two rows of it padding
        dict(name="shared_e4m3", op="shared", kv="e4m3", B=48, Hq=32, Hkv=8, D=128, bs=16, prefix=6000, rest=500,
             empty=2),
        # long-context heads of 256
        dict(name="shared_d256", op="shared", kv="bf16", B=24, Hq=16, Hkv=4, D=256, bs=16, prefix=16384, rest=333,
             empty=0),
        # many short answers of a one-KV-head model
        dict(name="shared_mqa", op="shared", kv="bf16", B=131, Hq=32, Hkv=1, D=128, bs=32, prefix=4096, rest=257,
             empty=1),
        # a large batch behind a book
        dict(name="shared_book", op="shared", kv="bf16", B=256, Hq=32, Hkv=8, D=128, bs=16, prefix=32768, rest=400,
             empty=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "shared", "shared"])
    Hq, Hkv, D = rng.choice([(32, 8, 128), (40, 8, 128), (32, 1, 128), (16, 4, 256), (16, 2, 64), (28, 4, 128),
                             (20, 1, 128), (64, 4, 128)])
    rot = rng.choice([D, D, D // 2, 32])
    interleaved = rng.random() < 0.3
    if op == "norm_rope":
        return dict(op=op, T=_log(rng, 1, 16000), Hq=Hq, Hkv=Hkv, D=D, rot=rot, interleaved=interleaved,
                    far=_log(rng, 500, 1000000))
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    bs = rng.choice([16, 16, 32, 8, 64])
    if op == "append":
        T = _log(rng, 1, 9000)
        B = T if T < 300 and rng.random() < 0.6 else rng.randint(1, min(T, 40))
        return dict(op=op, kv=kv, B=B, T=T, Hq=rng.choice([0, Hq]), Hkv=Hkv, D=D, rot=rot, interleaved=interleaved,
                    bs=bs, ctx=_log(rng, 64, 8192) if B < 64 else _log(rng, 64, 2048), norm=rng.random() < 0.5,
                    pad=rng.choice([0, 0, T // 7]))
    B = _log(rng, 2, 160)
    prefix = max(bs, _log(rng, 64, 20000) // bs * bs)
    return dict(op=op, kv=kv, B=B, Hq=Hq, Hkv=Hkv, D=D, bs=bs, prefix=prefix, rest=_log(rng, 1, 700),
                empty=rng.choice([0, 0, 1]))


# ---- inputs -------------------------------------------------------------------


def _inv_freq(rot, dev):
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    return (10000.0 ** (-i / rot)).to(torch.float32).to(dev)


def _heads(gen, T, H, D, dev):
    """Rows as a projection leaves them: channels of unlike size."""
    x = torch.randn(T, H, D, generator=gen, device=dev)
    x *= torch.exp(0.4 * torch.randn(1, H, D, generator=gen, device=dev))
    return x.to(torch.bfloat16)


def _weight(gen, D, dev):
    return (1.0 + 0.2 * torch.randn(D, generator=gen, device=dev)).to(torch.bfloat16)


def _pool(gen, blocks, Hkv, bs, D, kv, scale, dev):
    x = torch.randn(blocks, Hkv, bs, D, generator=gen, device=dev, dtype=torch.bfloat16)
    return x if kv == "bf16" else (x.float() / scale).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _lengths(gen, B, lo, hi, dev):
    return torch.randint(lo, hi + 1, (B,), generator=gen, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    c = dict(case)
    s = {"op": c["op"]}
    if c["op"] in ("norm_rope", "append"):
        T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
        qkv = _heads(gen, T, Hq + 2 * Hkv, D, dev)  # the fused projection's rows
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["inv_freq"] = _inv_freq(c["rot"], dev)
        s["interleaved"] = c["interleaved"]
        s["eps"] = 1e-6
    if c["op"] == "norm_rope":
        s["qw"], s["kw"] = _weight(gen, D, dev), _weight(gen, D, dev)
        start = torch.randint(0, c["far"], (1,), generator=gen, device=dev)
        s["positions"] = (start + torch.arange(T, device=dev)).to(torch.int32)
        return s
    bs, Hkv, D = c["bs"], c["Hkv"], c["D"]
    s["k_scale"], s["v_scale"] = (0.03125, 0.0234375) if c["kv"] == "e4m3" else (1.0, 1.0)
    if c["op"] == "append":
        B, T, ctx = c["B"], c["T"], c["ctx"]
        live = T - c["pad"]
        own_tokens = torch.full((B,), live // B, dtype=torch.int64)
        own_tokens[: live % B] += 1
        seq = torch.repeat_interleave(torch.arange(B), own_tokens)
        first = torch.cumsum(own_tokens, 0) - own_tokens
        place = torch.arange(live) - first[seq]
        width = -(-(ctx + int(own_tokens.max())) // bs)
        ctx_b = _lengths(gen, B, ctx // 2, ctx, dev).cpu()
        # the blocks this call writes, each sequence's own; the rest of the table is earlier context
        lo, hi = ctx_b // bs, (ctx_b + own_tokens - 1).clamp_min(0) // bs + 1
        need = (hi - lo).clamp_min(0)
        pool = B * (-(-int(own_tokens.max()) // bs) + 1)
        perm = torch.randperm(pool, generator=gen, device=dev).cpu()
        tables = torch.zeros(B, width, dtype=torch.int32)
        row = torch.repeat_interleave(torch.arange(B), need)
        at = torch.arange(int(need.sum())) - (torch.cumsum(need, 0) - need)[row] + lo[row]
        tables[row, at] = perm[: len(at)].to(torch.int32)
        pos = torch.cat([ctx_b[seq] + place, torch.zeros(c["pad"], dtype=torch.int64)])
        seq = torch.cat([seq, torch.full((c["pad"],), -1, dtype=torch.int64)])
        s["positions"], s["seq_ids"] = pos.to(torch.int32).to(dev), seq.to(torch.int32).to(dev)
        s["tables"] = tables.to(dev)
        s["k_cache"] = _pool(gen, len(perm), Hkv, bs, D, c["kv"], s["k_scale"], dev)
        s["v_cache"] = _pool(gen, len(perm), Hkv, bs, D, c["kv"], s["v_scale"], dev)
        s["qw"], s["kw"] = (_weight(gen, D, dev), _weight(gen, D, dev)) if c["norm"] else (None, None)
        if c["Hq"] == 0:
            s["q"] = s["qw"] = None
        return s
    B, n = c["B"], c["prefix"] // bs
    rest = _lengths(gen, B, 0, c["rest"], dev)
    rest[B // 2] = c["rest"]
    lens = rest + n * bs
    lens[1:1 + c["empty"]] = 0  # padding rows of the batch
    own_blocks = -(-c["rest"] // bs)
    blocks = n + B * own_blocks
    perm = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    s["shared"] = perm[:n].contiguous()
    s["tables"] = torch.cat([s["shared"].expand(B, n), perm[n:].view(B, own_blocks)], 1).contiguous()
    s["lens"] = lens.to(torch.int32)
    s["k_cache"] = _pool(gen, blocks, Hkv, bs, D, c["kv"], s["k_scale"], dev)
    s["v_cache"] = _pool(gen, blocks, Hkv, bs, D, c["kv"], s["v_scale"], dev)
    s["q"] = (1.5 * torch.randn(B, c["Hq"], D, generator=gen, device=dev)).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(D)
    return s


# ---- the plain forms ----------------------------------------------------------


def _norm(x, w, eps):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _rotate(x, positions, inv_freq, interleaved):
    """Rotation of fp32 rows [T, H, D]; angles in 64 bits."""
    a = positions.double()[:, None] * inv_freq.double()
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    R = 2 * inv_freq.numel()
    head, tail = x[..., :R], x[..., R:]
    if interleaved:
        x1, x2 = head[..., 0::2], head[..., 1::2]
        y = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    else:
        x1, x2 = head[..., : R // 2], head[..., R // 2:]
        y = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    return torch.cat([y, tail], -1)


def _prepared(s, name, w):
    return _rotate(_norm(s[name], w, s["eps"]), s["positions"], s["inv_freq"], s["interleaved"])


def _held(x, cache, scale):
    """fp32 values as the cache holds them."""
    if cache.dtype == torch.bfloat16:
        return x.to(torch.bfloat16).view(torch.int16)
    return (x / scale).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _append_plain(s):
    keep = (s["seq_ids"] >= 0).nonzero()[:, 0]
    seq, pos = s["seq_ids"][keep].long(), s["positions"][keep].long()
    bs = s["k_cache"].shape[2]
    block, slot = s["tables"][seq, pos // bs].long(), pos % bs
    k = _held(_prepared(s, "k", s["kw"])[keep], s["k_cache"], s["k_scale"])
    v = _held(s["v"].float()[keep], s["v_cache"], s["v_scale"])
    s["k_cache"].view(k.dtype)[block, :, slot] = k
    s["v_cache"].view(v.dtype)[block, :, slot] = v
    out = {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["q"] is not None:
        out["q"] = _prepared(s, "q", s["qw"]).to(torch.bfloat16)
    return out


def _shared_plain(s):
    q, kc, vc, n = s["q"], s["k_cache"], s["v_cache"], s["shared"].numel()
    (B, Hq, D), (_, Hkv, bs, _) = q.shape, kc.shape
    g, Lp = Hq // Hkv, n * bs
    qh = q.float().view(B, Hkv, g, D)
    kp = kc[s["shared"].long()].float().transpose(0, 1).reshape(Hkv, Lp, D) * s["k_scale"]
    vp = vc[s["shared"].long()].float().transpose(0, 1).reshape(Hkv, Lp, D) * s["v_scale"]
    pages = s["tables"][:, n:].long()
    ks = kc[pages].float().transpose(1, 2).reshape(B, Hkv, -1, D) * s["k_scale"]
    vs = vc[pages].float().transpose(1, 2).reshape(B, Hkv, -1, D) * s["v_scale"]
    lens = s["lens"].long()
    live = (Lp + torch.arange(ks.shape[2], device=q.device))[None] < lens[:, None]
    sp = (qh.transpose(0, 1).reshape(Hkv, B * g, D) @ kp.transpose(1, 2)) * s["scale"]
    ss = (qh @ ks.transpose(2, 3)) * s["scale"]
    ss = ss.masked_fill(~live[:, None, None], float("-inf")).transpose(0, 1).reshape(Hkv, B * g, -1)
    m = torch.maximum(sp.amax(-1, keepdim=True), ss.amax(-1, keepdim=True))
    sp, ss = torch.exp(sp - m), torch.exp(ss - m)
    total = sp.sum(-1, keepdim=True) + ss.sum(-1, keepdim=True)
    vs = vs.masked_fill(~live[:, None, :, None], 0.0)
    own_part = ss.view(Hkv, B, g, -1).transpose(0, 1) @ vs
    o = ((sp @ vp).view(Hkv, B, g, D).transpose(0, 1) + own_part) / total.view(Hkv, B, g, 1).transpose(0, 1)
    lse = (m + torch.log(total)).view(Hkv, B, g).transpose(0, 1).reshape(B, Hq)
    some = lens > 0
    o = torch.where(some[:, None, None], o.reshape(B, Hq, D), 0.0)
    return {"out": o.to(torch.bfloat16), "lse": torch.where(some[:, None], lse, float("-inf"))}


# ---- one pass -----------------------------------------------------------------


def run(s):
    if own:
        import paged_kv_attention_partition_b200 as pad

        if s["op"] == "norm_rope":
            q, k = pad.pad_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["positions"], s["inv_freq"],
                                        eps=s["eps"], interleaved=s["interleaved"])
            return {"q": q, "k": k}
        scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
        if s["op"] == "append":
            q = pad.pad_append_kv(s["k"], s["v"], s["positions"], s["tables"], s["k_cache"], s["v_cache"],
                                  seq_ids=s["seq_ids"], inv_freq=s["inv_freq"], interleaved=s["interleaved"],
                                  k_weight=s["kw"], q=s["q"], q_weight=s["qw"], eps=s["eps"], **scales)
            out = {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
            return out if q is None else {**out, "q": q}
        out, lse = pad.pad_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["shared"], s["tables"], s["lens"],
                                         s["scale"], lse=True, **scales)
        return {"out": out, "lse": lse}
    if s["op"] == "norm_rope":
        return {"q": _prepared(s, "q", s["qw"]).to(torch.bfloat16), "k": _prepared(s, "k", s["kw"]).to(torch.bfloat16)}
    return _append_plain(s) if s["op"] == "append" else _shared_plain(s)


def work(case):
    c = dict(case)
    if c["op"] == "norm_rope":
        rows = c["T"] * (c["Hq"] + c["Hkv"])
        return {"bytes": 4 * rows * c["D"] + 4 * c["T"] + 4 * c["D"] + 2 * c["rot"], "flops": 10 * rows * c["D"]}
    eb = 2 if c["kv"] == "bf16" else 1
    if c["op"] == "append":
        live = c["T"] - c["pad"]
        kv = live * c["Hkv"] * c["D"] * 2 * (2 + eb)
        q = 4 * c["T"] * c["Hq"] * c["D"]
        return {"bytes": kv + q + 12 * c["T"], "flops": 10 * c["T"] * (c["Hq"] + c["Hkv"]) * c["D"]}
    # lengths are spread evenly up to `rest`, one of them at it
    live = c["B"] - c["empty"]
    rest = live * c["rest"] / 2
    kv = 2 * eb * c["Hkv"] * c["D"] * (c["prefix"] + rest)
    io = c["B"] * c["Hq"] * (4 * c["D"] + 4)
    return {"bytes": kv + io + 4 * (c["prefix"] + rest) / c["bs"] + 4 * c["B"],
            "flops": 4 * c["Hq"] * c["D"] * (live * c["prefix"] + rest)}


# ---- the definitions in 64 bits -------------------------------------------------


def _exact_rows(x, w, eps, positions, inv_freq, interleaved):
    """Norm and rotation as complex products, in double."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + eps) * w.double()
    R = 2 * inv_freq.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       torch.outer(positions.double(), inv_freq.double()))[:, None]
    y = x.clone()
    if interleaved:
        y[..., :R] = torch.view_as_real(torch.view_as_complex(x[..., :R].unflatten(-1, (-1, 2)).contiguous()) * turn
                                        ).flatten(-2)
    else:
        z = torch.complex(x[..., : R // 2], x[..., R // 2: R]) * turn
        y[..., : R // 2], y[..., R // 2: R] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm_rope":
        return {n: _exact_rows(s[n], s[n + "w"], s["eps"], s["positions"], s["inv_freq"], s["interleaved"])
                for n in ("q", "k")}
    if s["op"] == "append":
        bs = s["k_cache"].shape[2]
        k = _exact_rows(s["k"], s["kw"], s["eps"], s["positions"], s["inv_freq"], s["interleaved"]) / s["k_scale"]
        v = s["v"].double() / s["v_scale"]
        out = {}
        ids, pos = s["seq_ids"].cpu(), s["positions"].cpu()
        t = torch.arange(len(ids))[ids >= 0]
        block = s["tables"].cpu()[ids[t].long(), torch.div(pos[t], bs, rounding_mode="floor").long()].long()
        flat = (block * bs + pos[t] % bs).to(k.device)
        for name, rows in (("k_cache", k), ("v_cache", v)):
            c = s[name].to(torch.float32).double().transpose(1, 2)  # block, slot, head, d
            d = c.reshape(-1, *c.shape[2:]).clone()
            d[flat] = rows[t.to(k.device)]
            out[name] = d.view(c.shape).transpose(1, 2).contiguous()
        if s["q"] is not None:
            out["q"] = _exact_rows(s["q"], s["qw"], s["eps"], s["positions"], s["inv_freq"], s["interleaved"])
        return out
    # each sequence by itself, over its own tokens in order
    q, bs = s["q"].double(), s["k_cache"].shape[2]
    B, Hq, D = q.shape
    Hkv = s["k_cache"].shape[1]
    out = torch.zeros_like(q)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    n = s["shared"].numel()

    def tokens(cache, table, scale):
        return cache[table.long()].to(torch.float32).double().transpose(0, 1).flatten(1, 2) * scale

    kp, vp = tokens(s["k_cache"], s["shared"], s["k_scale"]), tokens(s["v_cache"], s["shared"], s["v_scale"])
    for b, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        tail = s["tables"][b, n: -(-L // bs)]
        k = torch.cat([kp, tokens(s["k_cache"], tail, s["k_scale"])], 1)[:, :L]
        v = torch.cat([vp, tokens(s["v_cache"], tail, s["v_scale"])], 1)[:, :L]
        x = torch.einsum("hgd,htd->hgt", q[b].view(Hkv, -1, D), k) * s["scale"]
        lse[b] = torch.logsumexp(x, -1).flatten()
        out[b] = torch.einsum("hgt,htd->hgd", torch.softmax(x, -1), v).reshape(Hq, D)
    return {"out": out, "lse": lse}
