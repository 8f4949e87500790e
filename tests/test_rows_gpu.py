"""pad_qk_norm_rope and pad_append_kv on the GPU against their definitions in
64 bits: head layouts, partial and interleaved rotation, far positions, strides,
padding, refused places, both caches; and the decode that reads what was put."""
import math

import pytest
import torch

import paged_kv_attention_partition_b200 as pad
from operators_ref import close_bf16, close_e4m3, norm_rope, rand

pytestmark = pytest.mark.gpu

EPS = 1e-5


def inv_freq(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()


def heads(gen, T, H, D):
    return (rand(gen, T, H, D) * torch.exp(rand(gen, 1, 1, D))).to(torch.bfloat16)


NORM_CASES = [
    # T, Hq, Hkv, D, rot, interleaved, first position, weights
    (1, 32, 8, 128, 128, False, 0, "bf16"),
    (1, 1, 1, 64, 64, False, 7, "bf16"),
    (3, 40, 8, 128, 128, False, 8191, "f32"),
    (17, 5, 3, 128, 64, False, 100, "bf16"),
    (9, 16, 4, 256, 64, True, 1000000, "bf16"),
    (33, 7, 1, 64, 16, True, 50, "f32"),
    (5, 3, 2, 256, 256, False, 2**31 - 5, "bf16"),
    (4, 8, 2, 128, 96, False, -3, None),
    (1025, 4, 2, 128, 128, True, 12345, None),
    (300, 33, 5, 64, 0, False, 0, "bf16"),
    (2500, 40, 8, 128, 128, False, 3, "bf16"),
]


@pytest.mark.parametrize("case", NORM_CASES, ids=["-".join(map(str, c)) for c in NORM_CASES])
def test_norm_rope_matches_the_definition(cuda_device, case):
    T, Hq, Hkv, D, rot, inter, first, weights = case
    gen = torch.Generator().manual_seed(T + D)
    q, k = heads(gen, T, Hq, D), heads(gen, T, Hkv, D)
    wt = {"bf16": torch.bfloat16, "f32": torch.float32, None: None}[weights]
    qw, kw = (None, None) if wt is None else ((1 + 0.3 * rand(gen, D)).to(wt), (1 + 0.3 * rand(gen, D)).to(wt))
    pos = (torch.arange(T) + first).to(torch.int32) if rot else None
    f = inv_freq(rot) if rot else None
    d = lambda t: None if t is None else t.to(cuda_device)
    qo, ko = pad.pad_qk_norm_rope(d(q), d(k), d(qw), d(kw), d(pos), d(f), eps=EPS, interleaved=inter)
    for got, x, w, name in ((qo, q, qw, "q"), (ko, k, kw, "k")):
        ref, mag = norm_rope(x, w, EPS, pos, f, inter)
        close_bf16(got, ref, mag, name)


def test_norm_rope_in_place_on_slices_of_a_projection(cuda_device):
    # q and k as slices of one projection, written back in place: v's columns
    # and a token behind the slice stay as they were
    gen = torch.Generator().manual_seed(3)
    T, Hq, Hkv, D = 37, 10, 2, 128
    qkv = heads(gen, T + 1, Hq + 2 * Hkv, D).to(cuda_device)
    before = qkv.clone()
    w, f = torch.ones(D, dtype=torch.bfloat16, device=cuda_device), inv_freq(D).to(cuda_device)
    pos = torch.arange(T, dtype=torch.int32, device=cuda_device)
    q, k = qkv[:T, :Hq], qkv[:T, Hq:Hq + Hkv]
    pad.pad_qk_norm_rope(q, k, w, w, pos, f, eps=EPS, q_out=q, k_out=k)
    ref, mag = norm_rope(before[:T, :Hq + Hkv].cpu(), torch.ones(D), EPS, pos.cpu(), f.cpu(), False)
    close_bf16(qkv[:T, :Hq + Hkv], ref, mag)
    assert torch.equal(qkv[:T, Hq + Hkv:], before[:T, Hq + Hkv:]) and torch.equal(qkv[T], before[T])
    # q alone, into a layout with heads outermost
    out = torch.full((Hq, T, D), 7.0, dtype=torch.bfloat16, device=cuda_device).transpose(0, 1)
    got, none = pad.pad_qk_norm_rope(before[:T, :Hq], None, w, None, pos, f, eps=EPS, q_out=out)
    assert none is None and got is out
    close_bf16(out, ref[:, :Hq], mag[:, :Hq])


def test_norm_rope_rows_of_zeros_and_non_finite_rows(cuda_device):
    # a zero row under eps = 0 is 0 * inf = NaN in its own row only; infinities
    # and NaN stay in their rows
    x = torch.ones(4, 6, 128, dtype=torch.bfloat16)
    x[1, 2], x[2, 3, 5], x[3, 1, 100] = 0, float("inf"), float("nan")
    w = torch.ones(128, dtype=torch.bfloat16, device=cuda_device)
    out, _ = pad.pad_qk_norm_rope(x.to(cuda_device), None, w, eps=0.0)
    ref, _ = norm_rope(x, torch.ones(128), 0.0, None, None, False)
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(ref.to(torch.bfloat16)))
    fine = ~torch.isnan(ref)
    assert torch.equal(out.cpu()[fine], ref.to(torch.bfloat16)[fine])
    out, _ = pad.pad_qk_norm_rope(x.to(cuda_device), None, w, eps=1e-6)
    assert torch.equal(out[1, 2].cpu(), torch.zeros(128, dtype=torch.bfloat16))


class Put:
    """Tokens of a ragged batch and the cache they go to, NaN-free and distinct."""

    def __init__(self, B, counts, Hq, Hkv, D, bs, kv, seed, ctx, padding=0, shuffle=False):
        gen = torch.Generator().manual_seed(seed)
        seq = torch.cat([torch.full((n,), b) for b, n in enumerate(counts)] + [torch.full((padding,), -1)]).long()
        start = torch.randint(0, ctx + 1, (B,), generator=gen)
        pos = torch.cat([start[b] + torch.arange(n) for b, n in enumerate(counts)] + [torch.arange(padding)]).long()
        if shuffle:
            p = torch.randperm(len(seq), generator=gen)
            seq, pos = seq[p], pos[p]
        self.seq, self.pos, T = seq, pos, len(seq)
        self.W = (ctx + max(counts)) // bs + 1
        self.tables = torch.randperm(B * self.W + 3, generator=gen)[: B * self.W].view(B, self.W).to(torch.int32)
        self.k, self.v, self.q = heads(gen, T, Hkv, D), heads(gen, T, Hkv, D), heads(gen, T, max(Hq, 1), D)
        self.kv, self.bs, self.Hq = kv, bs, Hq
        self.scales = (0.05, 0.037) if kv == "e4m3" else (1.0, 1.0)
        dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
        shape = (B * self.W + 3, Hkv, bs, D)
        self.kc, self.vc = (rand(gen, *shape).to(dt) for _ in range(2))
        self.qw, self.kw = ((1 + 0.3 * rand(gen, D)).to(torch.bfloat16) for _ in range(2))

    def places(self):
        t = (self.seq >= 0).nonzero()[:, 0]
        return t, self.tables[self.seq[t], self.pos[t] // self.bs].long(), self.pos[t] % self.bs


def rest_untouched(after, before, block, slot):
    seen = torch.zeros(after.shape[0], after.shape[2], dtype=torch.bool)
    seen[block, slot] = True
    bits = torch.int16 if after.dtype == torch.bfloat16 else torch.uint8
    a, b = after.cpu().view(bits).transpose(1, 2), before.view(bits).transpose(1, 2)
    return torch.equal(a[~seen], b[~seen])


APPEND_CASES = [
    # counts, Hq, Hkv, D, bs, rot, interleaved, padding, norm, nhd
    ([1] * 5, 40, 8, 128, 16, 128, False, 0, True, False),
    ([1], 0, 1, 64, 1, 64, False, 0, False, False),
    ([3, 0, 17, 1], 8, 2, 128, 16, 64, False, 4, True, True),
    ([33, 65], 0, 4, 256, 32, 32, True, 3, False, False),
    ([200, 1, 1, 77], 5, 1, 64, 256, 0, False, 0, True, False),
    ([700, 800, 1100], 32, 8, 128, 16, 128, False, 11, True, False),
    ([2] * 100, 16, 4, 256, 8, 256, False, 1, False, True),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", APPEND_CASES, ids=["-".join(map(str, [sum(c[0]), *c[1:]])) for c in APPEND_CASES])
def test_append_matches_the_definition(cuda_device, case, kv):
    counts, Hq, Hkv, D, bs, rot, inter, padding, norm, nhd = case
    p = Put(len(counts), counts, Hq, Hkv, D, bs, kv, seed=sum(counts) + D, ctx=3 * bs + 2, padding=padding,
            shuffle=True)
    f = inv_freq(rot) if rot else None
    d = lambda t: None if t is None else t.to(cuda_device)
    kc, vc = (d(c.transpose(1, 2).contiguous()).transpose(1, 2) if nhd else d(c) for c in (p.kc, p.vc))
    q_out = pad.pad_append_kv(d(p.k), d(p.v), d(p.pos.int()), d(p.tables), kc, vc, seq_ids=d(p.seq.int()), inv_freq=d(f),
                              interleaved=inter, k_weight=d(p.kw) if norm else None, eps=EPS,
                              q=d(p.q) if Hq else None, q_weight=d(p.qw) if norm and Hq else None,
                              **(dict(k_scale=p.scales[0], v_scale=p.scales[1]) if kv == "e4m3" else {}))
    t, block, slot = p.places()
    for name, cache, before, x, w, freq, scale in (("k", kc, p.kc, p.k, p.kw if norm else None, f, p.scales[0]),
                                                   ("v", vc, p.vc, p.v, None, None, p.scales[1])):
        ref, mag = norm_rope(x[t], w, EPS, p.pos[t], freq, inter)
        got = cache.cpu()[block, :, slot]
        if kv == "bf16":
            close_bf16(got, ref, mag, name)
            assert name == "k" or torch.equal(got, p.v[t])  # V is copied bit for bit
        else:
            close_e4m3(got, ref, mag, scale, name)
        assert rest_untouched(cache, before, block, slot), name
    if Hq:
        ref, mag = norm_rope(p.q, p.qw if norm else None, EPS, p.pos, f, inter)
        close_bf16(q_out, ref, mag, "q")
    assert pad.pad_check_device_errors() == 0


def test_append_step_without_seq_ids(cuda_device):
    p = Put(6, [1] * 6, 0, 2, 128, 16, "bf16", seed=1, ctx=40)
    d = lambda t: t.to(cuda_device)
    kc, vc = d(p.kc), d(p.vc)
    assert pad.pad_append_kv(d(p.k), d(p.v), d(p.pos.int()), d(p.tables), kc, vc) is None
    t, block, slot = p.places()
    assert torch.equal(kc.cpu()[block, :, slot], p.k) and torch.equal(vc.cpu()[block, :, slot], p.v)


def test_append_e4m3_edges(cuda_device):
    # saturation, ties to even, subnormals, signed zeros, NaN, infinities
    vals = [448.0, 464.0, 480.0, 1e6, -1e6, float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 2.0**-9, 2.0**-10,
            1.5 * 2.0**-10, 2.0**-11, 17.0, 19.0, 18.0, -17.0, 240.0, 248.0]
    row = torch.zeros(64)
    row[: len(vals)] = torch.tensor(vals)
    k = row.to(torch.bfloat16).view(1, 1, 64).to(cuda_device)
    for scale in (1.0, 0.25):
        kc = torch.zeros(1, 1, 1, 64, dtype=torch.float8_e4m3fn, device=cuda_device)
        vc = torch.zeros_like(kc)
        zero = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        pad.pad_append_kv(k, k, zero, zero.view(1, 1), kc, vc, k_scale=scale, v_scale=scale)
        want = (k.float().cpu() / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        for c in (kc, vc):
            got = c.cpu().view(-1).float()
            assert torch.equal(got.isnan(), want.view(-1).float().isnan())
            assert torch.equal(got.nan_to_num(1.0), want.view(-1).float().nan_to_num(1.0))
            num = ~got.isnan()  # (a NaN code's sign is not specified)
            assert torch.equal(torch.signbit(got)[num], torch.signbit(want.view(-1).float())[num])


@pytest.mark.parametrize("scale", [1.0, 0.03125, 3.0 / 64, 0.7, 1e-3, 2.0 ** -100, 2.0 ** 100])
def test_append_e4m3_codes_of_every_bf16(cuda_device, scale):
    # the fp32 quotient rounded once, code for code
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    k = bits.view(torch.bfloat16).view(64, 8, 128)
    kc = torch.zeros(4, 8, 16, 128, dtype=torch.float8_e4m3fn, device=cuda_device)
    vc = torch.zeros_like(kc)
    pos = torch.arange(64, dtype=torch.int32, device=cuda_device)
    tables = torch.arange(4, dtype=torch.int32, device=cuda_device).view(1, 4)
    d = k.to(cuda_device)
    pad.pad_append_kv(d, d, pos, tables, kc, vc, seq_ids=torch.zeros_like(pos), k_scale=scale, v_scale=scale)
    s = torch.tensor(scale, dtype=torch.float32)
    want = (k.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).transpose(0, 1).reshape(8, 4, 16, 128).transpose(0, 1)
    num = ~want.float().isnan()
    for c in (kc.cpu(), vc.cpu()):
        assert torch.equal(c.float().isnan(), ~num)
        assert torch.equal(c.view(torch.uint8)[num], want.contiguous().view(torch.uint8)[num])


def test_norm_rope_of_the_largest_values(cuda_device):
    # the sum of squares passes fp32's range: rows of zeros, as rsqrt(inf) gives, not NaN
    q = torch.full((3, 4, 128), 3e38, dtype=torch.bfloat16, device=cuda_device)
    q[1] *= -1
    w = torch.full((128,), 8.0, device=cuda_device)
    pos = torch.tensor([0, 5, 1 << 30], dtype=torch.int32, device=cuda_device)
    f = torch.rand(64, generator=torch.Generator().manual_seed(0)).to(cuda_device)
    for inter in (False, True):
        out, _ = pad.pad_qk_norm_rope(q, None, w, None, pos, f, interleaved=inter)
        assert bool((out == 0).all())


def test_append_refuses_bad_places_token_by_token(cuda_device):
    # a position outside the table, a sequence that is not there, a block that is
    # not there: flagged and not written; every other token is
    gen = torch.Generator().manual_seed(5)
    B, W, bs, T = 3, 2, 16, 8
    k = heads(gen, T, 2, 128).to(cuda_device)
    tables = torch.tensor([[0, 1], [2, 99], [-5, 3]], dtype=torch.int32, device=cuda_device)
    for seq, pos, bits in (([0, 1, 2, 0], [32, 3, 20, 1], 0x2), ([0, 1, 2, 0], [-1, 3, 20, 1], 0x2),
                           ([3, 1, 2, 0], [0, 3, 20, 1], 0x1), ([1, 1, 2, 0], [16, 3, 20, 1], 0x1),
                           ([2, 1, 2, 0], [0, 3, 20, 1], 0x1)):
        kc = torch.zeros(5, 2, bs, 128, dtype=torch.bfloat16, device=cuda_device)
        vc = torch.zeros_like(kc)
        ids = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
        pad.pad_append_kv(k[:4], k[4:], ids(pos), tables, kc, vc, seq_ids=ids(seq))
        assert pad.pad_check_device_errors() == bits
        want = torch.zeros_like(kc)
        for t in (1, 2, 3):
            want[int(tables[seq[t], pos[t] // bs]), :, pos[t] % bs] = k[t]
        assert torch.equal(kc, want)


def test_append_then_decode(cuda_device):
    # prefill a ragged batch, then three decode steps, each one append (queries
    # beside it) and one decode: attention over exactly the tokens put so far
    gen = torch.Generator().manual_seed(11)
    B, Hq, Hkv, D, bs, W = 3, 8, 2, 128, 16, 6
    f, w = inv_freq(D).to(cuda_device), torch.ones(D, dtype=torch.bfloat16, device=cuda_device)
    tables = torch.randperm(B * W, generator=gen).view(B, W).to(torch.int32).to(cuda_device)
    for kv in (torch.bfloat16, torch.float8_e4m3fn):
        sc = dict(k_scale=0.03, v_scale=0.02) if kv != torch.bfloat16 else {}
        kc = torch.zeros(B * W, Hkv, bs, D, device=cuda_device).to(kv)
        vc = torch.zeros(B * W, Hkv, bs, D, device=cuda_device).to(kv)
        lens = [15, 1, 40]
        prompt = [heads(gen, n, 2 * Hkv, D) for n in lens]
        x = torch.cat(prompt).to(cuda_device)
        seq = torch.repeat_interleave(torch.arange(B), torch.tensor(lens)).int().to(cuda_device)
        pos = torch.cat([torch.arange(n) for n in lens]).int().to(cuda_device)
        pad.pad_append_kv(x[:, :Hkv], x[:, Hkv:], pos, tables, kc, vc, seq_ids=seq, inv_freq=f, k_weight=w, eps=EPS, **sc)
        ks = [norm_rope(p[:, :Hkv], torch.ones(D), EPS, torch.arange(n), f.cpu(), False)[0]
              for p, n in zip(prompt, lens)]
        vs = [p[:, Hkv:].double() for p in prompt]
        for _ in range(3):
            step = heads(gen, B, Hq + 2 * Hkv, D)
            xs, at = step.to(cuda_device), torch.tensor(lens, dtype=torch.int32)
            q = pad.pad_append_kv(xs[:, Hq:Hq + Hkv], xs[:, Hq + Hkv:], at.to(cuda_device), tables, kc, vc, inv_freq=f,
                                  k_weight=w, eps=EPS, q=xs[:, :Hq], q_weight=w, **sc)
            out, lse = pad.pad_decode(q, kc, vc, tables, (at + 1).to(cuda_device), 1 / math.sqrt(D), lse=True, **sc)
            kn = norm_rope(step[:, Hq:Hq + Hkv], torch.ones(D), EPS, at, f.cpu(), False)[0]
            qn = norm_rope(step[:, :Hq], torch.ones(D), EPS, at, f.cpu(), False)[0]
            for b in range(B):
                ks[b], vs[b] = torch.cat([ks[b], kn[b:b + 1]]), torch.cat([vs[b], step[b:b + 1, Hq + Hkv:].double()])
                lens[b] += 1
                for h in range(Hq):
                    k, v = ks[b][:, h // (Hq // Hkv)], vs[b][:, h // (Hq // Hkv)]
                    s = k @ qn[b, h] / math.sqrt(D)
                    e = torch.softmax(s, 0)
                    # q and every held row are off by half a step of their type: a score by u = (2^-8 + h) of
                    # sum |q k| scale, a weight by e^(2u) - 1, out by that and h of sum w |v|, and its own rounding
                    hk = 2.0 ** -8 if not sc else 2.0 ** -4
                    u = float(((k.abs() + (2.0**-10 * 0.03 / hk if sc else 0)) @ qn[b, h].abs()).max()) \
                        * (2.0 ** -8 + hk) / math.sqrt(D)
                    mag = e @ (v.abs() + (2.0**-10 * 0.02 / hk if sc else 0))
                    tol = mag * (math.expm1(2 * u) + hk * math.exp(2 * u) + 2.0 ** -7) + 2.0 ** -8 * (e @ v).abs()
                    assert ((out[b, h].double().cpu() - e @ v).abs() <= tol).all(), (kv, b, h)
                    assert abs(float(lse[b, h]) - float(torch.logsumexp(s, 0))) <= u + 1e-4
        assert pad.pad_check_device_errors() == 0


def test_rows_captured_and_replayed_with_new_inputs(cuda_device):
    gen = torch.Generator().manual_seed(7)
    p = Put(4, [1] * 4, 8, 2, 128, 16, "bf16", seed=2, ctx=30)
    d = lambda t: t.to(cuda_device)
    k, v, q, pos, tables, f = d(p.k), d(p.v), d(p.q), d(p.pos.int()), d(p.tables), d(inv_freq(128))
    kc, vc = d(p.kc), d(p.vc)
    q_out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # the first call of all: nothing to set up
        pad.pad_append_kv(k, v, pos, tables, kc, vc, inv_freq=f, q=q, q_out=q_out)
    for _ in range(2):
        k.copy_(heads(gen, 4, 2, 128))
        q.copy_(heads(gen, 4, 8, 128))
        pos.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        ref, mag = norm_rope(k.cpu(), None, 0, pos.cpu(), f.cpu(), False)
        at = pos.cpu().long()
        close_bf16(kc.cpu()[p.tables[torch.arange(4), at // 16].long(), :, at % 16], ref, mag)
        close_bf16(q_out, *norm_rope(q.cpu(), None, 0, pos.cpu(), f.cpu(), False))


def test_rows_on_another_stream(cuda_device):
    gen = torch.Generator().manual_seed(9)
    x = heads(gen, 3000, 12, 128).to(cuda_device)
    pos, f = torch.arange(3000, dtype=torch.int32, device=cuda_device), inv_freq(128).to(cuda_device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, _ = pad.pad_qk_norm_rope(x, None, None, None, pos, f, stream=side)
    with torch.cuda.stream(side):
        b, _ = pad.pad_qk_norm_rope(x, None, None, None, pos, f)
    side.synchronize()
    c, _ = pad.pad_qk_norm_rope(x, None, None, None, pos, f)
    assert torch.equal(a, c) and torch.equal(b, c)


def test_rows_without_tokens(cuda_device):
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=cuda_device)
    none = torch.empty(0, dtype=torch.int32, device=cuda_device)
    q, k = pad.pad_qk_norm_rope(e(0, 4, 128), e(0, 2, 128), None, None, none, inv_freq(128).to(cuda_device))
    assert q.shape == (0, 4, 128) and k.shape == (0, 2, 128)
    kc = torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16, device=cuda_device)
    assert pad.pad_append_kv(e(0, 2, 128), e(0, 2, 128), none, torch.zeros(1, 1, dtype=torch.int32, device=cuda_device),
                             kc, kc.clone(), seq_ids=none) is None
