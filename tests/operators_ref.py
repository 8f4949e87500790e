"""64-bit definitions and inputs for the tests of pad_qk_norm_rope, pad_append_kv
and pad_decode_shared: plain torch in float64 on the CPU, no library code."""
import math

import torch

F8_MAX = 448.0


def rand(gen, *shape):
    return torch.randn(*shape, generator=gen)


def norm_rope(x, w, eps, positions, inv_freq, interleaved):
    """(value, magnitude): the rows [T, H, D] in float64, and the sum of the
    magnitudes that each element's rotation adds or cancels."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if inv_freq is None:
        return x, x.abs()
    R = 2 * inv_freq.numel()
    a = positions.double()[:, None, None] * inv_freq.double()
    c, s = a.cos(), a.sin()
    y, mag = x.clone(), x.abs().clone()
    i1 = slice(0, R, 2) if interleaved else slice(0, R // 2)
    i2 = slice(1, R, 2) if interleaved else slice(R // 2, R)
    x1, x2 = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    mag[..., i1] = mag[..., i2] = x1.abs() + x2.abs()
    return y, mag


def close_bf16(got, ref, mag, what=""):
    """Half a bf16 step of the value, and the fp32 arithmetic before it: the norm's
    sum of D squares, its rsqrt and the rotation's four operations with a sine and
    cosine of 2 ulp -- under 32 fp32 half-steps (2^-24) of the terms' magnitude."""
    err = (got.double().cpu() - ref).abs()
    tol = ref.abs() * 2.0 ** -8 + mag * 2.0 ** -19 + 1e-37
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err / tol).max()):.3g} of the tolerance"


def close_e4m3(got, ref, mag, scale, what=""):
    """Half an E4M3 step of the value (2^-4 of it, or half a subnormal step 2^-10)
    and the same fp32 arithmetic; beyond the largest code, the largest code."""
    held = (ref / scale).clamp(-F8_MAX, F8_MAX)
    err = (got.float().double().cpu() - held).abs()
    tol = held.abs() * 2.0 ** -4 + 2.0 ** -10 + (mag / scale) * 2.0 ** -19
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err / tol).max()):.3g} of the tolerance"


class Batch:
    """A decode batch behind a shared prefix, on the CPU: the pages of every
    sequence, NaN wherever no live token is (dead slots, unused blocks), garbage in
    the table entries that may not be read."""

    def __init__(self, B, Hq, Hkv, D, bs, n, rests, kv="bf16", seed=0, empty=(), spare=2, k_amp=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.Hq, self.Hkv, self.D, self.bs, self.n, self.kv = Hq, Hkv, D, bs, n, kv
        rests = [int(r) for r in rests]
        assert len(rests) == B
        self.lens = torch.tensor([0 if b in empty else n * bs + r for b, r in enumerate(rests)], dtype=torch.int32)
        own = [-(-r // bs) if b not in empty else 0 for b, r in enumerate(rests)]
        self.W = max(1, n + max(own) + (1 if spare else 0)) if spare is not None else max(1, n + max(own))
        blocks = n + sum(own)
        nb = blocks + (spare or 0) + 1
        perm = torch.randperm(nb, generator=gen)[:blocks].to(torch.int32)
        dead = 1 << 30
        self.shared = perm[:n].clone()
        self.tables = torch.full((B, self.W), dead, dtype=torch.int32)
        at = n
        for b in range(B):
            self.tables[b, n:n + own[b]] = perm[at:at + own[b]]
            at += own[b]
        self.k_scale, self.v_scale = (3.0 / 64, 5.0 / 256) if kv == "e4m3" else (1.0, 1.0)
        self.k, self.v = (self._pool(gen, nb, sc, amp) for sc, amp in ((self.k_scale, k_amp), (self.v_scale, 1.0)))
        live = torch.zeros(nb, bs, dtype=torch.bool)
        live[self.shared.long()] = True
        for b in range(B):
            for t in range(n * bs, int(self.lens[b])):
                live[self.tables[b, t // bs].long(), t % bs] = True
        self.k.transpose(1, 2)[~live] = float("nan")
        self.v.transpose(1, 2)[~live] = float("nan")
        self.q = rand(gen, B, Hq, D).to(torch.bfloat16)
        self.scale = 1 / math.sqrt(D)

    def _pool(self, gen, nb, scale, amp):
        x = rand(gen, nb, self.Hkv, self.bs, self.D) * amp
        if self.kv == "bf16":
            return x.to(torch.bfloat16).float()
        return (x / scale).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn).float()

    def device(self, dev, nhd=False):
        dt = torch.bfloat16 if self.kv == "bf16" else torch.float8_e4m3fn

        def cache(x):
            return x.transpose(1, 2).contiguous().to(dt).to(dev).transpose(1, 2) if nhd else x.to(dt).to(dev)

        return dict(q=self.q.to(dev), k_cache=cache(self.k), v_cache=cache(self.v), shared_table=self.shared.to(dev),
                    block_tables=self.tables.to(dev), seq_lens=self.lens.to(dev), scale=self.scale,
                    **(dict(k_scale=self.k_scale, v_scale=self.v_scale) if self.kv == "e4m3" else {}))

    def rows(self, cache, b, scale):
        """[Hkv, L, D] of sequence b, float64."""
        L, bs = int(self.lens[b]), self.bs
        pages = torch.cat([self.shared, self.tables[b, self.n:]])[: -(-L // bs)].long()
        return cache[pages].double().transpose(0, 1).reshape(self.Hkv, -1, self.D)[:, :L] * scale

    def reference(self, sinks=None):
        """out, lse, and the tolerances of both, elementwise.

        out: every weight is rounded to 16 bits once (2^-8 of it for bf16), which
        moves out by at most 2^-8 of sum w |v|; out itself is rounded once more; the
        fp32 sums, exponentials (2^-22 each) and the merge stay below 2^-12 of sum w |v|
        for these lengths.  A score's error (a dot product of D terms in fp32, and
        the product with the scale) multiplies every weight: (D + 8) 2^-24 of
        scale sum |q k|; lse carries that and an fp32 logarithm's."""
        B, Hq, D = self.q.shape
        g = Hq // self.Hkv
        out = torch.zeros(B, Hq, D, dtype=torch.float64)
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
        tol_out, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
        for b in range(B):
            if int(self.lens[b]) == 0:
                if sinks is not None:
                    lse[b] = sinks.double()
                continue
            k, v = self.rows(self.k, b, self.k_scale), self.rows(self.v, b, self.v_scale)
            for h in range(Hq):
                q = self.q[b, h].double()
                s = k[h // g] @ q * self.scale
                e_s = (D + 8) * 2.0 ** -24 * float((k[h // g].abs() @ q.abs()).max()) * abs(self.scale) + 2.0 ** -21
                m = s.max() if sinks is None else max(s.max(), sinks[h].double())
                w = torch.exp(s - m)
                z = w.sum() + (torch.exp(sinks[h].double() - m) if sinks is not None else 0.0)
                out[b, h] = w @ v[h // g] / z
                lse[b, h] = m + torch.log(z)
                mag = w @ v[h // g].abs() / z
                tol_out[b, h] = mag * (2.0 ** -8 + 2.0 ** -12 + 2 * e_s) + out[b, h].abs() * 2.0 ** -8 + 1e-30
                tol_lse[b, h] = e_s + 2.0 ** -21 * (1 + lse[b, h].abs())
        return out, lse, tol_out, tol_lse


def check(got_out, got_lse, ref, what=""):
    out, lse, tol_out, tol_lse = ref
    got = got_out.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite out"
    err = (got - out).abs()
    assert (err <= tol_out).all(), f"{what}: out {float((err / tol_out.clamp_min(1e-30)).max()):.3g} of the tolerance"
    if got_lse is not None:
        g = got_lse.double().cpu()
        empty = torch.isneginf(lse)
        assert torch.equal(torch.isneginf(g), empty), f"{what}: -inf lse"
        err = (g - lse).abs()[~empty]
        assert (err <= tol_lse[~empty]).all(), f"{what}: lse off by {float(err.max()):.3g}"
