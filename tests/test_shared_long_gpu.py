"""pad_decode_shared over millions of tokens: one page's tokens again and again, so that
the definition is that page's softmax and the length only shows in the sums.

Where one accumulator took all of it the tensor core's additions, which cut off what
does not fit, lost 1.3 % (and up to 3 %) of the output over 5 million tokens."""
import math

import pytest
import torch

import paged_kv_attention_partition_b200 as pad
from operators_ref import rand

pytestmark = pytest.mark.gpu

BS = 256
PIECE = 65536  # tokens that one accumulator takes


def page(gen, H, D, kv, dev):
    k, v = rand(gen, 1, H, BS, D), rand(gen, 1, H, BS, D) + 2.0  # values of one sign: losses add up
    dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    return k.to(dt).to(dev), v.to(dt).to(dev)


def expect(q, kc, vc, scale, whole, rest=0):
    """out, lse and their tolerances for `whole` repeats of the page and its first
    `rest` tokens; q [B, H, g, D]."""
    s = torch.einsum("bhgd,hsd->bhgs", q.double(), kc[0].to(torch.float32).double()) * scale
    times = torch.full((BS,), float(whole), dtype=torch.float64, device=s.device)
    times[:rest] += 1
    m = s.amax(-1, keepdim=True)
    w = times * torch.exp(s - m)
    z = w.sum(-1, keepdim=True)
    v = vc[0].to(torch.float32).double()
    out = torch.einsum("bhgs,hsd->bhgd", w / z, v)
    mag = torch.einsum("bhgs,hsd->bhgd", w / z, v.abs())
    D = q.shape[-1]
    e_s = (D + 8) * 2.0 ** -24 * torch.einsum("bhgd,hsd->bhgs", q.double().abs(),
                                              kc[0].to(torch.float32).double().abs()).amax(-1, keepdim=True) * scale
    # weights of 16 bits (the same rounding at every repeat), a piece's products added 16 at a time and cut
    # off (2^-23 each), out's half step; scores as in operators_ref
    half = 2.0 ** -8 if kc.dtype == torch.bfloat16 else 2.0 ** -11
    tol = mag * (half + PIECE / 16 * 2.0 ** -23 + 2 * e_s) + out.abs() * 2.0 ** -8
    # a piece's sums of weights: an addition for every chunk of 64, rounded
    lse = (m + torch.log(z))[..., 0]
    return out, lse, tol, e_s[..., 0] + PIECE / 64 * 2.0 ** -24 + 2.0 ** -21 * (1 + lse.abs())


def check(out, lse, want):
    o, l, tol_o, tol_l = want
    assert (((out.double() - o).abs() - tol_o) <= 0).all(), float(((out.double() - o).abs() / tol_o).max())
    assert (((lse.double() - l).abs() - tol_l) <= 0).all(), float(((lse.double() - l).abs() / tol_l).max())
    assert pad.pad_check_device_errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D, B", [(64, 600), (128, 600), (256, 300)])
def test_a_prefix_of_millions(cuda_device, D, B, kv):
    # 64 heads of three row blocks: 1.3 of 192 items per CTA, two tiles of rows each
    H, n = 64, 1 << 13
    gen = torch.Generator().manual_seed(D)
    kc, vc = page(gen, H, D, kv, cuda_device)
    q = rand(gen, B, H, D).to(torch.bfloat16).to(cuda_device)
    zeros = torch.zeros(n, dtype=torch.int32, device=cuda_device)
    lens = torch.full((B,), n * BS, dtype=torch.int32, device=cuda_device)
    lens[B // 2] = 0
    out, lse = pad.pad_decode_shared(q, kc, vc, zeros, zeros.expand(B, n), lens, D ** -0.5, lse=True)
    assert bool((out[B // 2] == 0).all() and torch.isneginf(lse[B // 2]).all())
    some = lens > 0
    o, l, to, tl = expect(q[:, :, None], kc, vc, D ** -0.5, n)
    check(out[some], lse[some], (o[some, :, 0], l[some, :, 0], to[some, :, 0], tl[some, :, 0]))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("g", [4, 160])
def test_sequences_of_millions(cuda_device, D, g, kv):
    # behind an odd number of chunks, ending inside a page; a tile of rows and two (even and odd
    # chunks on an accumulator each, and a tile on each)
    H, n, W = 2, 3, 1 << 16
    gen = torch.Generator().manual_seed(D + g)
    kc, vc = page(gen, H, D, kv, cuda_device)
    q = rand(gen, 3, H * g, D).to(torch.bfloat16).to(cuda_device)
    zeros = torch.zeros(W, dtype=torch.int32, device=cuda_device)
    lens = torch.tensor([W * BS, (W // 2) * BS + 77, n * BS + 1], dtype=torch.int32, device=cuda_device)
    out, lse = pad.pad_decode_shared(q, kc, vc, zeros[:n], zeros.expand(3, W), lens, D ** -0.5, lse=True)
    for b, L in enumerate(lens.tolist()):
        o, l, to, tl = (x.flatten(1, 2) for x in expect(q[b:b + 1].view(1, H, g, D), kc, vc, D ** -0.5, L // BS, L % BS))
        check(out[b:b + 1], lse[b:b + 1], (o, l, to, tl))
