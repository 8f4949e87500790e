"""pad_decode_shared at values where a type's range ends: scales of zero and near
it, query rows at both ends of bf16, scores that are not numbers, weights far below
the largest, a maximum that rises with every chunk."""
import math

import pytest
import torch

import paged_kv_attention_partition_b200 as pad
from operators_ref import Batch, check, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.2, 1e-30, -1e-40, 1e-44])
def test_scales_of_either_sign_down_to_zero(cuda_device, scale, kv):
    # prefix and rests end inside a chunk: masked scores beside the live ones
    batch = Batch(3, 8, 2, 128, 16, 10, [0, 3, 200], kv=kv, seed=8)
    batch.scale = scale
    out, lse = pad.pad_decode_shared(**batch.device(cuda_device), lse=True)
    check(out, lse, batch.reference(), str(scale))
    assert pad.pad_check_device_errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("power", [-118, -112, 112, 118])
def test_query_rows_at_the_ends_of_bf16(cuda_device, kv, power):
    # rows of 2^power under a scale of 2^-power; one of zeros, and one far smaller than the rest
    batch = Batch(6, 8, 2, 128, 16, 9, [0, 1, 63, 64, 65, 200], kv=kv, seed=25)
    batch.q = (batch.q.float().clamp(-3.5, 3.5) * 2.0 ** power).to(torch.bfloat16)
    batch.q[2, 3] = 0
    batch.q[4, 1] = 2.0 ** min(power, -100)
    batch.scale *= 2.0 ** -power
    out, lse = pad.pad_decode_shared(**batch.device(cuda_device), lse=True)
    check(out, lse, batch.reference(), str(power))
    assert pad.pad_check_device_errors() == 0


@pytest.mark.parametrize("sink", [None, 0.5])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_scores_that_are_not_numbers(cuda_device, kv, sink):
    # from a query row (every score), or from one live token's K (one score): that
    # row's out and lse are NaN, every other row is what it was
    batch = Batch(7, 8, 2, 128, 16, 12, [9, 0, 100, 64, 1, 5, 30], kv=kv, seed=31, empty=(5,))
    sinks = None if sink is None else torch.full((8,), sink)
    ref = batch.reference(sinks)
    bad = torch.zeros(7, 8, dtype=torch.bool)
    for b, h in ((0, 0), (1, 2), (4, 7)):
        batch.q[b, h, 3] = float("nan")
        bad[b, h] = True
    batch.k[int(batch.tables[2, 12 + 5]), 1, 7, 11] = float("nan")  # token 192 + 87 of sequence 2, KV head 1
    bad[2, 4:] = True
    batch.q[5, 1] = float("nan")  # a padding row is not read
    out, lse = pad.pad_decode_shared(**batch.device(cuda_device), lse=True,
                                     sinks=None if sinks is None else sinks.to(cuda_device))
    on = bad.to(cuda_device)
    assert bool(out[on].isnan().all()) and bool(lse[on].isnan().all())
    out[on], ref[0][bad] = 0, 0
    lse[on], ref[1][bad] = 0, 0
    check(out, lse, ref, "other rows")
    assert pad.pad_check_device_errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D, B", [(64, 600), (256, 300)])
def test_one_token_before_a_hundred_thousand_others(cuda_device, D, B, kv):
    # The first token's score is e ln 2 and its value 0; N others have score 0 and value 1:
    # out = N 2^-e / (1 + N 2^-e).  Units of that whole prefix (more row blocks than CTAs), so
    # that one running maximum serves every weight.
    H, bs, n = 64, 256, 512
    N = n * bs - 1
    dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    kc = torch.zeros(2, H, bs, D)
    vc = torch.ones(2, H, bs, D)
    kc[0, :, 0, 0], vc[0, :, 0] = 8.0, 0.0
    q = rand(torch.Generator().manual_seed(1), B, H, D).to(torch.bfloat16)
    q[..., 0] = (math.log(2) * (16 + torch.arange(H) * 18 / H)).to(torch.bfloat16)  # e of 16 to 34
    d = lambda t: t.to(cuda_device)
    shared = torch.ones(n, dtype=torch.int32)
    shared[0] = 0
    tables = torch.zeros(1, n, dtype=torch.int32).expand(B, n)
    out, lse = pad.pad_decode_shared(d(q), d(kc.to(dt)), d(vc.to(dt)), d(shared), d(tables),
                                     torch.full((B,), n * bs, dtype=torch.int32, device=cuda_device), 0.125, lse=True)
    s = q[..., 0].double()
    w = N * torch.exp(-s)
    want = w / (1 + w)
    # N like weights: off by half a step of 16 bits (2^-8 bf16; f16 2^-11, or 2^-25 of a fixed point that stands
    # 2^7 above the largest); N / 16 fp32 additions of them (2^-23 each, if cut off); out's half step; exponentials and
    # scores of up to 34 below 2^-16
    tol = want * ((2.0 ** -8 if kv == "bf16" else 2.0 ** -11) + N / 16 * 2.0 ** -23 + 2.0 ** -8 + 2.0 ** -16)
    if kv == "e4m3":
        tol = tol + N * 2.0 ** -32
    err = (out.double().cpu() - want[..., None]).abs()
    assert (err <= tol[..., None]).all(), float((err / tol[..., None]).max())
    # l: N / 64 additions in fp32, and a logarithm
    assert ((lse.double().cpu() - s - torch.log1p(w)).abs() <= N / 64 * 2.0 ** -24 + 2.0 ** -16).all()
    assert pad.pad_check_device_errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_maximum_that_rises_with_every_chunk(cuda_device, D, kv):
    # the sums so far are rescaled, by 2^-9 and more, before every product but a unit's first
    batch = Batch(5, 8, 2, D, 16, 60, [1, 900, 64, 130, 0], kv=kv, seed=33)
    batch.scale = 1 / 16.0
    batch.q[..., 0] = 8 / (16 * batch.k_scale * batch.scale)
    for pages in [batch.shared] + [row[60:] for row in batch.tables]:
        for i, page in enumerate(pages.long().tolist()):
            if page < batch.k.shape[0]:
                x = batch.k[page, :, :, 0]
                x[~x.isnan()] = 16.0 * (i // 4 % 16)  # 8 more in the score each chunk
    out, lse = pad.pad_decode_shared(**batch.device(cuda_device), lse=True)
    check(out, lse, batch.reference(), "rising")
    assert pad.pad_check_device_errors() == 0
