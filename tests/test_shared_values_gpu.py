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
