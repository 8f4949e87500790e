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
