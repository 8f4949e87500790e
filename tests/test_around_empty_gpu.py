"""The calls around the decode without tokens or sequences: nothing to do is done, and
a call that is wrong beside an empty tensor is refused like any other (its outputs
would come back as they were allocated)."""
import pytest
import torch

import paged_kv_attention_partition_b200 as pad
from operators_ref import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture
def make(cuda_device):
    def bf16(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16, device=cuda_device)

    def i32(*shape):
        return torch.zeros(*shape, dtype=torch.int32, device=cuda_device)

    return bf16, i32


def refused(call, status=pad.PAD_ERR_INVALID_ARG):
    with pytest.raises(pad.PadError) as e:
        call()
    assert e.value.status == status


def test_rows(make):
    bf16, i32 = make
    q, k = pad.pad_qk_norm_rope(bf16(0, 4, 128), bf16(0, 2, 128), bf16(128), bf16(128))
    assert q.shape == (0, 4, 128) and k.shape == (0, 2, 128)
    refused(lambda: pad.pad_qk_norm_rope(bf16(5, 0, 128), bf16(5, 2, 128)), pad.PAD_ERR_UNSUPPORTED)  # no q heads
    refused(lambda: pad.pad_qk_norm_rope(bf16(5, 4, 128), bf16(5, 0, 128)), pad.PAD_ERR_UNSUPPORTED)
    refused(lambda: pad.pad_qk_norm_rope(bf16(0, 4, 128), bf16(5, 2, 128)))
    refused(lambda: pad.pad_qk_norm_rope(bf16(5, 4, 128), bf16(0, 2, 128)))
    refused(lambda: pad.pad_qk_norm_rope(bf16(0, 4, 128), None, bf16(64)))
    refused(lambda: pad.pad_qk_norm_rope(bf16(0, 4, 128), None, q_out=bf16(3, 4, 128)))
    refused(lambda: pad.pad_qk_norm_rope(bf16(0, 4, 96), None), pad.PAD_ERR_UNSUPPORTED)
    f = torch.zeros(0, device="cuda")
    refused(lambda: pad.pad_qk_norm_rope(bf16(5, 4, 128), None, None, None, i32(5), f))


def test_append(make):
    bf16, i32 = make
    kc, vc = bf16(4, 2, 16, 128), bf16(4, 2, 16, 128)
    put = lambda k, pos, **kw: pad.pad_append_kv(k, k, pos, kw.pop("tables", i32(2, 2)), kw.pop("kc", kc), vc, **kw)
    assert put(bf16(0, 2, 128), i32(0), seq_ids=i32(0)) is None
    assert put(bf16(0, 2, 128), i32(0), seq_ids=i32(0), q=bf16(0, 8, 128)).shape == (0, 8, 128)
    assert put(bf16(0, 2, 128), i32(0), tables=i32(0, 2)) is None  # a step of no sequences
    refused(lambda: put(bf16(0, 2, 128), i32(0), seq_ids=i32(0), q=bf16(4, 8, 128)))  # queries of no token
    refused(lambda: put(bf16(0, 2, 128), i32(0)))                                     # two sequences, no token
    refused(lambda: put(bf16(2, 0, 128), i32(2)), pad.PAD_ERR_UNSUPPORTED)
    refused(lambda: put(bf16(2, 2, 128), i32(0)))
    refused(lambda: put(bf16(0, 2, 128), i32(0), seq_ids=i32(0), kc=bf16(0, 2, 16, 128)))


def test_shared(make, cuda_device):
    bf16, i32 = make
    kc, vc = bf16(4, 2, 16, 128), bf16(4, 2, 16, 128)
    call = lambda q, tables, lens, shared=i32(1), **kw: pad.pad_decode_shared(q, kc, vc, shared, tables, lens, 0.1, **kw)
    out, lse = call(bf16(0, 8, 128), i32(0, 2), i32(0), lse=True)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    assert call(bf16(0, 8, 128), i32(0, 2), i32(0), shared=i32(0))[0].shape == (0, 8, 128)
    refused(lambda: call(bf16(0, 8, 128), i32(3, 2), i32(3)))
    refused(lambda: call(bf16(3, 0, 128), i32(3, 2), i32(3)))
    refused(lambda: call(bf16(0, 8, 128), i32(0, 2), i32(0), out=bf16(2, 8, 128)))
    refused(lambda: call(bf16(0, 8, 128), i32(0, 2), i32(0), shared=i32(3)))
    # a workspace of no bytes is too small, not none
    batch = Batch(3, 8, 2, 128, 16, 4, [20, 33, 7], seed=47)
    empty = torch.empty(0, dtype=torch.uint8, device=cuda_device)
    refused(lambda: pad.pad_decode_shared(**batch.device(cuda_device), workspace=empty))
