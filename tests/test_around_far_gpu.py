"""The calls around the decode where offsets pass 32 bits: pages at the end of a cache of
more than 2^32 elements, rows that lie 2^31 elements apart."""
import pytest
import torch

import paged_kv_attention_partition_b200 as pad
from operators_ref import Batch, check, close_bf16, norm_rope, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nhd", [False, True])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_pages_at_the_end_of_a_long_cache(cuda_device, kv, nhd):
    # 262207 pages of 16384 elements: the last ones start behind 2^32
    B, Hq, Hkv, D, bs, n = 5, 32, 8, 128, 16, 6
    NB = (1 << 18) + 63
    batch = Batch(B, Hq, Hkv, D, bs, n, [0, 3, 16, 40, 7], kv=kv, seed=51, spare=None)
    used = batch.k.shape[0]
    far = NB - used
    a = batch.device(cuda_device)
    for name in ("k_cache", "v_cache"):
        shape = (NB, bs, Hkv, D) if nhd else (NB, Hkv, bs, D)
        c = torch.empty(shape, dtype=a[name].dtype, device=cuda_device)
        c = c.transpose(1, 2) if nhd else c
        c[far:] = a[name]
        a[name] = c
    a["shared_table"] = a["shared_table"] + far
    a["block_tables"] = torch.where(a["block_tables"] < used, a["block_tables"] + far, a["block_tables"])
    out, lse = pad.pad_decode_shared(**a, lse=True)
    check(out, lse, batch.reference(), "far pages")

    # the next token of each sequence, where the append puts it
    gen = torch.Generator().manual_seed(52)
    k, v = (rand(gen, B, Hkv, D).to(torch.bfloat16) for _ in range(2))
    at = torch.tensor([0, 1, 15, 3, 7], dtype=torch.int32, device=cuda_device)  # slots of the last page
    page = torch.tensor([[NB - 1 - i] for i in range(B)], dtype=torch.int32, device=cuda_device)
    scales = {s: a[s] for s in ("k_scale", "v_scale") if s in a}
    pad.pad_append_kv(k.to(cuda_device), v.to(cuda_device), at, page, a["k_cache"], a["v_cache"], **scales)
    for x, name, s in ((k, "k_cache", scales.get("k_scale", 1.0)), (v, "v_cache", scales.get("v_scale", 1.0))):
        got = torch.stack([a[name][NB - 1 - i, :, int(at[i])] for i in range(B)]).cpu()
        want = x if kv == "bf16" else (x.float() / torch.tensor(s)).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), name
    assert pad.pad_check_device_errors() == 0


def test_rows_far_apart(cuda_device):
    # three tokens 2^31 + 64 elements apart, in and out
    T, H, D, step = 3, 5, 128, (1 << 31) + 64
    gen = torch.Generator().manual_seed(53)
    x = rand(gen, T, H, D).to(torch.bfloat16)
    room = torch.empty(2 * step + H * D, dtype=torch.bfloat16, device=cuda_device)
    q = room.as_strided((T, H, D), (step, D, 1))
    q.copy_(x)
    w = (1 + 0.1 * rand(gen, D)).to(torch.bfloat16)
    f = torch.rand(D // 2, generator=gen)
    pos = torch.tensor([0, 77, 1 << 20], dtype=torch.int32)
    d = lambda t: t.to(cuda_device)
    ref, mag = norm_rope(x, w, 1e-6, pos, f, False)
    out, _ = pad.pad_qk_norm_rope(q, None, d(w), None, d(pos), d(f))
    close_bf16(out, ref, mag, "from afar")
    pad.pad_qk_norm_rope(q, None, d(w), None, d(pos), d(f), q_out=q)
    close_bf16(q, ref, mag, "in place")
    # the same tokens' K and V, far apart too
    kc, vc = (torch.zeros(1, H, 4, D, dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    zero = torch.zeros(T, dtype=torch.int32, device=cuda_device)
    pad.pad_append_kv(q, q, torch.arange(T, dtype=torch.int32, device=cuda_device), zero[:1].view(1, 1), kc, vc, seq_ids=zero)
    assert torch.equal(kc[0, :, :T].transpose(0, 1), q) and torch.equal(vc[0, :, :T].transpose(0, 1), q)
    assert pad.pad_check_device_errors() == 0
