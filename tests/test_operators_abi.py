"""pad_qk_norm_rope, pad_append_kv and pad_decode_shared without a GPU: every
refusal comes before any device work, with a status and a message; the shared
plan; what the binding refuses by itself."""
import ctypes

import pytest
import torch

import paged_kv_attention_partition_b200 as pad
from paged_kv_attention_partition_b200 import _build

BF, F32, I32, F8 = pad.PAD_BF16, pad.PAD_F32, pad.PAD_I32, pad.PAD_FP8_E4M3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pad.load_library()


def desc(dtype, shape, strides=None, addr=0x100000):
    t = pad.PadTensor()
    t.data, t.dtype, t.ndim = addr, dtype, len(shape)
    acc = 1
    for i in reversed(range(len(shape))):
        t.shape[i] = shape[i]
        t.stride[i] = acc if strides is None else strides[i]
        acc *= shape[i]
    return t


def ref(t):
    return ctypes.addressof(t) if t is not None else None


class AppendOptions(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("interleaved", ctypes.c_int32), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("q", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


def refused(st, want):
    assert st == want and pad.pad_last_error(), (st, pad.pad_last_error())


NORM = dict(q=(BF, (5, 8, 128)), k=(BF, (5, 2, 128)), qw=(BF, (128,)), kw=(F32, (128,)), pos=(I32, (5,)),
            f=(F32, (64,)), qo=(BF, (5, 8, 128)), ko=(BF, (5, 2, 128)))


def call_norm(lib, eps=1e-6, **over):
    a = {n: desc(*v) if v is not None else None for n, v in {**NORM, **over}.items()}
    return lib.pad_qk_norm_rope(ref(a["q"]), ref(a["k"]), ref(a["qw"]), ref(a["kw"]), eps, ref(a["pos"]), ref(a["f"]), 0,
                                ref(a["qo"]), ref(a["ko"]), None)


@pytest.mark.parametrize("over, status", [
    (dict(q=None), pad.PAD_ERR_INVALID_ARG),
    (dict(q=(F32, (5, 8, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(q=(BF, (5, 8, 128, 1))), pad.PAD_ERR_INVALID_ARG),
    (dict(q=(BF, (5, 8, 128), (1024, 128, 2))), pad.PAD_ERR_INVALID_ARG),     # last dim not contiguous
    (dict(q=(BF, (5, 8, 128), (1028, 128, 1))), pad.PAD_ERR_INVALID_ARG),     # rows not 16-byte aligned
    (dict(q=(BF, (5, 8, 128), None, 0x100008)), pad.PAD_ERR_INVALID_ARG),
    (dict(qo=(BF, (5, 7, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(qo=(BF, (5, 8, 128), (0, 128, 1))), pad.PAD_ERR_INVALID_ARG),       # rows on one another
    (dict(qo=(BF, (5, 8, 128), (128, 128, 1))), pad.PAD_ERR_INVALID_ARG),
    (dict(ko=None), pad.PAD_ERR_INVALID_ARG),
    (dict(k=None, ko=None), pad.PAD_ERR_INVALID_ARG),                         # k_weight without k
    (dict(k=(BF, (4, 2, 128)), ko=(BF, (4, 2, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(k=(BF, (5, 2, 64)), ko=(BF, (5, 2, 64))), pad.PAD_ERR_INVALID_ARG),
    (dict(qw=(I32, (128,))), pad.PAD_ERR_INVALID_ARG),
    (dict(qw=(BF, (64,))), pad.PAD_ERR_INVALID_ARG),
    (dict(kw=(F32, (128,), (2,))), pad.PAD_ERR_INVALID_ARG),
    (dict(pos=None), pad.PAD_ERR_INVALID_ARG),
    (dict(pos=(I32, (6,))), pad.PAD_ERR_INVALID_ARG),
    (dict(f=None), pad.PAD_ERR_INVALID_ARG),
    (dict(f=(F32, (65,))), pad.PAD_ERR_INVALID_ARG),                          # more than head_dim / 2
    (dict(f=(F32, (0,))), pad.PAD_ERR_INVALID_ARG),
    (dict(f=(F32, (12,))), pad.PAD_ERR_UNSUPPORTED),                          # not a multiple of 8
    (dict(f=(F32, (8, 1))), pad.PAD_ERR_INVALID_ARG),
    (dict(eps=-1.0), pad.PAD_ERR_INVALID_ARG),
    (dict(eps=float("nan")), pad.PAD_ERR_INVALID_ARG),
    (dict(q=(BF, (5, 8, 96)), k=(BF, (5, 2, 96)), qo=(BF, (5, 8, 96)), ko=(BF, (5, 2, 96))), pad.PAD_ERR_UNSUPPORTED),
    (dict(q=(BF, (5, 65537, 128)), qo=(BF, (5, 65537, 128))), pad.PAD_ERR_UNSUPPORTED),
])
def test_norm_rope_refusals(lib, over, status):
    refused(call_norm(lib, **over), status)


APPEND = dict(k=(BF, (6, 2, 128)), v=(BF, (6, 2, 128)), pos=(I32, (6,)), seq=(I32, (6,)), t=(I32, (3, 4)),
              kc=(BF, (12, 2, 16, 128)), vc=(BF, (12, 2, 16, 128)), f=(F32, (64,)), kw=(BF, (128,)), q=(BF, (6, 8, 128)),
              qw=(BF, (128,)), qo=(BF, (6, 8, 128)))


def call_append(lib, eps=1e-6, ks=0.0, vs=0.0, **over):
    a = {n: desc(*v) if v is not None else None for n, v in {**APPEND, **over}.items()}
    o = AppendOptions(ref(a["f"]), 0, ref(a["kw"]), eps, ref(a["q"]), ref(a["qw"]), ref(a["qo"]), ks, vs)
    return lib.pad_append_kv(ref(a["k"]), ref(a["v"]), ref(a["pos"]), ref(a["seq"]), ref(a["t"]), ctypes.addressof(o),
                             ref(a["kc"]), ref(a["vc"]), None)


@pytest.mark.parametrize("over, status", [
    (dict(k=None), pad.PAD_ERR_INVALID_ARG),
    (dict(v=(BF, (6, 3, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(v=(BF, (5, 2, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(pos=None), pad.PAD_ERR_INVALID_ARG),
    (dict(pos=(I32, (5,))), pad.PAD_ERR_INVALID_ARG),
    (dict(seq=(I32, (7,))), pad.PAD_ERR_INVALID_ARG),
    (dict(seq=None), pad.PAD_ERR_INVALID_ARG),                                # 6 tokens, 3 sequences
    (dict(t=(I32, (3, 4), (8, 2))), pad.PAD_ERR_INVALID_ARG),
    (dict(t=(I32, (3, 0))), pad.PAD_ERR_INVALID_ARG),
    (dict(t=(I32, (3, 4), None, 0x100002)), pad.PAD_ERR_INVALID_ARG),
    (dict(t=(I32, (3, 1 << 28))), pad.PAD_ERR_UNSUPPORTED),
    (dict(kc=(F32, (12, 2, 16, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(kc=(F8, (12, 2, 16, 128))), pad.PAD_ERR_INVALID_ARG),               # V cache of another type
    (dict(kc=(BF, (12, 2, 16, 128), (4096, 2048, 132, 1))), pad.PAD_ERR_INVALID_ARG),
    (dict(kc=(BF, (12, 2, 16, 128), (4096, 0, 128, 1))), pad.PAD_ERR_INVALID_ARG),  # heads on one another
    (dict(kc=(BF, (12, 3, 16, 128)), vc=(BF, (12, 3, 16, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(vc=(BF, (11, 2, 16, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(kc=(BF, (12, 2, 12, 128)), vc=(BF, (12, 2, 12, 128))), pad.PAD_ERR_UNSUPPORTED),
    (dict(kc=(BF, (12, 2, 512, 128)), vc=(BF, (12, 2, 512, 128))), pad.PAD_ERR_UNSUPPORTED),
    (dict(kc=(BF, (0, 2, 16, 128)), vc=(BF, (0, 2, 16, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(qo=None), pad.PAD_ERR_INVALID_ARG),
    (dict(q=None, qo=None), pad.PAD_ERR_INVALID_ARG),                         # q_weight without q
    (dict(q=(BF, (5, 8, 128)), qo=(BF, (5, 8, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(kw=(BF, (127,))), pad.PAD_ERR_INVALID_ARG),
    (dict(f=(F32, (20,))), pad.PAD_ERR_UNSUPPORTED),
    (dict(ks=0.5), pad.PAD_ERR_INVALID_ARG),                                  # scales on a bf16 cache
    (dict(vs=-1.0), pad.PAD_ERR_INVALID_ARG),
    (dict(kc=(F8, (12, 2, 16, 128)), vc=(F8, (12, 2, 16, 128)), ks=float("inf")), pad.PAD_ERR_INVALID_ARG),
    (dict(eps=float("inf")), pad.PAD_ERR_INVALID_ARG),
    (dict(kc=(F8, (12, 2, 16, 128)), vc=(F8, (12, 2, 16, 128)), ks=2.0 ** -101), pad.PAD_ERR_UNSUPPORTED),
    (dict(kc=(F8, (12, 2, 16, 128)), vc=(F8, (12, 2, 16, 128)), vs=2.0 ** 101), pad.PAD_ERR_UNSUPPORTED),
    (dict(kw=(BF, (128,), None, 0x100008)), pad.PAD_ERR_INVALID_ARG),         # a weight off its 16 bytes
    (dict(qw=(F32, (128,), None, 0x100004)), pad.PAD_ERR_INVALID_ARG),
])
def test_append_refusals(lib, over, status):
    refused(call_append(lib, **over), status)


SHARED = dict(q=(BF, (2, 8, 128)), k=(BF, (10, 2, 16, 128)), v=(BF, (10, 2, 16, 128)), s=(I32, (3,)), t=(I32, (2, 5)),
              l=(I32, (2,)), out=(BF, (2, 8, 128)), lse=(F32, (2, 8)))


def call_shared(lib, scale=0.1, opts=None, ws=None, ws_bytes=0, **over):
    a = {n: desc(*v) if v is not None else None for n, v in {**SHARED, **over}.items()}
    return lib.pad_decode_shared(ref(a["q"]), ref(a["k"]), ref(a["v"]), ref(a["s"]), ref(a["t"]), ref(a["l"]), scale,
                                 ctypes.addressof(opts) if opts is not None else None, ref(a["out"]), ref(a["lse"]), ws,
                                 ws_bytes, None)


@pytest.mark.parametrize("over, status", [
    (dict(q=(F32, (2, 8, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(v=(BF, (10, 1, 16, 128))), pad.PAD_ERR_INVALID_ARG),
    (dict(s=None), pad.PAD_ERR_INVALID_ARG),
    (dict(s=(I32, (6,))), pad.PAD_ERR_INVALID_ARG),                           # more pages than a table row
    (dict(s=(I32, (3, 1))), pad.PAD_ERR_INVALID_ARG),
    (dict(s=(F32, (3,))), pad.PAD_ERR_INVALID_ARG),
    (dict(s=(I32, (3,), (2,))), pad.PAD_ERR_INVALID_ARG),
    (dict(s=(I32, (3,), None, 0)), pad.PAD_ERR_INVALID_ARG),
    (dict(t=(I32, (3, 5))), pad.PAD_ERR_INVALID_ARG),
    (dict(l=(I32, (3,))), pad.PAD_ERR_INVALID_ARG),
    (dict(out=(BF, (2, 8, 64))), pad.PAD_ERR_INVALID_ARG),
    (dict(lse=(F32, (2, 9))), pad.PAD_ERR_INVALID_ARG),
    (dict(scale=float("nan")), pad.PAD_ERR_INVALID_ARG),
    (dict(q=(BF, (2, 7, 128)), out=(BF, (2, 7, 128)), lse=(F32, (2, 7))), pad.PAD_ERR_INVALID_ARG),
    (dict(q=(BF, (2, 8, 96)), k=(BF, (10, 2, 16, 96)), v=(BF, (10, 2, 16, 96)), out=(BF, (2, 8, 96))),
     pad.PAD_ERR_UNSUPPORTED),
    (dict(k=(BF, (10, 2, 12, 128)), v=(BF, (10, 2, 12, 128))), pad.PAD_ERR_UNSUPPORTED),
    (dict(q=(BF, (2, 514, 128)), out=(BF, (2, 514, 128)), lse=(F32, (2, 514))), pad.PAD_ERR_UNSUPPORTED),
    (dict(opts=pad.PadOptions(5, None, 0, 0)), pad.PAD_ERR_UNSUPPORTED),      # a window shares no prefix
    (dict(opts=pad.PadOptions(-5, None, 0, 0)), pad.PAD_ERR_INVALID_ARG),
    (dict(opts=pad.PadOptions(0, None, 0.5, 0)), pad.PAD_ERR_INVALID_ARG),
    (dict(opts=pad.PadOptions(0, ctypes.pointer(desc(F32, (7,))), 0, 0)), pad.PAD_ERR_INVALID_ARG),
])
def test_shared_refusals(lib, over, status):
    refused(call_shared(lib, **over), status)


def test_shared_empty_batch_is_a_no_op(lib):
    assert call_shared(lib, q=(BF, (0, 8, 128)), t=(I32, (0, 5)), l=(I32, (0,)), out=(BF, (0, 8, 128)),
                       lse=(F32, (0, 8))) == pad.PAD_OK


def test_shared_plan(lib):
    p = pad.pad_decode_shared_plan(64, 40, 8, 128, 16, 560, 512, device=0)
    # 51 sequences x 5 heads share a pass (two 128-row tiles), 13 the second one
    assert (p["ctas"], p["chunk_tokens"], p["prefix_rows"], p["prefix_blocks"]) == (148, 64, 255, 2)
    # room for the partials of every (row block, KV head) and (sequence, KV head), each cut at
    # most once per CTA: fp32 rows of D + 1
    rows = (8 * 2 + 148) * 255 + (64 * 8 + 148) * 2 * 5
    assert rows * 129 * 4 <= p["workspace_bytes"] <= rows * 129 * 4 + 2 * 256
    # one tile of 128 rows at head_dim 256; a group above the rows is cut into head tiles
    p = pad.pad_decode_shared_plan(40, 16, 4, 256, 16, 100, 9, kv_dtype="e4m3")
    assert (p["chunk_tokens"], p["prefix_rows"], p["prefix_blocks"]) == (64, 128, 2)
    p = pad.pad_decode_shared_plan(3, 200, 1, 256, 16, 100, 9)
    assert (p["prefix_rows"], p["prefix_blocks"]) == (128, 6)
    assert pad.pad_decode_shared_plan(0, 8, 2, 128, 16, 10, 3)["workspace_bytes"] == 0
    # nothing shared: no room for a prefix
    a, b = (pad.pad_decode_shared_plan(8, 8, 2, 128, 16, 10, n)["workspace_bytes"] for n in (0, 1))
    assert a < b
    for bad in ((64, 40, 8, 128, 16, 560, 561), (64, 40, 8, 128, 16, 560, -1), (64, 41, 8, 128, 16, 560, 1)):
        with pytest.raises(pad.PadError) as e:
            pad.pad_decode_shared_plan(*bad)
        assert e.value.status == pad.PAD_ERR_INVALID_ARG
    with pytest.raises(pad.PadError):
        pad.pad_decode_shared_plan(64, 40, 8, 128, 16, 560, 512, kv_dtype="fp4")


def test_the_binding_refuses_what_it_cannot_describe():
    fast = pad._load_fast()
    for f, n in ((fast.qk_norm_rope, 11), (fast.append_kv, 17), (fast.decode_shared, 14)):
        with pytest.raises(TypeError):
            f()
        with pytest.raises(TypeError):
            f(*[None] * n)            # the first tensor is not optional
        with pytest.raises(ValueError):
            f(torch.zeros(1, 4, 128, dtype=torch.bfloat16), *[None] * (n - 1))  # not a CUDA tensor


def test_the_binding_has_no_cpu_path():
    x = torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    c = torch.zeros(1, 4, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pad.pad_qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        pad.pad_append_kv(x, x, i[0], i, c, c)
    with pytest.raises(ValueError):
        pad.pad_decode_shared(x, c, c, i[0], i, i[0], 0.1)
