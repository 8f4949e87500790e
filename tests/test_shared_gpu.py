"""pad_decode_shared on the GPU against attention over each sequence's own tokens
in 64 bits: row blocks of every kind, pages that end inside a chunk, prefixes that
many CTAs split, empty rows, both caches; then streams, graphs and bad data."""
import pytest
import torch

import paged_kv_attention_partition_b200 as pad
from operators_ref import Batch, check, norm_rope, rand

pytestmark = pytest.mark.gpu


def run(batch, dev, nhd=False, lse=True, **kw):
    a = batch.device(dev, nhd)
    a["out"] = torch.full(a["q"].shape, float("nan"), dtype=torch.bfloat16, device=dev)
    if lse:
        a["lse"] = torch.full(a["q"].shape[:2], float("nan"), device=dev)
    out, got_lse = pad.pad_decode_shared(**a, **kw)
    torch.cuda.synchronize()
    return out, got_lse


CASES = {
    # name: (B, Hq, Hkv, D, bs, shared pages, lengths behind them, options)
    "one": (1, 8, 2, 128, 16, 3, [5], {}),
    "one_token": (1, 4, 4, 128, 16, 0, [1], {}),
    "nothing_behind": (3, 8, 2, 128, 16, 9, [0, 0, 0], {"spare": None}),
    "nothing_shared": (4, 8, 2, 128, 16, 0, [1, 16, 17, 700], {}),
    "ragged": (5, 8, 2, 128, 16, 5, [0, 1, 16, 17, 300], {}),
    "chunk_edges": (6, 4, 1, 128, 16, 8, [127, 128, 129, 255, 256, 257], {}),
    "padding_rows": (6, 8, 2, 128, 16, 4, [9, 8, 7, 6, 5, 4], {"empty": (0, 3, 5)}),
    "all_padding": (3, 8, 2, 128, 16, 2, [1, 1, 1], {"empty": (0, 1, 2)}),
    "two_tiles_and_rest": (70, 5, 1, 128, 16, 12, [i % 19 for i in range(70)], {}),
    "exactly_one_tile": (32, 4, 1, 128, 16, 17, [3 * i for i in range(32)], {}),
    "one_row_over_a_tile": (129, 1, 1, 64, 16, 9, [i % 5 for i in range(129)], {}),
    "one_head_groups": (300, 2, 2, 64, 8, 3, [i % 7 for i in range(300)], {}),
    "group_3": (50, 6, 2, 64, 32, 6, [i % 40 for i in range(50)], {}),
    "group_160": (2, 160, 1, 128, 16, 9, [33, 1], {}),
    "group_256": (2, 256, 1, 64, 16, 9, [1, 140], {}),
    "d256": (5, 8, 2, 256, 16, 7, [0, 1, 63, 64, 65], {}),
    "d256_group_200": (2, 200, 1, 256, 16, 5, [17, 0], {}),
    "d256_many": (40, 16, 4, 256, 16, 9, [i % 23 for i in range(40)], {}),
    "pages_of_1": (3, 4, 2, 64, 1, 77, [0, 3, 40], {}),
    "pages_of_2": (3, 4, 2, 128, 2, 77, [0, 3, 200], {}),
    "pages_of_4": (2, 4, 1, 256, 4, 33, [7, 70], {}),
    "pages_of_64": (3, 8, 2, 128, 64, 5, [64, 1, 130], {}),
    "pages_of_256": (3, 8, 2, 128, 256, 2, [0, 300, 255], {}),
    "d256_pages_of_256": (2, 8, 2, 256, 256, 1, [70, 300], {}),
    "long_prefix": (4, 8, 2, 128, 16, 500, [20, 0, 1, 300], {}),
    "long_rest": (3, 8, 2, 128, 16, 2, [5000, 1, 0], {}),
    "many_long": (40, 40, 8, 128, 16, 0, [13 * i + 1 for i in range(40)], {}),
    "many_long_d64": (40, 16, 4, 64, 16, 5, [17 * i for i in range(40)], {}),
    "many_long_d256": (40, 16, 4, 256, 16, 0, [13 * i + 1 for i in range(40)], {}),
    "wide_scores": (4, 8, 2, 128, 16, 30, [200, 90, 0, 5], {"k_amp": 12.0}),
}


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", CASES)
def test_matches_the_definition(cuda_device, name, kv):
    B, Hq, Hkv, D, bs, n, rests, opt = CASES[name]
    batch = Batch(B, Hq, Hkv, D, bs, n, rests, kv=kv, seed=len(name) + B, **opt)
    out, lse = run(batch, cuda_device, nhd=len(name) % 2 == 1)
    check(out, lse, batch.reference(), f"{name}/{kv}")
    assert pad.pad_check_device_errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("bs", [2, 8, 16, 256])
@pytest.mark.parametrize("layout", ["heads outermost", "padded rows", "K and V unlike"])
def test_cache_layouts(cuda_device, layout, bs, kv):
    # block and head strides that make one coordinate and ones that do not
    batch = Batch(4, 8, 2, 128, bs, max(1, 160 // bs), [0, 3, 200, 77], kv=kv, seed=bs)
    a = batch.device(cuda_device)
    for name in ("k_cache", "v_cache"):
        c = a[name]
        if layout == "heads outermost":
            a[name] = c.transpose(0, 1).contiguous().transpose(0, 1)
        elif layout == "padded rows":
            wide = torch.zeros(*c.shape[:3], 160, dtype=torch.bfloat16, device=cuda_device).to(c.dtype)
            wide.view(torch.uint8).fill_(0x7F)
            wide[..., :128] = c
            a[name] = wide[..., :128]
        elif name == "v_cache":
            a[name] = c.transpose(1, 2).contiguous().transpose(1, 2)
    out, lse = pad.pad_decode_shared(**a, lse=True)
    check(out, lse, batch.reference(), layout)
    assert pad.pad_check_device_errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_same_as_pad_decode(cuda_device, kv):
    # what pad_decode gives for the same sequences, within both calls' tolerance
    batch = Batch(9, 16, 4, 128, 16, 20, [11 * i for i in range(9)], kv=kv, seed=4)
    a = batch.device(cuda_device)
    out, lse = pad.pad_decode_shared(**a, lse=True)
    tables = a["block_tables"].clone()
    tables[:, :20] = a["shared_table"]
    sc = {n: a[n] for n in ("k_scale", "v_scale") if n in a}
    o2, l2 = pad.pad_decode(a["q"], a["k_cache"], a["v_cache"], tables, a["seq_lens"], a["scale"], lse=True, **sc)
    ref = batch.reference()
    assert ((out.double() - o2.double()).abs().cpu() <= 2 * ref[2]).all()
    assert ((lse - l2).abs().cpu() <= 2 * ref[3]).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_sinks(cuda_device, kv):
    batch = Batch(4, 8, 2, 128, 16, 10, [0, 3, 200, 7], kv=kv, seed=6, empty=(3,))
    sinks = torch.tensor([0.5, -3.0, 25.0, -float("inf"), 2.0, 0.0, -100.0, 5.0])
    out, lse = run(batch, cuda_device, sinks=sinks.to(cuda_device))
    check(out, lse, batch.reference(sinks), "sinks")


def test_negative_and_zero_scale(cuda_device):
    for scale in (-0.2, 0.0):
        batch = Batch(3, 8, 2, 128, 16, 10, [0, 3, 200], seed=8)
        batch.scale = scale
        out, lse = run(batch, cuda_device)
        check(out, lse, batch.reference(), str(scale))


def test_scores_of_minus_infinity(cuda_device):
    # K rows of -inf along one positive q element: weight 0, whole chunks of them too
    batch = Batch(2, 4, 1, 128, 16, 24, [40, 200], seed=9)
    batch.q[..., 0] = 1.0
    ref_k = batch.k.clone()
    for pages in (batch.shared[:9], batch.tables[1, 24:26]):  # a chunk and more of the prefix
        batch.k[pages.long(), :, :, 0] = -float("inf")
    out, lse = run(batch, cuda_device)
    batch.k = ref_k
    batch.k[torch.cat([batch.shared[:9], batch.tables[1, 24:26]]).long(), :, :, 0] = -30000.0  # underflows to 0 too
    # scores of D = 128 terms of about 1: off by 136 * 2^-24 * 128 * scale at most, 1e-4
    for b in range(2):
        k, v = batch.rows(batch.k, b, 1.0)[0], batch.rows(batch.v, b, 1.0)[0]
        s = k @ batch.q[b].double().T * batch.scale
        w = torch.softmax(s, 0)
        want, mag = w.T @ v, w.T @ v.abs()
        assert ((out[b].double().cpu() - want).abs() <= mag * 2.0 ** -7 + want.abs() * 2.0 ** -8).all()
        assert ((lse[b].double().cpu() - torch.logsumexp(s, 0)).abs() <= 1e-4).all()


def test_bad_block_ids_read_as_zeros(cuda_device):
    batch = Batch(3, 8, 2, 128, 16, 6, [20, 40, 1], seed=10)
    batch.shared[2], batch.tables[1, 7] = 1 << 29, -7
    out, lse = run(batch, cuda_device)
    assert pad.pad_check_device_errors() == 0x1
    zero = batch.k.shape[0]
    for c in ("k", "v"):
        x = getattr(batch, c)
        setattr(batch, c, torch.cat([x, torch.zeros_like(x[:1])]))
    batch.shared[2], batch.tables[1, 7] = zero, zero
    check(out, lse, batch.reference(), "zero pages")


def test_bad_lengths_are_clamped_and_flagged(cuda_device):
    batch = Batch(5, 8, 2, 128, 16, 4, [20, 33, 7, 1, 30], seed=12, spare=None)
    cap = batch.W * 16
    a = batch.device(cuda_device)
    own = batch.tables.clone()
    own[:, 4:] = own[1, 4:]  # every row a full one
    a["block_tables"] = own.to(cuda_device)
    a["k_cache"], a["v_cache"] = a["k_cache"].nan_to_num(0.0), a["v_cache"].nan_to_num(0.0)
    for bad, as_if in ((-1, 0), (63, 0), (1, 0), (cap + 1, cap), (2**31 - 1, cap)):
        lens = batch.lens.clone()
        lens[2] = bad
        out, lse = pad.pad_decode_shared(**{**a, "seq_lens": lens.to(cuda_device)}, lse=True)
        assert pad.pad_check_device_errors() == 0x2, bad
        lens[2] = as_if
        o2, l2 = pad.pad_decode_shared(**{**a, "seq_lens": lens.to(cuda_device)}, lse=True)
        assert pad.pad_check_device_errors() == 0
        assert torch.equal(out, o2) and torch.equal(lse, l2), bad


def test_workspace_of_the_caller(cuda_device):
    batch = Batch(7, 8, 2, 128, 16, 30, [9 * i for i in range(7)], seed=13)
    a = batch.device(cuda_device)
    plan = pad.pad_decode_shared_plan(7, 8, 2, 128, 16, batch.W, 30)
    need = plan["workspace_bytes"]
    room = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=cuda_device)
    ws = room[: need]
    out, lse = pad.pad_decode_shared(**a, lse=True, workspace=ws)
    check(out, lse, batch.reference(), "workspace")
    assert bool((room[need:] == 0xA5).all())
    lib, _ = pad.pad_decode_shared(**a)
    assert torch.equal(out, lib)
    with pytest.raises(pad.PadError) as e:
        pad.pad_decode_shared(**a, workspace=ws[: need - 1])
    assert e.value.status == pad.PAD_ERR_INVALID_ARG
    with pytest.raises(pad.PadError):
        pad.pad_decode_shared(**a, workspace=room[1: need + 1])


def test_repeats_bit_for_bit(cuda_device):
    # no result depends on the order in which CTAs finish
    batch = Batch(33, 20, 4, 128, 16, 90, [13 * i % 400 for i in range(33)], seed=14)
    a = batch.device(cuda_device)
    first = pad.pad_decode_shared(**a, lse=True)
    for _ in range(5):
        again = pad.pad_decode_shared(**a, lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_captured_and_replayed_with_other_lengths(cuda_device):
    batch = Batch(6, 8, 2, 128, 16, 20, [100] * 6, seed=15)
    a = batch.device(cuda_device)
    out = torch.empty_like(a["q"])
    lse = torch.empty(a["q"].shape[:2], device=cuda_device)
    pad.pad_decode_shared(**a, out=out, lse=lse)  # scratch exists
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pad.pad_decode_shared(**a, out=out, lse=lse)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            pad.pad_decode_shared(**a, out=out, lse=lse)
        # a larger call on the capture's stream replaces the scratch; the graph's stays
        big = Batch(40, 8, 2, 128, 16, 3, [5] * 40, seed=16)
        o, l = pad.pad_decode_shared(**big.device(cuda_device), lse=True)
        side.synchronize()
        check(o, l, big.reference(), "larger call")
    for rests in ([0] * 6, [100, 1, 0, 50, 99, 16], [100] * 6):
        batch.lens = torch.tensor([320 + r for r in rests], dtype=torch.int32)
        a["seq_lens"].copy_(batch.lens)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(out, lse, batch.reference(), str(rests))
    assert pad.pad_check_device_errors() == 0


def test_scratch_does_not_grow_under_capture(cuda_device):
    batch = Batch(3, 8, 2, 128, 16, 4, [20, 33, 7], seed=17)
    a = batch.device(cuda_device)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        torch.cuda.synchronize()
        graph.capture_begin()
        try:
            with pytest.raises(pad.PadError) as e:
                pad.pad_decode_shared(**a)
        finally:
            graph.capture_end()
    assert e.value.status == pad.PAD_ERR_WORKSPACE


def test_two_streams_at_once(cuda_device):
    batches = [Batch(20, 8, 2, 128, 16, 60, [7 * i for i in range(20)], seed=s) for s in (18, 19)]
    args = [b.device(cuda_device) for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(pad.pad_decode_shared(**args[i], lse=True))
    torch.cuda.synchronize()
    for b, results in zip(batches, got):
        ref = b.reference()
        for out, lse in results:
            check(out, lse, ref, "two streams")


def test_two_threads_on_one_stream(cuda_device):
    # one scratch: the threads' kernels must not come between one another's
    import threading
    batches = [Batch(B, 8, 2, 128, 16, 30, [5 * i for i in range(B)], seed=s) for B, s in ((4, 22), (30, 23))]
    args = [b.device(cuda_device) for b in batches]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        for _ in range(30):
            got[i].append(pad.pad_decode_shared(**args[i], lse=True, stream=stream))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for b, results in zip(batches, got):
        assert len(results) == 30
        ref = b.reference()
        for out, lse in results:
            check(out, lse, ref, "two threads")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_non_finite_query_rows_stay_alone(cuda_device, kv):
    batch = Batch(20, 8, 2, 128, 16, 12, [9 * i for i in range(20)], kv=kv, seed=24)
    ref = batch.reference()
    bad = torch.zeros(20, 8, dtype=torch.bool)
    for b, h, x in ((0, 0, float("nan")), (7, 5, float("inf")), (19, 7, -float("inf"))):
        batch.q[b, h, 3] = x
        bad[b, h] = True
    out, lse = run(batch, cuda_device)
    assert bool(out.isnan().any(-1).cpu()[bad].all())
    ref[0][bad] = 0.0
    out[bad.to(cuda_device)] = 0
    lse = torch.where(bad.to(cuda_device), ref[1].float().to(cuda_device), lse)
    check(out, lse, ref, "other rows")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("power", [-90, 90])
def test_query_rows_far_from_one(cuda_device, kv, power):
    # rows of 2^power under a scale of 2^-power, some of zeros
    batch = Batch(6, 8, 2, 128, 16, 9, [0, 1, 63, 64, 65, 200], kv=kv, seed=25)
    batch.q = (batch.q.float() * 2.0 ** power).to(torch.bfloat16)
    batch.q[2, 3] = 0
    batch.scale *= 2.0 ** -power
    out, lse = run(batch, cuda_device)
    check(out, lse, batch.reference(), str(power))


def test_thousands_of_sequences(cuda_device):
    # many rounds of the schedule's sums, a row block of every kind, one-token items
    B = 2100
    batch = Batch(B, 2, 1, 64, 8, 3, [(7 * i) % 11 for i in range(B)], seed=26, empty=tuple(range(3, B, 17)))
    out, lse = run(batch, cuda_device)
    check(out, lse, batch.reference(), "thousands")


def test_strided_out_and_lse(cuda_device):
    batch = Batch(4, 8, 2, 128, 16, 10, [0, 3, 200, 7], seed=20)
    a = batch.device(cuda_device)
    wide = torch.full((4, 8, 3, 128), 7.0, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.full((8, 4), 7.0, device=cuda_device).t()
    q2 = torch.zeros(4, 12, 128, dtype=torch.bfloat16, device=cuda_device)
    q2[:, 2:10] = a["q"]
    a["q"] = q2[:, 2:10]
    pad.pad_decode_shared(**a, out=wide[:, :, 1], lse=lse)
    check(wide[:, :, 1], lse, batch.reference(), "strided")
    assert bool((wide[:, :, 0] == 7).all() and (wide[:, :, 2] == 7).all())


def test_a_serving_step(cuda_device):
    # prompt into the shared pages, each sequence's first tokens behind it, then a
    # step: append with its queries, decode behind the shared prefix -- the same as
    # pad_decode on the same cache
    gen = torch.Generator().manual_seed(21)
    B, Hq, Hkv, D, bs, n, W = 5, 16, 4, 128, 16, 7, 10
    f = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(cuda_device)
    w = (1 + 0.1 * rand(gen, D)).to(torch.bfloat16).to(cuda_device)
    blocks = torch.randperm(n + B * (W - n), generator=gen).to(torch.int32)
    tables = torch.cat([blocks[:n].expand(B, n), blocks[n:].view(B, W - n)], 1).contiguous().to(cuda_device)
    kc = torch.zeros(len(blocks), Hkv, bs, D, dtype=torch.bfloat16, device=cuda_device)
    vc = torch.zeros_like(kc)
    prompt = rand(gen, n * bs, 2 * Hkv, D).to(torch.bfloat16).to(cuda_device)
    pos = torch.arange(n * bs, dtype=torch.int32, device=cuda_device)
    pad.pad_append_kv(prompt[:, :Hkv], prompt[:, Hkv:], pos, tables, kc, vc, seq_ids=torch.zeros_like(pos), inv_freq=f,
                      k_weight=w)
    lens = torch.full((B,), n * bs, dtype=torch.int32, device=cuda_device)
    for _ in range(20):
        x = rand(gen, B, Hq + 2 * Hkv, D).to(torch.bfloat16).to(cuda_device)
        q = pad.pad_append_kv(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], lens, tables, kc, vc, inv_freq=f, k_weight=w,
                              q=x[:, :Hq], q_weight=w)
        close, _ = pad.pad_qk_norm_rope(x[:, :Hq], None, w, None, lens, f)
        assert torch.equal(q, close)
        lens = lens + 1
        out, lse = pad.pad_decode_shared(q, kc, vc, tables[0, :n], tables, lens, D ** -0.5, lse=True)
        o2, l2 = pad.pad_decode(q, kc, vc, tables, lens, D ** -0.5, lse=True)
        # both calls round each weight to bf16 once (2^-8 of sum w |v| <= max |v|) and out once
        assert (out.double() - o2.double()).abs().max() <= 2 * 2.0 ** -8 * (vc.abs().max() + o2.abs().max()).double()
        assert (lse - l2).abs().max() <= 1e-4
    assert pad.pad_check_device_errors() == 0


def test_a_captured_step_that_moves_its_lengths(cuda_device):
    # lengths, inputs and cache written by the kernels and copies just before: each call
    # starts beside its predecessor and must not read ahead of it
    gen = torch.Generator().manual_seed(27)
    B, Hq, Hkv, D, bs, n, W, steps = 6, 16, 4, 128, 16, 5, 9, 40
    blocks = torch.randperm(n + B * (W - n), generator=gen).to(torch.int32)
    tables = torch.cat([blocks[:n].expand(B, n), blocks[n:].view(B, W - n)], 1).contiguous().to(cuda_device)
    cache = rand(gen, 2, len(blocks), Hkv, bs, D).to(torch.bfloat16).to(cuda_device)
    f = torch.rand(D // 2, generator=gen).to(cuda_device)
    host = torch.stack([rand(gen, B, Hq + 2 * Hkv, D) for _ in range(steps)]).to(torch.bfloat16)
    rows = host.to(cuda_device)
    at = torch.zeros(1, dtype=torch.int64, device=cuda_device)
    lens = torch.full((B,), n * bs, dtype=torch.int32, device=cuda_device)
    x = torch.zeros(B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=cuda_device)
    outs = torch.zeros(steps, B, Hq, D, dtype=torch.bfloat16, device=cuda_device)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            x.copy_(rows.index_select(0, at)[0])
        main.wait_stream(side)
        q = pad.pad_append_kv(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], lens, tables, cache[0], cache[1], inv_freq=f,
                              q=x[:, :Hq])
        lens.add_(1)
        out, _ = pad.pad_decode_shared(q, cache[0], cache[1], tables[0, :n], tables, lens, D ** -0.5)
        outs.index_copy_(0, at, out[None])
        at.add_(1)

    start = (cache.clone(), lens.clone())
    for _ in range(steps):
        step()
    torch.cuda.synchronize()
    want, held = outs.clone(), cache.clone()
    cache.copy_(start[0])
    lens.copy_(start[1])
    at.zero_()
    outs.zero_()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        pad.pad_decode_shared(x[:, :Hq], cache[0], cache[1], tables[0, :n], tables, lens, D ** -0.5)  # its scratch
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache, held) and torch.equal(outs, want)
    q = pad.pad_qk_norm_rope(rows[-1][:, :Hq], None, None, None, lens - 1, f)[0]
    ref, _ = pad.pad_decode(q, cache[0], cache[1], tables, lens, D ** -0.5)
    # both calls round each weight to bf16 once (2^-8 of sum w |v| <= max |v|) and out once
    assert (outs[-1].double() - ref.double()).abs().max() <= 2 * 2.0 ** -8 * (cache[1].abs().max() + ref.abs().max()).double()
    assert pad.pad_check_device_errors() == 0
