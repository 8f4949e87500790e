"""The calls around the decode on streams of other owners: each thread's default
stream, streams given by the caller beside torch's current one."""
import threading

import pytest
import torch

import paged_kv_attention_partition_b200 as pad
from operators_ref import Batch, check

pytestmark = pytest.mark.gpu

PER_THREAD = 2  # cudaStreamPerThread: a stream in every thread behind one handle


def test_two_threads_on_their_default_streams(cuda_device):
    batches = [Batch(20, 8, 2, 128, 16, 60, [7 * i for i in range(20)], seed=s) for s in (41, 42, 43)]
    args = [b.device(cuda_device) for b in batches]
    for a in args:
        a["out"] = torch.empty_like(a["q"])
        a["lse"] = torch.empty(a["q"].shape[:2], device=cuda_device)
    tables = []
    for a in args:
        tables.append(a["block_tables"].clone())
        tables[-1][:, :60] = a["shared_table"]
    plain = [(torch.empty_like(a["q"]), torch.empty_like(a["lse"])) for a in args]
    torch.cuda.synchronize()
    barrier, errors = threading.Barrier(len(args)), []

    def work(i):
        try:
            torch.cuda.set_device(cuda_device)
            a = args[i]
            barrier.wait(timeout=60)
            for _ in range(30):
                pad.pad_decode_shared(**a, stream=PER_THREAD)
                pad.pad_decode(a["q"], a["k_cache"], a["v_cache"], tables[i], a["seq_lens"], a["scale"], num_splits=5,
                               out=plain[i][0], lse=plain[i][1], stream=PER_THREAD)
        except Exception as e:
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(args))]
    [t.start() for t in threads]
    [t.join(timeout=300) for t in threads]
    assert not errors, errors
    torch.cuda.synchronize()
    for b, a, (o, l) in zip(batches, args, plain):
        ref = b.reference()
        check(a["out"], a["lse"], ref, "shared")
        check(o, l, ref, "pad_decode")
    assert pad.pad_check_device_errors() == 0


def test_two_threads_with_workspaces_on_one_stream(cuda_device):
    # nothing of the library's is shared, so their kernels may come between one another's
    batches = [Batch(B, 8, 2, 128, 16, 30, [5 * i for i in range(B)], seed=s) for B, s in ((4, 44), (30, 45))]
    args = [b.device(cuda_device) for b in batches]
    for b, a in zip(batches, args):
        need = pad.pad_decode_shared_plan(len(b.lens), 8, 2, 128, 16, b.W, 30)["workspace_bytes"]
        a["workspace"] = torch.empty(need, dtype=torch.uint8, device=cuda_device)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        for _ in range(40):
            o = torch.empty_like(args[i]["q"])
            pad.pad_decode_shared(**args[i], out=o, stream=stream)
            got[i].append(o)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for b, results in zip(batches, got):
        assert len(results) == 40
        ref = b.reference()
        check(results[0], None, ref, "first")
        assert all(torch.equal(results[0], r) for r in results[1:])


def rows_call(dev, stream, **kw):
    x = torch.randn(3001, 12, 128, device=dev).to(torch.bfloat16)
    return [x], lambda: pad.pad_qk_norm_rope(x[:, :8], x[:, 8:], stream=stream, **kw)


def append_call(dev, stream, **kw):
    x = torch.randn(3001, 12, 128, device=dev).to(torch.bfloat16)
    pos = torch.arange(3001, dtype=torch.int32, device=dev)
    tables = torch.arange(188, dtype=torch.int32, device=dev).view(1, 188)
    kc, vc = (torch.zeros(188, 2, 16, 128, dtype=torch.bfloat16, device=dev) for _ in range(2))
    return [x, kc, vc], lambda: [pad.pad_append_kv(x[:, 8:10], x[:, 10:], pos, tables, kc, vc,
                                                   seq_ids=torch.zeros_like(pos), q=x[:, :8], stream=stream, **kw)]


def shared_call(dev, stream, **kw):
    batch = Batch(260, 64, 2, 128, 16, 30, [i % 7 for i in range(260)], seed=46)
    a = batch.device(dev)
    return [a["q"], a["k_cache"], a["v_cache"]], lambda: pad.pad_decode_shared(**a, lse=True, stream=stream, **kw)


@pytest.mark.parametrize("make", [rows_call, append_call, shared_call])
def test_tensors_dropped_while_another_stream_uses_them(cuda_device, make):
    # a block that the side stream still reads or writes is not given out again
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    tensors, call = make(cuda_device, side)
    call()  # (scratch, modules)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)
    outs = [t for t in call() if t is not None]
    held = {t.untyped_storage().data_ptr() for t in tensors + outs}
    sizes = [t.untyped_storage().nbytes() for t in tensors + outs for _ in range(3)]
    del tensors, outs, call
    fresh = [torch.empty(n, dtype=torch.uint8, device=cuda_device) for n in sizes]
    assert not side.query(), "the side stream was done too soon to see anything"
    assert not held & {t.untyped_storage().data_ptr() for t in fresh}
    side.synchronize()


@pytest.mark.parametrize("make", [rows_call, append_call, shared_call])
def test_outputs_dropped_while_the_current_stream_reads_them(cuda_device, make):
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    tensors, call = make(cuda_device, side)
    first = call()
    torch.cuda.synchronize()
    want = [t.clone() for t in first if t is not None]
    side.wait_stream(main)
    outs = [t for t in call() if t is not None]
    main.wait_stream(side)
    torch.cuda._sleep(400_000_000)
    copies = [t.clone() for t in outs]
    held, sizes = {t.data_ptr() for t in outs}, [t.untyped_storage().nbytes() for t in outs]
    del outs
    with torch.cuda.stream(side):
        fresh = [torch.empty(n, dtype=torch.uint8, device=cuda_device).fill_(0xFF) for n in sizes for _ in range(3)]
    assert not main.query(), "the current stream was done too soon to see anything"
    assert not held & {t.data_ptr() for t in fresh}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))


def test_the_per_thread_stream_takes_given_outputs_only(cuda_device):
    for make in (rows_call, append_call, shared_call):
        _, call = make(cuda_device, PER_THREAD)
        with pytest.raises(ValueError):
            call()
    x = torch.randn(5, 4, 128, device=cuda_device).to(torch.bfloat16)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    got, _ = pad.pad_qk_norm_rope(x, None, q_out=out, stream=PER_THREAD)
    torch.cuda.synchronize()
    assert got is out and torch.equal(out, x)


@pytest.mark.parametrize("mode", ["global", "thread_local", "relaxed"])
def test_a_call_beside_a_capture_on_another_stream(cuda_device, mode):
    # what the call asks about its own stream must not end the other's capture
    batches = [Batch(6, 8, 2, 128, 16, 20, [5 * i for i in range(6)], seed=s) for s in (48, 49)]
    args = [b.device(cuda_device) for b in batches]
    for a in args:
        a["out"] = torch.empty_like(a["q"])
        a["lse"] = torch.empty(a["q"].shape[:2], device=cuda_device)
    captured, others = torch.cuda.Stream(), (torch.cuda.Stream(), torch.cuda.default_stream())
    for s in (captured, *others):  # scratch exists
        pad.pad_decode_shared(**args[0], stream=s)
    torch.cuda.synchronize()
    for other in others:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=captured, capture_error_mode=mode):
            pad.pad_decode_shared(**args[0])
            pad.pad_decode_shared(**args[1], stream=other)
            pad.pad_decode_shared(**args[0])
        torch.cuda.synchronize()
        check(args[1]["out"], args[1]["lse"], batches[1].reference(), "beside")
        args[0]["out"].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(args[0]["out"], args[0]["lse"], batches[0].reference(), "captured")
