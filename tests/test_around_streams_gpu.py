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
