"""pad_decode_shared's host side and sources on the CPU: how its scratch is held and
locked, and what must hold of the kernel's text."""
import os
import re
import subprocess

import pytest

from paged_kv_attention_partition_b200 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")


def test_tensor_memory_loads_are_waited_for_by_their_values():
    # a wait that the loaded registers do not go through lets the compiler use them before it
    text = {f: open(os.path.join(_build.CSRC, f)).read() for f in ("pad_shared.cu", "pad_tc.cuh")}
    assert not re.search(r"wait_ld\(\)", "".join(text.values()))
    loads = re.findall(r"tc::ld(\d+)\([^;]*?(\w+)\);\s*(\S+);", text["pad_shared.cu"])
    assert len(loads) == text["pad_shared.cu"].count("tc::ld") >= 4
    for n, reg, following in loads:
        assert following == f"tc::wait_ld{n}({reg})", following


@pytest.fixture(scope="module")
def lane(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("lane") / "lane_scratch")
    src = [os.path.join(ROOT, "tests", "host_lane_scratch.cpp")] + \
          [os.path.join(_build.CSRC, f) for f in ("pad_api.cpp", "pad_shared_api.cpp")]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc())))
    res = subprocess.run(["g++", "-std=c++17", "-O1", "-g", *SAN, "-I", _build.INCLUDE, "-I", _build.CSRC, "-I",
                          os.path.join(cuda, "include"), *src, "-lpthread", "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return exe


def run_lane(lane, *args):
    res = subprocess.run([lane, *args], capture_output=True, text=True, env=ENV, timeout=120)
    assert res.returncode == 0 and "clean" in res.stdout, res.stdout + res.stderr


@pytest.mark.parametrize("ids", [[], ["no-ids"]])
def test_each_thread_has_its_own_scratch_on_the_per_thread_stream(lane, ids):
    run_lane(lane, "threads", *ids)


@pytest.mark.parametrize("scenario", ["reuse", "thread-reuse", "capture"])
def test_scratch_of_streams_that_are_gone(lane, scenario):
    run_lane(lane, scenario)


def test_only_calls_that_share_scratch_wait_for_one_another(lane):
    run_lane(lane, "locks")
