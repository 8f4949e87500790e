"""pad_decode_shared's host side and sources on the CPU: how its scratch is held and
locked, and what must hold of the kernel's text."""
import os
import re

from paged_kv_attention_partition_b200 import _build


def test_tensor_memory_loads_are_waited_for_by_their_values():
    # a wait that the loaded registers do not go through lets the compiler use them before it
    text = {f: open(os.path.join(_build.CSRC, f)).read() for f in ("pad_shared.cu", "pad_tc.cuh")}
    assert not re.search(r"wait_ld\(\)", "".join(text.values()))
    loads = re.findall(r"tc::ld(\d+)\([^;]*?(\w+)\);\s*(\S+);", text["pad_shared.cu"])
    assert len(loads) == text["pad_shared.cu"].count("tc::ld") >= 4
    for n, reg, following in loads:
        assert following == f"tc::wait_ld{n}({reg})", following
