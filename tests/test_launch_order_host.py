"""The order of the two halves of a programmatic dependent launch in the kernels' sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_kv_long_sfi_gb300", "csrc")


def _source():
    text = "".join(open(os.path.join(CSRC, f)).read() for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh")))
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def _kernels():
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\s*\(.*?\n}\n", _source(), re.S):
        yield m.group(1), m.group(0)


def test_the_kernels_are_found():
    names = {n for n, _ in _kernels()}
    assert {"kv4_attn_kernel", "kv4_append_kernel", "kv4_read_kernel", "kv4_compact_kernel", "page_copy_kernel",
            "qk_norm_rope_kernel"} <= names


@pytest.mark.parametrize("name,body", [pytest.param(n, b, id=n) for n, b in _kernels()])
def test_dependents_are_released_after_the_wait(name, body):
    """A kernel that releases its dependents before its own wait lets the next kernel start while
    the one before it still runs. An attention launch with SFI_ATTN_EARLY_KV_PREFETCH reads its
    pages at once then, although only its direct predecessor is known not to write them. (A kernel
    that is launched the ordinary way starts when all before it has finished, and needs no wait.)"""
    calls = re.findall(r"grid_(launch_dependents|dependency_wait)\(\)", body)
    ordinary = "dependency_wait" not in calls
    if ordinary and calls:
        # the launch of an ordinary kernel: kernel<<<...>>>, by its name or a variable set from it
        assert re.search(name + r"<[^;]*;\s*kernel<<<", _source()) or name + "<<<" in _source(), name
    waited = ordinary
    for c in calls:
        if c == "launch_dependents":
            assert waited, f"{name} releases its dependents before its wait"
        waited |= c == "dependency_wait"
