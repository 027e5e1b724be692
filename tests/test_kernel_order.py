"""What every kernel of the library keeps to so that its dependents may start early, read from
the sources: nothing at run time shows a breach until two kernels happen to share a
multiprocessor.

A dependent launch may begin once every block has signalled. The tensor-core GEMM allocates
all of a multiprocessor's tensor memory in its prologue, before it waits for the kernel
ahead of it. A block that signalled first and allocated afterwards could find that memory
taken by a GEMM block that waits for it to end, and wait for it in turn, without a limit."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "group_wise_int4_b200", "csrc")


def _kernels():
    """(file:name, body) of every kernel that signals its dependents."""
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            name = re.search(r"(\w+)\s*\(", re.sub(r"__launch_bounds__\s*\((?:[^()]|\([^()]*\))*\)", "", text[m.end():m.end() + 400])).group(1)
            at = text.index("{", m.end())
            depth, end = 0, at
            for end in range(at, len(text)):
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                if depth == 0:
                    break
            body = text[at:end]
            if "pdl_trigger(" in body:
                out.append(pytest.param(body, id=f"{os.path.basename(path)}:{name}"))
    return out


def test_the_kernels_are_found():
    names = [p.id for p in _kernels()]
    assert len(names) == len(set(names)) and len(names) >= 15
    assert sum("tmem_alloc(" in p.values[0] for p in _kernels()) == 3, "both GEMMs and the attention tiles"


@pytest.mark.parametrize("body", _kernels())
def test_tensor_memory_is_allocated_before_dependents_may_start(body):
    if "tmem_alloc(" in body:
        assert body.index("tmem_alloc(") < body.index("pdl_trigger(")


@pytest.mark.parametrize("body", _kernels())
def test_dependents_may_start_only_after_the_kernels_own_wait(body):
    """The GEMM's early weight loads count on it: when its grid runs, all that came before the
    kernel directly ahead of it is complete."""
    assert body.index("pdl_wait(") < body.index("pdl_trigger(")
