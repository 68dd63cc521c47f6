"""Every kernel is launched as a programmatic dependent of the kernel before it on the stream, so memory order rests
on its own wait: before anything else it waits, unconditionally, and only then lets its own dependent start."""
import glob
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "rotated_kv_cache_gb300", "csrc")


def _kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__ void(?: __launch_bounds__\((?:[^()]|\([^()]*\))*\))?\s+(\w+)\s*\(", text):
            at, depth = text.index("{", m.end()), 0
            for end in range(at, len(text)):
                depth += (text[end] == "{") - (text[end] == "}")
                if depth == 0:
                    break
            yield os.path.basename(path), m.group(1), text[at:end]


def test_kernels_are_found():
    assert len(list(_kernels())) >= 18


@pytest.mark.parametrize("file,name,body", [pytest.param(*k, id=k[1]) for k in _kernels()])
def test_a_kernel_waits_before_it_does_anything(file, name, body):
    if name == "wait_timeout_kernel":  # (reads and writes nothing of other kernels but the error word, and is no dependent)
        return
    calls = re.findall(r"pdl_wait_primary\(\)|pdl_allow_dependents\(\)", body)
    assert calls[:2] == ["pdl_wait_primary()", "pdl_allow_dependents()"], calls
    before = body[:body.index("pdl_wait_primary();")]
    # nothing conditional, and no load or store, ahead of the wait
    last = before.rstrip().rsplit("\n", 1)[-1] if before.strip("{ \n") else ""
    assert not re.search(r"\bif\b[^;]*$", before), last
    assert "= *" not in before and "atomic" not in before and "ld_global" not in before
