"""How the single-token operators' kernels read memory.

They are launched while the kernel in front of them still runs (programmatic dependent
launch), so what they read may be written during their own lifetime.  The non-coherent loads
(ld.global.nc: __ldg, and what the compiler makes of a const pointer marked __restrict__) ask for
memory that nothing writes as long as the kernel lives, and may be moved in front of the
wait; results would be stale only now and then, which no run shows for certain."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a4_post_quantized_b200", "csrc")


@pytest.mark.parametrize("name", ["group.cu", "kv.cu", "decode.cuh"])
def test_no_non_coherent_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    for form in (r"__ldg\b", r"\.nc\b", r"const\s+\w+\s*\*\s*__restrict__", r"\w+\s+const\s*\*\s*__restrict__"):
        assert not re.findall(form, code), form


@pytest.mark.parametrize("name", ["group.cu", "kv.cu"])
def test_every_kernel_waits(name):
    """Each kernel waits for the one in front exactly once on every path: at its top, or in its loop's first round."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    kernels = re.split(r"__global__", code)[1:]
    assert len(kernels) >= 3
    for k in kernels:
        assert k.count("griddep_wait()") == 1, k[:200]
        assert k.index("griddep_wait()") < k.index("griddep_launch_dependents()")
