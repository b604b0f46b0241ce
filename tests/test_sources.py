"""What the kernels' sources have to keep to, where a wrong result would show by chance only."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "vision_transformer_attention_psapackqkv_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_no_read_only_loads_while_an_earlier_kernel_may_write(path):
    """Programmatic dependent launch makes a kernel resident while the one before it still writes what it
    reads.  Loads of the read-only path (and const __restrict__ parameters, which become such loads) promise
    memory that nobody writes during the kernel, and nothing keeps them behind the wait."""
    code = _code(path)
    assert not re.search(r"__ldg\s*\(|ld\.global[\w.:]*\.nc\b", code)
    for kernel in code.split("__global__")[1:]:
        if "pdl_wait()" in kernel:
            assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", kernel.split("{")[0])
