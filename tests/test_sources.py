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


def test_what_the_prefix_kernel_reads_before_its_wait():
    """The kernel over a shared prefix runs beside the end of the one before it, whose own wait covers all
    that came earlier: the lengths are read past L1 then, where an older copy of them could lie."""
    code = _code(os.path.join(CSRC, "prefix_attn.cu"))
    kernel = code.split("prefix_tc_kernel(")[1].split("prefix_join_kernel(")[0]
    assert kernel.rstrip().count("pdl_wait()") == 1 and "a.lens[" not in kernel
    in_use = code.split("bool in_use(")[1].split("};")[0]
    assert "ld_global_l2(lens +" in in_use and "lens[" not in in_use
