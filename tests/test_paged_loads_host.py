"""The paged kernels are launched while the kernel before them still runs, so none of what they read is constant for
their whole duration: no load of theirs may promise that (ld.global.nc), whatever wait stands before it."""
import os
import re

import pytest

from attention_kl_divergence_02_b200 import build


@pytest.mark.parametrize("name", ["cache_kernels.cuh", "paged.cuh", "paged_attn_kernel.cuh", "paged_kl_kernel.cuh"])
def test_no_read_only_loads(name):
    with open(os.path.join(build.CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc|__restrict__", code)
