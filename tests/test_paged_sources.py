"""What the paged kernels' sources must not contain: they begin while the kernel
before them still writes, so loads through the read-only path, which nothing
orders behind that kernel's stores, have no place in them."""
import os
import re

import pytest

from exact_io_aware_online_b200 import _build


@pytest.mark.parametrize("name", ["cache_sm100.cuh", "paged_sm100.cuh"])
def test_no_read_only_loads(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg|__restrict__|global\.nc", code)
