"""What the experts' operators do on the host, without a GPU."""

import glob
import os
import re

import pytest

from combine_moe_layout_02_gb300 import build as moe_build
from combine_moe_layout_02_gb300 import moe


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe_build.build()
    return moe.lib()


@pytest.mark.parametrize("cycles,warp", [(0, -1), (1, -2), (1, 12)])
def test_product_wait_hook_refuses(cycles, warp):
    with pytest.raises(moe.MoeError):
        moe.moe_test_product_wait(cycles, warp)


def test_no_load_is_multicast_across_a_cluster():
    """The library takes any device pointer and is loaded by processes that use several GPUs: its loads are plain."""
    sources = glob.glob(os.path.join(os.path.dirname(moe.__file__), "csrc", "*.cu*"))
    assert len(sources) > 10
    for path in sources:
        text = re.sub(r'"\s*"', "", open(path, encoding="utf-8").read())  # adjacent literals are one string
        for line in re.findall(r'"[^"]*cp\.async\.bulk[^"]*"', text):
            assert "multicast" not in line, (path, line)
