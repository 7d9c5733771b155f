"""What the experts' operators do on the host, without a GPU."""

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
