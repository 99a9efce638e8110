"""The operators' argument checks at the ends of their ranges, without a GPU."""
import pytest

from tests.conftest import gpu_available
from tests.test_ops_cpu import O, _combine  # noqa: F401 (O is a fixture)


@pytest.mark.skipif(gpu_available(), reason="goes on to the launch, which finds no device")
def test_combine_gradient_without_rows(O):  # noqa: F811
    """With no rows there is no drows to give, and the call is not refused."""
    import mxfp4_moe_expert_02_amd as M
    none = dict(rows=0, drows=0, dweights=0)
    assert _combine(O, "moe_combine_backward", **none) == M.MOE_E_NULL
    assert _combine(O, "moe_combine_backward", num_rows=0, **none) == M.MOE_E_HIP
    assert _combine(O, "moe_combine_backward", num_rows=0, dout=0, **none) == M.MOE_E_NULL
