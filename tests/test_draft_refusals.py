"""Refusals of the draft-verification entry points at the ends of fp32, on the
CPU (empty batches: nothing is launched whatever the answer)."""
import pytest

from prefix_shared_kv_radixattention_gb300 import binding as rx
from tests.test_draft_oracle import _tree


@pytest.mark.parametrize("bad", [dict(scale=1e-39, k_scale=1.0), dict(scale=3.4e38, k_scale=1.0)], ids=str)
def test_tree_refuses_a_scale_outside_the_normal_range(bad):
    assert set(_tree(rx.library(), batch=0, **bad)) == {rx.RX_ERR_INVALID}


@pytest.mark.parametrize("bad", [dict(scale=0.125, k_scale=1e-38), dict(scale=1e-20, k_scale=1e-20),
                                 dict(scale=10.0, k_scale=3e38)], ids=str)
def test_tree_refuses_a_product_of_scales_outside_the_normal_range(bad):
    """0 times the -inf of a masked place would be NaN.  The bf16 call has
    no K scale."""
    assert _tree(rx.library(), batch=0, **bad)[0] == rx.RX_ERR_INVALID
