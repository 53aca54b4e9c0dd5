"""Softmax weights far below the largest in rx_attn_tree and rx_attn_tree_fp8:
one key takes nearly all of the weight and has a V of zero (an attention sink),
so the result is the sum over the others, whose weights are 2^-17 to 2^-37 of
the sink's.  Bounds: tests/_draft.check_tree, whose sum p |v| leaves the sink
out."""
import numpy as np
import pytest

from tests import _draft
from tests.test_gpu_draft_tree import Run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("where", ["first", "last", "drafted"])
@pytest.mark.parametrize("gap", [12.0, 13.8, 16.2, 17.3, 26.0])
def test_one_dominant_key_without_a_value(gap, where, f8):
    """Every q is one in all d = 64 places, so a key that is c everywhere has
    the score 64 c / 8 = 8 c: the sink's is `gap` nats above the others' 0."""
    prefixes, trees = [1000, 8192, 40], [3, 5, 2]
    b = _draft.TreeBatch(41, 4, 2, 64, prefixes, trees, masks="chain")
    b.q[:] = 1.0
    b.k[:] = 0.0
    for i, p in enumerate(prefixes):
        at = {"first": 0, "last": p - 1, "drafted": p}[where]
        slot = int(b.rtt[b.req_idx[i], at])
        b.k[slot] = gap / 8
        b.v[slot] = 0.0
    r = Run(b, f8)
    o, lse = r()
    assert int(r.status.item()) == 0
    _draft.check_tree(o, lse, r.reference(), f"gap {gap}, {where}")
    assert np.abs(o).max() > 0
