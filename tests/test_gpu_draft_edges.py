"""Arguments at the edge of what the draft-verification calls take: scales near
the ends of fp32."""
import numpy as np
import pytest

from tests import _draft
from tests.test_gpu_draft_tree import Run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("ks", [1e-13, 1e-30, 1e25])
def test_query_rows_of_zeros_and_scales_near_the_ends(ks):
    """Over FP8 pools a row's score factor is the product of sm_scale, the
    pool's scale and the row's power of two: it must not vanish (a masked
    place is -inf times it).  With K codes of order one the scores are
    about ks: every weight is the same for the small scales; for the large
    one only the rows of zeros are looked at."""
    b = _draft.TreeBatch(63, 4, 2, 64, [200, 0, 127], [7, 5, 1])
    b.q[::2] = 0.0
    if ks < 1:
        b.q[1::4] *= np.float32(1e-30)
    r = Run(b, True)             # codes of k / 0.07
    r.ks = ks
    r.k64 = r.k64 / 0.07 * ks
    o, lse = r()
    assert int(r.status.item()) == 0
    keep = slice(None) if ks < 1 else slice(0, None, 2)
    _draft.check_tree(o[keep], lse[keep], tuple(x[keep] for x in r.reference()), f"scale {ks}")
