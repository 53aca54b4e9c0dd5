"""That the bounds of the step's test tell a right step from a wrong one, on the
CPU: a last position that attention did not see yet, a window or a context that is
off by one, a row that was stored in another's place."""
import numpy as np
import pytest

from prefix_shared_kv_radixattention_gb300 import inputs
from tests._chain import HKV, D, Chain


def _round(x):
    return inputs.bf16_to_f32(inputs.bf16_round(np.asarray(x, np.float32))).astype(np.float64)


@pytest.mark.parametrize("window", [0, 48])
@pytest.mark.parametrize("seed", range(5))
def test_a_wrong_step_shows(seed, window):
    c = Chain(100 + seed, window)
    k, v = np.zeros((c.num_slots, HKV, D)), np.zeros((c.num_slots, HKV, D))
    for new in ([70, 60], [1, 1]):
        s = c.step(new)
        q, kn, vn = (_round(x) for x in c.rotated(s))
        old = k.copy(), v.copy()
        k[s.lists[3]], v[s.lists[3]] = kn, vn
    right = c.attention(s, q, k, v)
    good = _round(right[0]), right[1].astype(np.float32)
    c.check(s, q, *good, right)                                  # as the calls round it
    swapped = k.copy(), v.copy()
    for x, y in zip(swapped, (kn, vn)):
        x[s.lists[3]] = y[::-1]
    wrong = {"the newest rows not stored yet": c.attention(s, q, *old), "stored in one another's place": c.attention(s, q, *swapped),
             "the newest position not seen": c.attention(s, q, k, v, prefix=s.prefix - 1)}
    if window:
        wrong["a window of one less"] = c.attention(s, q, k, v, window=window - 1)
        wrong["a window of one more"] = c.attention(s, q, k, v, window=window + 1)
    for what, (o, lse, _) in wrong.items():
        for row in range(s.n):                                   # every token's row by itself
            mixed = good[0].copy(), good[1].copy()
            mixed[0][row], mixed[1][row] = _round(o[row]), lse[row]
            with pytest.raises(AssertionError):
                c.check(s, q, *mixed, right)
                pytest.fail(what, pytrace=False)
