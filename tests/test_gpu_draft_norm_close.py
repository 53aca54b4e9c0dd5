"""rx_qk_norm_rope_store and its FP8 form to the arithmetic of the kernel: a
result may differ from the nearest value of its type only where the exact
value lies within the fp32 arithmetic's error of a tie.

That error, of y' = the rotated value, in units of 2^-24 (|y_c| + |y_c+d/2|):
the sum of squares is 13 roundings deep (four packed multiply-adds of two
pairs, the join, three shuffles; the mean and eps), half of which the root
passes on: 6.5; the root's Newton step 1; the products with it and with the
weight 2; sine and cosine, below half a place plus the series' remainder, 1;
the product and the multiply-add of the rotation 2; together under 13.  For far
positions the table's frequencies, and the oracle's, are off by 2^-53 of
themselves: pos * 2^-53 each, 2.3e-16 |pos| together.  The FP8 division adds a
place."""
import numpy as np
import pytest

from oracle import fp8
from prefix_shared_kv_radixattention_gb300 import inputs
from tests.test_gpu_draft_norm import CASES, _case, _g, _heads

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BASE, EPS = 10000.0, 1e-6


def _slack(y, pos):
    h = y.shape[-1] // 2
    m = np.abs(y[..., :h]) + np.abs(y[..., h:])
    m = m * (13 * 2.0 ** -24 + 2.3e-16 * np.abs(pos.astype(np.float64)))[:, None, None]
    return np.concatenate([m, m], -1)


def _between(got, lo, hi, what):
    """got is nearest to some value in [lo, hi]: rounding is monotonic."""
    assert ((got >= lo) & (got <= hi)).all(), f"{what}: {((got < lo) | (got > hi)).sum()} of {got.size}"


@pytest.mark.parametrize("n,hq,hkv,d", [*CASES, (4099, 32, 8, 128)])
def test_results_are_the_nearest_but_for_near_ties(n, hq, hkv, d):
    g = _g()
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = _case(3 * n + d, n, hq, hkv, d, True, True)
    slots, pos = g.i32(c["slots"]), g.i32(c["pos"])
    qo = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    kp, vp = (torch.zeros(c["S"], hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rx.rx_qk_norm_rope_store(kp, vp, c["q"], qo, c["k"], c["v"], *c["wd"], slots, pos, BASE, EPS)

    def bf16(x):
        return inputs.bf16_to_f32(inputs.bf16_round(x.astype(np.float32))).astype(np.float64)

    # through fp32 (another rounding: one more place of slack on either side)
    for got, which in ((qo, "q"), (kp[slots.long()], "k")):
        y, ref = _heads(c, which, BASE, EPS)
        s = _slack(y, c["pos"]) + 2.0 ** -23 * np.abs(ref) + 1e-37
        _between(got.double().cpu().numpy(), bf16(ref - s), bf16(ref + s), which)

    scale = np.float32(0.0523)
    k8, v8 = (torch.zeros(c["S"], hkv, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    rx.rx_qk_norm_rope_store_fp8(k8, v8, float(scale), float(scale), c["q"], qo, c["k"], c["v"], *c["wd"], slots, pos, BASE, EPS)
    y, ref = _heads(c, "k", BASE, EPS)
    s = (_slack(y, c["pos"]) + 2.0 ** -23 * np.abs(ref)) / float(scale) + 1e-37
    got = fp8.decode(k8[slots.long()].cpu().numpy())
    lo, hi = (fp8.decode(fp8.encode(ref / float(scale) + e)) for e in (-s, s))
    _between(got, lo, hi, "codes")
    # what the interval leaves open, a matter of the oracle alone: it is some 3e-6
    # of the value wide, a step 2^-4 to 2^-3 of it, so one code in 10,000 or so
    assert (lo != hi).sum() <= 3 + 2.5e-4 * lo.size
