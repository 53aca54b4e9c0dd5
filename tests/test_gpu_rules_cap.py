"""The capped score itself, by tokens that see one position, their own: the
log-sum-exp is the score.  Against cap tanh(s / cap) in 64 bits, with the error
that include/rx.h states."""
import numpy as np
import pytest

from tests._rules import RulesBatch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("path", ["split", "staged", "decode"])
@pytest.mark.parametrize("cap,slopes", [(5.0, False), (30.0, False), (50.0, False), (80.0, False), (1e3, False), (20.0, True)])
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 1, 128)], ids=str)
def test_capped_scores(heads, cap, slopes, path, f8):
    from tests.test_gpu_rules import STAGED, Run
    new = [1] * 40 if path == "decode" else [40, 3, 65]
    for top in (0.37, 0.99, 10.0):                       # of the cap: within 3/8, within it, beyond
        b = RulesBatch(61, *heads, [100 + 7 * i for i in range(len(new))], new, cap=cap, window=1, slopes=slopes)
        b.k[:] = 0.0
        b.k[:, :, 0] = 1.0                               # every product is q's first value
        rng = np.random.default_rng(62)
        b.q[:] = 0.0
        b.q[:, :, 0] = rng.uniform(-0.998 * top, 0.998 * top, b.q.shape[:2]) * cap / b.scale   # 0.998: q is rounded to bf16
        run = Run(b, f8, ks=1.0)
        _, lse = run("decode" if path == "decode" else "extend", STAGED if path == "staged" else None)
        assert int(run.status.item()) == 0
        s = run.q64[:, :, 0] * float(np.float32(b.scale))
        t = cap * np.tanh(s / cap)
        beyond = np.abs(s).max() > cap or (path == "decode" and heads[2] == 128 and cap <= 150)   # the exponential's form
        score = 5 * 2.0 ** -23 * cap if beyond else 2.0 ** -21 * np.abs(t) + 2.0 ** -24 * cap
        # the log-sum-exp is (m + log2 l) ln 2: the product and the constant, 2^-24 each; with a fixed base m and l are
        # not the score and 1: 2^(x - m) is off by 2^-22 of itself, its logarithm, below 128, by one step of 2^-17, the
        # sum by half a one of 2^-17
        fixed = cap <= 50.0 and not slopes
        off = 2.0 ** -23 * np.abs(t) + (np.log(2) * (2.0 ** -22 / np.log(2) + 1.5 * 2.0 ** -17) if fixed else 0.0)
        assert (np.abs(lse - t) <= score + off).all(), (top, (np.abs(lse - t) / (score + off)).max())
