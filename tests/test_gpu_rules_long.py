"""Attention with rules over dozens of position tiles, with scores that rise, fall
or go up and down along the context: the running maximum is raised again and again,
the results rescaled, the parts of many CTAs joined.  Bounds: tests/_rules.check."""
import numpy as np
import pytest

from tests._rules import RulesBatch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _trend(b, kind):
    """q's first value times k's is a score that moves between -40 and 40 along each context.  What check() allows for
    the scores' sums, 3e-4 times a quarter of the largest q, holds: sum |q k| scale stays under 40 + 0.64 sqrt(d) + 1 (the
    other products are of order one), times d 2^-24 that is 3.7e-4 at d = 128, and the largest q is 8."""
    top = 40.0 * np.sqrt(b.d) / 8.0
    b.q[:, :, 0] = 8.0
    for r in range(len(b.new_len)):
        n = int(b.prefix_len[r] + b.new_len[r])
        x = np.linspace(-1, 1, n)
        x = {"rising": x, "falling": -x, "waves": np.sin(17 * x)}[kind]
        b.k[b.rtt[b.req_idx[r], :n], :, 0] = (top * x)[:, None]


RULES = [dict(slopes=True), dict(cap=80.0), dict(cap=50.0), dict(cap=80.0, slopes=True), dict(), dict(window=4500), dict(window=3000, slopes=True)]


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("kind", ["rising", "falling", "waves"])
@pytest.mark.parametrize("rules", RULES, ids=str)
@pytest.mark.parametrize("heads", [(8, 1, 128), (16, 1, 128), (4, 2, 64)], ids=str)
def test_decode(heads, rules, kind, f8):
    from tests.test_gpu_rules import Run
    b = RulesBatch(81, *heads, [7000, 5111, 640, 63], [1, 1, 1, 1], **rules)
    _trend(b, kind)
    if rules.get("slopes"):
        b.see_from = np.array([300, 0, 5, 0], np.int32)
    Run(b, f8, ks=0.2).check("decode", what=kind)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("kind", ["rising", "falling"])
@pytest.mark.parametrize("path", ["split", "staged"])
@pytest.mark.parametrize("rules", RULES + [dict(mask="spans", slopes=True), dict(mask="any")], ids=str)
@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 4, 64)], ids=str)
def test_extend(heads, rules, path, kind, f8):
    from tests.test_gpu_rules import STAGED, Run
    b = RulesBatch(82, *heads, [5100, 1999], [41, 9], **rules)
    _trend(b, kind)
    Run(b, f8, ks=0.2).check(max_len=STAGED if path == "staged" else None, what=kind)


@pytest.mark.parametrize("kind", ["rising", "falling"])
@pytest.mark.parametrize("path", ["split", "staged"])
@pytest.mark.parametrize("rules", [dict(slopes=True), dict(cap=80.0), dict()], ids=str)
def test_extend_with_two_row_tiles(rules, path, kind):
    """More than 128 rows a kv head: a K and V tile serves two row tiles."""
    from tests.test_gpu_rules import STAGED, Run
    b = RulesBatch(83, 16, 1, 64, [4000], [50], **rules)
    _trend(b, kind)
    Run(b).check(max_len=STAGED if path == "staged" else None, what=kind)
