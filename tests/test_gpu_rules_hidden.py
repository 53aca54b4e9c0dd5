"""What no token of a request sees does not change a bit of its results, whatever
K and V hold there, nor does it change how exact they are."""
import numpy as np
import pytest

from tests import _rules
from tests._rules import RulesBatch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FROM = 150          # every token sees from here on: the tile of positions 128 .. 255 is seen in part


def _run(path, heads, f8, fill, rules, seed=51):
    """Outputs, and the oracle's for the pools as they were before `fill` went to what is hidden."""
    from tests.test_gpu_rules import STAGED, Run
    new = [1, 1, 1] if path == "decode" else [40, 33, 70]
    b = RulesBatch(seed, *heads, [300, 160, 420], new, **rules)
    if not rules.get("window"):
        b.see_from = np.full(sum(new), FROM, np.int32)
    hidden = []
    for r in range(3):
        first = FROM if not rules.get("window") else max(0, int(b.prefix_len[r]) - rules["window"] + 1)
        hidden += b.rtt[b.req_idx[r], :first].tolist()

    def edit(run, k, v):
        if fill is None:
            return
        at = torch.tensor(hidden, device="cuda")
        for t in (k, v):
            if f8:      # 0x7E: the largest code, 0x7F: NaN
                t[at] = {"large": 0x7E, "inf": 0x7F, "nan": 0x7F}[fill]
            elif fill == "inf":  # scores of plus or minus infinity, V infinite throughout
                t[at] = 0.0 if t is k else float("inf")
                t[at, :, 0] = float("inf")
            else:
                t[at] = {"large": 1e4, "nan": float("nan")}[fill]

    run = Run(b, f8, edit=edit)
    o, lse = run("decode" if path == "decode" else "extend", STAGED if path == "staged" else None)
    assert int(run.status.item()) == 0
    return o, lse, b, b.oracle(run.q64, run.k64, run.v64)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("path", ["split", "staged", "decode"])
@pytest.mark.parametrize("rules", [dict(cap=50.0), dict(cap=80.0), dict(cap=20.0, slopes=True), dict(cap=30.0, window=70), dict(slopes=True),
                                   dict(window=70)], ids=str)
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 1, 128), (32, 1, 128)], ids=str)
def test_hidden_keys_do_not_change_a_bit(heads, rules, path, f8):
    o, lse, b, ref = _run(path, heads, f8, None, rules)
    _rules.check(o, lse, ref, b)
    for fill in ("large", "inf", "nan"):
        again = _run(path, heads, f8, fill, rules)
        assert np.array_equal(o, again[0]) and np.array_equal(lse, again[1]), fill


@pytest.mark.parametrize("path", ["split", "staged", "decode"])
@pytest.mark.parametrize("fill", ["large", "inf", "nan"])
def test_a_large_cap_stays_exact_beside_hidden_keys(fill, path):
    """The exponential's form is off by a few 2^-23 of the cap: with a cap of 1e6, 0.3 and more."""
    for heads, f8 in (((8, 2, 64), False), ((32, 1, 128), True)):
        o, lse, b, ref = _run(path, heads, f8, fill, dict(cap=1e6))
        _rules.check(o, lse, ref, b, cap=30.0)
