"""Batches of every size with rules: more requests than the scheduling warp holds
at a time and than a thread each, empty ones among them; and windowed calls in the
workspace that the header says is enough for them."""
import numpy as np
import pytest

from tests import _rules
from tests._rules import RulesBatch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("rules", [dict(window=17, cap=50.0), dict(slopes=True), dict()], ids=str)
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 1, 128), (18, 1, 128)], ids=str)
@pytest.mark.parametrize("B", [31, 33, 70, 769, 1603])
def test_decode(B, heads, rules, f8):
    from tests.test_gpu_rules import Run
    rng = np.random.default_rng(B)
    ctx = np.where(rng.random(B) < 0.05, rng.integers(100, 300, B), rng.integers(1, 20, B))
    b = RulesBatch(91, *heads, list(ctx - 1), [1] * B, **rules)
    b.see_from = np.where(rng.random(B) < 0.5, rng.integers(0, ctx + 2), 0).astype(np.int32)
    none = rng.random(B) < 0.2                                   # no context: left out
    none[[0, B - 1]] = True
    run = Run(b, f8)
    run.seq[torch.from_numpy(none).cuda()] = 0
    o, lse = run("decode")
    assert int(run.status.item()) == 0
    assert np.isnan(o[none]).all() and np.isnan(lse[none]).all()
    ref = b.oracle(run.q64, run.k64, run.v64)
    _rules.check(o[~none], lse[~none], tuple(x[~none] for x in ref), b)


@pytest.mark.parametrize("path", ["split", "staged"])
@pytest.mark.parametrize("rules", [dict(window=17, cap=50.0, mask="any"), dict(slopes=True), dict(mask="docs")], ids=str)
@pytest.mark.parametrize("B", [33, 70, 800])
def test_extend(B, rules, path):
    from tests.test_gpu_rules import STAGED, Run
    rng = np.random.default_rng(B + 1)
    new = np.where(rng.random(B) < 0.3, 0, rng.integers(1, 5, B))
    new[[0, B - 1]] = 0
    b = RulesBatch(92, 4, 2, 64, list(rng.integers(0, 60, B)), list(new), **rules)
    Run(b).check(max_len=STAGED if path == "staged" else None)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("shared", [0, 512])
@pytest.mark.parametrize("window", [1, 2, 100, 127, 128, 129, 130, 257, 400])
def test_windowed_calls_in_the_least_workspace(window, shared, f8):
    """Contexts count with their last window + max_extend_len + 128 positions."""
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    from tests.test_gpu_rules import STAGED, Run
    for prefixes in ([126, 127, 128, 129, 254, 255, 256, 257, 0], [640, 639, 641, 1023, 1024, 1025, 513, 2000, 767]):
        new = [33, 1, 2, 30, 17, 33, 32, 31, 5]
        b = RulesBatch(93, 4, 2, 64, prefixes, new, window=window, cap=50.0, shared=shared)
        for r in range(len(new)):                                # nothing before a window is read
            b.rtt[b.req_idx[r], :max(0, prefixes[r] - window + 1)] = -1
        context = sum(min(p + n, window + 33 + 128) for p, n in zip(prefixes, new))
        run = Run(b, f8)
        ws = torch.empty(rx.rx_attn_rules_workspace(context, len(new), b.hq, b.hkv, b.d, 33), dtype=torch.uint8, device="cuda")
        o, lse = torch.full_like(run.q, float("nan")), torch.full(run.q.shape[:2], float("nan"), device="cuda")
        run.extend(o, lse, ws, STAGED)
        torch.cuda.synchronize()
        assert int(run.status.item()) == 0
        _rules.check(o.float().cpu().numpy(), lse.cpu().numpy(), b.oracle(run.q64, run.k64, run.v64), b)
