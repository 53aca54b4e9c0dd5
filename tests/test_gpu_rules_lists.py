"""The lists of a step in front of the attention calls: lists that were cut, or
that leave a request out, and what the calls behind them then read and write."""
import numpy as np
import pytest

from tests._rules import RulesBatch, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

CALLS = ["rules split", "rules staged", "rules split fp8", "rules staged fp8", "plain gathered", "plain staged", "plain fp8"]


def _run(call, b, n, plen, nlen, tokens, pages=None, size=0):
    """The lists cut at `tokens`, then the attention call over n rows of which only the first `tokens` are the caller's.
    Returns o and lse of all n rows (NaN where nothing was written), the status and qo_indptr."""
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    from tests import _gpu as g
    from tests.test_gpu_rules import STAGED, Run
    run = Run(b, "fp8" in call)
    e = lambda m: torch.full((m,), -5, dtype=torch.int32, device="cuda")  # noqa: E731
    indptr, seq, pos, slots = e(len(nlen) + 1), e(len(nlen)), e(tokens), e(tokens)
    plen, nlen = g.i32(plen), g.i32(nlen)
    rx.rx_step_maps(run.req, plen, nlen, run.rtt, b.num_slots, indptr, seq, pos, slots, dev_status=run.status,
                    pages=None if pages is None else g.i32(pages), page_size=size)
    o, lse = torch.full_like(run.q, float("nan")), torch.full(run.q.shape[:2], float("nan"), device="cuda")
    most = STAGED if "staged" in call else int(nlen.max())
    ws = run.workspace(most)
    args = (run.q, o, lse, indptr, run.req, plen, nlen, run.rtt, most, b.scale)
    if call.startswith("rules"):
        if run.f8:
            rx.rx_attn_extend_rules_fp8(run.k, run.v, run.ks, run.vs, *args, run.rules, ws, run.status)
        else:
            rx.rx_attn_extend_rules(run.k, run.v, *args, run.rules, ws, run.status)
    elif run.f8:
        rx.rx_attn_extend_fp8(run.k, run.v, run.ks, run.vs, *args, None, run.status)
    else:
        rx.rx_attn_extend(run.k, run.v, *args, run.status, workspace=ws if "staged" in call else None)
    torch.cuda.synchronize()
    return o.float().cpu().numpy(), lse.cpu().numpy(), int(run.status.item()), indptr.tolist(), run


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("tokens", [102, 101, 60, 31, 0])
def test_requests_whose_rows_were_cut_are_left_out(call, tokens):
    """q and o have rows behind the lists' end; they are not the call's."""
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    new = [31, 0, 70, 1]
    b = RulesBatch(41, 8, 2, 64, [130, 20, 257, 63], new, cap=50.0 if call.startswith("rules") else 0.0)
    o, lse, status, indptr, run = _run(call, b, 102, b.prefix_len, b.new_len, tokens)
    assert indptr == [min(x, tokens) for x in b.indptr.tolist()]
    assert status == (rx.RX_DEV_BAD_LEN if tokens < 102 else 0)
    ref = b.oracle(run.q64, run.k64, run.v64)
    for r, (s, e) in enumerate(zip(b.indptr, b.indptr[1:])):
        if e <= tokens:
            check(o[s:e], lse[s:e], tuple(x[s:e] for x in ref), b, f"request {r}")
        else:
            assert np.isnan(o[s:e]).all() and np.isnan(lse[s:e]).all(), f"request {r}"


@pytest.mark.parametrize("call", CALLS)
def test_a_request_that_the_lists_leave_out(call):
    """A request past the pages' positions, though not past the slot lists' stride: its tokens have no rows."""
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    from tests import _gpu as g
    new = [20, 33, 9]
    b = RulesBatch(42, 8, 2, 64, [30, 40, 12], new, cap=30.0 if call.startswith("rules") else 0.0)
    size = 8
    wide = 8                                                     # 64 positions; request 1 wants 73
    pages = np.random.default_rng(1).permutation(b.rtt.shape[0] * wide).reshape(-1, wide)
    b.num_slots = pages.size * size
    rng = np.random.default_rng(2)
    b.k, b.v = (rng.standard_normal((b.num_slots, 2, 64)).astype(np.float32) for _ in range(2))
    for r in (0, 2):                                             # the cached positions; the new ones come from the call
        p = np.arange(b.prefix_len[r] + new[r])
        b.rtt[b.req_idx[r], :len(p)] = pages[b.req_idx[r], p // size] * size + p % size
    b.rtt[b.req_idx[1], :73] = np.arange(73)
    o, lse, status, indptr, run = _run(call, b, 62, b.prefix_len, b.new_len, 62, pages, size)
    assert status == rx.RX_DEV_BAD_LEN and indptr == [0, 20, 20, 29]
    assert g is not None
    q64 = run.q64.copy()
    q64[53:62] = q64[20:29]                                      # request 2's rows are where the lists put them
    ref = b.oracle(q64, run.k64, run.v64)
    check(o[:20], lse[:20], tuple(x[:20] for x in ref), b, "request 0")
    check(o[20:29], lse[20:29], tuple(x[53:62] for x in ref), b, "request 2")
    assert np.isnan(o[29:]).all() and np.isnan(lse[29:]).all()
