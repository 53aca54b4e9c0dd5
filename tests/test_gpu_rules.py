"""GPU parity of rx_attn_extend_rules, rx_attn_decode_rules and their FP8 forms
against the fp64 oracle.  Bounds: tests/_rules.check."""
import numpy as np
import pytest

from oracle import fp8
from prefix_shared_kv_radixattention_gb300 import inputs
from tests import _rules
from tests._rules import RulesBatch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

STAGED = 1025      # a host bound that makes the call copy the contexts, however short the requests are


def _g():
    from tests import _gpu
    return _gpu


class Run:
    """One batch on the device, bf16 or E4M3 pools."""

    def __init__(self, b, f8=False, ks=0.07, vs=0.03, layers=0, layer=0, edit=None):
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        g = _g()
        self.b, self.f8, self.ks, self.vs, self.layer = b, f8, ks, vs, layer
        if f8:
            kc, vc = fp8.encode(b.k / np.float32(ks)), fp8.encode(b.v / np.float32(vs))
            self.k64, self.v64 = fp8.decode(kc) * ks, fp8.decode(vc) * vs
            k, v = (torch.from_numpy(np.ascontiguousarray(c.astype(np.uint8))).cuda() for c in (kc, vc))
        else:
            kc, vc = inputs.bf16_round(b.k), inputs.bf16_round(b.v)
            self.k64, self.v64 = (inputs.bf16_to_f32(c).astype(np.float64) for c in (kc, vc))
            k, v = g.to_dev(kc), g.to_dev(vc)
        if edit is not None:
            edit(self, k, v)
        if layers:   # the other layers hold junk
            full = [torch.full((layers, *k.shape), 37, dtype=k.dtype, device="cuda") for _ in range(2)]
            full[0][layer], full[1][layer] = k, v
            k, v = full
        self.k, self.v = k, v
        qb = inputs.bf16_round(b.q)
        self.q64 = inputs.bf16_to_f32(qb).astype(np.float64)
        self.q = g.to_dev(qb)
        self.indptr, self.req, self.plen, self.nlen = (g.i32(x) for x in (b.indptr, b.req_idx, b.prefix_len, b.new_len))
        self.rtt = g.i32(b.rtt)
        self.seq = g.i32(b.prefix_len + b.new_len)
        dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
        self.rules = rx.AttnRules(b.cap, b.window, dev(b.slopes), dev(b.see_from), dev(b.see_to))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def workspace(self, max_len=None):
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        b = self.b
        context = int((b.prefix_len + b.new_len).sum())
        return torch.empty(rx.rx_attn_rules_workspace(context, len(b.new_len), b.hq, b.hkv, b.d,
                                                      max_len or max(1, int(b.new_len.max()))), dtype=torch.uint8,
                           device="cuda")

    def extend(self, o, lse, ws, max_len=None, stream=None):
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        b = self.b
        args = (self.q, o, lse, self.indptr, self.req, self.plen, self.nlen, self.rtt,
                max_len or max(1, int(b.new_len.max())), b.scale, self.rules, ws, self.status)
        if self.f8:
            rx.rx_attn_extend_rules_fp8(self.k, self.v, self.ks, self.vs, *args, stream=stream, layer=self.layer)
        else:
            rx.rx_attn_extend_rules(self.k, self.v, *args, stream=stream, layer=self.layer)

    def decode(self, o, lse, ws, stream=None):
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        args = (self.q, o, lse, self.req, self.seq, self.rtt, self.b.scale, self.rules, ws, self.status)
        if self.f8:
            rx.rx_attn_decode_rules_fp8(self.k, self.v, self.ks, self.vs, *args, stream=stream, layer=self.layer)
        else:
            rx.rx_attn_decode_rules(self.k, self.v, *args, stream=stream, layer=self.layer)

    def __call__(self, call="extend", max_len=None, with_lse=True):
        g = _g()
        og = g.Guarded(self.q.shape, torch.bfloat16)
        lg = g.Guarded(self.q.shape[:2], torch.float32) if with_lse else None
        ws = self.workspace(max_len)
        if call == "extend":
            self.extend(og.t, lg.t if with_lse else None, ws, max_len)
        else:
            self.decode(og.t, lg.t if with_lse else None, ws)
        torch.cuda.synchronize()
        og.check("o")
        if with_lse:
            lg.check("lse")
        return og.t.float().cpu().numpy(), (lg.t.cpu().numpy() if with_lse else None)

    def check(self, call="extend", max_len=None, what="", with_lse=True):
        o, lse = self(call, max_len, with_lse)
        assert int(self.status.item()) == 0, what
        return _rules.check(o, lse, self.b.oracle(self.q64, self.k64, self.v64), self.b, what)


HEADS = [(4, 4, 64), (8, 2, 128), (8, 1, 64), (16, 1, 128)]
RULES = [dict(cap=30.0), dict(cap=50.0, spread=12.0), dict(cap=80.0, spread=12.0), dict(window=17), dict(window=150, cap=5.0),
         dict(slopes=True), dict(slopes=True, cap=20.0, window=200), dict(mask="docs"), dict(mask="prefix", cap=50.0),
         dict(mask="spans"), dict(mask="spans", window=64, slopes=True), dict(mask="any", cap=50.0), dict(mask="any", window=40),
         dict(mask="any", slopes=True), dict()]


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("path", ["split", "staged"])
@pytest.mark.parametrize("rules", RULES, ids=str)
@pytest.mark.parametrize("heads", HEADS[:2], ids=str)
def test_extend(heads, rules, path, f8):
    b = RulesBatch(11, *heads, [130, 0, 257, 63], [31, 70, 1, 64], **rules)
    Run(b, f8).check(max_len=STAGED if path == "staged" else None)


@pytest.mark.parametrize("path", ["split", "staged"])
@pytest.mark.parametrize("heads", HEADS[2:] + [(32, 1, 64), (128, 1, 128)], ids=str)
def test_extend_many_heads(heads, path):
    b = RulesBatch(12, *heads, [140, 3], [5, 9], cap=50.0, window=100, mask="prefix")
    Run(b).check(max_len=STAGED if path == "staged" else None)


@pytest.mark.parametrize("path", ["split", "staged"])
@pytest.mark.parametrize("rules", [dict(cap=50.0), dict(window=100, mask="spans"), dict(window=300, slopes=True)], ids=str)
def test_extend_several_row_groups(rules, path):
    """More query rows than a CTA takes, contexts that end inside tiles."""
    b = RulesBatch(13, 8, 1, 64, [515, 128], [97, 129], **rules)
    Run(b).check(max_len=STAGED if path == "staged" else None)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("window", [0, 1, 40, 129, 300, 5000])
def test_extend_shared_prefixes(window, f8):
    """Requests that share their first positions: staged once, with and without a window that begins inside them."""
    b = RulesBatch(14, 4, 2, 64, [400, 390, 700, 200], [20, 33, 5, 9], window=window, cap=50.0, shared=390)
    Run(b, f8).check(max_len=STAGED)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("rules", [dict(cap=30.0), dict(cap=80.0, spread=10.0), dict(window=1), dict(window=128), dict(window=200),
                                   dict(slopes=True, cap=50.0), dict(mask="docs"), dict()], ids=str)
@pytest.mark.parametrize("heads", HEADS + [(6, 2, 64), (5, 1, 128), (128, 1, 64)], ids=str)
def test_decode(heads, rules, f8):
    """One token a request, contexts from one position on; see_from at every place."""
    ctx = [1, 2, 127, 128, 129, 640, 1000]
    docs = rules.get("mask") == "docs"
    b = RulesBatch(15, *heads, [n - 1 for n in ctx], [1] * len(ctx), **{k: v for k, v in rules.items() if k != "mask"})
    if docs:
        b.see_from = np.array([0, 1, 127, 64, -3, 300, 999], np.int32)     # request 2 sees nothing
    Run(b, f8).check("decode")


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
def test_decode_over_many_ctas(f8):
    """A context cut among all CTAs, joined from their parts."""
    b = RulesBatch(16, 2, 1, 128, [40000, 17], [1, 1], cap=50.0)
    Run(b, f8).check("decode")


@pytest.mark.parametrize("path", ["split", "staged", "decode"])
@pytest.mark.parametrize("rules", [dict(cap=2.0, spread=12.0), dict(cap=50.0, spread=40.0), dict(cap=80.0, spread=60.0),
                                   dict(cap=1e-3)], ids=str)
def test_scores_far_beyond_the_cap(rules, path):
    """Scores of every size against the cap: within it, around it, many times it."""
    new = [1, 1, 1] if path == "decode" else [40, 70, 3]
    for heads, f8 in ((HEADS[0], False), (HEADS[1], False), (HEADS[1], True)):
        b = RulesBatch(27, *heads, [100, 3, 260], new, **rules)
        b.q[::2] *= np.float32(0.02)                                   # rows with small scores next to rows with large ones
        Run(b, f8).check("decode" if path == "decode" else "extend", STAGED if path == "staged" else None)


@pytest.mark.parametrize("path", ["split", "staged", "decode"])
@pytest.mark.parametrize("cap", [1e3, 1e6])
def test_large_caps_cost_nothing(cap, path):
    new = [1, 1] if path == "decode" else [40, 7]
    for heads, f8 in ((HEADS[0], False), (HEADS[1], False), (HEADS[1], True)):
        b = RulesBatch(28, *heads, [100, 260], new, cap=cap)
        run = Run(b, f8)
        o, lse = run("decode" if path == "decode" else "extend", STAGED if path == "staged" else None)
        _rules.check(o, lse, b.oracle(run.q64, run.k64, run.v64), b, cap=30.0)


def test_without_lse():
    b = RulesBatch(17, 8, 2, 64, [100], [9], cap=50.0)
    Run(b).check(with_lse=False)
    b = RulesBatch(17, 8, 2, 64, [100], [1], cap=50.0)
    Run(b).check("decode", with_lse=False)


@pytest.mark.parametrize("path", ["split", "staged"])
def test_layers(path):
    b = RulesBatch(18, 4, 2, 64, [200, 50], [20, 7], window=90, cap=50.0)
    for f8 in (False, True):
        Run(b, f8, layers=3, layer=2).check(max_len=STAGED if path == "staged" else None)


@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 2, 128)], ids=str)
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("path", ["split", "staged", "decode"])
@pytest.mark.parametrize("rules", [dict(window=70), dict(mask="docs"), dict(cap=50.0, window=70)], ids=str)
def test_not_finite_where_a_token_does_not_see(rules, path, f8, heads):
    """NaN and infinities of K and V reach the tokens that see their position, and no other."""
    new = [1, 1] if path == "decode" else [60, 12]
    b = RulesBatch(19, *heads, [300, 90], new, **{**rules, **({"mask": ""} if path == "decode" else {})})
    if path == "decode" and "mask" in rules:
        b.see_from = np.array([280, 40], np.int32)
    at = [(0, 231), (0, 240), (0, 20), (0, 299), (0, 300 + new[0] - 1), (1, 30)]   # (request, position)
    bad = [float("nan"), float("inf"), float("nan"), float("-inf"), float("inf"), float("nan")]

    def edit(run, k, v):
        for (r, p), x in zip(at, bad):
            s = int(b.rtt[b.req_idx[r], p])
            v[s, 1, 5] = 0x7F if f8 else x
            if p < 30:                                  # its K as well
                k[s] = 0x7F if f8 else x

    run = Run(b, f8, edit=edit)
    o, lse = run("decode" if path == "decode" else "extend", STAGED if path == "staged" else None)
    assert int(run.status.item()) == 0
    ref_o, ref_l, ref_a = b.oracle(run.q64, run.k64, run.v64)
    from oracle import rules as oracle_rules
    row = 0
    for r in range(2):
        for i in range(new[r]):
            p = int(b.prefix_len[r]) + i
            lo, hi = oracle_rules.seen(p, int(b.prefix_len[r]) + new[r], b.window,
                                       0 if b.see_from is None else int(b.see_from[row]))
            hit = {x if not f8 else float("nan") for (rr, pp), x in zip(at, bad) if rr == r and lo <= pp < hi}
            if any(rr == r and lo <= pp < hi and pp < 30 for rr, pp in at):   # a score that is not a number
                assert np.isnan(o[row]).all() and np.isnan(lse[row]).all()
                o[row], lse[row] = ref_o[row], ref_l[row]
                hit = set()
            for h in range(heads[0] // 2, heads[0]):    # the heads of kv head 1
                got = o[row, h, 5]
                if hit:
                    want_nan = any(np.isnan(x) for x in hit) or len(hit) > 1
                    assert np.isnan(got) if want_nan else got == next(iter(hit)), (r, i, h, got, hit)
                    o[row, h, 5] = ref_o[row, h, 5]
            row += 1
    _rules.check(o, lse, (ref_o, ref_l, ref_a), b)


@pytest.mark.parametrize("path", ["split", "staged"])
def test_bad_slots_and_lengths(path):
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    max_len = STAGED if path == "staged" else None
    b = RulesBatch(20, 4, 2, 64, [200, 60], [10, 12], cap=50.0)
    b.rtt[b.req_idx[0], 150] = b.num_slots
    b.rtt[b.req_idx[1], 3] = -1
    run = Run(b)
    o, lse = run(max_len=max_len)
    assert int(run.status.item()) == rx.RX_DEV_BAD_SLOT
    _rules.check(o, lse, b.oracle(run.q64, run.k64, run.v64), b)       # such rows read as zeros
    b = RulesBatch(21, 4, 2, 64, [200, 60], [10, 12], cap=50.0)
    run = Run(b)
    run.plen[0] = b.rtt.shape[1] - 9                                   # one position past the stride
    o, lse = run(max_len=max_len)
    assert int(run.status.item()) == rx.RX_DEV_BAD_LEN
    assert np.isnan(o[:10]).all() and not np.isnan(o[10:]).any()       # left as they were


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("path", ["split", "staged", "decode"])
def test_slots_before_the_window_may_be_anything(path, f8):
    new = [1, 1, 1] if path == "decode" else [60, 12, 30]
    for heads in ((4, 2, 64), (8, 2, 128)):
        b = RulesBatch(29, *heads, [300, 90, 260], new, window=70, cap=50.0, shared=280)
        for r in range(3):
            b.rtt[b.req_idx[r], :max(0, int(b.prefix_len[r]) - 69)] = (-1, b.num_slots, -(2 ** 31))[r]
        Run(b, f8).check("decode" if path == "decode" else "extend", STAGED if path == "staged" else None)


@pytest.mark.parametrize("window", [100, 130, 150, 200])
def test_shared_tiles_with_windows_that_begin_apart(window):
    """Requests that share their text, the windows' starts inside one tile and across tiles, in either order."""
    for prefixes in ([400, 380, 390, 130], [380, 400, 130, 390]):
        b = RulesBatch(30, 4, 2, 64, prefixes, [20, 33, 5, 9], window=window, shared=384)
        Run(b).check(max_len=STAGED)


def test_decode_leaves_out_requests_without_a_context():
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    b = RulesBatch(22, 4, 2, 64, [99, 20, 30], [1, 1, 1], cap=50.0)
    run = Run(b)
    run.seq[1] = 0
    o, lse = run("decode")
    assert int(run.status.item()) == 0 and np.isnan(o[1]).all() and np.isnan(lse[1]).all()
    r = b.oracle(run.q64, run.k64, run.v64)
    _rules.check(o[[0, 2]], lse[[0, 2]], tuple(x[[0, 2]] for x in r), b)
    run.seq[1] = -1
    o, lse = run("decode")
    assert int(run.status.item()) == rx.RX_DEV_BAD_LEN and np.isnan(o[1]).all()


def test_staged_contexts_past_the_workspace():
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    b = RulesBatch(23, 4, 2, 64, [500, 600], [10, 12], cap=50.0)
    run = Run(b)
    ws = run.workspace()[:900 * b.hkv * b.d * 4]        # room for 900 rows of K and V less its head (1,280 are needed)
    o, lse = torch.full_like(run.q, float("nan")), torch.full(run.q.shape[:2], float("nan"), device="cuda")
    run.extend(o, lse, ws, STAGED)
    torch.cuda.synchronize()
    assert int(run.status.item()) == rx.RX_DEV_BAD_LEN and bool(torch.isnan(o).all())


@pytest.mark.parametrize("max_len", [None, STAGED], ids=["split", "staged"])
def test_captured_calls_on_a_stream(max_len):
    """A captured call replayed on changed inputs, two graphs with workspaces of their own in flight at once."""
    runs, outs, graphs = [], [], []
    for seed in (24, 25):
        run = Run(RulesBatch(seed, 8, 2, 64, [300, 40], [20, 33], cap=50.0, window=128, mask="prefix"))
        ws = run.workspace(max_len)
        o, lse = torch.zeros_like(run.q), torch.zeros(run.q.shape[:2], device="cuda")
        run.extend(o, lse, ws, max_len)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run.extend(o, lse, ws, max_len)
        runs.append((run, ws))
        outs.append((o, lse))
        graphs.append(graph)
    for run, _ in runs:
        run.v.mul_(-2)
        run.v64 = run.v64 * -2
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (run, _), (o, lse) in zip(runs, outs):
        _rules.check(o.float().cpu().numpy(), lse.cpu().numpy(), run.b.oracle(run.q64, run.k64, run.v64), run.b)


def test_results_do_not_depend_on_the_run():
    """The same call gives the same bits: nothing is joined in an order that varies."""
    for call, new, max_len in (("decode", [1, 1], None), ("extend", [40, 21], None), ("extend", [40, 21], STAGED)):
        run = Run(RulesBatch(26, 8, 2, 128, [3000, 777], new, cap=50.0))
        first = run(call, max_len)
        for _ in range(3):
            again = run(call, max_len)
            assert all(np.array_equal(x, y) for x, y in zip(first, again))
