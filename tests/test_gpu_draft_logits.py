"""rx_logits_process against the oracle, bit for bit: every step of the
definition is one fp32 rounding, so nothing may differ."""
import numpy as np
import pytest

from oracle import draft
from prefix_shared_kv_radixattention_gb300 import inputs
from tests import _draft

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _g():
    from tests import _gpu
    return _gpu


class Case:
    def __init__(self, seed, n_req, vocab, hist=0, bias=0, trees=None, masks="tree", states=0, penalties=True, bf16=False,
                 pad=0, prompt=0.7):
        rng = np.random.default_rng(seed)
        self.n_req, self.vocab, self.bf16 = n_req, vocab, bf16
        self.trees = trees
        self.indptr = None if trees is None else np.concatenate([[0], np.cumsum(trees)]).astype(np.int32)
        self.rows = n_req if trees is None else int(self.indptr[-1])
        x = (4 * rng.standard_normal((self.rows, vocab + pad))).astype(np.float32)
        self.bits = inputs.bf16_round(x)
        if bf16:
            x = inputs.bf16_to_f32(self.bits)
        self.x = x
        low = max(1, vocab // 20)
        self.hist = [np.where(rng.random(m) < 0.5, rng.integers(0, low, m), rng.integers(0, vocab, m)).astype(np.int32)
                     for m in (rng.integers(0, hist + 1, n_req) if hist else [0] * n_req)]
        self.prompt = np.array([int(len(h) * prompt) for h in self.hist], np.int32)
        f = np.float32
        self.rep = (1 + rng.random(n_req)).astype(f) if penalties else None
        self.freq = rng.random(n_req).astype(f) if penalties else None
        self.pres = rng.random(n_req).astype(f) if penalties else None
        if penalties and n_req > 2:
            self.rep[1], self.freq[1], self.pres[1] = 1, 0, 0    # a request without penalties among the others
        self.bias = None
        if bias:
            self.bias = []
            for _ in range(n_req):
                m = int(rng.integers(0, bias + 1))
                t = np.sort(rng.integers(0, vocab, m))
                if m > 3:
                    t[1:3] = t[0]                                # the same id three times
                    t = np.sort(t)
                self.bias.append((t.astype(np.int32), (5 * rng.standard_normal(m)).astype(f)))
        self.draft = self.see = None
        if trees is not None:
            self.draft = [rng.integers(0, vocab, t).astype(np.int32) for t in trees]
            for d in self.draft:
                d[1:] = np.where(rng.random(len(d) - 1) < 0.4, d[:-1], d[1:]) if len(d) > 1 else d[1:]
            self.see = [draft.tree_mask(_draft.random_parents(rng, t)) if masks == "tree" else
                        np.tril(np.ones((t, t), bool)) if masks == "chain" else rng.random((t, t)) < 0.4 for t in trees]
            self.words = (max(max(trees), 1) + 31) // 32
            m = np.ones((self.rows, self.words * 32), bool)      # bits past a tree: ignored
            for b, t in enumerate(trees):
                m[self.indptr[b]:self.indptr[b + 1], :t] = self.see[b]
            self.mask = None if masks == "chain" else _draft.pack(m, self.words)
        self.allow = self.allow_row = None
        if states:
            share = rng.choice([0.0005, 0.3, 0.97], states)
            self.allow = rng.random((states, vocab)) < share[:, None]
            self.allow[0] = False                                # a state that allows nothing
            self.allow_row = rng.integers(-1, states, self.rows).astype(np.int32)

    def reference(self):
        rows = None if self.trees is None else [range(self.indptr[b], self.indptr[b + 1]) for b in range(self.n_req)]
        out = draft.logits_process(self.x, self.vocab, self.hist, self.prompt, self.rep, self.freq, self.pres, self.bias, rows,
                                   self.draft, self.see, self.allow, self.allow_row)
        return np.stack([out[r] for r in range(self.rows)]) if self.rows else np.zeros((0, self.vocab), np.float32)

    def rules(self):
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        dev = lambda a, dt: None if a is None else torch.from_numpy(np.ascontiguousarray(a, dt)).cuda()  # noqa: E731
        ptr = lambda lists: np.concatenate([[0], np.cumsum([len(t) for t in lists])])  # noqa: E731
        kw = dict(hist=dev(np.concatenate(self.hist), np.int32), hist_ptr=dev(ptr(self.hist), np.int64),
                  prompt_len=dev(self.prompt, np.int32), repetition=dev(self.rep, np.float32),
                  frequency=dev(self.freq, np.float32), presence=dev(self.pres, np.float32))
        if self.bias is not None:
            kw |= dict(bias_tok=dev(np.concatenate([t for t, _ in self.bias]), np.int32),
                       bias_val=dev(np.concatenate([v for _, v in self.bias]), np.float32),
                       bias_ptr=dev(ptr([t for t, _ in self.bias]), np.int64))
        if self.trees is not None:
            kw |= dict(qo_indptr=dev(self.indptr, np.int32), draft_tok=dev(np.concatenate(self.draft), np.int32),
                       tree_mask=dev(self.mask, np.int32))
        if self.allow is not None:
            kw |= dict(allow=dev(_draft.pack(self.allow, (self.vocab + 127) // 128 * 4), np.int32),
                       allow_row=dev(self.allow_row, np.int32))
        return rx.LogitsRules(self.n_req, self.vocab, **kw)

    def logits(self):
        return _g().to_dev(self.bits) if self.bf16 else torch.from_numpy(self.x.copy()).cuda()


def _same(got, ref):
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got, ref, equal_nan=True), f"{(got != ref).sum()} of {ref.size} differ"


def _run(c, out=None, **kw):
    g = _g()
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    og = g.Guarded((c.rows, c.vocab), torch.float32)
    rx.rx_logits_process(c.rules(), c.logits(), og.t, status, **kw)
    torch.cuda.synchronize()
    og.check("out")
    return og.t.cpu().numpy(), int(status.item())


CASES = {
    "one_row": dict(n_req=1, vocab=32000, hist=500, bias=8),
    "one_id": dict(n_req=3, vocab=1, hist=4, states=2),
    "small": dict(n_req=7, vocab=130, hist=300, bias=20, states=3),
    "odd_vocab": dict(n_req=5, vocab=5003, hist=900, bias=30, states=4),
    "odd_vocab_bf16": dict(n_req=5, vocab=5003, hist=900, bias=30, states=4, bf16=True),
    "padded_rows": dict(n_req=4, vocab=4999, hist=900, bias=30, states=4, pad=13),
    "padded_rows_bf16": dict(n_req=4, vocab=4997, hist=900, bias=30, states=4, pad=11, bf16=True),
    "wide": dict(n_req=3, vocab=128256, hist=20000, bias=300, states=5),
    "wide_bf16": dict(n_req=9, vocab=70000, hist=3000, bias=300, states=5, bf16=True),
    "batch": dict(n_req=200, vocab=9000, hist=100, bias=5, states=4),
    "only_mask": dict(n_req=6, vocab=3333, penalties=False, states=6),
    "only_bias": dict(n_req=6, vocab=3333, penalties=False, bias=40),
    "nothing": dict(n_req=6, vocab=3333, penalties=False),
    "no_prompt": dict(n_req=6, vocab=333, hist=900, prompt=0.0),
    "all_prompt": dict(n_req=6, vocab=333, hist=900, prompt=1.0),
    "tree": dict(n_req=4, vocab=6000, hist=800, bias=20, states=5, trees=[5, 0, 33, 1]),
    "tree_bf16": dict(n_req=3, vocab=20001, hist=800, bias=20, states=5, trees=[16, 70, 3], bf16=True),
    "tree_chain": dict(n_req=3, vocab=6000, hist=80, trees=[5, 9, 1], masks="chain"),
    "tree_any": dict(n_req=3, vocab=40, hist=80, trees=[64, 9, 31], masks="any", states=3, bias=9),
    "tree_one": dict(n_req=1, vocab=128256, hist=5000, trees=[20], states=3),
}


@pytest.mark.parametrize("name", CASES)
def test_parity(name):
    c = Case(sum(map(ord, name)), **CASES[name])
    got, status = _run(c)
    assert status == 0
    _same(got, c.reference())


def test_in_place():
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    for kw in (dict(pad=0), dict(pad=3), dict(trees=[3, 30, 2])):
        c = Case(3, 3, 5000, hist=400, bias=20, states=3, **kw)
        x = c.logits()
        rx.rx_logits_process(c.rules(), x, x)
        _same(x.cpu().numpy()[:, :5000], c.reference())
        assert np.array_equal(x.cpu().numpy()[:, 5000:], c.x[:, 5000:])   # padding is left as it was


def test_values_that_are_not_finite():
    """NaN and infinities pass through the rules as fp32 arithmetic has them;
    a masked place is -inf whatever it held."""
    c = Case(4, 4, 700, hist=300, bias=10, states=3)
    rng = np.random.default_rng(1)
    for v in (np.nan, np.inf, -np.inf, -0.0, 3.4e38):
        c.x[rng.random(c.x.shape) < 0.05] = v
    got, status = _run(c)
    assert status == 0
    _same(got, c.reference())


def test_rows_behind_the_last_are_left_alone():
    g = _g()
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = Case(5, 2, 900, hist=30, states=2, trees=[4, 3])
    r = c.rules()
    for t in r.row_tensors:      # padded row tensors
        assert t.shape[0] == 7
    x = torch.cat([c.logits(), torch.ones(5, 900, device="cuda")])
    out = torch.full((12, 900), 7.0, device="cuda")
    pad = lambda t: torch.cat([t, torch.zeros(5, *t.shape[1:], dtype=t.dtype, device="cuda")])  # noqa: E731
    kw = {k: getattr(c, k) for k in ()}
    rules = rx.LogitsRules(2, 900, hist=g.i32(np.concatenate(c.hist)),
                           hist_ptr=torch.tensor([0, len(c.hist[0]), len(c.hist[0]) + len(c.hist[1])], device="cuda"),
                           prompt_len=g.i32(c.prompt), repetition=torch.from_numpy(c.rep).cuda(),
                           frequency=torch.from_numpy(c.freq).cuda(), presence=torch.from_numpy(c.pres).cuda(),
                           qo_indptr=g.i32(c.indptr), draft_tok=pad(g.i32(np.concatenate(c.draft))),
                           tree_mask=pad(torch.from_numpy(c.mask).cuda()),
                           allow=torch.from_numpy(_draft.pack(c.allow, (900 + 127) // 128 * 4)).cuda(),
                           allow_row=pad(g.i32(c.allow_row)), **kw)
    rx.rx_logits_process(rules, x, out)
    _same(out.cpu().numpy()[:7], c.reference())
    assert (out[7:] == 7.0).all()


@pytest.mark.parametrize("where", ["hist", "draft", "bias"])
def test_token_ids_outside_the_vocabulary(where):
    c = Case(6, 3, 3000, hist=60, bias=9, trees=[4, 5, 6], prompt=0.5)
    if where == "hist":
        c.hist[0] = np.concatenate([c.hist[0], [3000, -5, 2**31 - 1, -2**31]]).astype(np.int32)
    elif where == "draft":
        c.draft[2][:] = [-1, 3000, 5, 5, -9, 2]
    else:
        t, v = c.bias[0]
        c.bias[0] = (np.concatenate([[-3], t, [3000, 4000]]).astype(np.int32), np.concatenate([[1], v, [2, 3]]).astype(np.float32))
    got, status = _run(c)
    assert status == 32       # RX_DEV_BAD_TOKEN
    _same(got, c.reference())


def test_bias_lists_out_of_order_and_mask_rows_out_of_range_are_flagged():
    c = Case(7, 2, 3000, bias=9, penalties=False)
    c.bias[1] = (np.array([9, 8, 7], np.int32), np.ones(3, np.float32))
    got, status = _run(c)
    assert status == 32
    _same(got[:1], c.reference()[:1])
    c = Case(8, 4, 3000, states=3)
    c.allow_row[:] = [1, 3, -2, -1]
    got, status = _run(c)
    assert status == 16       # RX_DEV_BAD_STATE
    _same(got, c.reference())
    assert np.isneginf(got[1:3]).all()


def test_long_history_of_one_token_and_repeated_calls():
    """Counts are whole numbers whatever the order they are added in."""
    c = Case(9, 2, 50000, hist=10, prompt=0.0)
    c.hist = [np.full(100000, 77, np.int32), np.arange(50000, dtype=np.int32)]
    c.prompt = np.array([3, 0], np.int32)
    got, status = _run(c)
    assert status == 0
    _same(got, c.reference())
    assert np.array_equal(_run(c)[0], got)


def test_captured_call_sees_new_history():
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = Case(10, 3, 4000, hist=200, bias=10, states=3)
    rules, x = c.rules(), c.logits()
    out = torch.zeros(3, 4000, device="cuda")
    graph = torch.cuda.CUDAGraph()
    rx.rx_logits_process(rules, x, out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rx.rx_logits_process(rules, x, out)
    hist = rules._keep[0]
    new = np.random.default_rng(0).integers(0, 4000, hist.numel()).astype(np.int32)
    hist.copy_(torch.from_numpy(new))
    at = np.concatenate([[0], np.cumsum([len(h) for h in c.hist])])
    c.hist = [new[at[i]:at[i + 1]] for i in range(3)]
    graph.replay()
    torch.cuda.synchronize()
    _same(out.cpu().numpy(), c.reference())


def test_binding_refuses_wrong_tensors():
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = Case(11, 3, 400, hist=20, states=2)
    rules, x = c.rules(), c.logits()
    out = torch.zeros(3, 400, device="cuda")
    for a, b in ((x.half(), out), (x, out.bfloat16()), (x[:, :399], out), (x, out[:2]), (x.cpu(), out), (x.t(), out),
                 (x[:2], out[:2])):
        with pytest.raises((TypeError, ValueError, rx.RxError)):
            rx.rx_logits_process(rules, a, b)
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (dict(hist=i), dict(repetition=torch.ones(2, device="cuda")), dict(prompt_len=i.long()), dict(bias_tok=i),
                dict(allow=i[None]), dict(draft_tok=i), dict(allow=torch.zeros(2, 12, dtype=torch.int32, device="cuda"),
                                                             allow_row=i)):
        with pytest.raises((TypeError, ValueError)):
            rx.LogitsRules(3, 400, **bad)
