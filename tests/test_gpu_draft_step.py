"""The verification step of drafted tokens as a serving loop runs it: norm,
rotation and store of the drafted tokens' rows, attention of their trees, the
rules on their logits, the constrained step that picks each node's next token;
eager, and captured and replayed with other requests in the same tensors.
Then the calls at the edges of the logits rules and of the FP8 codes."""
import numpy as np
import pytest

from oracle import draft, fp8
from prefix_shared_kv_radixattention_gb300 import inputs
from tests import _draft
from tests.test_gpu_draft_logits import Case, _same
from tests.test_gpu_draft_norm import _check_bf16, _check_codes

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HQ, HKV, D, VOCAB, BASE, EPS = 8, 2, 64, 300, 10000.0, 1e-6
KS, VS = 0.02, 0.03
STATES = 5


def _g():
    from tests import _gpu
    return _gpu


def _machine(seed):
    """A state machine in which every state allows about half of the ids."""
    rng = np.random.default_rng(seed)
    lists = [np.sort(rng.choice(VOCAB, 150, replace=False)) for _ in range(STATES)]
    ptr = np.concatenate([[0], np.cumsum([len(t) for t in lists])]).astype(np.int32)
    tok = np.concatenate(lists).astype(np.int32)
    return ptr, tok, rng.integers(0, STATES, len(tok)).astype(np.int32), lists


class Inputs:
    """Host inputs of one step: requests with a cached prefix, a drafted tree
    each, its projected rows, the tokens so far."""

    def __init__(self, seed, prefixes, trees):
        rng = np.random.default_rng(seed)
        self.trees, self.prefixes = trees, np.array(prefixes, np.int32)
        self.indptr = np.concatenate([[0], np.cumsum(trees)]).astype(np.int32)
        n, B = int(self.indptr[-1]), len(trees)
        self.parents = [_draft.random_parents(rng, t) for t in trees]
        self.see = [draft.tree_mask(p) for p in self.parents]
        self.x = inputs.bf16_round(rng.standard_normal((n, HQ + 2 * HKV, D)).astype(np.float32))
        self.slots_of = rng.permutation(1000)[:sum(prefixes) + n].astype(np.int32)
        self.rtt = np.full((B + 1, 400), -1, np.int32)
        self.req = rng.permutation(B + 1)[:B].astype(np.int32)
        at = 0
        self.slots = []
        for b in range(B):
            m = prefixes[b] + trees[b]
            self.rtt[self.req[b], :m] = self.slots_of[at:at + m]
            self.slots.append(self.slots_of[at + prefixes[b]:at + m])
            at += m
        self.slots = np.concatenate(self.slots)
        self.k = rng.standard_normal((1000, HKV, D)).astype(np.float32)
        self.v = rng.standard_normal((1000, HKV, D)).astype(np.float32)
        self.hist = [rng.integers(0, VOCAB, 50).astype(np.int32) for _ in range(B)]
        self.prompt = rng.integers(0, 50, B).astype(np.int32)
        self.draft = [rng.integers(0, VOCAB, t).astype(np.int32) for t in trees]
        self.rules = [f.astype(np.float32) for f in (1 + rng.random(B), rng.random(B), rng.random(B))]
        self.state = rng.integers(0, STATES, n).astype(np.int32)


class Step:
    """The device tensors of a step, and the step itself."""

    def __init__(self, s, f8, machine):
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        g = _g()
        self.f8, self.B, n = f8, len(s.trees), int(s.indptr[-1])
        self.fsm = rx.Fsm(STATES, VOCAB, *machine[:3], 4)
        rng = np.random.default_rng(99)
        self.w = [g.to_dev(inputs.bf16_round((1 + 0.2 * rng.standard_normal(D)).astype(np.float32))) for _ in range(2)]
        self.head = torch.from_numpy((rng.standard_normal((HQ * D, VOCAB)) / 8).astype(np.float32)).cuda().bfloat16()
        kv = torch.uint8 if f8 else torch.bfloat16
        self.kp, self.vp = (torch.zeros(1000, HKV, D, dtype=kv, device="cuda") for _ in range(2))
        self.x = torch.zeros(n, HQ + 2 * HKV, D, dtype=torch.bfloat16, device="cuda")
        self.q, self.o = (torch.zeros(n, HQ, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.lse = torch.zeros(n, HQ, device="cuda")
        i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
        self.slots, self.pos, self.indptr, self.req, self.plen = i32(n), i32(n), i32(self.B + 1), i32(self.B), i32(self.B)
        self.rtt, self.mask, self.draft, self.state0, self.state = i32(self.B + 1, 400), i32(n, 1), i32(n), i32(n), i32(n)
        self.hist, self.prompt = i32(50 * self.B), i32(self.B)
        self.hist_ptr = 50 * torch.arange(self.B + 1, device="cuda")
        self.pen = [torch.ones(self.B, device="cuda") for _ in range(3)]
        self.raw, self.logits = (torch.zeros(n, VOCAB, device="cuda") for _ in range(2))
        self.tok, self.count = i32(n, 5), i32(n)
        self.fsm_ws = rx.fsm_workspace(n)
        self.status = i32(1)
        self.ws = torch.empty(rx.rx_attn_tree_workspace(self.B, HQ, HKV, D, 32), dtype=torch.uint8, device="cuda")
        self.rules = rx.LogitsRules(self.B, VOCAB, hist=self.hist, hist_ptr=self.hist_ptr, prompt_len=self.prompt,
                                    repetition=self.pen[0], frequency=self.pen[1], presence=self.pen[2],
                                    qo_indptr=self.indptr, draft_tok=self.draft, tree_mask=self.mask, allow=self.fsm.mask,
                                    allow_row=self.state0)

    def set(self, s):
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        built = [rx.rx_tree_mask_build(p, 1) for p in s.parents]
        self.depth = np.concatenate([d for _, d in built])
        pos = np.repeat(s.prefixes, s.trees) + self.depth
        kv = (lambda a, sc: fp8.encode(a / np.float32(sc)).astype(np.uint8)) if self.f8 else (lambda a, sc: inputs.bf16_round(a))
        for dst, src in ((self.kp, kv(s.k, KS)), (self.vp, kv(s.v, VS)), (self.x, s.x), (self.slots, s.slots), (self.pos, pos),
                         (self.indptr, s.indptr), (self.req, s.req), (self.plen, s.prefixes), (self.rtt, s.rtt),
                         (self.mask, np.concatenate([m for m, _ in built])), (self.draft, np.concatenate(s.draft)),
                         (self.state0, s.state), (self.hist, np.concatenate(s.hist)), (self.prompt, s.prompt),
                         *zip(self.pen, s.rules)):
            t = _g().to_dev(src) if src.dtype == np.uint16 else torch.from_numpy(np.ascontiguousarray(src)).cuda()
            dst.copy_(t.view(dst.dtype) if t.dtype != dst.dtype and t.element_size() == dst.element_size() else t)
        self.at = pos

    def run(self):
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        q, k, v = self.x[:, :HQ], self.x[:, HQ:HQ + HKV], self.x[:, HQ + HKV:]
        rest = (*self.w, self.slots, self.pos, BASE, EPS, self.status)
        tree = (self.q, self.o, self.lse, self.indptr, self.req, self.plen, self.mask, self.rtt, 32, D ** -0.5, self.ws, self.status)
        if self.f8:
            rx.rx_qk_norm_rope_store_fp8(self.kp, self.vp, KS, VS, q, self.q, k, v, *rest)
            rx.rx_attn_tree_fp8(self.kp, self.vp, KS, VS, *tree)
        else:
            rx.rx_qk_norm_rope_store(self.kp, self.vp, q, self.q, k, v, *rest)
            rx.rx_attn_tree(self.kp, self.vp, *tree)
        self.raw.copy_(self.o.view(len(self.o), HQ * D) @ self.head)
        rx.rx_logits_process(self.rules, self.raw, self.logits, self.status)
        self.state.copy_(self.state0)
        rx.rx_fsm_step(self.fsm, self.logits, self.state, self.tok, self.count, self.fsm_ws, self.status)

    def results(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        return [t.clone() for t in (self.q, self.kp, self.vp, self.o, self.lse, self.raw, self.logits, self.tok, self.count,
                                    self.state)]


def _check(s, step, res, machine):
    q, kp, vp, o, lse, raw, logits, tok, _, _ = res
    f64 = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    x = inputs.bf16_to_f32(s.x).astype(np.float64)
    w = [f64(t) for t in step.w]
    _check_bf16(f64(q), draft.qk_norm(x[:, :HQ], w[0], EPS), draft.qk_norm_rope(x[:, :HQ], w[0], step.at, BASE, EPS), "q")
    y, ref = (fn(x[:, HQ:HQ + HKV], w[1], *a) for fn, a in ((draft.qk_norm, (EPS,)),
                                                          (draft.qk_norm_rope, (step.at, BASE, EPS))))
    kn, vn = kp.cpu()[torch.from_numpy(s.slots).long()], vp.cpu()[torch.from_numpy(s.slots).long()]
    if step.f8:
        _check_codes(kn.numpy(), y, ref, float(np.float32(KS)), "k")
        k64, v64 = (fp8.decode(t.cpu().numpy()) * float(np.float32(sc)) for t, sc in ((kp, KS), (vp, VS)))
    else:
        _check_bf16(f64(kn), y, ref, "k")
        assert np.array_equal(f64(vn), x[:, HQ + HKV:])
        k64, v64 = f64(kp), f64(vp)
    ref = draft.tree_attention(f64(q), k64, v64, s.rtt, s.req, s.prefixes, s.indptr, s.see, D ** -0.5)
    _draft.check_tree(f64(o), lse.cpu().numpy(), ref)
    allow = np.zeros((STATES, VOCAB), bool)
    for i, t in enumerate(machine[3]):
        allow[i, t] = True
    rows = [range(s.indptr[b], s.indptr[b + 1]) for b in range(len(s.trees))]
    want = draft.logits_process(raw.cpu().numpy(), VOCAB, s.hist, s.prompt, *s.rules, None, rows, s.draft, s.see, allow, s.state)
    want = np.stack([want[r] for r in range(len(s.x))])
    _same(logits.cpu().numpy(), want)
    assert np.array_equal(tok.cpu().numpy()[:, 0], want.argmax(1))   # the first of the largest
    assert allow[s.state, tok.cpu().numpy()[:, 0]].all()


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
def test_verification_step(f8):
    machine = _machine(7)
    first, second = Inputs(1, [130, 0, 77, 256], [9, 1, 17, 5]), Inputs(2, [3, 200, 128, 31], [4, 20, 2, 6])
    step = Step(first, f8, machine)
    eager = []
    for s in (first, second):
        step.set(s)
        step.run()
        eager.append(step.results())
        _check(s, step, eager[-1], machine)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for s, want in zip((first, second, first), (*eager, eager[0])):
        step.set(s)
        graph.replay()
        for a, b in zip(step.results(), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_trees_too_large_for_the_rules_get_their_mask_only():
    """1,025 drafted tokens, and more of them than the mask has bits."""
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    for trees, words in (([1025, 3], None), ([33, 3], 1)):
        c = Case(12, 2, 90, hist=40, bias=5, states=3, trees=trees)
        if words:
            c.mask = np.ascontiguousarray(c.mask[:, :words])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.zeros(c.rows, 90, device="cuda")
        rx.rx_logits_process(c.rules(), c.logits(), out, status)
        assert int(status.item()) == rx.RX_DEV_BAD_LEN
        c.rep[0], c.freq[0], c.pres[0] = 1, 0, 0
        c.bias[0] = (np.zeros(0, np.int32), np.zeros(0, np.float32))
        _same(out.cpu().numpy(), c.reference())


def test_lists_that_descend_and_drafts_without_penalties():
    """A request whose list pointers descend is flagged and gets its mask only;
    a drafted token outside the vocabulary is reported although no penalty
    asks for it."""
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = Case(15, 3, 500, hist=60, states=3)
    rules, status = c.rules(), torch.zeros(1, dtype=torch.int32, device="cuda")
    at = [0, len(c.hist[0]), 0, 0]                               # request 1 from the end of 0's back to its start
    rules._keep[1].copy_(torch.tensor(at))
    out = torch.zeros(3, 500, device="cuda")
    rx.rx_logits_process(rules, c.logits(), out, status)
    assert int(status.item()) == rx.RX_DEV_BAD_LEN
    c.hist[1] = c.hist[2] = np.zeros(0, np.int32)
    _same(out.cpu().numpy(), c.reference())
    c = Case(16, 2, 500, trees=[4, 3], penalties=False)
    c.draft[1][2] = 500
    out = torch.zeros(7, 500, device="cuda")
    status.zero_()
    rx.rx_logits_process(c.rules(), c.logits(), out, status)
    assert int(status.item()) == rx.RX_DEV_BAD_TOKEN
    _same(out.cpu().numpy(), c.reference())


@pytest.mark.parametrize("in_place", [False, True])
def test_quotients_of_every_size(in_place):
    """Repetition factors and logits of every exponent: the quotient is the
    correctly rounded one."""
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    rng = np.random.default_rng(3)
    n = 48
    c = Case(13, n, 2000, hist=4000, prompt=0.5)
    bits = rng.integers(0, 1 << 31, c.x.shape, dtype=np.uint32) | (rng.integers(0, 4, c.x.shape) == 0).astype(np.uint32) << 31
    near = rng.random(c.x.shape) < 0.5
    c.x = np.where(near, (20 * rng.standard_normal(c.x.shape)).astype(np.float32), bits.view(np.float32))
    c.x = np.where(np.isnan(c.x), np.float32(1), c.x).astype(np.float32)
    c.rep = np.exp2(rng.uniform(-80, 80, n)).astype(np.float32)
    c.rep[:20] = 1 + rng.random(20)
    c.freq[:], c.pres[:] = 0, 0
    x = c.logits()
    out = x if in_place else torch.empty_like(x)
    rx.rx_logits_process(c.rules(), x, out)
    with np.errstate(all="ignore"):
        _same(out.cpu().numpy(), c.reference())


def test_two_captured_calls_of_the_same_rules_at_once():
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = Case(14, 5, 30000, hist=3000, bias=20, states=3)
    rules, x, want = c.rules(), c.logits(), c.reference()
    outs = [torch.zeros(5, 30000, device="cuda") for _ in range(2)]
    graphs = []
    for o in outs:
        rx.rx_logits_process(rules, x, o)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rx.rx_logits_process(rules, x, o)
        graphs.append(g)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, (torch.cuda.Stream(), torch.cuda.Stream())):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        _same(o.cpu().numpy(), want)


@pytest.mark.parametrize("scale", [1.0, 0.037, 1.7e-3, 3e-25, 1e25, 2.0 ** -60, 2.0 ** 61, 1e-38])
def test_codes_are_those_of_the_slot_scatter(scale):
    """V through the fused call and through rx_kv_store_fp8: the same codes,
    whatever the values and the scale (a quotient is rounded correctly in both)."""
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    g = _g()
    rng = np.random.default_rng(5)
    n, hkv, d = 300, 3, 128
    bits = rng.integers(0, 1 << 16, (n, hkv, d)).astype(np.uint16)        # any bf16 value, NaN and infinities among them
    some = rng.random((n, hkv, 1)) < 0.7
    bits = np.where(some, inputs.bf16_round((300 * scale * rng.standard_normal(bits.shape)).astype(np.float32)), bits)
    bits[0, 0, :4] = [0x8000, 0, 1, 0x8001]                               # zeros and the least subnormals
    v, k = g.to_dev(bits), torch.zeros(n, hkv, d, dtype=torch.bfloat16, device="cuda")
    slots = g.i32(rng.permutation(n).astype(np.int32))
    pools = [[torch.zeros(n, hkv, d, dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2)]
    q = torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda")
    rx.rx_qk_norm_rope_store_fp8(*pools[0], 1.0, scale, q, torch.empty_like(q), k, v, None, None, slots, slots, BASE, EPS)
    rx.rx_kv_store_fp8(*pools[1], 1.0, scale, k, v, slots)
    assert torch.equal(pools[0][1], pools[1][1])


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv,most", [(16, 1, 20), (4, 2, 6)], ids=["two_row_tiles", "one_row_tile"])
def test_a_request_with_a_nan_value_leaves_the_next_ones_alone(hq, hkv, most, f8):
    """Many requests a CTA, every third with a NaN V at its last drafted token,
    which only that token sees."""
    from tests.test_gpu_draft_tree import Run
    rng = np.random.default_rng(8)
    B = 700
    trees = [int(t) for t in rng.integers(1, most + 1, B)]
    prefixes = [int(p) for p in rng.integers(0, 150, B)]
    b = _draft.TreeBatch(9, hq, hkv, 64, prefixes, trees, masks="chain")
    ref = Run(b, f8).reference()
    last = b.indptr[1:] - 1
    bad = last[::3]
    for i in range(0, B, 3):
        b.v[b.rtt[b.req_idx[i], prefixes[i] + trees[i] - 1]] = np.nan
    r = Run(b, f8)
    o, lse = r()
    assert int(r.status.item()) == 0
    keep = np.setdiff1d(np.arange(int(b.indptr[-1])), bad)
    _draft.check_tree(o[keep], lse[keep], tuple(x[keep] for x in ref), "the others")
    assert np.isnan(o[bad]).all()
