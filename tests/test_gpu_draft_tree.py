"""GPU parity of rx_attn_tree and rx_attn_tree_fp8 against the fp64 oracle.
Bounds: tests/_draft.check_tree."""
import numpy as np
import pytest

from oracle import fp8
from prefix_shared_kv_radixattention_gb300 import inputs
from tests import _draft

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _g():
    from tests import _gpu
    return _gpu


class Run:
    """One batch on the device, bf16 or E4M3 pools."""

    def __init__(self, b, f8=False, ks=0.07, vs=0.03, layers=0, layer=0):
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
        if layers:   # the other layers hold junk
            full = [torch.full((layers, *k.shape), 37, dtype=k.dtype, device="cuda") for _ in range(2)]
            full[0][layer], full[1][layer] = k, v
            k, v = full
        self.k, self.v = k, v
        qb = inputs.bf16_round(b.q)
        self.q64 = inputs.bf16_to_f32(qb).astype(np.float64)
        self.q = g.to_dev(qb)
        self.indptr, self.req, self.plen, self.rtt = g.i32(b.indptr), g.i32(b.req_idx), g.i32(b.prefix_len), g.i32(b.rtt)
        self.mask = None if b.mask is None else torch.from_numpy(b.mask.copy()).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        self.ws = torch.empty(rx.rx_attn_tree_workspace(len(b.trees), b.hq, b.hkv, b.d, b.max_tree), dtype=torch.uint8,
                              device="cuda")

    def launch(self, o, lse, stream=None, max_tree=None, ws=None):
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        b = self.b
        args = (self.q, o, lse, self.indptr, self.req, self.plen, self.mask, self.rtt, max_tree or b.max_tree, b.scale,
                self.ws if ws is None else ws, self.status)
        if self.f8:
            rx.rx_attn_tree_fp8(self.k, self.v, self.ks, self.vs, *args, stream=stream, layer=self.layer)
        else:
            rx.rx_attn_tree(self.k, self.v, *args, stream=stream, layer=self.layer)

    def __call__(self, with_lse=True, **kw):
        g = _g()
        og = g.Guarded(tuple(self.q.shape), torch.bfloat16)
        lg = g.Guarded(tuple(self.q.shape[:2]), torch.float32)
        self.ws.fill_(0xFF)    # NaN patterns: nothing may be read that the call did not write
        self.launch(og.t, lg.t if with_lse else None, **kw)
        torch.cuda.synchronize()
        og.check("o")
        lg.check("lse")
        return og.t.float().cpu().numpy(), lg.t.cpu().numpy()

    def reference(self):
        return self.b.oracle(self.q64, self.k64, self.v64)


SHAPES = [
    # hq, hkv, d, prefixes, trees
    (4, 4, 64, [0, 1, 63, 64, 65], [1, 1, 2, 3, 7]),
    (8, 2, 128, [127, 128, 129, 0, 300], [5, 0, 33, 17, 1]),
    (32, 8, 128, [700, 0, 1], [16, 3, 64]),
    (7, 1, 128, [200, 255, 257], [19, 18, 1]),                   # 7 q heads a kv head: rows that do not fill a tile
    (32, 32, 128, [90, 511], [4, 1]),
    (64, 8, 128, [1300], [64]),                                  # 512 rows a kv head
    (16, 1, 64, [40, 1000], [130, 65]),
    (128, 1, 64, [50, 129], [3, 2]),                             # 128 q heads on one kv head
    (6, 2, 64, [0, 0, 0], [1, 31, 200]),                         # no prefix at all
    (8, 8, 64, [5000, 4999, 3, 2], [2, 1, 1, 2]),
]


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("masks", ["tree", "any", "chain"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_parity(shape, masks, f8):
    hq, hkv, d, prefixes, trees = SHAPES[shape]
    r = Run(_draft.TreeBatch(11 + shape, hq, hkv, d, prefixes, trees, masks=masks), f8)
    o, lse = r()
    assert int(r.status.item()) == 0
    _draft.check_tree(o, lse, r.reference(), f"{SHAPES[shape]} {masks}")
    o2, lse2 = r()
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2), "two calls differ"
    assert np.array_equal(r(with_lse=False)[0], o)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
def test_many_requests(f8):
    """More requests than CTAs, lengths from nothing to some tiles."""
    rng = np.random.default_rng(5)
    B = 300
    trees = [int(t) for t in rng.integers(0, 6, B)]
    prefixes = [int(p) for p in rng.integers(0, 400, B)]
    r = Run(_draft.TreeBatch(6, 4, 2, 64, prefixes, trees), f8)
    o, lse = r()
    assert int(r.status.item()) == 0
    _draft.check_tree(o, lse, r.reference())


def test_layered_pool_and_wider_mask_rows():
    b = _draft.TreeBatch(21, 8, 2, 64, [77, 130], [9, 40], words=4)
    for f8 in (False, True):
        r = Run(b, f8, layers=3, layer=1)
        o, lse = r()
        _draft.check_tree(o, lse, r.reference())


def test_rows_behind_the_last_are_left_alone():
    b = _draft.TreeBatch(22, 4, 2, 64, [77, 130], [9, 4])
    r = Run(b)
    n = int(b.indptr[-1])
    r.q = torch.cat([r.q, torch.ones(5, *r.q.shape[1:], dtype=r.q.dtype, device="cuda")])
    r.mask = torch.cat([r.mask, torch.full((5, b.words), -1, dtype=torch.int32, device="cuda")])
    o, lse = r()
    assert np.isnan(o[n:]).all() and np.isnan(lse[n:]).all()
    _draft.check_tree(o[:n], lse[:n], r.reference())


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_what_a_token_does_not_see_takes_no_part(bad, f8):
    """K and V of drafted tokens that some rows do not see, and pool rows
    nobody lists, hold NaN or infinities: those rows are as without them."""
    if f8 and not np.isnan(bad):
        pytest.skip("E4M3 has no infinities")
    for hq, hkv, d, prefixes, trees in ((8, 2, 128, [200, 0, 120], [40, 6, 20]), (4, 4, 64, [3, 127], [9, 2])):
        b = _draft.TreeBatch(23, hq, hkv, d, prefixes, trees, masks="any")
        clean = Run(b, f8)
        ref = clean.reference()
        seen_by_none = np.zeros(int(b.indptr[-1]), bool)
        spoiled = {}
        for i, t in enumerate(trees):
            j = t // 2
            spoiled[i] = j
            slot = int(b.rtt[b.req_idx[i], prefixes[i] + j])
            if i % 2 == 0:
                b.k[slot] = bad
            b.v[slot] = bad
            seen_by_none[b.indptr[i]:b.indptr[i + 1]] = ~b.see[i][:, j]
        used = np.concatenate([b.rtt[b.req_idx[i], :prefixes[i] + t] for i, t in enumerate(trees)])
        rest = np.setdiff1d(np.arange(b.num_slots), used)
        b.k[rest] = b.v[rest] = bad
        r = Run(b, f8)
        o, lse = r()
        assert int(r.status.item()) == 0
        keep = seen_by_none
        _draft.check_tree(o[keep], lse[keep], tuple(x[keep] for x in ref), "unseen")
        assert not np.isfinite(o[~keep]).any(), "a seen NaN or infinity in V reaches every value of the row"


def test_bad_slots_read_as_zeros():
    b = _draft.TreeBatch(24, 8, 2, 64, [150, 5], [7, 3])
    for col, val in ((3, -1), (149, b.num_slots), (152, 2**31 - 1)):
        b.rtt[b.req_idx[0], col] = val
    for f8 in (False, True):
        r = Run(b, f8)
        o, lse = r()
        assert int(r.status.item()) == 1    # RX_DEV_BAD_SLOT
        _draft.check_tree(o, lse, r.reference())


def test_bad_lengths_leave_their_rows_unwritten():
    b = _draft.TreeBatch(25, 8, 2, 64, [150, 20, 30], [7, 3, 5])
    for what in ("tree", "stride", "negative"):
        r = Run(b)
        if what == "tree":
            o, lse = r(max_tree=5)
        else:
            p = b.prefix_len.copy()
            p[0] = b.rtt.shape[1] - 6 if what == "stride" else -1
            r.plen = _g().i32(p)
            o, lse = r()
        assert int(r.status.item()) == 2    # RX_DEV_BAD_LEN
        assert np.isnan(o[:7]).all() and np.isnan(lse[:7]).all()
        _draft.check_tree(o[7:], lse[7:], tuple(x[7:] for x in r.reference()))


def test_one_token_equals_decode():
    """A tree of one node is the decode step."""
    g = _g()
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    b = _draft.TreeBatch(26, 32, 8, 128, [1000, 3, 129], [1, 1, 1])
    r = Run(b)
    o, lse = r()
    od, ld = torch.empty_like(r.q), torch.empty(3, 32, device="cuda")
    sl = g.i32(b.prefix_len + 1)
    ws = torch.empty(max(1, rx.rx_attn_decode_workspace(3, 32, 8, 128, 1001)), dtype=torch.uint8, device="cuda")
    rx.rx_attn_decode(r.k, r.v, r.q, od, ld, r.req, sl, r.rtt, 1001, b.scale, None, ws, r.status)
    _, _, ra = r.reference()
    # both round the weights and the result to bf16
    assert (np.abs(o - od.float().cpu().numpy()) <= 2 * (_draft.HALF_STEP * np.abs(o) + (_draft.HALF_STEP + 2e-4) * ra)).all()
    assert np.abs(lse - ld.cpu().numpy()).max() <= 1e-3


def test_streams_and_a_captured_call_with_new_lengths():
    """Calls on two streams with their own workspaces, and a captured call
    replayed after the lengths, slots and masks in its tensors changed."""
    b1 = _draft.TreeBatch(27, 16, 4, 128, [900, 33], [12, 30])
    b2 = _draft.TreeBatch(28, 16, 4, 128, [40, 700], [30, 2], words=b1.words)
    r1, r2 = Run(b1), Run(b2)
    want = [r1(), r2()]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for r, s in ((r1, s1), (r2, s2)):
        o, lse = torch.empty_like(r.q), torch.empty(r.q.shape[:2], device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        r.launch(o, lse, stream=s)
        outs.append((o, lse))
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in zip(outs, want):
        assert np.array_equal(o.float().cpu().numpy(), wo) and np.array_equal(lse.cpu().numpy(), wl)

    n, stride, slots = 42, 1200, 4000
    rc = Run(b1)
    rc.q = torch.zeros(n, 16, 128, dtype=torch.bfloat16, device="cuda")
    rc.rtt = torch.zeros(4, stride, dtype=torch.int32, device="cuda")
    rc.k, rc.v = (torch.zeros(slots, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rc.mask = torch.zeros(n, b1.words, dtype=torch.int32, device="cuda")
    o, lse = torch.zeros_like(rc.q), torch.zeros(n, 16, device="cuda")
    rc.launch(o, lse, max_tree=32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rc.launch(o, lse, max_tree=32)
    for r, (wo, wl) in ((r1, want[0]), (r2, want[1]), (r1, want[0])):
        b = r.b
        m = int(b.indptr[-1])
        for dst, src in ((rc.q[:m], r.q), (rc.rtt[:, :b.rtt.shape[1]], r.rtt), (rc.k[:b.num_slots], r.k),
                         (rc.v[:b.num_slots], r.v), (rc.mask[:m], r.mask), (rc.indptr, r.indptr), (rc.req, r.req),
                         (rc.plen, r.plen)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(o[:m].float().cpu().numpy(), wo) and np.array_equal(lse[:m].cpu().numpy(), wl)
    assert int(rc.status.item()) == 0


def test_binding_refuses_wrong_tensors():
    b = _draft.TreeBatch(29, 4, 2, 64, [10], [3])
    r = Run(b)
    o, lse = torch.empty_like(r.q), torch.empty(r.q.shape[:2], device="cuda")
    for name, val in (("q", r.q.float()), ("req", r.req.long()), ("mask", r.mask[:2]), ("plen", r.plen.repeat(2)),
                      ("rtt", r.rtt.cpu()), ("q", r.q.transpose(0, 1)), ("ws", r.ws.view(torch.int32))):
        keep = getattr(r, name)
        setattr(r, name, val)
        with pytest.raises((TypeError, ValueError)):
            r.launch(o, lse)
        setattr(r, name, keep)
    with pytest.raises(ValueError):
        r.launch(o, lse[:2])
