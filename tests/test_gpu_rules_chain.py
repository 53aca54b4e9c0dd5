"""One layer's attention step, its calls one behind the other: each call against
the oracle on what the calls before it left on the device, so that a position, a
row or a slot that one of them has wrong shows."""
import numpy as np
import pytest

from oracle import fp8
from tests._chain import BASE, CAP, D, HKV, HQ, PAGE, Chain
from tests.test_gpu_draft_norm import _check_bf16, _check_codes

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


class Device:
    def __init__(self, chain, f8):
        from tests import _gpu as g
        self.g, self.c, self.f8, self.scales = g, chain, f8, (0.021, 0.0173)
        self.pools = [torch.zeros(chain.num_slots, HKV, D, dtype=torch.uint8 if f8 else torch.bfloat16, device="cuda") for _ in range(2)]
        self.rtt, self.pages, self.req = g.i32(chain.rtt), g.i32(chain.pages), g.i32(chain.req)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def values(self):
        """The pools in 64 bits."""
        if self.f8:
            return [fp8.decode(p.cpu().numpy()) * float(np.float32(x)) for p, x in zip(self.pools, self.scales)]
        return [p.double().cpu().numpy() for p in self.pools]

    def run(self, new, see_to=None, captured=False, decode=False):
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        g, c = self.g, self.c
        before = self.values()
        s = c.step(new, see_to)
        qkv, pos_axes = g.to_dev(s.x), g.i32(s.pos).view(3, s.n)
        q = torch.zeros(s.n, HQ, D, dtype=torch.bfloat16, device="cuda")
        og, lg = g.Guarded((s.n, HQ, D), torch.bfloat16), g.Guarded((s.n, HQ), torch.float32)
        e = lambda m: torch.full((m,), -9, dtype=torch.int32, device="cuda")  # noqa: E731
        indptr, seq, pos, slots = e(c.B + 1), e(c.B), e(s.n), e(s.n)
        plen, nlen = g.i32(s.prefix), g.i32(s.new)
        rules = rx.AttnRules(cap=CAP, window=c.window, see_to=None if see_to is None else g.i32(see_to))
        most = int(s.new.max())
        ws = torch.empty(rx.rx_attn_rules_workspace(int(c.lens.sum()), c.B, HQ, HKV, D, most), dtype=torch.uint8, device="cuda")
        pool = (*self.pools, *self.scales) if self.f8 else tuple(self.pools)
        store = rx.rx_qk_rope_axes_store_fp8 if self.f8 else rx.rx_qk_rope_axes_store
        ext = rx.rx_attn_extend_rules_fp8 if self.f8 else rx.rx_attn_extend_rules
        dec = rx.rx_attn_decode_rules_fp8 if self.f8 else rx.rx_attn_decode_rules

        def calls():
            rx.rx_step_maps(self.req, plen, nlen, self.rtt, c.num_slots, indptr, seq, pos, slots, pages=self.pages, page_size=PAGE,
                            dev_status=self.status)
            store(*pool, qkv[:, :HQ], q, qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], None, None, slots, pos_axes, c.axis, BASE,
                  dev_status=self.status)
            if decode:
                dec(*pool, q, og.t, lg.t, self.req, seq, self.rtt, D ** -0.5, rules, ws, self.status)
            else:
                ext(*pool, q, og.t, lg.t, indptr, self.req, plen, nlen, self.rtt, most, D ** -0.5, rules, ws, self.status)

        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                calls()
            graph.replay()
        else:
            calls()
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        # the lists
        assert indptr.tolist() == s.lists[0] and seq.tolist() == s.lists[1] and pos.tolist() == s.lists[2] and slots.tolist() == s.lists[3]
        assert np.array_equal(self.rtt.cpu().numpy(), c.rtt)
        # the rotation and what it stored, the rest of the pools as it was
        after, at = self.values(), np.array(s.lists[3])
        q_want, k_want, v_want = c.rotated(s)
        _check_bf16(q.float().cpu().numpy(), s.x64[:, :HQ], q_want, "q")
        if self.f8:
            raw = [p.cpu().numpy()[at] for p in self.pools]
            _check_codes(raw[0], s.x64[:, HQ:HQ + HKV], k_want, float(np.float32(self.scales[0])), "k")
            _check_codes(raw[1], v_want, v_want, float(np.float32(self.scales[1])), "v")
        else:
            _check_bf16(after[0][at].astype(np.float32), s.x64[:, HQ:HQ + HKV], k_want, "k")
            assert np.array_equal(after[1][at], v_want)
        rest = np.setdiff1d(np.arange(c.num_slots), at)
        assert all(np.array_equal(x[rest], y[rest]) for x, y in zip(before, after))
        # the attention, over what the device holds
        og.check("o")
        lg.check("lse")
        q64 = q.double().cpu().numpy()
        c.check(s, q64, og.t.float().cpu().numpy(), lg.t.cpu().numpy(), c.attention(s, q64, *after), str(new))


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
@pytest.mark.parametrize("window", [0, 48])
def test_prompt_text_and_tokens(window, captured, f8):
    d = Device(Chain(71, window), f8)
    see_to = np.zeros(103, np.int32)
    see_to[10:40] = 40                                           # an image of request 0, positions 10 .. 39
    see_to[70 + 5:70 + 30] = 30                                  # one of request 1
    d.run([70, 33], see_to, captured)
    d.run([20, 1], np.zeros(21, np.int32), captured)             # text behind them
    for _ in range(3):
        d.run([1, 1], None, captured, decode=True)
    d.run([1, 1], None, captured)                                # single tokens by the other call


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
def test_many_requests(f8):
    """40 requests, some of them with nothing new."""
    rng = np.random.default_rng(72)
    d = Device(Chain(73, 20, B=40, wide=6), f8)
    d.run(rng.integers(0, 50, 40), None)
    d.run(np.where(rng.random(40) < 0.3, 0, 5), None, True)
    d.run([1] * 40, None, True, decode=True)
