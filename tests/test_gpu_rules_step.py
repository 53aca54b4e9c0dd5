"""One layer's attention step of a model that reads images and text, its calls
one behind the other as a program makes them, eager and captured: the lists of
the step, rotation on several axes with store, prompt attention in which an
image's tokens see one another, then decode steps of the same requests."""
import numpy as np
import pytest

from oracle import rules as ref
from prefix_shared_kv_radixattention_gb300 import inputs
from tests._draft import HALF_STEP

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HQ, HKV, D, PAGE, BASE = 8, 2, 64, 16, 1e4


class Layer:
    """Two requests over a paged pool, capped scores, a window, three axes."""

    def __init__(self, seed, window):
        from tests import _gpu as g
        rng = np.random.default_rng(seed)
        self.g, self.rng, self.window = g, rng, window
        self.lens = np.zeros(2, np.int64)                        # tokens in the pool
        self.wide, self.rows = 16, 4
        pages = rng.permutation(self.rows * self.wide).reshape(self.rows, self.wide)
        self.pages, self.num_slots = g.i32(pages), pages.size * PAGE
        self.req = np.array([2, 0])
        self.rtt = torch.full((self.rows, self.wide * PAGE), -1, dtype=torch.int32, device="cuda")
        self.rtt_host = np.full((self.rows, self.wide * PAGE), -1)
        self.pages_host = pages
        self.axis = [c % 3 for c in range(D // 2)]
        self.k = torch.zeros(self.num_slots, HKV, D, dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.k64, self.v64 = np.zeros((self.num_slots, HKV, D)), np.zeros((self.num_slots, HKV, D))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, new, see_to=None, captured=False):
        from prefix_shared_kv_radixattention_gb300 import binding as rx
        g, n = self.g, int(np.sum(new))
        x = inputs.bf16_round(self.rng.standard_normal((n, HQ + 2 * HKV, D)).astype(np.float32))
        text = np.concatenate([np.arange(p, p + t) for p, t in zip(self.lens, new)])
        pos3 = np.stack([text, text + self.rng.integers(0, 9, n), text + self.rng.integers(0, 9, n)])
        qkv, pos_axes = g.to_dev(x), g.i32(pos3).view(3, n)
        q = torch.empty(n, HQ, D, dtype=torch.bfloat16, device="cuda")
        o, lse = torch.empty_like(q), torch.empty(n, HQ, device="cuda")
        e = lambda m: torch.empty(m, dtype=torch.int32, device="cuda")  # noqa: E731
        indptr, seq, pos, slots = e(3), e(2), e(n), e(n)
        req, plen, nlen = g.i32(self.req), g.i32(self.lens), g.i32(new)
        decode = see_to is None and max(new) == 1
        rules = rx.AttnRules(cap=50.0, window=self.window, see_to=None if see_to is None else g.i32(see_to))
        context = int(self.lens.sum()) + n
        ws = torch.empty(rx.rx_attn_rules_workspace(context, 2, HQ, HKV, D, max(new)), dtype=torch.uint8, device="cuda")

        def calls():
            rx.rx_step_maps(req, plen, nlen, self.rtt, self.num_slots, indptr, seq, pos, slots, pages=self.pages,
                            page_size=PAGE, dev_status=self.status)
            rx.rx_qk_rope_axes_store(self.k, self.v, qkv[:, :HQ], q, qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], None, None, slots,
                                     pos_axes, self.axis, BASE, dev_status=self.status)
            if decode:
                rx.rx_attn_decode_rules(self.k, self.v, q, o, lse, req, seq, self.rtt, D ** -0.5, rules, ws, self.status)
            else:
                rx.rx_attn_extend_rules(self.k, self.v, q, o, lse, indptr, req, plen, nlen, self.rtt, max(new), D ** -0.5, rules,
                                        ws, self.status)

        if captured:
            calls()                                              # writes what the replay writes again
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                calls()
            o.zero_()
            graph.replay()
        else:
            calls()
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0

        # the oracle's step
        want = ref.step_maps(self.req, self.lens, new, self.rtt_host, self.num_slots, n, self.pages_host, PAGE)
        self.rtt_host = want[4]
        assert pos.tolist() == want[2] and slots.tolist() == want[3] and np.array_equal(self.rtt.cpu().numpy(), self.rtt_host)
        x64 = inputs.bf16_to_f32(x).astype(np.float64)
        self.k64[want[3]] = ref.rope_axes(x64[:, HQ:HQ + HKV], pos3, self.axis, BASE)
        self.v64[want[3]] = x64[:, HQ + HKV:]
        q64 = ref.rope_axes(x64[:, :HQ], pos3, self.axis, BASE)
        r = ref.attention(q64, self.k64, self.v64, self.rtt_host, self.req, self.lens, new, D ** -0.5, 50.0, self.window, None,
                          None, see_to)
        self.lens = self.lens + np.asarray(new)
        # q and K were rounded to bf16 on the way: a score is off by at most 2 2^-8 sum |q k| scale, which for 64
        # values of order one (at most 5, products 0.64 on average) stays below 2 2^-8 0.64 64 1.6 / 8 = 0.064;
        # every weight moves by at most that twice, and V is of order sum p |v|
        ro, rl, ra = r
        err = np.abs(o.float().cpu().numpy() - ro)
        bound = HALF_STEP * np.abs(ro) + (HALF_STEP + 2 * 0.064) * ra
        assert (err <= bound).all(), (err / bound).max()
        assert np.abs(lse.cpu().numpy() - rl).max() <= 0.064 + 1e-3


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
@pytest.mark.parametrize("window", [0, 48])
def test_prompt_with_images_then_decode(window, captured):
    layer = Layer(61, window)
    new = [70, 33]
    see_to = np.zeros(103, np.int32)
    see_to[10:40] = 40                                           # an image of request 0, positions 10 .. 39
    see_to[70 + 5:70 + 30] = 30                                  # one of request 1
    layer.step(new, see_to, captured)
    layer.step([20, 1], np.zeros(21, np.int32), captured)        # text behind them
    for _ in range(3):
        layer.step([1, 1], None, captured)
