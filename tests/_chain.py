"""The host's side of the tests of a whole attention step (lists, rotation on
several axes with store, attention with rules): inputs, and what each call of the
step has to have done, from what the calls before it left behind."""
from types import SimpleNamespace

import numpy as np

from oracle import rules as ref
from prefix_shared_kv_radixattention_gb300 import inputs
from tests import _rules

HQ, HKV, D, PAGE, BASE, CAP = 8, 2, 64, 16, 1e4, 50.0


class Chain:
    """Requests over a paged pool, capped scores, a window, three axes."""

    def __init__(self, seed, window, B=2, wide=16):
        self.rng, self.window, self.B = np.random.default_rng(seed), window, B
        self.lens = np.zeros(B, np.int64)                        # tokens in the pool
        self.pages = self.rng.permutation((B + 2) * wide).reshape(B + 2, wide)
        self.num_slots = self.pages.size * PAGE
        self.req = self.rng.permutation(B + 2)[:B]
        self.rtt = np.full((B + 2, wide * PAGE), -1)
        self.axis = np.array([c % 3 for c in range(D // 2)], np.uint8)

    def step(self, new, see_to=None):
        """The inputs of the next step, as bf16 bits where they are values."""
        new = np.asarray(new)
        n = int(new.sum())
        text = np.concatenate([np.arange(p, p + t) for p, t in zip(self.lens, new)])
        s = SimpleNamespace(new=new, n=n, see_to=see_to, prefix=self.lens.copy(),
                            x=inputs.bf16_round(self.rng.standard_normal((n, HQ + 2 * HKV, D)).astype(np.float32)),
                            pos=np.stack([text, text + self.rng.integers(0, 9, n), text + self.rng.integers(0, 9, n)]))
        s.lists = ref.step_maps(self.req, self.lens, new, self.rtt, self.num_slots, n, self.pages, PAGE)
        self.rtt = s.lists[4]
        s.x64 = inputs.bf16_to_f32(s.x).astype(np.float64)
        self.lens = self.lens + new
        return s

    def rotated(self, s):
        """q and the new rows of K and V in 64 bits."""
        return (ref.rope_axes(s.x64[:, :HQ], s.pos, self.axis, BASE), ref.rope_axes(s.x64[:, HQ:HQ + HKV], s.pos, self.axis, BASE),
                s.x64[:, HQ + HKV:])

    def attention(self, s, q, k, v, window=None, prefix=None):
        """The oracle over q and the pools as the calls before left them."""
        return ref.attention(q, k, v, self.rtt, self.req, s.prefix if prefix is None else prefix, s.new, D ** -0.5, CAP,
                             self.window if window is None else window, None, None, s.see_to)

    def check(self, s, q, o, lse, want, what=""):
        """Bounds of tests/_rules.check; the log-sum-exp tighter: scores of d exact products summed in fp32 are off by
        at most d 2^-24 of sum |q k| scale, for 64 products of order one (0.64 on average; twice that here) under
        64 2^-24 64 1.28 / 8 = 4e-5, the cap adds 2^-24 of itself, the sum and its logarithm under 2e-5."""
        _rules.check(o, lse, want, SimpleNamespace(q=q, cap=CAP), what)
        assert np.abs(lse - want[1]).max() <= 1e-4, what
