"""Inputs, calls and error bounds shared by the tests of the attention with
rules on the scores (tests/test_gpu_rules*.py)."""
import numpy as np

from oracle import rules as ref
from tests._draft import HALF_STEP


class RulesBatch:
    """A ragged batch over a random pool: fp32 values (the caller rounds them),
    slot lists, rules."""

    def __init__(self, seed, hq, hkv, d, prefixes, news, cap=0.0, window=0, slopes=False, mask="", spread=1.0, spare=64,
                 shared=0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d = hq, hkv, d
        B = len(news)
        self.prefix_len, self.new_len = np.array(prefixes, np.int32), np.array(news, np.int32)
        self.indptr = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        n = int(self.indptr[-1])
        stride = max(p + t for p, t in zip(prefixes, news)) + 5
        self.num_slots = sum(p + t for p, t in zip(prefixes, news)) + spare
        perm = rng.permutation(self.num_slots).astype(np.int32)
        self.rtt = np.full((B + 2, stride), -7, np.int32)       # unused entries are bad slots: never read
        self.req_idx = rng.permutation(B + 2)[:B].astype(np.int32)
        at = 0
        for b in range(B):
            m = prefixes[b] + news[b]
            self.rtt[self.req_idx[b], :m] = perm[at:at + m]
            at += m
        for b in range(1, B):                                   # the first `shared` positions are request 0's
            m = min(shared, prefixes[0], prefixes[b])
            self.rtt[self.req_idx[b], :m] = self.rtt[self.req_idx[0], :m]
        self.k = rng.standard_normal((self.num_slots, hkv, d)).astype(np.float32)
        self.v = rng.standard_normal((self.num_slots, hkv, d)).astype(np.float32)
        self.q = (spread * rng.standard_normal((n, hq, d))).astype(np.float32)
        self.cap, self.window, self.scale = cap, window, 1.0 / np.sqrt(d)
        self.slopes = (2.0 ** (-8.0 * (1 + np.arange(hq)) / hq)).astype(np.float32) if slopes else None
        self.see_from = self.see_to = None
        lo, hi = np.zeros(n, np.int64), np.zeros(n, np.int64)
        for b in range(B):
            P, T, s = prefixes[b], news[b], int(self.indptr[b])
            i = np.arange(T)
            if mask == "docs":
                k = i // 23
                lo[s:s + T] = np.where(k > 0, P + 23 * k, 0)
            elif mask == "prefix":
                hi[s:s + T] = np.where(i < (T + 1) // 2, P + (T + 1) // 2, 0)
            elif mask == "spans":
                hi[s:s + T] = np.where(i // 40 % 2 == 0, P + 40 * (i // 40 + 1), 0)   # may end past the context
            elif mask == "any":                                  # whatever a program may put there, rows left empty
                lo[s:s + T] = np.where(rng.random(T) < 0.5, rng.integers(-5, P + T + 9, T), 0)
                hi[s:s + T] = np.where(rng.random(T) < 0.5, rng.integers(-5, P + T + 9, T), 0)
        if mask in ("docs", "any"):
            self.see_from = lo.astype(np.int32)
        if mask in ("prefix", "spans", "any"):
            self.see_to = hi.astype(np.int32)

    def oracle(self, q, k, v):
        return ref.attention(q, k, v, self.rtt, self.req_idx, self.prefix_len, self.new_len, self.scale, self.cap,
                             self.window, self.slopes, self.see_from, self.see_to)


def check(o, lse, r, b, what="", cap=None):
    """Bounds of the attention with rules.  o: the softmax weights are rounded to
    bf16 before P V (2^-8 of sum p |v|; divided by the sum of the rounded weights,
    sum p (1 + e) v / sum p (1 + e) is off from o by at most max |e| sum p |v - o|, under
    2^-8 (sum p |v| + |o|)) and the result once more (2^-8 of |o|).
    The scores are fp32 sums of d exact products, off by at most d 2^-24 sum |q
    k| scale; with spread s of the queries that sum is under 0.8 s sqrt(d) times
    1.5: under 3e-4 s for d up to 128.  A cap adds under 4 2^-23 cap log2(e) log2
    units: 1e-6 cap; a bias is rounded to 2^-24 of scores that count, under 64:
    1e-5.  Each moves every weight by at most that, twice with the sum.  cap: where
    every score is far within the cap its share is 2^-21 of a score, under 64 (and
    2^-25 of the cap): less than 1e-6 of 30 whatever the cap."""
    ro, rl, ra = r
    s = max(1.0, float(np.abs(b.q).max()) / 4.0)
    off = 2 * (3e-4 * s + 1e-6 * (b.cap if cap is None else cap) + 1e-5)
    bound = 2 * HALF_STEP * np.abs(ro) + (HALF_STEP * (1 + HALF_STEP) + off) * ra + 1e-30
    err = np.abs(np.asarray(o, np.float64) - ro)
    assert not np.isnan(o).any(), f"{what}: NaN"
    worst = (err / bound).max() if err.size else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3f} of its bound"
    if lse is not None:
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse), empty), f"{what}: empty rows"
        assert np.abs(np.where(empty, 0, lse - np.where(empty, 0, rl)))[~empty].max(initial=0) <= off + 1e-4, f"{what}: lse"
        assert (np.asarray(o)[empty] == 0).all(), f"{what}: an empty row's output"
    return float(worst)
