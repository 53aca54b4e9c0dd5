"""Inputs and error bounds shared by the tests of the draft-verification
operators (tests/test_draft_oracle.py, tests/test_gpu_draft_*.py)."""
import numpy as np

HALF_STEP = 2.0 ** -8          # bf16: half a step of a rounding, relative


def random_parents(rng, n):
    return np.array([-1] + [int(rng.integers(-1 if rng.random() < 0.1 else 0, i)) for i in range(1, n)], np.int32)[:n]


def pack(see, words):
    """bool [n, m] -> int32 [n, words]."""
    n, m = see.shape
    bits = np.zeros((n, words * 32), np.uint64)
    bits[:, :min(m, words * 32)] = see[:, :words * 32]
    w = (bits.reshape(n, words, 32) << np.arange(32, dtype=np.uint64)).sum(2).astype(np.uint32)
    return w.view(np.int32)


class TreeBatch:
    """A ragged batch of drafted trees over a random pool: fp32 values (the
    caller rounds them), slot lists, masks."""

    def __init__(self, seed, hq, hkv, d, prefixes, trees, masks="tree", words=None, spare=64):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d = hq, hkv, d
        B = len(trees)
        self.prefix_len = np.array(prefixes, np.int32)
        self.indptr = np.concatenate([[0], np.cumsum(trees)]).astype(np.int32)
        self.trees = list(trees)
        n = int(self.indptr[-1])
        stride = max(p + t for p, t in zip(prefixes, trees)) + 5
        self.num_slots = sum(p + t for p, t in zip(prefixes, trees)) + spare
        perm = rng.permutation(self.num_slots).astype(np.int32)
        self.rtt = np.full((B + 2, stride), -7, np.int32)       # unused entries are bad slots: never read
        self.req_idx = rng.permutation(B + 2)[:B].astype(np.int32)
        at = 0
        for b in range(B):
            m = prefixes[b] + trees[b]
            self.rtt[self.req_idx[b], :m] = perm[at:at + m]
            at += m
        self.k = rng.standard_normal((self.num_slots, hkv, d)).astype(np.float32)
        self.v = rng.standard_normal((self.num_slots, hkv, d)).astype(np.float32)
        self.q = rng.standard_normal((n, hq, d)).astype(np.float32)
        self.max_tree = max(max(trees), 1)
        self.words = (self.max_tree + 31) // 32 if words is None else words
        self.see = []
        for t in trees:
            if masks == "tree":
                from oracle.draft import tree_mask
                s = tree_mask(random_parents(rng, t))
            elif masks == "chain":
                s = np.tril(np.ones((t, t), bool))
            else:                                                # any mask, some rows empty
                s = rng.random((t, t)) < 0.3
                s[rng.random(t) < 0.3] = False
            self.see.append(s)
        # bits at and past T are garbage: they must be ignored
        m = np.zeros((n, self.words * 32), bool)
        m[:] = rng.random(m.shape) < 0.5
        for b, t in enumerate(trees):
            m[self.indptr[b]:self.indptr[b + 1], :t] = self.see[b]
        self.mask = None if masks == "chain" else pack(m, self.words)
        self.scale = 1.0 / np.sqrt(d)

    def oracle(self, q, k, v):
        from oracle.draft import tree_attention
        return tree_attention(q, k, v, self.rtt, self.req_idx, self.prefix_len, self.indptr, self.see, self.scale)


def check_tree(o, lse, ref, what=""):
    """Bounds of the tree attention kernels.  o: the softmax weights are
    rounded to bf16 before P V (2^-8 of sum p |v|) and the result once more
    (2^-8 of |o|); the scores are fp32 sums of d exact products, off by at
    most d 2^-24 sum |q k| scale, under 1e-4 for values of order one, which
    moves every weight by at most that.  lse: 1e-3 as for the other attention
    entry points."""
    ro, rl, ra = ref
    bound = HALF_STEP * np.abs(ro) + (HALF_STEP + 2e-4) * ra + 1e-30
    err = np.abs(np.asarray(o, np.float64) - ro)
    assert not np.isnan(o).any(), f"{what}: NaN"
    worst = (err / bound).max() if err.size else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3f} of its bound"
    if lse is not None:
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse), empty), f"{what}: empty rows"
        assert np.abs(np.where(empty, 0, lse - np.where(empty, 0, rl)))[~empty].max(initial=0) <= 1e-3, f"{what}: lse"
        assert (np.asarray(o)[empty] == 0).all(), f"{what}: an empty row's output"
    return float(worst)
