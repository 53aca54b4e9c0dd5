"""rx_attn_tree and rx_attn_tree_fp8 where a CTA walks many tiles of a
request: scores that rise along the context (the running maximum moves and the
accumulated output is scaled), dozens of tiles a segment, a request cut into
more than 32 parts, and trees up to the largest."""
import numpy as np
import pytest

from tests import _draft
from tests.test_gpu_draft_tree import Run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _check(o, lse, ref, slack, what):
    """Bound: half a step of bf16 for the result and for the weights, and a
    weight's relative error from its score's (numerator and denominator:
    twice `slack`, the largest error of a score)."""
    ro, rl, ra = ref
    assert not np.isnan(o).any(), f"{what}: NaN"
    h = _draft.HALF_STEP
    bound = h * np.abs(ro) + (h + 2 * slack) * ra + 1e-30
    err = np.abs(o.astype(np.float64) - ro)
    assert (err <= bound).all(), f"{what}: error {(err / bound).max():.3f} of its bound"
    assert np.abs(lse - rl).max() <= 1e-3 + slack, f"{what}: lse"


def _score_slack(r):
    """fp32 scores: d products summed, off by at most d 2^-24 sum |q k| scale;
    their scaling and the difference from the maximum round thrice more, 2^-24
    of at most twice the largest score each."""
    b = r.b
    top = b.scale * np.abs(r.q64).sum(-1).max() * np.abs(r.k64).max()
    return (b.d + 6) * 2.0 ** -24 * top


SHAPES = {
    # hq, hkv, d, requests, prefix, tree
    "one_row_tile": (4, 2, 64, 24, 4000, 4),
    "one_row_tile_d128": (8, 4, 128, 16, 3000, 3),
    "two_row_tiles": (16, 1, 64, 40, 4000, 20),
    "two_row_tiles_d128": (32, 2, 128, 16, 3000, 7),
}


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("step", [3, 1])
@pytest.mark.parametrize("shape", SHAPES)
def test_scores_that_rise_along_the_context(shape, step, f8):
    """Every q is a factor f of (1, .., 1) plus noise, f by row; every key c (1,
    .., 1) plus noise, c rising by about 6 nats of f = 1 (8.7 in log2 units, more
    than the running maximum may lag) each `step` tiles of 128 for the first
    eight rises, then level.  So rows with f 1 scale their output, those with
    0, 1/2 and -1 do not, or not in the same tiles.  V shrinks as the scores
    rise, so that what came before still shows in the result."""
    hq, hkv, d, B, prefix, tree = SHAPES[shape]
    rng = np.random.default_rng(7)
    prefixes = [prefix - int(x) for x in rng.integers(0, 300, B)]
    trees = [max(1, tree - i % 3) for i in range(B)]
    b = _draft.TreeBatch(51, hq, hkv, d, prefixes, trees)
    n = int(b.indptr[-1])
    f = np.array([1.0, 0.0, 0.5, -1.0, 1.0])[rng.integers(0, 5, (n, hq))]
    b.q = (f[:, :, None] + 0.02 * b.q).astype(np.float32)
    unit = 1 / (d * b.scale)                                    # c of one nat
    rise = np.zeros(b.num_slots, np.float32)
    for i, (p, t) in enumerate(zip(prefixes, trees)):
        at = np.arange(p + t)
        rise[b.rtt[b.req_idx[i], :p + t]] = np.minimum(at // (128 * step), 8)
    b.k = ((6 * unit * rise)[:, None, None] + 0.05 * b.k).astype(np.float32)
    b.v = (b.v * np.exp2(-rise)[:, None, None]).astype(np.float32)
    r = Run(b, f8)
    o, lse = r()
    assert int(r.status.item()) == 0
    ref = r.reference()
    _check(o, lse, ref, _score_slack(r), f"{shape}, {step}")
    o2, lse2 = r()
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2), "two calls differ"


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("shape", [(4, 1, 64, [20000], [5]), (32, 1, 128, [20010, 5], [7, 1]), (8, 1, 64, [40000, 300, 0], [2, 9, 3])],
                         ids=str)
def test_a_request_in_more_than_32_parts(shape, f8):
    """One kv head and 157 tiles or more: every CTA has one or two of them."""
    r = Run(_draft.TreeBatch(52, *shape), f8)
    o, lse = r()
    assert int(r.status.item()) == 0
    _draft.check_tree(o, lse, r.reference(), str(shape))


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("shape", [(8, 8, 64, 16, 5000, 6), (64, 4, 128, 16, 5200, 10)], ids=["one_row_tile", "two_row_tiles"])
def test_dozens_of_tiles_a_segment(shape, f8):
    hq, hkv, d, B, prefix, tree = shape
    rng = np.random.default_rng(9)
    prefixes = [prefix - int(x) for x in rng.integers(0, 700, B)]
    r = Run(_draft.TreeBatch(53, hq, hkv, d, prefixes, [max(1, tree - i % 4) for i in range(B)]), f8)
    o, lse = r()
    assert int(r.status.item()) == 0
    _draft.check_tree(o, lse, r.reference(), str(shape))
    o2, lse2 = r()
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2), "two calls differ"


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv,prefixes,trees", [(4, 1, [100, 0], [513, 3]), (2, 2, [0, 77, 300], [1024, 1, 640]),
                                                   (16, 1, [129], [1024])], ids=str)
def test_the_largest_trees(hq, hkv, prefixes, trees, f8):
    """Any masks, and NaN in V at a drafted token far along each tree: the rows
    that do not see it are as without it."""
    b = _draft.TreeBatch(54, hq, hkv, 64, prefixes, trees, masks="any")
    ref = Run(b, f8).reference()
    sees = np.zeros(int(b.indptr[-1]), bool)
    for i, t in enumerate(trees):
        if t > 512:
            b.v[b.rtt[b.req_idx[i], prefixes[i] + t - 1]] = np.nan
            b.v[b.rtt[b.req_idx[i], prefixes[i] + 510]] = np.nan
            sees[b.indptr[i]:b.indptr[i + 1]] = b.see[i][:, t - 1] | b.see[i][:, 510]
    r = Run(b, f8)
    o, lse = r()
    assert int(r.status.item()) == 0
    _draft.check_tree(o[~sees], lse[~sees], tuple(x[~sees] for x in ref), str(trees))
    assert np.isnan(o[sees]).all()
    assert sees.any() and not sees.all()
