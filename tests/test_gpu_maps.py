"""GPU parity of rx_step_maps against the oracle, bit for bit."""
import numpy as np
import pytest

from oracle import rules as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def _run(req, plen, nlen, rtt, num_slots, tokens, pages=None, size=0, seq=True, graph=False):
    """(qo_indptr, seq_len, pos, slots, rtt, status); entries that the call leaves alone are -77."""
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    B = len(req)
    new = lambda n: torch.full((n + 64,), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    bufs = [new(B + 1), new(B), new(tokens), new(tokens)]
    indptr, sl, pos, slots = (b[:n] for b, n in zip(bufs, (B + 1, B, tokens, tokens)))
    rt, status = _i32(rtt), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (_i32(req), _i32(plen), _i32(nlen), rt, num_slots, indptr, sl if seq else None, pos, slots)
    more = dict(pages=None if pages is None else _i32(pages), page_size=size, dev_status=status)
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rx.rx_step_maps(*args, **more)
        g.replay()
    else:
        rx.rx_step_maps(*args, **more)
    torch.cuda.synchronize()
    for b, n in zip(bufs, (B + 1, B if seq else 0, tokens, tokens)):
        assert bool((b[n:] == -77).all()), "written outside"
    return [x.cpu().numpy() for x in (indptr, sl, pos, slots, rt)] + [int(status.item())]


def _check(req, plen, nlen, rtt, num_slots, tokens, pages=None, size=0, **kw):
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    indptr, seq, pos, slots, rt, status = _run(req, plen, nlen, rtt, num_slots, tokens, pages, size, **kw)
    want = ref.step_maps(req, plen, nlen, rtt, num_slots, tokens, pages, size)
    assert indptr.tolist() == want[0]
    if kw.get("seq", True):
        assert seq.tolist() == want[1]
    n = len(want[2])
    assert pos[:n].tolist() == want[2] and slots[:n].tolist() == want[3]
    assert (pos[n:] == -77).all() and (slots[n:] == -77).all()          # behind the last token
    assert np.array_equal(rt, want[4])
    assert status == (rx.RX_DEV_BAD_LEN if want[5] else 0) | (rx.RX_DEV_BAD_SLOT if want[6] else 0)


def _batch(seed, B, most, spare=3, empty=0.2, long=200):
    rng = np.random.default_rng(seed)
    plen = rng.integers(0, long, B)
    nlen = np.where(rng.random(B) < empty, 0, rng.integers(0, most + 1, B))
    stride = int((plen + nlen).max(initial=0)) + spare
    rows = B + 3
    req = rng.permutation(rows)[:B]
    rtt = rng.integers(0, 100000, (rows, stride))
    return req, plen, nlen, rtt, rng


@pytest.mark.parametrize("B,most", [(1, 1), (1, 0), (1, 3000), (5, 7), (64, 1), (255, 3), (256, 40), (257, 40), (1000, 1), (3000, 5),
                                    (65535, 1)])
def test_slot_lists(B, most):
    req, plen, nlen, rtt, _ = _batch(B + most, B, most, long=200 if B < 4000 else 3)
    n = int(nlen.sum())
    _check(req, plen, nlen, rtt, 100000, n)
    _check(req, plen, nlen, rtt, 100000, n + 500, seq=False, graph=B < 100)


@pytest.mark.parametrize("size", [1, 7, 16, 64])
@pytest.mark.parametrize("B,most", [(1, 1), (6, 100), (300, 20), (2, 3000)])
def test_pages(B, most, size):
    req, plen, nlen, rtt, rng = _batch(7 * B + size, B, most)
    wide = -(-rtt.shape[1] // size)
    pages = rng.permutation(rtt.shape[0] * wide).reshape(rtt.shape[0], wide)
    _check(req, plen, nlen, rtt, rtt.shape[0] * wide * size, int(nlen.sum()) + 9, pages, size)


def test_nothing():
    _check([], [], [], np.zeros((2, 5), int), 10, 0)
    _check([1, 0], [3, 0], [0, 0], np.zeros((2, 5), int), 10, 0)
    _check([1, 0], [3, 0], [0, 0], np.zeros((2, 5), int), 10, 6)


def test_lengths_out_of_range_and_too_many_tokens():
    rtt = np.arange(80).reshape(4, 20)
    _check([0, 1, 2, 3], [-1, 3, 5, 0], [2, -2, 16, 20], rtt, 80, 40)        # only the last is sound
    _check([0, 1, 2, 3], [2**31 - 1, 3, 5, 0], [2**31 - 1, 4, 15, 2], rtt, 80, 40)
    _check([0, 1, 2], [1, 2, 3], [10, 10, 10], rtt, 80, 15)
    _check([0, 1, 2], [1, 2, 3], [10, 10, 10], rtt, 80, 0)
    pages = np.arange(8).reshape(4, 2)
    _check([0, 1], [0, 0], [8, 9], rtt, 80, 40, pages, 4)                    # past the pages' positions


def test_slots_and_pages_outside_the_pool():
    rtt = np.arange(80).reshape(4, 20)
    rtt[1, 3], rtt[2, 0], rtt[2, 19] = -5, 80, 79
    _check([0, 1, 2, 3], [0, 0, 0, 0], [20, 20, 20, 20], rtt, 80, 80)
    pages = np.array([[0, 1], [-1, 4], [2**27, 3], [5, -(2**31)]])
    _check([0, 1, 2, 3], [0, 0, 0, 0], [8, 7, 6, 5], np.arange(80).reshape(4, 20), 20, 40, pages, 4)


def test_refused_tensors():
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    t = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    rtt = torch.zeros(2, 9, dtype=torch.int32, device="cuda")
    for bad in ((t(2), t(3), t(2), rtt, 10, t(3), t(2), t(4), t(4)), (t(2), t(2), t(2), rtt, 10, t(2), t(2), t(4), t(4)),
                (t(2), t(2), t(2), rtt, 10, t(3), t(1), t(4), t(4)), (t(2), t(2), t(2), rtt, 10, t(3), t(2), t(4), t(5)),
                (t(2), t(2), t(2), t(9), 10, t(3), t(2), t(4), t(4))):
        with pytest.raises(ValueError):
            rx.rx_step_maps(*bad)
    with pytest.raises(TypeError):
        rx.rx_step_maps(t(2), t(2).long(), t(2), rtt, 10, t(3), t(2), t(4), t(4))
