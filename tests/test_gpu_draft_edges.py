"""Arguments at the edge of what the draft-verification calls take: tensors
without a word, a row or a token, and scales near the ends of fp32."""
import numpy as np
import pytest

from tests import _draft
from tests.test_gpu_draft_tree import Run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _rx():
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    return rx


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
def test_mask_rows_without_words_are_not_a_chain(f8):
    """A mask tensor of no words is too narrow for any tree; only None is a chain."""
    b = _draft.TreeBatch(61, 4, 2, 64, [10, 3], [3, 1])
    r = Run(b, f8)
    o, lse = torch.empty_like(r.q), torch.empty(r.q.shape[:2], device="cuda")
    r.mask = _i32(4, 0)
    with pytest.raises(ValueError):
        r.launch(o, lse)


def test_rules_without_words_or_mask_rows():
    """No words of a tree mask, no row of an allow table: refused, neither a
    chain nor rows without a grammar."""
    rx = _rx()
    indptr = torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        rx.LogitsRules(2, 400, qo_indptr=indptr, draft_tok=_i32(3), tree_mask=_i32(3, 0))
    with pytest.raises(ValueError):
        rx.LogitsRules(3, 400, allow=_i32(0, 16), allow_row=_i32(3))


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
def test_nothing_drafted(f8):
    """No request has a drafted token, or there is no request: nothing to do."""
    b = _draft.TreeBatch(62, 4, 2, 64, [10, 3], [1, 1])
    r = Run(b, f8)
    r.q, r.mask, r.indptr = r.q[:0], r.mask[:0], _i32(3)
    r.launch(torch.empty_like(r.q), None)
    r.indptr, r.req, r.plen = _i32(1), r.req[:0], r.plen[:0]
    r.launch(torch.empty_like(r.q), torch.empty(0, 4, device="cuda"))
    torch.cuda.synchronize()
    assert int(r.status.item()) == 0


@pytest.mark.parametrize("ks", [1e-13, 1e-30, 1e25])
def test_query_rows_of_zeros_and_scales_near_the_ends(ks):
    """Over FP8 pools a row's score factor is the product of sm_scale, the
    pool's scale and the row's power of two: it must not vanish (a masked
    place is -inf times it).  With K codes of order one the scores are
    about ks: every weight is the same for the small scales; for the large
    one only the rows of zeros are looked at."""
    b = _draft.TreeBatch(63, 4, 2, 64, [200, 0, 127], [7, 5, 1])
    b.q[::2] = 0.0
    if ks < 1:
        b.q[1::4] *= np.float32(1e-30)
    r = Run(b, True)             # codes of k / 0.07
    r.ks = ks
    r.k64 = r.k64 / 0.07 * ks
    o, lse = r()
    assert int(r.status.item()) == 0
    keep = slice(None) if ks < 1 else slice(0, None, 2)
    _draft.check_tree(o[keep], lse[keep], tuple(x[keep] for x in r.reference()), f"scale {ks}")


def test_calls_of_several_threads_at_once():
    """Every thread with a stream and outputs of its own: the results are those
    of the same calls one after the other."""
    import threading

    from tests.test_gpu_draft_logits import Case
    rx = _rx()
    c = Case(64, 5, 9001, hist=500, bias=20, states=3)
    rules, x = c.rules(), c.logits()
    runs = [Run(_draft.TreeBatch(65, 8, 2, 64, [300, 7, 129], [9, 4, 17]), f8) for f8 in (False, True)]

    def step(out, stream):
        for r, (o, lse, ws) in zip(runs, out[1:]):
            r.launch(o, lse, stream=stream, ws=ws)
        rx.rx_logits_process(rules, x, out[0], stream=stream)

    def outputs():
        return [torch.zeros(5, 9001, device="cuda")] + [
            (torch.zeros_like(r.q), torch.zeros(r.q.shape[:2], device="cuda"), torch.empty_like(r.ws)) for r in runs]

    want, outs = outputs(), [outputs() for _ in range(8)]
    step(want, None)
    torch.cuda.synchronize()
    streams, gate, bad = [torch.cuda.Stream() for _ in outs], threading.Barrier(len(outs)), []

    def work(out, stream):
        try:
            gate.wait(60)
            for _ in range(10):
                step(out, stream)
        except Exception as e:  # noqa: BLE001 -- reported by the test's thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(outs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad
    for out in outs:
        assert torch.equal(out[0], want[0])
        for (o, lse, _), (wo, wl, _) in zip(out[1:], want[1:]):
            assert torch.equal(o, wo) and torch.equal(lse, wl)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
def test_pools_past_32_bits_of_offset(f8):
    """The same rows in slots whose byte offset passes 2^32: the same bits.  The
    norm, rotation and store writes there too."""
    rx = _rx()
    b = _draft.TreeBatch(66, 32, 16, 128, [300, 0, 129], [9, 4, 17])
    r = Run(b, f8)
    want = r()
    rows = (2 ** 32 + 2 ** 28) // (16 * 128 * r.k.element_size())
    first = rows - b.num_slots
    k, v = (torch.zeros(rows, 16, 128, dtype=r.k.dtype, device="cuda") for _ in range(2))
    k[first:], v[first:] = r.k, r.v
    small = r.k, r.v
    r.k, r.v, r.rtt = k, v, torch.where(r.rtt < 0, r.rtt, r.rtt + first)
    got = r()
    assert int(r.status.item()) == 0
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])

    n = 40
    x = torch.randn(n, 64, 128, generator=torch.Generator().manual_seed(5)).cuda().bfloat16()
    slots = torch.randperm(b.num_slots, generator=torch.Generator().manual_seed(6))[:n].int().cuda()
    pos, q = torch.arange(n, dtype=torch.int32, device="cuda"), torch.empty(n, 32, 128, dtype=torch.bfloat16, device="cuda")
    for pools, at in ((small, slots), ((k, v), slots + first)):
        args = (x[:, :32], q, x[:, 32:48], x[:, 48:], None, None, at, pos, 10000.0, 1e-6, r.status)
        if f8:
            rx.rx_qk_norm_rope_store_fp8(*pools, 0.05, 0.05, *args)
        else:
            rx.rx_qk_norm_rope_store(*pools, *args)
    assert int(r.status.item()) == 0
    for big, little in zip((k, v), small):
        assert torch.equal(big[first:], little) and not big[:first].any()


def test_logits_past_32_bits_of_offset():
    """17,000 rows of 128,256 ids (2^31 elements and more): the last rows as
    those of a call of their own."""
    rx = _rx()
    n, V, m = 17000, 128256, 3
    x = torch.zeros(n, V, dtype=torch.bfloat16, device="cuda")
    x[-m:] = torch.randn(m, V, generator=torch.Generator().manual_seed(7)).cuda()
    out = torch.empty(n, V, device="cuda")
    pres = torch.linspace(0, 1, n, device="cuda")
    hist = torch.arange(n, dtype=torch.int32, device="cuda") % V
    ptr = torch.arange(n + 1, device="cuda")
    rx.rx_logits_process(rx.LogitsRules(n, V, hist=hist, hist_ptr=ptr, presence=pres), x, out)
    few = torch.empty(m, V, device="cuda")
    rx.rx_logits_process(rx.LogitsRules(m, V, hist=hist[-m:].contiguous(), hist_ptr=ptr[:m + 1].contiguous(),
                                        presence=pres[-m:].contiguous()), x[-m:], few)
    assert torch.equal(out[-m:], few)
    assert (few != x[-m:].float()).sum() == m and (out[:-m] != 0).sum() == n - m - 1   # the first row's presence is 0
