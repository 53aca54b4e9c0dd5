"""The draft-verification operators on the CPU: pins of oracle/draft.py, the
host mask builder against it, and the refusals of the device entry points
(returned before any launch: the pointers here are never dereferenced)."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import draft
from prefix_shared_kv_radixattention_gb300 import binding as rx
from prefix_shared_kv_radixattention_gb300 import inputs
from tests import _draft

FAKE = 0x100000


def test_tree_mask_pin():
    #      0
    #    1   2      (3 follows the text so far)
    #    4
    see = draft.tree_mask([-1, 0, 0, -1, 1])
    assert see.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [0, 0, 0, 1, 0],
                                        [1, 1, 0, 0, 1]]


def test_tree_attention_of_a_chain_is_extend():
    """A chain of drafted tokens is the causal extend pass (the pinned C oracle)."""
    b = _draft.TreeBatch(3, 4, 2, 64, [17, 0, 40], [5, 3, 1], masks="chain")
    qb, kb, vb = (inputs.bf16_round(x) for x in (b.q, b.k, b.v))
    w = inputs.bf16_to_f32
    o, lse, a = b.oracle(w(qb), w(kb).astype(np.float64), w(vb).astype(np.float64))
    ro, rl = oracle.extend(qb, kb, vb, b.rtt, b.req_idx, b.prefix_len, np.array(b.trees), b.indptr, b.scale)
    assert np.abs(o - ro).max() < 1e-12 and np.abs(lse - rl).max() < 1e-12
    assert (a >= np.abs(o) - 1e-12).all()


def test_tree_attention_empty_row_and_single_key():
    q = np.ones((2, 1, 2))
    k, v = np.ones((3, 1, 2)), np.arange(6.0).reshape(3, 1, 2)
    o, lse, _ = draft.tree_attention(q, k, v, np.array([[2, 1]]), [0], [0], [0, 2], [np.array([[0, 0], [1, 0]], bool)], 0.5)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all()
    assert np.allclose(o[1, 0], v[2, 0]) and np.isclose(lse[1, 0], 1.0)   # 0.5 * (1 + 1)


def test_qk_norm_pins():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])                               # mean square 25 / 4
    assert np.allclose(draft.qk_norm(x, None, 0.0), x / 2.5)
    assert np.allclose(draft.qk_norm(x, [1, 2, 3, 4], 0.0), x / 2.5 * [1, 2, 3, 4])
    assert np.allclose(draft.qk_norm(x, None, 25 / 4 * 3), x / 5)        # eps inside the root
    assert np.array_equal(draft.qk_norm_rope(x, None, [0], 10000.0, 0.0), draft.qk_norm(x, None, 0.0))


def test_logits_pins():
    x = np.array([[1.0, -1.0, 2.0, 3.0, 0.5]], np.float32)
    out = draft.logits_process(x, 5, hist=[[0, 1, 2, 2]], prompt_len=[2], repetition=[2.0], frequency=[0.25],
                               presence=[0.5], bias=[([3, 3], [1.0, 0.5])], allow=np.array([[1, 1, 1, 1, 0]], bool),
                               allow_row=[0])[0]
    # 0 and 1 are in the prompt, 2 was made twice: 2 / 2 - 2 * 0.25 - 0.5
    assert out.tolist() == [0.5, -2.0, 0.0, 4.5, -np.inf]
    # a node's path counts too; a row whose mask allows nothing is all -inf
    out = draft.logits_process(np.repeat(x, 2, 0), 5, hist=[[]], frequency=[1.0], rows_of=[range(2)], draft=[[4, 4]],
                               see=[np.array([[1, 0], [1, 1]], bool)], allow=np.zeros((1, 5), bool), allow_row=[-1, 0])
    assert out[0].tolist() == [1.0, -1.0, 2.0, 3.0, -0.5] and np.isneginf(out[1]).all()


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 200])
def test_tree_mask_build(n):
    rng = np.random.default_rng(n)
    for words in ((n + 31) // 32, (n + 31) // 32 + 2):
        parent = _draft.random_parents(rng, n)
        mask, depth = rx.rx_tree_mask_build(parent, words)
        see = draft.tree_mask(parent)
        assert np.array_equal(mask, _draft.pack(see, words))
        assert np.array_equal(depth, see.sum(1) - 1)


def test_tree_mask_build_refusals():
    assert rx.rx_tree_mask_build([])[0].shape == (0, 0)
    for parent, words in (([0], 1), ([-1, 1], 1), ([-2], 1), ([-1] * 33, 1), ([-1, 5, 0], 1)):
        with pytest.raises(rx.RxError) as e:
            rx.rx_tree_mask_build(parent, words)
        assert e.value.code == rx.RX_ERR_INVALID


def _tree(lib, **kw):
    a = dict(k=FAKE, v=FAKE, slots=64, hkv=2, d=64, L=0, layer=0, q=FAKE, o=FAKE, lse=None, hq=4, indptr=FAKE, req=FAKE,
             plen=FAKE, mask=FAKE, words=2, rtt=FAKE, stride=100, batch=3, max_tree=40, ws=FAKE, ws_bytes=1 << 30,
             scale=0.125, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    P = ctypes.c_void_p
    rest = (P(a["q"]), P(a["o"]), P(a["lse"]), a["hq"], P(a["indptr"]), P(a["req"]), P(a["plen"]), P(a["mask"]),
            a["words"], P(a["rtt"]), a["stride"], a["batch"], a["max_tree"], P(a["ws"]), a["ws_bytes"], a["scale"],
            None, None)
    pool = rx.KVPool(a["k"], a["v"], a["slots"], a["hkv"], a["d"], a["L"], a["layer"])
    p8 = rx.KVPoolFp8(a["k"], a["v"], a["slots"], a["hkv"], a["d"], a["k_scale"], a["v_scale"], a["L"], a["layer"])
    out = [lib.rx_attn_tree_fp8(ctypes.byref(p8), *rest)]
    if a["k_scale"] > 0 and a["v_scale"] > 0:
        out.append(lib.rx_attn_tree(ctypes.byref(pool), *rest))
    return out


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(o=None), dict(indptr=None), dict(req=None), dict(plen=None), dict(rtt=None), dict(k=None),
    dict(stride=0), dict(stride=1 << 31), dict(batch=-1), dict(max_tree=0), dict(scale=0.0), dict(scale=float("nan")),
    dict(words=1), dict(words=0), dict(hq=0), dict(slots=0), dict(q=FAKE + 8), dict(o=FAKE + 2), dict(ws=FAKE + 16),
    dict(k=FAKE + 4), dict(mask=FAKE + 2), dict(lse=FAKE + 2), dict(L=2, layer=2), dict(k_scale=0.0),
    dict(v_scale=-1.0)], ids=str)
def test_tree_refuses_invalid_arguments(bad):
    assert set(_tree(rx.library(), **bad)) == {rx.RX_ERR_INVALID}
    assert rx.last_error()


@pytest.mark.parametrize("bad", [dict(d=96), dict(d=256), dict(hq=5), dict(hq=258, hkv=2), dict(max_tree=1025, words=40),
                                 dict(batch=65536), dict(hq=8193, hkv=8193)], ids=str)
def test_tree_refuses_unsupported_shapes(bad):
    assert set(_tree(rx.library(), **bad)) == {rx.RX_ERR_UNSUPPORTED}


def test_tree_refuses_a_short_workspace():
    need = rx.rx_attn_tree_workspace(3, 4, 2, 64, 40)
    assert need > 0
    assert set(_tree(rx.library(), ws_bytes=need - 1)) == {rx.RX_ERR_CAPACITY}
    assert set(_tree(rx.library(), ws=None)) == {rx.RX_ERR_CAPACITY}
    assert set(_tree(rx.library(), batch=0, ws_bytes=1 << 30)) == {rx.RX_OK}   # nothing to do: no launch
    for bad in ((3, 5, 2, 64, 40), (3, 4, 2, 96, 40), (-1, 4, 2, 64, 40), (3, 4, 2, 64, 0), (3, 4, 0, 64, 1)):
        with pytest.raises(rx.RxError):
            rx.rx_attn_tree_workspace(*bad)


def _norm(lib, **kw):
    a = dict(k=FAKE, v=FAKE, slots=64, hkv=2, d=64, L=0, layer=0, q=FAKE, qs=256, out=FAKE, kn=FAKE, vn=FAKE, kvs=256,
             qw=None, kw=None, sl=FAKE, pos=FAKE, n=3, hq=4, base=10000.0, eps=1e-6, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    P = ctypes.c_void_p
    rest = (P(a["q"]), a["qs"], P(a["out"]), P(a["kn"]), P(a["vn"]), a["kvs"], P(a["qw"]), P(a["kw"]), P(a["sl"]),
            P(a["pos"]), a["n"], a["hq"], a["base"], a["eps"], None, None)
    pool = rx.KVPool(a["k"], a["v"], a["slots"], a["hkv"], a["d"], a["L"], a["layer"])
    p8 = rx.KVPoolFp8(a["k"], a["v"], a["slots"], a["hkv"], a["d"], a["k_scale"], a["v_scale"], a["L"], a["layer"])
    out = [lib.rx_qk_norm_rope_store_fp8(ctypes.byref(p8), *rest)]
    if a["k_scale"] > 0 and a["v_scale"] > 0:
        out.append(lib.rx_qk_norm_rope_store(ctypes.byref(pool), *rest))
    return out


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(out=None), dict(kn=None), dict(vn=None), dict(sl=None), dict(pos=None), dict(k=None), dict(n=-1),
    dict(hq=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(qs=255), dict(qs=248), dict(kvs=120),
    dict(kvs=260), dict(q=FAKE + 8), dict(out=FAKE + 8), dict(kn=FAKE + 2), dict(vn=FAKE + 8), dict(qw=FAKE + 8),
    dict(kw=FAKE + 2), dict(k=FAKE + 4), dict(qs=512), dict(slots=0), dict(L=2, layer=-1), dict(k_scale=0.0)], ids=str)
def test_norm_refuses_invalid_arguments(bad):
    # qs=512 with q_out = q: rows that are not contiguous cannot be written in place
    assert set(_norm(rx.library(), **bad)) == {rx.RX_ERR_INVALID}


@pytest.mark.parametrize("bad", [dict(d=96, qs=512, out=FAKE + 4096), dict(base=1.0), dict(base=float("nan")),
                                 dict(hq=65536, qs=65536 * 64)], ids=str)
def test_norm_refuses_unsupported_shapes(bad):
    assert set(_norm(rx.library(), **bad)) == {rx.RX_ERR_UNSUPPORTED}


def test_norm_of_nothing_is_a_noop():
    assert set(_norm(rx.library(), n=0, q=None, out=None, kn=None, vn=None, sl=None, pos=None)) == {rx.RX_OK}


def _logits(lib, **kw):
    a = dict(n_req=4, vocab=100, rows=4, logits=FAKE, bf16=0, ls=100, out=FAKE + 4096, os=100, null=False)
    rules = {k: kw.pop(k) for k in list(kw) if k not in a}
    a.update(kw)
    r = rx.LogitsRulesStruct(n_req=a["n_req"], vocab=a["vocab"], **rules)
    P = ctypes.c_void_p
    return lib.rx_logits_process(None if a["null"] else ctypes.byref(r), P(a["logits"]), a["bf16"], a["ls"], P(a["out"]),
                                 a["os"], a["rows"], None, None)


@pytest.mark.parametrize("bad", [
    dict(null=True), dict(n_req=-1), dict(vocab=0), dict(rows=-1), dict(rows=5), dict(bf16=2), dict(logits=None),
    dict(out=None), dict(ls=99), dict(os=99), dict(logits=FAKE + 2), dict(out=FAKE + 2), dict(logits=FAKE + 1, bf16=1),
    dict(out=FAKE, ls=104), dict(out=FAKE, bf16=1), dict(hist=FAKE), dict(bias_ptr=FAKE), dict(bias_ptr=FAKE, bias_tok=FAKE),
    dict(allow=FAKE, n_allow=1), dict(allow=FAKE, allow_row=FAKE), dict(draft_tok=FAKE),
    dict(draft_tok=FAKE, qo_indptr=FAKE, tree_mask=FAKE)], ids=str)
def test_logits_refuses_invalid_arguments(bad):
    assert _logits(rx.library(), **bad) == rx.RX_ERR_INVALID


def test_logits_other_answers_without_a_launch():
    lib = rx.library()
    assert _logits(lib, n_req=70000, rows=70000) == rx.RX_ERR_UNSUPPORTED
    assert _logits(lib, vocab=(1 << 30) + 1, ls=1 << 31, os=1 << 31) == rx.RX_ERR_UNSUPPORTED
    assert _logits(lib, n_req=0, rows=0, logits=None, out=None) == rx.RX_OK
    assert _logits(lib, n_req=3, rows=0, qo_indptr=FAKE, logits=None, out=None) == rx.RX_OK
