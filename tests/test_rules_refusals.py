"""Refusals of the calls with rules on the scores, of the rotation on several
axes and of the lists of a step, on the CPU: nothing is launched."""
import ctypes

import numpy as np
import pytest

from prefix_shared_kv_radixattention_gb300 import binding as rx

FAKE = 1 << 20
P = ctypes.c_void_p


def _pools(a):
    pool = rx.KVPool(a["k"], a["v"], a["slots"], a["hkv"], a["d"], a["L"], a["layer"])
    p8 = rx.KVPoolFp8(a["k"], a["v"], a["slots"], a["hkv"], a["d"], a["k_scale"], a["v_scale"], a["L"], a["layer"])
    return pool, p8


BASE = dict(k=FAKE, v=FAKE, slots=64, hkv=2, d=64, L=0, layer=0, k_scale=1.0, v_scale=1.0)


def _attn(decode=False, **kw):
    """Codes of the FP8 and the bf16 call."""
    lib = rx.library()
    a = dict(BASE, q=FAKE, o=FAKE, lse=None, hq=4, indptr=FAKE, req=FAKE, plen=FAKE, elen=FAKE, rtt=FAKE, stride=100, batch=3,
             max_len=40, ws=FAKE, ws_bytes=1 << 30, scale=0.125, cap=50.0, window=0, slope=None, see_from=None, see_to=None,
             rules=True)
    a.update(kw)
    rules = ctypes.byref(rx.AttnRulesStruct(a["cap"], a["window"], a["slope"], a["see_from"], a["see_to"])) if a["rules"] else None
    pool, p8 = _pools(a)
    head = (P(a["q"]), P(a["o"]), P(a["lse"]), a["hq"])
    tail = (rules, P(a["ws"]), a["ws_bytes"], a["scale"], None, None)
    if decode:
        rest = (*head, P(a["req"]), P(a["plen"]), P(a["rtt"]), a["stride"], a["batch"], *tail)
        out = [lib.rx_attn_decode_rules_fp8(ctypes.byref(p8), *rest)]
    else:
        rest = (*head, P(a["indptr"]), P(a["req"]), P(a["plen"]), P(a["elen"]), P(a["rtt"]), a["stride"], a["batch"],
                a["max_len"], *tail)
        out = [lib.rx_attn_extend_rules_fp8(ctypes.byref(p8), *rest)]
    if a["k_scale"] == 1.0 and a["v_scale"] == 1.0:
        out.append((lib.rx_attn_decode_rules if decode else lib.rx_attn_extend_rules)(ctypes.byref(pool), *rest))
    return set(out)


INVALID = [dict(q=None), dict(o=None), dict(req=None), dict(plen=None), dict(rtt=None), dict(k=None), dict(v=None), dict(stride=0),
           dict(stride=1 << 31), dict(batch=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=1e-39),
           dict(scale=3e38, cap=0.0, slope=FAKE), dict(hq=0), dict(slots=0), dict(hkv=0), dict(q=FAKE + 8), dict(o=FAKE + 2),
           dict(ws=FAKE + 16), dict(k=FAKE + 4), dict(v=FAKE + 8), dict(lse=FAKE + 2), dict(L=2, layer=2), dict(k_scale=0.0),
           dict(v_scale=-1.0), dict(k_scale=float("nan")), dict(rules=False), dict(cap=-1.0), dict(cap=float("nan")),
           dict(window=-1), dict(slope=FAKE + 2), dict(see_from=FAKE + 1)]


@pytest.mark.parametrize("decode", [False, True], ids=["extend", "decode"])
@pytest.mark.parametrize("bad", INVALID, ids=str)
@pytest.mark.parametrize("max_len", [40, 2000])
def test_attention_refuses_invalid_arguments(bad, decode, max_len):
    if bad == dict(scale=3e38, cap=0.0, slope=FAKE):
        bad = dict(bad, k_scale=2.0)                     # only the product is out of range
    assert _attn(decode, max_len=max_len, **bad) == {rx.RX_ERR_INVALID}
    assert rx.last_error()


@pytest.mark.parametrize("bad", [dict(indptr=None), dict(elen=None), dict(see_to=FAKE + 2), dict(max_len=-1)], ids=str)
def test_extend_refuses_invalid_arguments(bad):
    assert _attn(**bad) == {rx.RX_ERR_INVALID}


def test_decode_refuses_a_bound_behind_its_token():
    assert _attn(True, see_to=FAKE) == {rx.RX_ERR_INVALID}


@pytest.mark.parametrize("decode", [False, True], ids=["extend", "decode"])
@pytest.mark.parametrize("bad", [dict(d=96), dict(d=256), dict(hq=5), dict(hq=258), dict(cap=1e-4), dict(cap=2e6),
                                 dict(cap=float("inf")), dict(batch=65536)], ids=str)
def test_attention_refuses_unsupported_shapes(bad, decode):
    assert _attn(decode, **bad) == {rx.RX_ERR_UNSUPPORTED}


def test_extend_wants_head_groups_that_divide_its_tiles():
    assert _attn(hq=6) == {rx.RX_ERR_UNSUPPORTED}
    assert _attn(hq=6, max_len=2000) == {rx.RX_ERR_UNSUPPORTED}


def test_attention_refuses_a_short_workspace():
    need = rx.rx_attn_rules_workspace(0, 3, 4, 2, 64, 1)
    assert _attn(True, ws_bytes=need - 1) == {rx.RX_ERR_CAPACITY}
    for decode in (False, True):
        assert _attn(decode, ws=None) == {rx.RX_ERR_CAPACITY}
        assert _attn(decode, batch=0) == {rx.RX_OK}                      # nothing to do: no launch
    assert _attn(max_len=0) == {rx.RX_OK}
    need = rx.rx_attn_rules_workspace(1000, 3, 4, 2, 64, 40)
    assert _attn(ws_bytes=1 << 16, max_len=40) == {rx.RX_ERR_CAPACITY}
    assert _attn(ws_bytes=1 << 14, max_len=2000) == {rx.RX_ERR_CAPACITY}
    assert need >= 1000 * 2 * 64 * 4
    for bad in ((-1, 3, 4, 2, 64, 1), (0, 0, 4, 2, 64, 1), (0, 3, 5, 2, 64, 1), (0, 3, 4, 2, 96, 1), (0, 3, 4, 2, 64, 0),
                (0, 65536, 4, 2, 64, 1), (1 << 31, 3, 4, 2, 64, 9), (0, 3, 258, 2, 64, 1)):
        with pytest.raises(rx.RxError):
            rx.rx_attn_rules_workspace(*bad)


def test_rules_refuse_other_tensors():
    torch = pytest.importorskip("torch")
    with pytest.raises(TypeError):
        rx.AttnRules(slopes=torch.zeros(4))                              # not on the GPU
    with pytest.raises(ValueError):
        rx.AttnRules(window=-1)
    with pytest.raises(ValueError):
        rx.AttnRules(window=1 << 31)


def _axes(**kw):
    lib = rx.library()
    a = dict(BASE, q=FAKE, qs=256, out=FAKE, kn=FAKE, vn=FAKE, kvs=256, norm=0, qw=None, kw=None, sl=FAKE, pos=FAKE, ps=3, axes=3,
             pair=[c % 3 for c in range(64)], n=3, hq=4, base=10000.0, eps=0.0)
    a.update(kw)
    pair = None if a["pair"] is None else (ctypes.c_uint8 * 64)(*a["pair"])
    rest = (P(a["q"]), a["qs"], P(a["out"]), P(a["kn"]), P(a["vn"]), a["kvs"], a["norm"], P(a["qw"]), P(a["kw"]), P(a["sl"]),
            P(a["pos"]), a["ps"], a["axes"], pair, a["n"], a["hq"], a["base"], a["eps"], None, None)
    pool, p8 = _pools(a)
    out = [lib.rx_qk_rope_axes_store_fp8(ctypes.byref(p8), *rest)]
    if a["k_scale"] == 1.0:
        out.append(lib.rx_qk_rope_axes_store(ctypes.byref(pool), *rest))
    return set(out)


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(kn=None), dict(sl=None), dict(pos=None), dict(n=-1), dict(hq=-1),
                                 dict(qs=255), dict(kvs=120), dict(q=FAKE + 8), dict(k=FAKE + 4), dict(qs=512), dict(pair=None),
                                 dict(ps=2), dict(pair=[0] * 31 + [3] + [0] * 32), dict(axes=2), dict(qw=FAKE), dict(kw=FAKE),
                                 dict(norm=1, eps=-1.0), dict(norm=1, eps=float("nan")), dict(L=2, layer=5), dict(k_scale=0.0)],
                         ids=lambda b: str(b)[:40])
def test_axes_refuse_invalid_arguments(bad):
    assert _axes(**bad) == {rx.RX_ERR_INVALID}
    assert rx.last_error()


@pytest.mark.parametrize("bad", [dict(d=96, qs=512, out=FAKE + 4096), dict(base=1.0), dict(axes=0), dict(axes=9)], ids=str)
def test_axes_refuse_unsupported_shapes(bad):
    assert _axes(**bad) == {rx.RX_ERR_UNSUPPORTED}


def test_axes_of_nothing_are_a_noop():
    assert _axes(n=0, q=None, out=None, kn=None, vn=None, sl=None, pos=None) == {rx.RX_OK}
    assert _axes(n=0, eps=float("nan")) == {rx.RX_OK}                     # not looked at without a norm


def _maps(**kw):
    a = dict(req=FAKE, plen=FAKE, nlen=FAKE, batch=3, rtt=FAKE, stride=100, pages=None, ps=0, size=0, slots=640, indptr=FAKE,
             seq=FAKE + 64, pos=FAKE, out=FAKE, n=30)
    a.update(kw)
    return rx.library().rx_step_maps(P(a["req"]), P(a["plen"]), P(a["nlen"]), a["batch"], P(a["rtt"]), a["stride"], P(a["pages"]),
                                     a["ps"], a["size"], a["slots"], P(a["indptr"]), P(a["seq"]), P(a["pos"]), P(a["out"]), a["n"],
                                     None, None)


@pytest.mark.parametrize("bad", [dict(req=None), dict(plen=None), dict(nlen=None), dict(rtt=None), dict(indptr=None), dict(pos=None),
                                 dict(out=None), dict(batch=-1), dict(n=-1), dict(n=1 << 31), dict(stride=0), dict(stride=1 << 31),
                                 dict(slots=0), dict(slots=1 << 31), dict(pages=FAKE), dict(pages=FAKE, ps=4),
                                 dict(pages=FAKE, ps=4, size=-1), dict(pages=FAKE, size=16), dict(seq=FAKE)], ids=str)
def test_maps_refuse_invalid_arguments(bad):
    assert _maps(**bad) == rx.RX_ERR_INVALID
    assert rx.last_error()


def test_pair_axis_has_an_entry_a_pair():
    """The binding's own checks come before any use of the device."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("host tensors")
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        rx.rx_qk_rope_axes_store(x, x, x, x, x, x, None, None, None, None, np.zeros(32, np.uint8), 1e4)


@pytest.mark.parametrize("bad", [256, -1, 1.5, float("nan"), 1 << 40])
def test_pair_axis_is_not_cut_to_a_byte(bad):
    for make in (list, np.array):
        with pytest.raises(ValueError):
            rx._pair_axis(make([0] * 31 + [bad]))
    for good in ([0, 1, 255], np.array([0, 1, 255]), np.array([0., 1., 255.]), np.array([0, 1, 255], np.uint8)):
        axis, _, size = rx._pair_axis(good)
        assert axis.dtype == np.uint8 and axis.tolist() == [0, 1, 255] and size == 3


def _shared(f8, hq, hkv, batch, max_len):
    """Whether rx_attn_extend_rules shares the contexts among CTAs (else it copies them): the two refuse a workspace of
    one byte in words of their own."""
    lib, kw = rx.library(), dict(BASE, d=128, hkv=hkv)
    pool = _pools(kw)[1 if f8 else 0]
    rules = rx.AttnRulesStruct(50.0, 0, None, None, None)
    call = lib.rx_attn_extend_rules_fp8 if f8 else lib.rx_attn_extend_rules
    rc = call(ctypes.byref(pool), P(FAKE), P(FAKE), None, hq, P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), 100, batch, max_len,
              ctypes.byref(rules), P(FAKE), 1, 0.125, None, None)
    assert rc == rx.RX_ERR_CAPACITY
    words = rx.last_error()
    assert words.endswith("needed") != words.endswith("too small"), words
    return words.endswith("needed")


@pytest.mark.parametrize("f8,hq,hkv,batch,max_len,shared", [
    # few rows, any number of requests
    (False, 32, 8, 512, 16, True), (False, 32, 8, 64, 64, True), (False, 32, 8, 1, 64, True),
    # many rows: only where few CTAs would be left with long contexts
    (False, 64, 8, 4, 64, True), (False, 64, 8, 5, 64, False), (False, 32, 8, 8, 128, False), (False, 64, 8, 1, 256, True),
    # few kv heads: 4,096 rows and more at 64 CTAs and more take up to a third longer when shared
    (False, 8, 1, 1, 512, True), (False, 8, 1, 2, 512, True), (False, 8, 1, 5, 512, False), (False, 16, 1, 1, 1024, False),
    (False, 16, 2, 1, 1024, False), (False, 8, 2, 5, 512, False), (False, 8, 1, 5, 256, True), (False, 16, 1, 1, 512, True),
    (False, 8, 1, 1, 1025, False),
    # E4M3: every row tile gathers for itself
    (True, 32, 8, 8, 16, True), (True, 32, 8, 9, 16, False), (True, 64, 8, 4, 16, True), (True, 64, 8, 8, 16, False),
    (True, 32, 8, 2, 64, True), (True, 32, 8, 4, 64, False), (True, 8, 1, 16, 64, False), (True, 8, 1, 4, 64, True),
    (True, 8, 1, 1, 512, True), (True, 16, 1, 1, 512, False)])
def test_which_calls_share_their_contexts(f8, hq, hkv, batch, max_len, shared):
    assert _shared(f8, hq, hkv, batch, max_len) == shared
