"""GPU parity of rx_qk_norm_rope_store and rx_qk_norm_rope_store_fp8 against
the fp64 oracle.

Bound of a value y' = rotation of y: the sum of squares (128 positive terms,
19 roundings deep), the root, the quotient and the products are 26 roundings
of 2^-24, 1.6e-6 relative on y; the angle is off by at most 2^-22 (its fp32
rounding near pi) plus 2^-31; the rotation adds three roundings.  Together
under 2.5e-6 (|y_c| + |y_c+d/2|).  Then half a step of the result's type."""
import numpy as np
import pytest

from oracle import draft, fp8
from prefix_shared_kv_radixattention_gb300 import inputs
from tests import _draft

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SLACK = 2.5e-6


def _g():
    from tests import _gpu
    return _gpu


def _case(seed, n, hq, hkv, d, packed, weights, size=2.0):
    g = _g()
    rng = np.random.default_rng(seed)
    R = hq + 2 * hkv
    x = inputs.bf16_round((size * rng.standard_normal((n, R, d))).astype(np.float32))
    if n:
        x[0, 0] = 0                                              # a head of zeros
        x[-1, hq] = inputs.bf16_round(np.full(d, 1e-20, np.float32))
    xd = g.to_dev(x)
    q, k, v = xd[:, :hq], xd[:, hq:hq + hkv], xd[:, hq + hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    w = [inputs.bf16_round((1 + 0.3 * rng.standard_normal(d)).astype(np.float32)) if weights else None for _ in range(2)]
    wd = [None if t is None else g.to_dev(t) for t in w]
    w64 = [None if t is None else inputs.bf16_to_f32(t).astype(np.float64) for t in w]
    pos = rng.integers(0, 200000, n).astype(np.int32)
    for i, p in zip(range(1, n), (10_000_000, 2**31 - 1, -7, -(2**31), 0)):
        pos[i] = p
    S = n + 37
    slots = rng.permutation(S)[:n].astype(np.int32)
    x64 = inputs.bf16_to_f32(x).astype(np.float64)
    return dict(x=x, x64=x64, q=q, k=k, v=v, wd=wd, w64=w64, pos=pos, S=S, slots=slots, hq=hq, hkv=hkv, d=d, n=n)


def _bound(y, half):
    """SLACK (|y_c| + |y_c+d/2|), y before the rotation."""
    h = y.shape[-1] // 2
    m = SLACK * (np.abs(y[..., :h]) + np.abs(y[..., h:]))
    return np.concatenate([m, m], -1) + half


def _heads(c, which, base, eps):
    hq, hkv = c["hq"], c["hkv"]
    x = c["x64"][:, :hq] if which == "q" else c["x64"][:, hq:hq + hkv]
    w = c["w64"][0 if which == "q" else 1]
    y = draft.qk_norm(x, w, eps)
    return y, draft.qk_norm_rope(x, w, c["pos"], base, eps)


def _check_bf16(got, y, ref, what):
    err = np.abs(got.astype(np.float64) - ref)
    assert (err <= _bound(y, _draft.HALF_STEP * np.abs(ref) + 1e-38)).all(), f"{what}: {err.max()}"


def _check_codes(codes, y, ref, scale, what):
    want, got = np.clip(ref / scale, -448, 448), fp8.decode(codes)
    half = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10)      # half a step; subnormals are 2^-9 apart
    err = np.abs(got - want)
    assert (err <= _bound(y / scale, half)).all(), f"{what}: {err.max()}"


CASES = [(1, 4, 4, 64), (3, 32, 8, 128), (67, 7, 1, 128), (130, 64, 8, 128), (641, 4, 4, 64), (33, 32, 32, 128),
         (1000, 5, 3, 64)]


@pytest.mark.parametrize("weights", [True, False], ids=["w", "no_w"])
@pytest.mark.parametrize("packed", [True, False], ids=["packed", "apart"])
@pytest.mark.parametrize("n,hq,hkv,d", CASES)
def test_parity(n, hq, hkv, d, packed, weights):
    g = _g()
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    base, eps = (10000.0, 1e-6) if packed else (500000.0, 1e-5)
    c = _case(n + d, n, hq, hkv, d, packed, weights)
    qo = g.Guarded((n, hq, d), torch.bfloat16)
    kp, vp = (g.Guarded((c["S"], hkv, d), torch.bfloat16) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rx.rx_qk_norm_rope_store(kp.t, vp.t, c["q"], qo.t, c["k"], c["v"], *c["wd"], g.i32(c["slots"]), g.i32(c["pos"]), base,
                             eps, status)
    torch.cuda.synchronize()
    for t in (qo, kp, vp):
        t.check("norm")
    assert int(status.item()) == 0
    _check_bf16(qo.t.float().cpu().numpy(), *_heads(c, "q", base, eps), "q")
    k = kp.t.float().cpu().numpy()
    _check_bf16(k[c["slots"]], *_heads(c, "k", base, eps), "k")
    assert np.array_equal(g.to_host_u16(vp.t)[c["slots"]], c["x"][:, hq + hkv:])
    rest = np.setdiff1d(np.arange(c["S"]), c["slots"])
    assert np.isnan(k[rest]).all() and np.isnan(vp.t.float().cpu().numpy()[rest]).all()
    # position 0 is the norm alone


@pytest.mark.parametrize("size", [2.0, 60.0])
@pytest.mark.parametrize("n,hq,hkv,d", CASES)
def test_parity_fp8(n, hq, hkv, d, size):
    g = _g()
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    base, eps, ks, vs = 10000.0, 1e-6, 0.0071, 0.13              # some K values and V values saturate
    c = _case(n + d, n, hq, hkv, d, True, True, size)
    qo = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    kp, vp = (torch.full((2, c["S"], hkv, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rx.rx_qk_norm_rope_store_fp8(kp, vp, ks, vs, c["q"], qo, c["k"], c["v"], *c["wd"], g.i32(c["slots"]), g.i32(c["pos"]),
                                 base, eps, status, layer=1)
    assert int(status.item()) == 0
    _check_bf16(qo.float().cpu().numpy(), *_heads(c, "q", base, eps), "q")
    k, v = kp.cpu().numpy(), vp.cpu().numpy()
    assert (k[0] == 0x7F).all() and (v[0] == 0x7F).all()         # the other layer
    _check_codes(k[1][c["slots"]], *_heads(c, "k", base, eps), float(np.float32(ks)), "k")
    # V: exactly what rx_kv_store_fp8 stores
    k2, v2 = torch.zeros_like(kp[1]), torch.zeros_like(vp[1])
    rx.rx_kv_store_fp8(k2, v2, ks, vs, c["k"].contiguous(), c["v"].contiguous(), g.i32(c["slots"]), status)
    assert np.array_equal(v[1][c["slots"]], v2.cpu().numpy()[c["slots"]])
    rest = np.setdiff1d(np.arange(c["S"]), c["slots"])
    assert (k[1][rest] == 0x7F).all() and (v[1][rest] == 0x7F).all()


def test_in_place_and_without_q_heads():
    g = _g()
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = _case(5, 77, 8, 2, 128, False, True)
    kp, vp = (torch.zeros(c["S"], 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k2, v2 = torch.zeros_like(kp), torch.zeros_like(vp)
    qo, q_in = torch.empty_like(c["q"]), c["q"].clone()
    tail = (c["k"], c["v"], *c["wd"], g.i32(c["slots"]), g.i32(c["pos"]), 10000.0, 1e-6)
    rx.rx_qk_norm_rope_store(kp, vp, c["q"], qo, *tail)
    assert torch.equal(c["q"], q_in)
    rx.rx_qk_norm_rope_store(k2, v2, q_in, q_in, *tail)
    assert torch.equal(q_in, qo) and torch.equal(kp, k2) and torch.equal(vp, v2)
    none = torch.empty(77, 0, 128, dtype=torch.bfloat16, device="cuda")
    k2.zero_(), v2.zero_()
    rx.rx_qk_norm_rope_store(k2, v2, none, none, *tail)
    assert torch.equal(kp, k2) and torch.equal(vp, v2)


def test_position_zero_and_unit_weights_is_the_norm():
    g = _g()
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = _case(6, 9, 4, 2, 64, True, False)
    qo = torch.empty(9, 4, 64, dtype=torch.bfloat16, device="cuda")
    kp, vp = (torch.zeros(c["S"], 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rx.rx_qk_norm_rope_store(kp, vp, c["q"], qo, c["k"], c["v"], None, None, g.i32(c["slots"]),
                             torch.zeros(9, dtype=torch.int32, device="cuda"), 10000.0, 1e-6)
    ref = draft.qk_norm(c["x64"][:, :4], None, 1e-6)
    _check_bf16(qo.float().cpu().numpy(), ref, ref, "norm")


def test_bad_slots_are_flagged_and_skipped():
    g = _g()
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = _case(7, 40, 4, 2, 64, True, True)
    slots = c["slots"].copy()
    slots[[3, 17, 39]] = [-1, c["S"], 2**31 - 1]
    qo = torch.empty(40, 4, 64, dtype=torch.bfloat16, device="cuda")
    kp, vp = (g.Guarded((c["S"], 2, 64), torch.bfloat16) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rx.rx_qk_norm_rope_store(kp.t, vp.t, c["q"], qo, c["k"], c["v"], *c["wd"], g.i32(slots), g.i32(c["pos"]), 10000.0, 1e-6,
                             status)
    assert int(status.item()) == 1
    kp.check(), vp.check()
    _check_bf16(qo.float().cpu().numpy(), *_heads(c, "q", 10000.0, 1e-6), "q")
    good = np.setdiff1d(np.arange(40), [3, 17, 39])
    y, ref = _heads(c, "k", 10000.0, 1e-6)
    _check_bf16(kp.t.float().cpu().numpy()[slots[good]], y[good], ref[good], "k")
    unwritten = np.setdiff1d(np.arange(c["S"]), slots[good])
    assert np.isnan(kp.t.float().cpu().numpy()[unwritten]).all()


def test_stream_graph_and_empty_call():
    g = _g()
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = _case(8, 50, 8, 2, 128, True, True)
    qo = torch.empty(50, 8, 128, dtype=torch.bfloat16, device="cuda")
    kp, vp = (torch.zeros(c["S"], 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots, pos = g.i32(c["slots"]), g.i32(c["pos"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rx.rx_qk_norm_rope_store(kp, vp, c["q"], qo, c["k"], c["v"], *c["wd"], slots, pos, 10000.0, 1e-6)
    pos.copy_(torch.flip(pos, [0]))
    c["pos"] = c["pos"][::-1].copy()
    graph.replay()
    torch.cuda.synchronize()
    _check_bf16(qo.float().cpu().numpy(), *_heads(c, "q", 10000.0, 1e-6), "q")
    e = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    i0 = torch.empty(0, dtype=torch.int32, device="cuda")
    rx.rx_qk_norm_rope_store(kp, vp, e, e, e[:, :2], e[:, :2], None, None, i0, i0, 10000.0, 1e-6)


def test_binding_refuses_wrong_tensors():
    g = _g()
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = _case(9, 6, 4, 2, 64, True, True)
    kp, vp = (torch.zeros(c["S"], 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    good = dict(q=c["q"], q_out=torch.empty(6, 4, 64, dtype=torch.bfloat16, device="cuda"), k_new=c["k"], v_new=c["v"],
                q_weight=c["wd"][0], k_weight=c["wd"][1], slots=g.i32(c["slots"]), pos=g.i32(c["pos"]))
    for name, val in (("q", c["q"].float()), ("q", c["q"][:, :, ::2]), ("q_out", good["q_out"][:5]), ("k_new", c["k"][:5]),
                      ("v_new", c["v"].contiguous()), ("q_weight", c["wd"][0][:32]), ("slots", good["slots"].long()),
                      ("pos", good["pos"][:3]), ("q_out", good["q_out"].transpose(0, 1))):
        with pytest.raises((TypeError, ValueError)):
            rx.rx_qk_norm_rope_store(kp, vp, base=10000.0, eps=1e-6, **{**good, name: val})
