"""GPU parity of rx_qk_rope_axes_store and its FP8 form against the fp64 oracle.

Bound: that of tests/test_gpu_draft_norm.py with the norm (2.5e-6 of |y_c| +
|y_c+d/2|, then half a step of the result's type), and without it too, where
the angle's and the rotation's share of it remains."""
import numpy as np
import pytest

from oracle import draft, fp8
from oracle import rules as ref
from prefix_shared_kv_radixattention_gb300 import inputs
from tests.test_gpu_draft_norm import _case, _check_bf16, _check_codes, _g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

CASES = [(1, 4, 4, 64), (3, 32, 8, 128), (67, 7, 1, 128), (130, 64, 8, 128), (641, 4, 4, 64), (33, 32, 32, 128)]


def _axes_case(seed, shape, axes, packed, norm, weights, size=2.0):
    c = _case(seed, *shape, packed, weights and norm, size=size)
    rng = np.random.default_rng(seed + 1)
    n, d = c["n"], c["d"]
    pos = np.stack([c["pos"]] + [rng.integers(-3000, 150000, n).astype(np.int32) for _ in range(axes - 1)])
    return c, pos, rng.integers(0, axes, d // 2).astype(np.uint8)


def _call(c, pos, axis, base, eps, pools, scales=None, q_out=None, layer=0):
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    g = _g()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (c["q"], q_out, c["k"], c["v"], *c["wd"], g.i32(c["slots"]), g.i32(pos).view(pos.shape), axis, base, eps, status)
    if scales is None:
        rx.rx_qk_rope_axes_store(*pools, *args, layer=layer)
    else:
        rx.rx_qk_rope_axes_store_fp8(*pools, *scales, *args, layer=layer)
    torch.cuda.synchronize()
    return int(status.item())


def _want(c, pos, axis, base, eps, which):
    x = c["x64"][:, :c["hq"]] if which == "q" else c["x64"][:, c["hq"]:c["hq"] + c["hkv"]]
    w = c["w64"][0 if which == "q" else 1]
    y = x if eps is None else draft.qk_norm(x, w, eps)
    return y, ref.rope_axes(x, pos, axis, base, w, eps)


@pytest.mark.parametrize("eps", [None, 1e-6], ids=["plain", "norm"])
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("shape", CASES, ids=str)
def test_bf16(shape, packed, eps):
    g = _g()
    for axes in (1, 3, 8):
        c, pos, axis = _axes_case(31 + axes, shape, axes, packed, eps is not None, weights=axes != 3)
        n, hq, hkv, d = shape
        pools = [torch.full((c["S"], hkv, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        out = g.Guarded((n, hq, d), torch.bfloat16)
        assert _call(c, pos, axis, 1e6, eps, pools, q_out=out.t) == 0
        out.check("q_out")
        _check_bf16(out.t.float().cpu().numpy(), *_want(c, pos, axis, 1e6, eps, "q"), "q")
        k, v = (p.float().cpu().numpy() for p in pools)
        _check_bf16(k[c["slots"]], *_want(c, pos, axis, 1e6, eps, "k"), "k")
        assert np.array_equal(v[c["slots"]], c["x64"][:, hq + hkv:].astype(np.float32))
        rest = np.setdiff1d(np.arange(c["S"]), c["slots"])
        assert (k[rest] == 9).all() and (v[rest] == 9).all()


@pytest.mark.parametrize("size", [2.0, 1e13, 1e-20])
@pytest.mark.parametrize("eps", [None, 1e-6], ids=["plain", "norm"])
@pytest.mark.parametrize("shape", CASES, ids=str)
def test_fp8(shape, eps, size):
    if size != 2.0 and eps is not None:
        pytest.skip("sizes matter without a norm")
    c, pos, axis = _axes_case(41, shape, 3, True, eps is not None, True, size=size)
    n, hq, hkv, d = shape
    scales = (0.021 * size, 0.0173 * size)
    pools = [torch.full((c["S"], hkv, d), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    assert _call(c, pos, axis, 1e4, eps, pools, scales, q_out=out) == 0
    _check_bf16(out.float().cpu().numpy(), *_want(c, pos, axis, 1e4, eps, "q"), "q")
    k, v = (p.cpu().numpy() for p in pools)
    sc = [float(np.float32(s)) for s in scales]
    _check_codes(k[c["slots"]], *_want(c, pos, axis, 1e4, eps, "k"), sc[0], "k")
    x = c["x64"][:, hq + hkv:]
    _check_codes(v[c["slots"]], x, x, sc[1], "v")
    rest = np.setdiff1d(np.arange(c["S"]), c["slots"])
    assert (k[rest] == 9).all() and (v[rest] == 9).all()


def test_one_axis_is_the_norm_rotation_and_store():
    """Bit for bit, with the norm and equal positions on the axes."""
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    g = _g()
    c, pos, axis = _axes_case(51, (130, 16, 4, 128), 3, True, True, True)
    pos[:] = pos[0]
    got, want = ([torch.zeros(c["S"], 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)] +
                 [torch.empty(130, 16, 128, dtype=torch.bfloat16, device="cuda")] for _ in range(2))
    assert _call(c, pos, axis, 1e4, 1e-6, got[:2], q_out=got[2]) == 0
    rx.rx_qk_norm_rope_store(*want[:2], c["q"], want[2], c["k"], c["v"], *c["wd"], g.i32(c["slots"]), g.i32(pos[0]), 1e4, 1e-6)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_in_place_layers_bad_slots_and_strided_positions():
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c, pos, axis = _axes_case(52, (40, 8, 2, 64), 3, False, False, False)
    c["slots"][3], c["slots"][7] = -1, c["S"]
    pools = [torch.zeros((3, c["S"], 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert _call(c, pos, axis, 1e4, None, pools, q_out=c["q"], layer=1) == rx.RX_DEV_BAD_SLOT
    _check_bf16(c["q"].float().cpu().numpy(), *_want(c, pos, axis, 1e4, None, "q"), "q")    # their q rows are written
    ok = [i for i in range(40) if i not in (3, 7)]
    y, want = _want(c, pos, axis, 1e4, None, "k")
    _check_bf16(pools[0][1].float().cpu().numpy()[c["slots"][ok]], y[ok], want[ok], "k")
    assert not pools[0][0].any() and not pools[0][2].any()
    assert int((pools[0][1] != 0).any(-1).any(-1).sum()) == 38


def test_refused_tensors():
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c, pos, axis = _axes_case(53, (4, 4, 2, 64), 3, False, False, False)
    g = _g()
    pools = [torch.zeros((c["S"], 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = torch.empty_like(c["q"])

    def call(p=pos, a=axis, o=out):
        rx.rx_qk_rope_axes_store(*pools, c["q"], o, c["k"], c["v"], None, None, g.i32(c["slots"]), g.i32(p), a, 1e4)

    call()
    for bad in (dict(p=pos[:, :3]), dict(p=pos[0]), dict(a=axis[:31]), dict(o=out[:3]), dict(a=torch.zeros(33, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(TypeError):
        call(a=torch.zeros(32, dtype=torch.int32))
    with pytest.raises(rx.RxError):
        call(a=np.full(32, 3, np.uint8))
