"""The bindings of the calls with rules, of the rotation on several axes and of
the lists of a step refuse a tensor that is not on the current device, whichever
it is.  On the CPU: the tensors are fakes without memory."""
import pytest

from prefix_shared_kv_radixattention_gb300 import binding as rx

torch = pytest.importorskip("torch")
fake = pytest.importorskip("torch._subclasses.fake_tensor")


@pytest.fixture
def on_device_0(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(fake.FakeTensor, "data_ptr", lambda self: 4096, raising=False)

    class Called(Exception):
        pass

    def launch(*a):
        raise Called

    for name in ("rx_attn_extend_rules", "rx_attn_extend_rules_fp8", "rx_attn_decode_rules", "rx_attn_decode_rules_fp8",
                 "rx_qk_rope_axes_store", "rx_qk_rope_axes_store_fp8", "rx_step_maps"):
        monkeypatch.setattr(rx._lib, name, launch)
    monkeypatch.setattr(rx, "_stream", lambda *a: 0)
    with fake.FakeTensorMode():
        yield Called


def _args(away):
    """Every tensor of the calls by its name; `away` on device 1, the others on 0."""
    bf16, i32, u8, f32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
    shapes = dict(k_pool=(bf16, 64, 2, 64), v_pool=(bf16, 64, 2, 64), k_code=(u8, 64, 2, 64), v_code=(u8, 64, 2, 64),
                  q=(bf16, 3, 4, 64), o=(bf16, 3, 4, 64), lse=(f32, 3, 4), indptr=(i32, 4), req=(i32, 3), plen=(i32, 3), nlen=(i32, 3),
                  rtt=(i32, 5, 20), ws=(u8, 1 << 20), status=(i32, 1), slopes=(f32, 4), see_from=(i32, 3), see_to=(i32, 3),
                  k_new=(bf16, 3, 2, 64), v_new=(bf16, 3, 2, 64), qw=(bf16, 64), kw=(bf16, 64), slots=(i32, 3), axes=(i32, 2, 3),
                  pos=(i32, 3), seq=(i32, 3), pages=(i32, 5, 4))
    return {n: torch.empty(s, dtype=t, device="cuda:1" if n == away else "cuda:0") for n, (t, *s) in shapes.items()}


def _rules(a, to=True):
    return rx.AttnRules(30.0, 8, a["slopes"], a["see_from"], a["see_to"] if to else None)


def _extend(a, f8):
    pool = (a["k_code"], a["v_code"], 1.0, 1.0) if f8 else (a["k_pool"], a["v_pool"])
    (rx.rx_attn_extend_rules_fp8 if f8 else rx.rx_attn_extend_rules)(
        *pool, a["q"], a["o"], a["lse"], a["indptr"], a["req"], a["plen"], a["nlen"], a["rtt"], 1, 0.125, _rules(a), a["ws"], a["status"])


def _decode(a, f8):
    pool = (a["k_code"], a["v_code"], 1.0, 1.0) if f8 else (a["k_pool"], a["v_pool"])
    (rx.rx_attn_decode_rules_fp8 if f8 else rx.rx_attn_decode_rules)(
        *pool, a["q"], a["o"], a["lse"], a["req"], a["seq"], a["rtt"], 0.125, _rules(a, False), a["ws"], a["status"])


def _axes(a, f8):
    pool = (a["k_code"], a["v_code"], 1.0, 1.0) if f8 else (a["k_pool"], a["v_pool"])
    (rx.rx_qk_rope_axes_store_fp8 if f8 else rx.rx_qk_rope_axes_store)(
        *pool, a["q"], a["o"], a["k_new"], a["v_new"], a["qw"], a["kw"], a["slots"], a["axes"], [0] * 32, 1e4, 1e-6, a["status"])


def _maps(a, f8):
    rx.rx_step_maps(a["req"], a["plen"], a["nlen"], a["rtt"], 64, a["indptr"], a["seq"], a["pos"], a["slots"], a["pages"], 16, a["status"])


POOL = ["k_pool", "v_pool"]
CASES = [(_extend, POOL + ["q", "o", "lse", "indptr", "req", "plen", "nlen", "rtt", "ws", "status", "slopes", "see_from", "see_to"]),
         (_decode, POOL + ["q", "o", "lse", "req", "seq", "rtt", "ws", "status", "slopes", "see_from"]),
         (_axes, POOL + ["q", "o", "k_new", "v_new", "qw", "kw", "slots", "axes", "status"])]
NAMED = [(call, n, False) for call, names in CASES for n in names]
NAMED += [(call, n.replace("_pool", "_code"), True) for call, names in CASES for n in names]
NAMED += [(_maps, n, False) for n in ("req", "plen", "nlen", "rtt", "indptr", "seq", "pos", "slots", "pages", "status")]


@pytest.mark.parametrize("call,name,f8", NAMED, ids=lambda x: x.__name__ if callable(x) else str(x))
def test_a_tensor_elsewhere_is_refused(call, name, f8, on_device_0):
    with pytest.raises(ValueError, match="current CUDA device"):
        call(_args(name), f8)


@pytest.mark.parametrize("call", [_extend, _decode, _axes, _maps])
def test_tensors_here_are_taken(call, on_device_0):
    with pytest.raises(on_device_0):
        call(_args(None), False)
