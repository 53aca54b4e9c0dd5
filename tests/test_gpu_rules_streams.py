"""The calls with rules, the rotation on several axes and the lists of a step on a
stream of the caller's own, whose inputs are written there just before, and two
captured decode calls in flight; lists with more room than tokens."""
import numpy as np
import pytest

from oracle import rules as ref
from tests import _rules
from tests._chain import BASE, D, HKV, HQ, PAGE, Chain
from tests._rules import RulesBatch
from tests.test_gpu_draft_norm import _check_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _late(stream, *tensors):
    """Zeroes for the tensors, whose contents come back on `stream` some milliseconds later: a call on another stream
    reads the zeroes."""
    kept = [t.clone() for t in tensors]
    for t in tensors:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(10_000_000)
        for t, k in zip(tensors, kept):
            t.copy_(k)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("path", ["split", "staged", "decode", "decode 64"])
def test_attention_on_a_stream(path, f8):
    from tests.test_gpu_rules import STAGED, Run
    decode = path.startswith("decode")
    new = [1, 1] if decode else [20, 33]
    b = RulesBatch(95, 8, 2, 64 if path == "decode 64" else 128, [300, 40], new, cap=50.0, window=128)
    run, s = Run(b, f8), torch.cuda.Stream()
    ws = run.workspace(STAGED)
    o, lse = torch.zeros_like(run.q), torch.zeros(run.q.shape[:2], device="cuda")
    _late(s, run.q, run.rtt, run.seq, run.plen, run.nlen, run.indptr)
    if decode:
        run.decode(o, lse, ws, stream=s)
    else:
        run.extend(o, lse, ws, STAGED if path == "staged" else None, stream=s)
    s.synchronize()
    assert int(run.status.item()) == 0
    _rules.check(o.float().cpu().numpy(), lse.cpu().numpy(), b.oracle(run.q64, run.k64, run.v64), b)


def test_lists_and_rotation_on_a_stream_with_room_to_spare():
    """Lists longer than the tokens: what is behind the last one stays as it was, here slots that are none, whose rows
    are turned, flagged and not stored."""
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    from tests import _gpu as g
    c = Chain(96, 0)
    s = c.step([21, 12])
    room, st = s.n + 9, torch.cuda.Stream()
    rtt, pages, req, plen, nlen = (g.i32(x) for x in (np.full(c.rtt.shape, -1), c.pages, c.req, s.prefix, s.new))
    indptr, seq = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (3, 2))
    pos, slots = (torch.full((room,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    x = torch.zeros(room, HQ + 2 * HKV, D, dtype=torch.bfloat16, device="cuda")
    x[:s.n] = g.to_dev(s.x)
    axes = torch.zeros(3, room, dtype=torch.int32, device="cuda")
    axes[:, :s.n] = g.i32(s.pos).view(3, s.n)
    k, v = (torch.full((c.num_slots, HKV, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.full((room, HQ, D), 7.0, dtype=torch.bfloat16, device="cuda")
    listed, status = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    _late(st, nlen, pages, x, axes)
    rx.rx_step_maps(req, plen, nlen, rtt, c.num_slots, indptr, seq, pos, slots, pages=pages, page_size=PAGE, dev_status=listed, stream=st)
    rx.rx_qk_rope_axes_store(k, v, x[:, :HQ], q, x[:, HQ:HQ + HKV], x[:, HQ + HKV:], None, None, slots, axes, c.axis, BASE,
                             dev_status=status, stream=st)
    st.synchronize()
    assert int(listed.item()) == 0 and int(status.item()) == rx.RX_DEV_BAD_SLOT
    assert indptr.tolist() == s.lists[0] and pos.tolist() == s.lists[2] + [-1] * 9 and slots.tolist() == s.lists[3] + [-1] * 9
    q_want, k_want, v_want = c.rotated(s)
    _check_bf16(q[:s.n].float().cpu().numpy(), s.x64[:, :HQ], q_want, "q")
    at = np.array(s.lists[3])
    _check_bf16(k.float().cpu().numpy()[at], s.x64[:, HQ:HQ + HKV], k_want, "k")
    assert np.array_equal(v.double().cpu().numpy()[at], v_want)
    rest = np.setdiff1d(np.arange(c.num_slots), at)
    assert bool((k[torch.from_numpy(rest).cuda()] == 7).all()) and bool((v[torch.from_numpy(rest).cuda()] == 7).all())
    # attention over the first rows; those behind stay as they were
    o = torch.full_like(q, 5.0)
    ws = torch.empty(rx.rx_attn_rules_workspace(s.n, 2, HQ, HKV, D, 21), dtype=torch.uint8, device="cuda")
    rx.rx_attn_extend_rules(k, v, q, o, None, indptr, req, plen, nlen, rtt, 21, D ** -0.5, rx.AttnRules(cap=50.0), ws, listed)
    torch.cuda.synchronize()
    assert int(listed.item()) == 0 and bool((o[s.n:] == 5).all())
    q64, k64, v64 = (t.double().cpu().numpy() for t in (q[:s.n], k, v))
    r = ref.attention(q64, k64, v64, c.rtt, c.req, s.prefix, s.new, D ** -0.5, 50.0)
    _rules.check(o[:s.n].float().cpu().numpy(), None, r, type("B", (), dict(q=q64, cap=50.0)))


@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 2, 64)], ids=str)
def test_two_captured_decode_calls_in_flight(heads):
    from tests.test_gpu_rules import Run
    runs, graphs = [], []
    for seed in (97, 98):
        run = Run(RulesBatch(seed, *heads, [3000, 40, 700], [1, 1, 1], slopes=True, window=900))
        ws = run.workspace()
        o, lse = torch.zeros_like(run.q), torch.zeros(run.q.shape[:2], device="cuda")
        run.decode(o, lse, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run.decode(o, lse, ws)
        runs.append((run, ws, o, lse))
        graphs.append(graph)
    for run, *_ in runs:
        run.v.mul_(-2)
        run.v64 = run.v64 * -2
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for run, _, o, lse in runs:
        assert int(run.status.item()) == 0
        _rules.check(o.float().cpu().numpy(), lse.cpu().numpy(), run.b.oracle(run.q64, run.k64, run.v64), run.b)
