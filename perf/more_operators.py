"""One layer's attention step of a model that reads images and text, as cases to measure.

Next to the model's own matrix products, such a step runs four operators of
this library:

  maps    rx_step_maps: the lists that the other calls take (where each
          request's new tokens start, their positions and slots), built on
          the GPU from the requests' lengths, from slot lists or from pages;
  rotate  rx_qk_rope_axes_store(_fp8): rotary embedding of every q and k head
          with positions on several axes (time, height, width), after an
          optional RMS norm, and the scatter of K and V into the slot pool;
  extend  rx_attn_extend_rules(_fp8): attention of the new tokens over their
          slot lists with rules on the scores: a tanh cap, a bias that falls
          with the distance, a window, and for each token the positions that
          it sees (documents, images whose tokens see one another, prefixes);
  decode  rx_attn_decode_rules(_fp8): the same rules for one token a request.

``run`` computes them in elementary torch operations, or through the
library's binding where ``own`` is set.  Head counts, head sizes and lengths
are those of the library's workloads (32/32, 32/8 and 64/8 heads of 128, 4/4
of 64; 1,280, 8,192 and 32,768 tokens of context).
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
PAGE = 16  # tokens of a page

HEADS = [(32, 32, 128), (32, 8, 128), (64, 8, 128), (4, 4, 64)]


def listed():
    return [
        # the tiny extend batch: latency counts
        dict(name="extend_tiny", op="extend", batch=4, hq=4, hkv=4, d=64, prefix=64, new=16, group=4, cap=30.0, window=0,
             slopes=False, mask="prefix", span=0, fp8=False),
        # prompts with images over a cached prefix, four requests to a prefix: an image's tokens see all of it
        dict(name="extend_images", op="extend", batch=32, hq=32, hkv=8, d=128, prefix=2048, new=512, group=4, cap=0.0,
             window=0, slopes=False, mask="spans", span=144, fp8=False),
        # the extend part of the long chat step, capped scores
        dict(name="extend_capped", op="extend", batch=16, hq=64, hkv=8, d=128, prefix=4096, new=1024, group=1, cap=50.0,
             window=0, slopes=False, mask="", span=0, fp8=False),
        # a windowed layer of capped scores, documents packed into odd lengths, E4M3 pools
        dict(name="extend_window_fp8", op="extend", batch=7, hq=32, hkv=8, d=128, prefix=8191, new=1531, group=1, cap=50.0,
             window=1024, slopes=False, mask="docs", span=700, fp8=True),
        # one user's next token
        dict(name="decode_one", op="decode", batch=1, hq=32, hkv=8, d=128, ctx=333, cap=50.0, window=0, slopes=False,
             mask="", fp8=False),
        # few-shot batch, scores that fall with the distance
        dict(name="decode_few_shot", op="decode", batch=64, hq=32, hkv=32, d=128, ctx=1281, cap=0.0, window=0, slopes=True,
             mask="", fp8=False),
        # long multi-turn chat, capped scores
        dict(name="decode_long_chat", op="decode", batch=16, hq=64, hkv=8, d=128, ctx=32768, cap=50.0, window=0,
             slopes=False, mask="", fp8=False),
        # a windowed layer over long contexts, E4M3 pools
        dict(name="decode_window_fp8", op="decode", batch=64, hq=32, hkv=8, d=128, ctx=32768, cap=50.0, window=4096,
             slopes=False, mask="docs", fp8=True),
        # the projections of one small batch: latency counts
        dict(name="rotate_small_batch", op="rotate", n=16, hq=32, hkv=8, d=128, axes=3, mixed=False, norm=False, fp8=False,
             packed=True),
        # the extend part of the long chat step, with the norm of each head
        dict(name="rotate_extend", op="rotate", n=16384, hq=64, hkv=8, d=128, axes=3, mixed=True, norm=True, fp8=False,
             packed=True),
        # a decode batch: one new token a request
        dict(name="maps_decode", op="maps", batch=64, prefix=1280, new=1, paged=False),
        # a large batch of prompts over pages
        dict(name="maps_extend", op="maps", batch=256, prefix=4096, new=1024, paged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "extend", "decode", "decode", "rotate", "maps"])
    if op == "maps":
        batch, new = _log(rng, 1, 1024), _log(rng, 1, 4096)
        return dict(op=op, batch=batch, prefix=_log(rng, 1, 32768), new=max(1, min(new, 256 * 1024 // batch)),
                    paged=rng.random() < 0.5)
    hq, hkv, d = rng.choice(HEADS)
    if op == "rotate":
        n = min(_log(rng, 1, 16384), 16384 * 80 * 128 // ((hq + 2 * hkv) * d))
        return dict(op=op, n=n, hq=hq, hkv=hkv, d=d, axes=rng.choice([2, 3, 3, 4]), mixed=rng.random() < 0.5,
                    norm=rng.random() < 0.5, fp8=rng.random() < 0.4, packed=rng.random() < 0.7)
    cap = rng.choice([0.0, 0.0, 30.0, 50.0, 80.0])
    window = rng.choice([0, 0, _log(rng, 16, 8192)])
    slopes, fp8 = rng.random() < 0.3, rng.random() < 0.4
    if op == "decode":
        batch, ctx = _log(rng, 1, 64), _log(rng, 1, 32768)
        ctx = max(1, min(ctx, 16 * 32768 * 8 * 128 // (batch * hkv * d)))
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, ctx=ctx, cap=cap, window=window, slopes=slopes,
                    mask=rng.choice(["", "", "docs"]), fp8=fp8)
    batch, new, prefix = _log(rng, 1, 32), _log(rng, 1, 2048), _log(rng, 1, 16384)
    # no more cached values and scores than the long chat's extend part has
    new = max(1, min(new, 16 * 64 * 1024 * 5120 // (batch * hq * (prefix + 2048))))
    prefix = max(1, min(prefix, 16 * 5120 * 8 * 128 // (batch * hkv * d) - new, 16 * 64 * 1024 * 5120 // (batch * hq * new) - new))
    return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, prefix=prefix, new=new, group=rng.choice([1, 1, 4]), cap=cap,
                window=window, slopes=slopes, mask=rng.choice(["", "prefix", "spans", "docs"]), span=_log(rng, 16, 1024),
                fp8=fp8)


# --------------------------------------------------------------------------- inputs


def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1000003 + salt) % (1 << 62))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def _sizes(c):
    """New tokens of each request: from half of the most up to it."""
    return [c["new"] - 37 * i % (c["new"] // 2 + 1) for i in range(c["batch"])]


def _seen(c, i, P, T):
    """What new token i of T (numpy) may see beside the rules that need no list: from which position, up to which."""
    lo, hi = np.zeros_like(i), np.zeros_like(i)
    if c["mask"] == "prefix":     # the first half of the new tokens is a prefix whose tokens all see one another
        hi = np.where(i < (T + 1) // 2, P + (T + 1) // 2, 0)
    elif c["mask"] == "spans":    # every other span is an image
        k = i // c["span"]
        hi = np.where(k % 2 == 0, P + np.minimum(T, (k + 1) * c["span"]), 0)
    elif c["mask"] == "docs":     # the first document goes on from the cached text
        k = i // c["span"]
        lo = np.where(k > 0, P + k * c["span"], 0)
    return lo, hi


def _pools(s, g, slots, hkv, d, fp8):
    k, v = _randn(g, slots, hkv, d), _randn(g, slots, hkv, d)
    if fp8:
        s["k_scale"], s["v_scale"] = 0.0517, 0.0423
        s["k"] = (k / s["k_scale"]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["v"] = (v / s["v_scale"]).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["k"], s["v"] = k.to(torch.bfloat16), v.to(torch.bfloat16)


def _slopes(c):
    """A head's score falls by its slope a token: 2^(-8/Hq) and its powers."""
    h = torch.arange(1, c["hq"] + 1, device=DEV, dtype=torch.float64)
    return torch.exp2(-8 * h / c["hq"]).float() if c["slopes"] else None


def _prepare_extend(c, seed):
    g, rng = _gen(seed, 1), random.Random(seed * 7 + 1)
    B, hq, hkv, d, G = c["batch"], c["hq"], c["hkv"], c["d"], c["group"]
    new = _sizes(c)
    heads = -(-B // G)
    pre = [rng.randint((c["prefix"] + 1) // 2, c["prefix"]) for _ in range(heads)]
    pre[0] = c["prefix"]
    plen = [pre[b // G] for b in range(B)]
    slots = sum(pre) + sum(new)
    perm = torch.randperm(slots, generator=g, device=DEV).to(torch.int32)
    rtt = torch.full((B, c["prefix"] + c["new"]), -1, dtype=torch.int32, device=DEV)
    at, own_at = 0, sum(pre)
    for b in range(B):
        if b and b % G == 0:
            at += pre[b // G - 1]
        rtt[b, :plen[b]] = perm[at:at + plen[b]]
        rtt[b, plen[b]:plen[b] + new[b]] = perm[own_at:own_at + new[b]]
        own_at += new[b]
    lo, hi = zip(*[_seen(c, np.arange(new[b]), plen[b], new[b]) for b in range(B)])
    n = sum(new)
    # queries whose scores spread as a trained model's: some reach the cap
    q = (3 * _randn(g, n, hq, d)).to(torch.bfloat16)
    s = dict(c=c, q=q, rtt=rtt, plen=_i32(plen), elen=_i32(new), indptr=_i32(np.cumsum([0] + new)),
             req=torch.arange(B, dtype=torch.int32, device=DEV), scale=1 / math.sqrt(d), slopes=_slopes(c),
             see_from=_i32(np.concatenate(lo)) if c["mask"] == "docs" else None,
             see_to=_i32(np.concatenate(hi)) if c["mask"] in ("prefix", "spans") else None,
             context=sum(plen) + n, o=torch.empty_like(q), lse=torch.empty(n, hq, device=DEV),
             status=torch.zeros(1, dtype=torch.int32, device=DEV), kept={})
    _pools(s, g, slots, hkv, d, c["fp8"])
    return s


def _prepare_decode(c, seed):
    g, rng = _gen(seed, 2), random.Random(seed * 7 + 2)
    B, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
    n = [rng.randint((c["ctx"] + 1) // 2, c["ctx"]) for _ in range(B)]
    n[0] = c["ctx"]
    perm = torch.randperm(B * c["ctx"], generator=g, device=DEV).to(torch.int32)
    q = (3 * _randn(g, B, hq, d)).to(torch.bfloat16)
    s = dict(c=c, q=q, rtt=perm.view(B, c["ctx"]), seq=_i32(n), req=torch.arange(B, dtype=torch.int32, device=DEV),
             scale=1 / math.sqrt(d), slopes=_slopes(c),
             see_from=_i32([rng.randint(0, x // 2) for x in n]) if c["mask"] == "docs" else None, see_to=None,
             o=torch.empty_like(q), lse=torch.empty(B, hq, device=DEV),
             status=torch.zeros(1, dtype=torch.int32, device=DEV), kept={})
    _pools(s, g, B * c["ctx"], hkv, d, c["fp8"])
    return s


def _pair_axis(c):
    """The axis that turns each pair: the axes in turn, or sections one behind the other (with three axes 16, 24 and 24
    of 64 pairs)."""
    half, a = c["d"] // 2, c["axes"]
    if c["mixed"]:
        return [i % a for i in range(half)]
    first = half // (a + 1)
    return [0] * first + [1 + i * (a - 1) // (half - first) for i in range(half - first)]


def _prepare_rotate(c, seed):
    g = _gen(seed, 3)
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    # the model's projection: one row a token, q heads, k heads, v heads
    qkv = (2 * _randn(g, n, hq + 2 * hkv, d)).to(torch.bfloat16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if not c["packed"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    slots = n + n // 2 + 64
    pool = torch.uint8 if c["fp8"] else torch.bfloat16
    # text far into a long conversation: the same position on every axis; images: a frame, and places in it
    pos = torch.randint(0, 131072, (n,), generator=g, device=DEV, dtype=torch.int32).expand(c["axes"], n).contiguous()
    image = torch.rand(n, generator=g, device=DEV) < 0.6
    pos[1:] += torch.where(image, torch.randint(0, 96, (c["axes"] - 1, n), generator=g, device=DEV, dtype=torch.int32), 0)
    w = [(1 + 0.2 * _randn(g, d)).to(torch.bfloat16) if c["norm"] else None for _ in range(2)]
    return dict(c=c, q=q, k_new=k, v_new=v, q_out=torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV), qw=w[0], kw=w[1],
                k=torch.zeros(slots, hkv, d, dtype=pool, device=DEV), v=torch.zeros(slots, hkv, d, dtype=pool, device=DEV),
                slots=torch.randperm(slots, generator=g, device=DEV)[:n].to(torch.int32), pos=pos,
                axis=torch.tensor(_pair_axis(c), dtype=torch.uint8), axis_dev=torch.tensor(_pair_axis(c), device=DEV),
                base=1000000.0, eps=1e-6 if c["norm"] else None, k_scale=0.0523, v_scale=0.0517,
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_maps(c, seed):
    g, rng = _gen(seed, 4), random.Random(seed * 7 + 4)
    B = c["batch"]
    new = _sizes(c)
    pre = [rng.randint(0, c["prefix"]) for _ in range(B)]
    total, n = c["prefix"] + c["new"], sum(new)
    req = list(range(B + B // 4))
    rng.shuffle(req)
    s = dict(c=c, plen=_i32(pre), new=_i32(new), req=_i32(req[:B]), n=n,
             indptr=torch.empty(B + 1, dtype=torch.int32, device=DEV), seq=torch.empty(B, dtype=torch.int32, device=DEV),
             pos=torch.empty(n, dtype=torch.int32, device=DEV), slots=torch.empty(n, dtype=torch.int32, device=DEV),
             status=torch.zeros(1, dtype=torch.int32, device=DEV), pages=None)
    if c["paged"]:
        s["rtt"] = torch.full((len(req), total), -1, dtype=torch.int32, device=DEV)
        wide = -(-total // PAGE)
        s["pages"] = torch.randperm(len(req) * wide, generator=g, device=DEV).to(torch.int32).view(len(req), wide)
        s["num_slots"] = len(req) * wide * PAGE
    else:
        s["rtt"] = torch.randperm(len(req) * total, generator=g, device=DEV).to(torch.int32).view(len(req), total)
        s["num_slots"] = len(req) * total
    return s


def prepare(case, seed):
    return {"extend": _prepare_extend, "decode": _prepare_decode, "rotate": _prepare_rotate,
            "maps": _prepare_maps}[case["op"]](case, seed)


# --------------------------------------------------------------------------- plain forms, in 32 bits


def _values(pool, scale):
    return pool.float() if pool.dtype == torch.bfloat16 else pool.view(torch.float8_e4m3fn).float() * scale


def _plain_attention(s, q, pos, there, lo, hi, lens):
    """Every request padded to the longest context.  q [B, T, hq, d] in 32 bits; pos, there, lo, hi [B, T]: a query
    token's position, whether there is one, and the positions lo <= j < hi that it may see; lens [B]."""
    c = s["c"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    G, L, (B, T) = hq // hkv, s["rtt"].shape[1], pos.shape
    key = torch.arange(L, device=DEV)
    if c["window"]:
        lo = torch.maximum(lo, pos - c["window"] + 1)
    see = (key >= lo[..., None]) & (key < hi[..., None]) & there[..., None]            # [B, T, L]
    at = s["rtt"].long().clamp(min=0).view(-1)
    k = _values(s["k"][at], s.get("k_scale")).view(B, L, hkv, d)
    v = _values(s["v"][at], s.get("v_scale")).view(B, L, hkv, d)
    v = torch.where((key < lens[:, None])[:, :, None, None], v, 0)
    q = q.view(B, T, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * T, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, hkv, G, T, L)
    if c["cap"]:
        x.div_(c["cap"]).tanh_().mul_(c["cap"])
    if s["slopes"] is not None:
        far = (pos[..., None] - key).abs().float()
        x.sub_(s["slopes"].view(1, hkv, G, 1, 1) * far[:, None, None])
    x.masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, hkv, G * T, L), v.permute(0, 2, 1, 3)).view(B, hkv, G, T, d)
    o = torch.where(total > 0, o / total, 0).permute(0, 3, 1, 2, 4).reshape(B, T, hq, d)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, T, hq)
    return o.to(torch.bfloat16), lse


def _plain_extend(s):
    T = s["c"]["new"]
    plen, elen, start = s["plen"].long(), s["elen"].long(), s["indptr"].long()
    i = torch.arange(T, device=DEV)
    there = i < elen[:, None]
    row = torch.where(there, start[:-1, None] + i, 0)
    pos = plen[:, None] + i
    lo, hi = torch.zeros_like(pos), pos + 1
    if s["see_from"] is not None:
        lo = s["see_from"].long()[row]
    if s["see_to"] is not None:
        hi = torch.maximum(hi, torch.minimum(s["see_to"].long()[row], (plen + elen)[:, None]))
    o, lse = _plain_attention(s, s["q"][row].float(), pos, there, lo, hi, plen + elen)
    return o[there], lse[there]


def _plain_decode(s):
    seq = s["seq"].long()[:, None]
    lo = torch.zeros_like(seq) if s["see_from"] is None else s["see_from"].long()[:, None]
    o, lse = _plain_attention(s, s["q"][:, None].float(), seq - 1, seq > 0, lo, seq, seq[:, 0])
    return o[:, 0], lse[:, 0]


def _plain_rotate(s):
    d = s["c"]["d"]
    turn = s["base"] ** (-2 * torch.arange(d // 2, device=DEV, dtype=torch.float64) / d)
    a = s["pos"].double()[s["axis_dev"]].t() * turn                                     # [n, d / 2]
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]

    def rotate(x, w):
        x = x.float()
        if s["eps"] is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        lo, hi = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)

    q, k, v = rotate(s["q"], s["qw"]).to(torch.bfloat16), rotate(s["k_new"], s["kw"]), s["v_new"].float()
    at = s["slots"].long()
    if s["c"]["fp8"]:
        s["k"][at] = (k / s["k_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["v"][at] = (v / s["v_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return q, s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
    s["k"][at] = k.to(torch.bfloat16)
    s["v"][at] = s["v_new"]
    return q, s["k"], s["v"]


def _plain_maps(s):
    new, plen, req = s["new"].long(), s["plen"].long(), s["req"].long()
    end = torch.cumsum(new, 0)
    indptr = torch.cat([torch.zeros_like(end[:1]), end])
    who = torch.repeat_interleave(torch.arange(len(new), device=DEV), new, output_size=s["n"])
    pos = torch.arange(s["n"], device=DEV) - indptr[who] + plen[who]
    if s["pages"] is None:
        slots = s["rtt"][req[who], pos].long()
    else:
        slots = s["pages"][req[who], pos // PAGE].long() * PAGE + pos % PAGE
        s["rtt"][req[who], pos] = slots.to(torch.int32)
    i32 = torch.int32
    return indptr.to(i32), (plen + new).to(i32), pos.to(i32), slots.to(i32), s["rtt"]


# --------------------------------------------------------------------------- the library's calls


def _own(s):
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = s["c"]
    if c["op"] == "maps":
        rx.rx_step_maps(s["req"], s["plen"], s["new"], s["rtt"], s["num_slots"], s["indptr"], s["seq"], s["pos"], s["slots"],
                        pages=s["pages"], page_size=PAGE if c["paged"] else 0, dev_status=s["status"])
        return s["indptr"], s["seq"], s["pos"], s["slots"], s["rtt"]
    if c["op"] == "rotate":
        if c["fp8"]:
            rx.rx_qk_rope_axes_store_fp8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["q"], s["q_out"], s["k_new"],
                                         s["v_new"], s["qw"], s["kw"], s["slots"], s["pos"], s["axis"], s["base"], s["eps"],
                                         s["status"])
            return s["q_out"], s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
        rx.rx_qk_rope_axes_store(s["k"], s["v"], s["q"], s["q_out"], s["k_new"], s["v_new"], s["qw"], s["kw"], s["slots"],
                                 s["pos"], s["axis"], s["base"], s["eps"], s["status"])
        return s["q_out"], s["k"], s["v"]
    keep = s["kept"]
    if not keep:  # the rules and the workspace, kept for the batch as a serving program does
        keep["rules"] = rx.AttnRules(cap=c["cap"], window=c["window"], slopes=s["slopes"], see_from=s["see_from"],
                                     see_to=s["see_to"])
        new, context = (c["new"], s["context"]) if c["op"] == "extend" else (1, 0)
        keep["ws"] = torch.empty(rx.rx_attn_rules_workspace(context, c["batch"], c["hq"], c["hkv"], c["d"], new),
                                 dtype=torch.uint8, device=DEV)
    if c["op"] == "extend":
        args = (s["q"], s["o"], s["lse"], s["indptr"], s["req"], s["plen"], s["elen"], s["rtt"], c["new"], s["scale"],
                keep["rules"], keep["ws"], s["status"])
        if c["fp8"]:
            rx.rx_attn_extend_rules_fp8(s["k"], s["v"], s["k_scale"], s["v_scale"], *args)
        else:
            rx.rx_attn_extend_rules(s["k"], s["v"], *args)
    else:
        args = (s["q"], s["o"], s["lse"], s["req"], s["seq"], s["rtt"], s["scale"], keep["rules"], keep["ws"], s["status"])
        if c["fp8"]:
            rx.rx_attn_decode_rules_fp8(s["k"], s["v"], s["k_scale"], s["v_scale"], *args)
        else:
            rx.rx_attn_decode_rules(s["k"], s["v"], *args)
    return s["o"], s["lse"]


def run(state):
    if own:
        return _own(state)
    return {"extend": _plain_extend, "decode": _plain_decode, "rotate": _plain_rotate,
            "maps": _plain_maps}[state["c"]["op"]](state)


# --------------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "maps":
        B, n = c["batch"], sum(_sizes(c))
        by = B * 20 + n * 8 + (n / PAGE * 4 + n * 4 if c["paged"] else n * 4)
        return dict(bytes=by, flops=n)
    if c["op"] == "rotate":
        n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
        by = n * d * (2 * (hq + 2 * hkv) + 2 * hq + 2 * hkv * (1 if c["fp8"] else 2)) + 4 * n * (1 + c["axes"])
        return dict(bytes=by, flops=n * d * (7 if c["norm"] else 3) * (hq + hkv))
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    row = hkv * d * 2 * (1 if c["fp8"] else 2) + 4
    window = c["window"] or 1 << 30
    if c["op"] == "decode":
        most = 0.75 * c["ctx"] * (0.75 if c["mask"] == "docs" else 1)
        keys = c["batch"] * min(window, most)
        return dict(bytes=keys * row + c["batch"] * hq * (4 * d + 4), flops=4 * d * hq * keys)
    pairs, keys, P = 0.0, 0.0, int(0.75 * c["prefix"])
    for b, T in enumerate(_sizes(c)):
        i = np.arange(T)
        lo, hi = _seen(c, i, P, T)
        lo = np.maximum(lo, P + i - window + 1).clip(0)
        pairs += float((np.maximum(hi, P + i + 1) - lo).sum())
        first = int(lo.min())
        keys += max(0, P - first) / c["group"] + P + T - max(P, first)
    n = sum(_sizes(c))
    return dict(bytes=keys * row + n * hq * (4 * d + 4), flops=4 * d * hq * pairs)


# --------------------------------------------------------------------------- the definition, in 64 bits


def _exact_rows(s, b, q, pos, lo, hi, length):
    """One request: its query tokens q [n, hq, d] at pos [n], each over positions lo <= j < hi."""
    c = s["c"]
    hq, hkv = c["hq"], c["hkv"]
    G = hq // hkv
    code = torch.float8_e4m3fn if c["fp8"] else torch.bfloat16
    at = s["rtt"][b, :length].long()
    k = s["k"][at].view(code).double() * (s["k_scale"] if c["fp8"] else 1.0)
    v = s["v"][at].view(code).double() * (s["v_scale"] if c["fp8"] else 1.0)
    j = torch.arange(length, device=DEV)
    if c["window"]:
        lo = torch.maximum(lo, pos - (c["window"] - 1))
    hidden = (j[None] < lo[:, None]) | (j[None] >= hi[:, None])
    far = (j[None] - pos[:, None]).abs().double()
    o, l = [], []
    for g in range(hkv):
        x = torch.einsum("tgc,lc->gtl", q[:, g * G:(g + 1) * G].double(), k[:, g]) * s["scale"]
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        if s["slopes"] is not None:
            x = x - s["slopes"][g * G:(g + 1) * G].double()[:, None, None] * far
        x = x.masked_fill(hidden[None], -math.inf)
        l.append(torch.logsumexp(x, -1).t())
        o.append(torch.einsum("gtl,lc->tgc", torch.softmax(x, -1).nan_to_num(0.0), v[:, g]))
    return torch.cat(o, 1), torch.cat(l, 1)


def _exact_extend(s):
    out = []
    for b in range(s["c"]["batch"]):
        i, e, P = int(s["indptr"][b]), int(s["indptr"][b + 1]), int(s["plen"][b])
        pos = P + torch.arange(e - i, device=DEV)
        lo = torch.zeros_like(pos) if s["see_from"] is None else s["see_from"][i:e].long()
        hi = pos + 1
        if s["see_to"] is not None:
            hi = torch.maximum(hi, s["see_to"][i:e].long().clamp(max=P + e - i))
        out.append(_exact_rows(s, b, s["q"][i:e], pos, lo, hi, P + e - i))
    return torch.cat([x[0] for x in out]), torch.cat([x[1] for x in out])


def _exact_decode(s):
    out = []
    for b in range(s["c"]["batch"]):
        n = int(s["seq"][b])
        pos = torch.tensor([n - 1], device=DEV)
        lo = torch.zeros_like(pos) if s["see_from"] is None else s["see_from"][b:b + 1].long()
        out.append(_exact_rows(s, b, s["q"][b:b + 1], pos, lo, pos + 1, n))
    return torch.cat([x[0] for x in out]), torch.cat([x[1] for x in out])


def _exact_rotate(s):
    c = s["c"]
    d, n = c["d"], c["n"]
    h = d // 2
    freq = torch.pow(torch.tensor(s["base"], dtype=torch.float64, device=DEV),
                     torch.arange(h, dtype=torch.float64, device=DEV) * (-2.0 / d))
    angle = torch.stack([s["pos"][int(a)].double() * freq[i] for i, a in enumerate(s["axis"])], 1)
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)

    def f(x, w):
        x = x.double()
        if s["eps"] is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + s["eps"]) * w.double()
        z = torch.complex(x[..., :h].contiguous(), x[..., h:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)

    def codes(x, scale):  # the nearest of E4M3's values: three fraction bits, exponents from -6
        x = x / scale
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(x / step) * step).clamp(-448, 448)

    k, v = f(s["k_new"], s["kw"]), s["v_new"].double()
    if c["fp8"]:
        k, v = codes(k, s["k_scale"]), codes(v, s["v_scale"])
    kp = torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV)
    vp = torch.zeros_like(kp)
    kp.index_copy_(0, s["slots"].long(), k.reshape(n, *kp.shape[1:]))
    vp.index_copy_(0, s["slots"].long(), v.reshape(n, *vp.shape[1:]))
    return f(s["q"], s["qw"]), kp, vp


def exact(case, seed):
    if case["op"] == "maps":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"extend": _exact_extend, "decode": _exact_decode, "rotate": _exact_rotate}[case["op"]](s)
