"""The operators of one speculative decoding step, as cases to measure.

A step that verifies drafted tokens runs, next to the model's own matrix
products, three operators of this library:

  norm    rx_qk_norm_rope_store(_fp8): RMS norm of every q and k head, the
          rotary embedding, and the scatter of K and V into the slot pool;
  tree    rx_attn_tree(_fp8): attention of each request's tree of drafted
          tokens over its slot list -- the cached prefix, which every node
          sees, and the tree's own tokens, which a node sees where its mask
          row says so;
  logits  rx_logits_process: penalties for repeated tokens, logit biases and
          grammar masks on the logits of every request or drafted node.

``run`` computes them in elementary torch operations, or through the
library's binding where ``own`` is set.  Head counts, head sizes and lengths
are those of the library's workloads (32/32, 32/8 and 64/8 heads of 128, 4/4
of 64; 1,280, 8,192 and 32,768 tokens of context; 128,256 ids).
"""
import math

import torch

own = False

DEV = "cuda"
WORKSPACE = 64 << 20  # the scratch memory a serving program lends to every attention call

HEADS = [(32, 32, 128), (32, 8, 128), (64, 8, 128), (4, 4, 64)]


def listed():
    return [
        # one user's request, a short prompt and a handful of drafted tokens: latency counts
        dict(name="tree_one_request", op="tree", batch=1, hq=32, hkv=8, d=128, ctx=333, shared=0, tree=5, fp8=False),
        # few-shot batch, one q head per kv head, a few drafted tokens each
        dict(name="tree_few_shot", op="tree", batch=64, hq=32, hkv=32, d=128, ctx=1281, shared=0, tree=4, fp8=False),
        # long multi-turn chat: 16 requests of up to 32k tokens, a quarter of them a shared system prompt
        dict(name="tree_long_chat", op="tree", batch=16, hq=64, hkv=8, d=128, ctx=32768, shared=8192, tree=16, fp8=False),
        # the same lengths over E4M3 pools, smaller trees
        dict(name="tree_long_chat_fp8", op="tree", batch=16, hq=32, hkv=8, d=128, ctx=32768, shared=0, tree=13, fp8=True),
        # wide trees: 64 nodes times 8 q heads are 512 query rows a kv head
        dict(name="tree_wide", op="tree", batch=8, hq=64, hkv=8, d=128, ctx=8192, shared=0, tree=64, fp8=False),
        # the verification step's projections of one small batch: latency counts
        dict(name="norm_small_batch", op="norm", n=16, hq=32, hkv=8, d=128, fp8=False, packed=True),
        # an odd number of tokens into E4M3 pools
        dict(name="norm_fp8", op="norm", n=4099, hq=32, hkv=8, d=128, fp8=True, packed=True),
        # the extend part of the long chat step: 16 requests of 1,024 new tokens
        dict(name="norm_extend", op="norm", n=16384, hq=64, hkv=8, d=128, fp8=False, packed=True),
        # one request's next token
        dict(name="logits_one_row", op="logits", batch=1, tree=0, vocab=32000, bf16=False, hist=700, bias=8, grammar=False),
        # constrained decoding of a batch, one row a request
        dict(name="logits_constrained", op="logits", batch=64, tree=0, vocab=128256, bf16=False, hist=8192, bias=32,
             grammar=True),
        # every node of 16 drafted trees, long histories, the model's bf16 logits
        dict(name="logits_tree", op="logits", batch=16, tree=16, vocab=128256, bf16=True, hist=32768, bias=32,
             grammar=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "norm", "logits"])
    if op == "tree":
        hq, hkv, d = rng.choice(HEADS)
        batch, tree, ctx = _log(rng, 1, 64), _log(rng, 1, 64), _log(rng, 16, 32768)
        # no more cached values than the long chat holds, no more scores than it has
        ctx = max(16, min(ctx, 16 * 32768 * 8 * 128 // (batch * hkv * d), 16 * 32768 * 64 * 16 // (batch * hq * tree)))
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, ctx=ctx, shared=rng.choice([0, 0, ctx // 4]), tree=tree,
                    fp8=rng.random() < 0.4)
    if op == "norm":
        hq, hkv, d = rng.choice(HEADS)
        n = min(_log(rng, 1, 16384), 16384 * 80 * 128 // ((hq + 2 * hkv) * d))
        return dict(op=op, n=n, hq=hq, hkv=hkv, d=d, fp8=rng.random() < 0.4, packed=rng.random() < 0.7)
    vocab = rng.choice([4000, 32000, 50257, 128256])
    batch, tree = _log(rng, 1, 64), rng.choice([0, 0, rng.randint(1, 16)])
    batch = max(1, min(batch, 256 * 128256 // (vocab * max(1, tree))))
    return dict(op=op, batch=batch, tree=tree, vocab=vocab, bf16=rng.random() < 0.5, hist=_log(rng, 1, 32768),
                bias=rng.choice([0, rng.randint(1, 300)]), grammar=rng.random() < 0.6)


# --------------------------------------------------------------------------- inputs


def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1000003 + salt) % (1 << 62))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _lengths(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV)


def _sizes(c):
    """Nodes of each request's tree: from half of the widest up to it."""
    return [c["tree"] - 5 * i % (c["tree"] // 2 + 1) for i in range(c["batch"])]


def _tree_masks(g, sizes):
    """Mask rows of random trees: node 0 is the root; every node sees itself
    and its ancestors.  Returns bool [nodes, widest tree]."""
    top = max(sizes)
    parent = (torch.rand((len(sizes), top), generator=g, device=DEV) * torch.arange(top, device=DEV)).long()
    see = torch.eye(top, dtype=torch.bool, device=DEV).repeat(len(sizes), 1, 1)
    at = torch.arange(len(sizes), device=DEV)
    for i in range(1, top):
        see[:, i] |= see[at, parent[:, i]]
    keep = torch.arange(top, device=DEV)[None, :] < torch.tensor(sizes, device=DEV)[:, None]
    return (see & keep[:, None, :])[keep]


def _pack_bits(see):
    """bool [rows, n] -> int32 words [rows, ceil(n / 32)], bit j % 32 of word j / 32."""
    rows, n = see.shape
    words = -(-n // 32)
    wide = torch.zeros((rows, words * 32), dtype=torch.int64, device=see.device)
    wide[:, :n] = see
    w = (wide.view(rows, words, 32) << torch.arange(32, device=see.device)).sum(2)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _indptr(sizes):
    t = torch.zeros(len(sizes) + 1, dtype=torch.int64)
    t[1:] = torch.cumsum(torch.tensor(sizes), 0)
    return t


def _prepare_tree(c, seed):
    g = _gen(seed, 1)
    B, hq, hkv, d, ctx = c["batch"], c["hq"], c["hkv"], c["d"], c["ctx"]
    shared = c["shared"]
    plen = _lengths(g, B, max(shared, (ctx + 1) // 2), ctx)
    plen[0] = ctx
    sizes = _sizes(c)
    indptr = _indptr(sizes)
    see = _tree_masks(g, sizes)
    stride = ctx + c["tree"]
    private = stride - shared
    slots = shared + B * private
    perm = torch.randperm(slots, generator=g, device=DEV).to(torch.int32)
    rtt = torch.cat([perm[:shared].expand(B, shared), perm[shared:].view(B, private)], 1).contiguous()
    q = _randn(g, sum(sizes), hq, d).to(torch.bfloat16)
    k, v = _randn(g, slots, hkv, d), _randn(g, slots, hkv, d)
    s = dict(c=c, q=q, rtt=rtt, plen=plen.to(torch.int32), indptr=indptr.to(torch.int32).to(DEV),
             mask=_pack_bits(see), req=torch.arange(B, dtype=torch.int32, device=DEV), scale=1 / math.sqrt(d),
             o=torch.empty_like(q), lse=torch.empty(sum(sizes), hq, device=DEV),
             status=torch.zeros(1, dtype=torch.int32, device=DEV),
             ws=torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV))
    if c["fp8"]:
        s["k_scale"], s["v_scale"] = 0.0517, 0.0423
        s["k"] = (k / s["k_scale"]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["v"] = (v / s["v_scale"]).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["k"], s["v"] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    return s


def _prepare_norm(c, seed):
    g = _gen(seed, 2)
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    # the model's projection: one row a token, q heads, k heads, v heads
    qkv = (2 * _randn(g, n, hq + 2 * hkv, d)).to(torch.bfloat16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if not c["packed"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    slots = n + n // 2 + 64
    pool = torch.uint8 if c["fp8"] else torch.bfloat16
    return dict(c=c, q=q, k_new=k, v_new=v, q_out=torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV),
                qw=(1 + 0.2 * _randn(g, d)).to(torch.bfloat16), kw=(1 + 0.2 * _randn(g, d)).to(torch.bfloat16),
                k=torch.zeros(slots, hkv, d, dtype=pool, device=DEV),
                v=torch.zeros(slots, hkv, d, dtype=pool, device=DEV),
                slots=torch.randperm(slots, generator=g, device=DEV)[:n].to(torch.int32),
                pos=torch.randint(0, 131072, (n,), generator=g, device=DEV, dtype=torch.int32),
                base=500000.0, eps=1e-6, k_scale=0.0523, v_scale=0.0517,
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_logits(c, seed):
    g = _gen(seed, 3)
    B, V = c["batch"], c["vocab"]
    hl = _lengths(g, B, (c["hist"] + 1) // 2, c["hist"])
    hl[0] = c["hist"]
    hist_ptr = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    hist_ptr[1:] = torch.cumsum(hl, 0)
    total = int(hist_ptr[-1])
    # repeated tokens: low ids are common, as in text
    hist = (V * torch.rand(total, generator=g, device=DEV).pow(3)).long().clamp_(0, V - 1).to(torch.int32)
    s = dict(c=c, hist=hist, hist_ptr=hist_ptr, prompt=(hl * 3 // 4).to(torch.int32),
             rep=1 + 0.3 * torch.rand(B, generator=g, device=DEV), freq=0.4 * torch.rand(B, generator=g, device=DEV),
             pres=0.6 * torch.rand(B, generator=g, device=DEV), status=torch.zeros(1, dtype=torch.int32, device=DEV))
    rows = B
    for name in ("bias_ptr", "bias_tok", "bias_val", "indptr", "draft", "tree_mask", "allow", "allow_row"):
        s[name] = None
    if c["tree"]:
        sizes = _sizes(c)
        rows = sum(sizes)
        s["indptr"] = _indptr(sizes).to(torch.int32).to(DEV)
        s["draft"] = (V * torch.rand(rows, generator=g, device=DEV).pow(3)).long().clamp_(0, V - 1).to(torch.int32)
        s["tree_mask"] = _pack_bits(_tree_masks(g, sizes))
    if c["bias"]:
        n = c["bias"]
        s["bias_ptr"] = torch.arange(B + 1, device=DEV) * n
        s["bias_tok"] = torch.sort(torch.randint(0, V, (B, n), generator=g, device=DEV), 1)[0].to(torch.int32).view(-1)
        s["bias_val"] = 4 * _randn(g, B * n)
    if c["grammar"]:
        # states of a grammar: every other one has a few allowed ids (its fixed text), the others most of the vocabulary
        states = 32
        share = torch.where(torch.arange(states, device=DEV) % 2 == 0, 0.0005, 0.97)
        words = -(-V // 128) * 4
        ok = torch.zeros((states, words * 32), dtype=torch.bool, device=DEV)
        ok[:, :V] = torch.rand((states, V), generator=g, device=DEV) < share[:, None]
        s["allow"] = _pack_bits(ok)
        s["allow_row"] = torch.randint(0, states, (rows,), generator=g, device=DEV, dtype=torch.int32)
        s["allow_row"][1::8] = -1  # requests without a grammar
    x = 3 * _randn(g, rows, V)
    s["logits"] = x.to(torch.bfloat16) if c["bf16"] else x
    s["out"] = torch.empty(rows, V, device=DEV)
    s["rules"] = None
    return s


def prepare(case, seed):
    return {"tree": _prepare_tree, "norm": _prepare_norm, "logits": _prepare_logits}[case["op"]](case, seed)


# --------------------------------------------------------------------------- plain forms, in 32 bits


def _values(pool, scale):
    return pool.float() if pool.dtype == torch.bfloat16 else pool.view(torch.float8_e4m3fn).float() * scale


def _plain_tree(s):
    """Every request padded to the longest context and the widest tree."""
    c = s["c"]
    B, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
    G, T, L = hq // hkv, c["tree"], s["rtt"].shape[1]
    plen, start = s["plen"].long(), s["indptr"].long()
    tlen = start[1:] - start[:-1]
    node = torch.arange(T, device=DEV)
    row = start[:-1, None] + node                       # [B, T]
    there = node < tlen[:, None]
    row = torch.where(there, row, 0)
    pos = torch.arange(L, device=DEV)
    rel = pos[None, :] - plen[:, None]                  # key position within the tree
    bit = rel.clamp(0, T - 1)                           # [B, L]
    words = s["mask"][row]                              # [B, T, W]
    word = torch.gather(words, 2, (bit // 32)[:, None, :].expand(B, T, L))
    seen = ((word >> (bit % 32)[:, None, :].to(torch.int32)) & 1).bool()
    see = (rel < 0)[:, None, :] | (seen & ((rel >= 0) & (rel < tlen[:, None]))[:, None, :])   # [B, T, L]
    at = s["rtt"].long()
    k = _values(s["k"][at.view(-1)], s.get("k_scale")).view(B, L, hkv, d)
    v = _values(s["v"][at.view(-1)], s.get("v_scale")).view(B, L, hkv, d)
    v = torch.where((rel < tlen[:, None])[:, :, None, None], v, 0)
    q = s["q"][row.view(-1)].float().view(B, T, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * T, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, hkv, G, T, L)
    x.masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, hkv, G * T, L), v.permute(0, 2, 1, 3)).view(B, hkv, G, T, d) / total
    lse = (top + total.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, hq, d)[there].to(torch.bfloat16)
    return o, lse.permute(0, 3, 1, 2).reshape(B, T, hq)[there]


def _plain_norm(s):
    d = s["c"]["d"]
    turn = s["base"] ** (-2 * torch.arange(d // 2, device=DEV, dtype=torch.float64) / d)
    a = s["pos"].double()[:, None] * turn
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]

    def norm_rope(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        lo, hi = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)

    q, k, v = norm_rope(s["q"], s["qw"]).to(torch.bfloat16), norm_rope(s["k_new"], s["kw"]), s["v_new"].float()
    at = s["slots"].long()
    if s["c"]["fp8"]:
        s["k"][at] = (k / s["k_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["v"][at] = (v / s["v_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return q, s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
    s["k"][at] = k.to(torch.bfloat16)
    s["v"][at] = s["v_new"]
    return q, s["k"], s["v"]


def _rows_of(s):
    """The request of every logits row."""
    if s["indptr"] is None:
        return torch.arange(s["c"]["batch"], device=DEV)
    start = s["indptr"].long()
    return torch.repeat_interleave(torch.arange(len(start) - 1, device=DEV), start[1:] - start[:-1])


def _unpack_bits(words, n):
    return ((words[..., None] >> torch.arange(32, dtype=torch.int32, device=words.device)) & 1).view(
        words.shape[0], -1)[:, :n].bool()


def _plain_logits(s):
    V, B = s["c"]["vocab"], s["c"]["batch"]
    req = _rows_of(s)
    ptr = s["hist_ptr"]
    who = torch.repeat_interleave(torch.arange(B, device=DEV), ptr[1:] - ptr[:-1])
    made = torch.arange(len(who), device=DEV) - ptr[who] >= s["prompt"][who]     # behind the prompt
    seen = torch.zeros(B * V, dtype=torch.int32, device=DEV)
    seen.index_add_(0, who * V + s["hist"], torch.ones_like(who, dtype=torch.int32))
    count = torch.zeros(B * V, dtype=torch.int32, device=DEV)
    count.index_add_(0, who * V + s["hist"], made.to(torch.int32))
    seen, count = seen.view(B, V)[req], count.view(B, V)[req]
    if s["draft"] is not None:  # the drafted tokens on each node's path
        path = _unpack_bits(s["tree_mask"], s["c"]["tree"])
        r, j = path.nonzero(as_tuple=True)
        tok = s["draft"][s["indptr"].long()[req[r]] + j].long()
        one = torch.ones_like(r, dtype=torch.int32)
        seen.view(-1).index_add_(0, r * V + tok, one)
        count.view(-1).index_add_(0, r * V + tok, one)
    x = s["logits"].float()
    rep = s["rep"][req][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["freq"][req][:, None] * count - s["pres"][req][:, None] * (count > 0)
    if s["bias_tok"] is not None:
        n = s["c"]["bias"]
        add = torch.zeros(B * V, device=DEV)
        add.index_add_(0, torch.arange(B * n, device=DEV) // n * V + s["bias_tok"], s["bias_val"])
        x = x + add.view(B, V)[req]
    if s["allow"] is not None:
        ok = _unpack_bits(s["allow"], V)[s["allow_row"].long()] | (s["allow_row"] < 0)[:, None]
        x = torch.where(ok, x, -math.inf)
    return x


# --------------------------------------------------------------------------- the library's calls


def _own(s):
    from prefix_shared_kv_radixattention_gb300 import binding as rx
    c = s["c"]
    if c["op"] == "tree":
        if c["fp8"]:
            rx.rx_attn_tree_fp8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["q"], s["o"], s["lse"], s["indptr"],
                                s["req"], s["plen"], s["mask"], s["rtt"], c["tree"], s["scale"], s["ws"], s["status"])
        else:
            rx.rx_attn_tree(s["k"], s["v"], s["q"], s["o"], s["lse"], s["indptr"], s["req"], s["plen"], s["mask"],
                            s["rtt"], c["tree"], s["scale"], s["ws"], s["status"])
        return s["o"], s["lse"]
    if c["op"] == "norm":
        if c["fp8"]:
            rx.rx_qk_norm_rope_store_fp8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["q"], s["q_out"], s["k_new"],
                                         s["v_new"], s["qw"], s["kw"], s["slots"], s["pos"], s["base"], s["eps"],
                                         s["status"])
            return s["q_out"], s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
        rx.rx_qk_norm_rope_store(s["k"], s["v"], s["q"], s["q_out"], s["k_new"], s["v_new"], s["qw"], s["kw"],
                                 s["slots"], s["pos"], s["base"], s["eps"], s["status"])
        return s["q_out"], s["k"], s["v"]
    if s["rules"] is None:  # kept for the batch, as a serving program does
        s["rules"] = rx.LogitsRules(c["batch"], c["vocab"], hist=s["hist"], hist_ptr=s["hist_ptr"],
                                    prompt_len=s["prompt"], repetition=s["rep"], frequency=s["freq"],
                                    presence=s["pres"], bias_tok=s["bias_tok"], bias_val=s["bias_val"],
                                    bias_ptr=s["bias_ptr"], qo_indptr=s["indptr"], draft_tok=s["draft"],
                                    tree_mask=s["tree_mask"], allow=s["allow"], allow_row=s["allow_row"])
    rx.rx_logits_process(s["rules"], s["logits"], s["out"], s["status"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"tree": _plain_tree, "norm": _plain_norm, "logits": _plain_logits}[state["c"]["op"]](state)


# --------------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "tree":
        B, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
        mean_t = sum(_sizes(c)) / B
        mean_p = (max(c["shared"], c["ctx"] / 2) + c["ctx"]) / 2
        rows = B * mean_t
        keys = c["shared"] + B * (mean_p - c["shared"] + mean_t)  # a shared slot is read once
        by = keys * hkv * d * 2 * (1 if c["fp8"] else 2) + rows * hq * (d * 4 + 4) + B * (mean_p + mean_t) * 4
        return dict(bytes=by, flops=4 * d * hq * rows * (mean_p + mean_t / 2))
    if c["op"] == "norm":
        n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
        by = n * d * (2 * (hq + 2 * hkv) + 2 * hq + 2 * hkv * (1 if c["fp8"] else 2)) + 8 * n
        return dict(bytes=by, flops=n * d * 7 * (hq + hkv))
    rows = sum(_sizes(c)) if c["tree"] else c["batch"]
    read = 0.5625 if c["grammar"] else 1.0  # 7 rows of 16 allow hardly any id: their logits need no read
    by = rows * c["vocab"] * (4 + read * (2 if c["bf16"] else 4) + (0.125 if c["grammar"] else 0))
    by += c["batch"] * (c["hist"] * 0.75 * 4 + c["bias"] * 8)
    return dict(bytes=by, flops=rows * c["vocab"] * 4)


# --------------------------------------------------------------------------- the definition, in 64 bits


def _exact_tree(s):
    """Request by request, head by head group, over the listed slots."""
    c = s["c"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    G = hq // hkv
    start, plen = s["indptr"].tolist(), s["plen"].tolist()
    code = torch.float8_e4m3fn if c["fp8"] else torch.bfloat16
    outs, lses = [], []
    for b in range(c["batch"]):
        n, p = start[b + 1] - start[b], plen[b]
        at = s["rtt"][b, :p + n].long()
        k = s["k"][at].view(code).double() * (s["k_scale"] if c["fp8"] else 1.0)
        v = s["v"][at].view(code).double() * (s["v_scale"] if c["fp8"] else 1.0)
        q = s["q"][start[b]:start[b + 1]].double()
        m = s["mask"][start[b]:start[b + 1]].cpu().tolist()
        see = torch.ones((n, p + n), dtype=torch.bool)
        for i in range(n):
            for j in range(n):
                see[i, p + j] = bool((m[i][j // 32] >> (j % 32)) & 1)
        see = see.to(DEV)
        o, l = [], []
        for g in range(hkv):
            x = torch.einsum("tgc,lc->gtl", q[:, g * G:(g + 1) * G], k[:, g]) * s["scale"]
            x = torch.where(see[None], x, torch.full_like(x, -math.inf))
            l.append(torch.logsumexp(x, -1).t())
            o.append(torch.einsum("gtl,lc->tgc", torch.softmax(x, -1), v[:, g]))
        outs.append(torch.cat(o, 1))
        lses.append(torch.cat(l, 1))
    return torch.cat(outs), torch.cat(lses)


def _exact_norm(s):
    d = s["c"]["d"]
    n = s["c"]["n"]
    h = d // 2
    angle = torch.outer(s["pos"].double(), torch.pow(torch.tensor(s["base"], dtype=torch.float64, device=DEV),
                                                     torch.arange(h, dtype=torch.float64, device=DEV) * (-2.0 / d)))
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)

    def f(x, w):
        x = x.double()
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + s["eps"]) * w.double()
        z = torch.complex(x[..., :h].contiguous(), x[..., h:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)

    def codes(x, scale):  # the nearest of E4M3's values: three fraction bits, exponents from -6
        x = x / scale
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(x / step) * step).clamp(-448, 448)

    k, v = f(s["k_new"], s["kw"]), s["v_new"].double()
    if s["c"]["fp8"]:
        k, v = codes(k, s["k_scale"]), codes(v, s["v_scale"])
    kp = torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV)
    vp = torch.zeros_like(kp)
    kp.index_copy_(0, s["slots"].long(), k.reshape(n, *kp.shape[1:]))
    vp.index_copy_(0, s["slots"].long(), v.reshape(n, *vp.shape[1:]))
    return f(s["q"], s["qw"]), kp, vp


def _exact_logits(s):
    """Row by row."""
    c = s["c"]
    V = c["vocab"]
    ptr, prompt = s["hist_ptr"].tolist(), s["prompt"].tolist()
    start = list(range(c["batch"] + 1)) if s["indptr"] is None else s["indptr"].tolist()
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["batch"]):
        h = s["hist"][ptr[b]:ptr[b + 1]].long()
        said = torch.bincount(h[prompt[b]:], minlength=V)
        asked = torch.bincount(h[:prompt[b]], minlength=V)
        rep, freq, pres = (float(s[k][b]) for k in ("rep", "freq", "pres"))
        for r in range(start[b], start[b + 1]):
            n = said
            if s["draft"] is not None:
                words = s["tree_mask"][r].tolist()
                on = [j for j in range(start[b + 1] - start[b]) if (words[j // 32] >> (j % 32)) & 1]
                n = n + torch.bincount(s["draft"][start[b]:start[b + 1]].long()[on], minlength=V)
            x = s["logits"][r].double()
            x = torch.where((n + asked) > 0, torch.where(x > 0, x / rep, x * rep), x)
            x = x - freq * n - pres * (n > 0).double()
            if s["bias_tok"] is not None:
                i, j = int(s["bias_ptr"][b]), int(s["bias_ptr"][b + 1])
                x = x.index_add(0, s["bias_tok"][i:j].long(), s["bias_val"][i:j].double())
            if s["allow"] is not None and int(s["allow_row"][r]) >= 0:
                words = s["allow"][int(s["allow_row"][r])].long()
                ids = torch.arange(V, device=DEV)
                x[((words[ids // 32] >> (ids % 32)) & 1) == 0] = -math.inf
            out[r] = x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "norm": _exact_norm, "logits": _exact_logits}[case["op"]](s)
