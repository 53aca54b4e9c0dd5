"""Verification of drafted tokens -- oracle.

TEST INFRASTRUCTURE ONLY.  Plain numpy in fp64; it imports nothing from the
CUDA path.  The pages do not speak of speculative decoding; the definitions
are those written in ``include/rx.h``:

* ``tree_mask``: a drafted token sees itself and its ancestors;
* ``tree_attention``: softmax(scale q K^T) V over the prefix and the drafted
  tokens a mask row names; a row that sees nothing gives 0 and -inf;
* ``qk_norm_rope``: x / sqrt(mean x^2 + eps) * w, rotated;
* ``logits_process``: penalties, biases and grammar masks, every step
  rounded to fp32 (the result is exact, so tests compare bits).

Pinned in ``tests/test_draft_oracle.py``.
"""
from __future__ import annotations

import numpy as np

from oracle import rope_f64


def tree_mask(parent):
    """bool [n, n]: row i holds i and its ancestors."""
    n = len(parent)
    out = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            out[i, j] = True
            j = parent[j]
    return out


def tree_attention(q, k_pool, v_pool, rtt, req_idx, prefix_len, qo_indptr, see, sm_scale):
    """q fp64 [n, Hq, d]; pools fp64 [S, Hkv, d]; see: a bool [T_b, T_b] per
    request.  Slots outside the pool read as zero rows.  Returns (o [n, Hq,
    d], lse [n, Hq], a [n, Hq, d]), a = sum_j p_j |v_j| (for error bounds)."""
    q = np.asarray(q, np.float64)
    n, hq, d = q.shape
    S, hkv, _ = k_pool.shape
    G = hq // hkv
    o = np.zeros((n, hq, d))
    a = np.zeros((n, hq, d))
    lse = np.full((n, hq), -np.inf)
    for b in range(len(req_idx)):
        s, e = int(qo_indptr[b]), int(qo_indptr[b + 1])
        P, T = int(prefix_len[b]), e - s
        if T == 0:
            continue
        slots = np.asarray(rtt[req_idx[b], :P + T], np.int64)
        ok = (slots >= 0) & (slots < S)
        k = np.where(ok[:, None, None], k_pool[np.where(ok, slots, 0)], 0.0)
        v = np.where(ok[:, None, None], v_pool[np.where(ok, slots, 0)], 0.0)
        for i in range(T):
            seen = np.concatenate([np.ones(P, bool), np.asarray(see[b][i], bool)])
            if not seen.any():
                continue
            for g in range(hkv):
                x = sm_scale * (q[s + i, g * G:(g + 1) * G] @ k[seen, g].T)       # [G, seen]
                m = x.max(1, keepdims=True)
                w = np.exp(x - m)
                tot = w.sum(1, keepdims=True)
                o[s + i, g * G:(g + 1) * G] = (w / tot) @ v[seen, g]
                a[s + i, g * G:(g + 1) * G] = (w / tot) @ np.abs(v[seen, g])
                lse[s + i, g * G:(g + 1) * G] = (m + np.log(tot))[:, 0]
    return o, lse, a


def qk_norm(x, w, eps):
    """x / sqrt(mean x^2 + eps) * w over the last axis, fp64 (w: [d] or None)."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if w is None else y * np.asarray(w, np.float64)


def qk_norm_rope(x, w, pos, base, eps):
    return rope_f64(qk_norm(x, w, eps), pos, base)


def logits_process(logits, vocab, hist=None, prompt_len=None, repetition=None, frequency=None, presence=None,
                   bias=None, rows_of=None, draft=None, see=None, allow=None, allow_row=None):
    """fp32 rows after the rules.  logits fp32 [rows, >= vocab]; hist: token
    list per request; bias: (ids, values) per request; rows_of: the rows of
    each request (default: row r is request r); draft: drafted token lists and
    see: bool [T, T] per request; allow: bool [mask rows, vocab], allow_row
    [rows].  Ids outside the vocabulary are left out."""
    f = np.float32
    n_req = len(rows_of) if rows_of is not None else len(logits)
    rows_of = [range(i, i + 1) for i in range(n_req)] if rows_of is None else rows_of
    out = {}
    for b in range(n_req):
        h = np.asarray(hist[b] if hist is not None else [], np.int64)
        hp = int(prompt_len[b]) if prompt_len is not None else 0
        for i, r in enumerate(rows_of[b]):
            x = np.array(logits[r, :vocab], f)
            made = list(h[hp:]) + ([draft[b][j] for j in range(len(draft[b])) if see[b][i][j]] if draft is not None else [])
            made = np.array([t for t in made if 0 <= t < vocab], np.int64)
            asked = np.array([t for t in h[:hp] if 0 <= t < vocab], np.int64)
            count = np.bincount(made, minlength=vocab)
            seen = (count + np.bincount(asked, minlength=vocab)) > 0
            rep = f(repetition[b]) if repetition is not None else f(1)
            fr = f(frequency[b]) if frequency is not None else f(0)
            pr = f(presence[b]) if presence is not None else f(0)
            with np.errstate(invalid="ignore"):
                x = np.where(seen, np.where(x > 0, x / rep, x * rep), x).astype(f)
                x = np.where(count > 0, x - fr * count.astype(f), x).astype(f)
                x = np.where(count > 0, x - pr, x).astype(f)
                if bias is not None:
                    add = {}
                    for t, v in zip(*bias[b]):
                        if 0 <= t < vocab:
                            add[int(t)] = f(v) if int(t) not in add else f(add[int(t)] + f(v))
                    for t, v in add.items():
                        x[t] = f(x[t] + v)
            if allow is not None and allow_row[r] != -1:
                a = int(allow_row[r])
                ok = allow[a] if 0 <= a < len(allow) else np.zeros(vocab, bool)
                x = np.where(ok, x, f(-np.inf))
            out[r] = x
    return out
