"""Rules on attention scores, rotation on several axes, lists of a step -- oracle.

TEST INFRASTRUCTURE ONLY.  Plain numpy in fp64; it imports nothing from the
CUDA path.  The definitions are those written in ``include/rx.h``:

* ``attention``: a tanh cap, a bias that falls with the distance, a window and
  bounds of each query token;
* ``rope_axes``: rotation whose pairs take their positions from several axes;
* ``step_maps``: where new tokens start, their positions and slots.

Pinned in ``tests/test_rules_oracle.py``.
"""
from __future__ import annotations

import numpy as np


def seen(p, n, window=0, see_from=0, see_to=0):
    """The positions [lo, hi) that the token at p of a context of n sees."""
    lo = max(0, see_from, p - window + 1 if window else 0)
    return lo, max(p + 1, min(see_to, n))


def attention(q, k_pool, v_pool, rtt, req_idx, prefix_len, new_len, sm_scale, cap=0.0, window=0, slopes=None,
              see_from=None, see_to=None):
    """q fp64 [n, Hq, d] (request after request); pools fp64 [S, Hkv, d].  Slots
    outside the pool read as zero rows.  Returns (o, lse, a): a = sum_j p_j |v_j|
    (for error bounds)."""
    q = np.asarray(q, np.float64)
    n, hq, d = q.shape
    S, hkv, _ = k_pool.shape
    G = hq // hkv
    o, a = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse = np.full((n, hq), -np.inf)
    row = 0
    for b in range(len(req_idx)):
        P, T = int(prefix_len[b]), int(new_len[b])
        for i in range(T):
            p = P + i
            lo, hi = seen(p, P + T, window, 0 if see_from is None else int(see_from[row]),
                          0 if see_to is None else int(see_to[row]))
            if lo < hi:
                slots = np.asarray(rtt[req_idx[b], lo:hi], np.int64)
                ok = (slots >= 0) & (slots < S)
                k = np.where(ok[:, None, None], k_pool[np.where(ok, slots, 0)], 0.0)
                v = np.where(ok[:, None, None], v_pool[np.where(ok, slots, 0)], 0.0)
                far = np.abs(p - np.arange(lo, hi))
                for h in range(hq):
                    x = sm_scale * (k[:, h // G] @ q[row, h])
                    if cap:
                        x = cap * np.tanh(x / cap)
                    if slopes is not None:
                        x = x - float(slopes[h]) * far
                    top = x.max()
                    w = np.exp(x - top)
                    lse[row, h] = top + np.log(w.sum())
                    w = w / w.sum()
                    o[row, h] = w @ v[:, h // G]
                    a[row, h] = w @ np.abs(v[:, h // G])
            row += 1
    return o, lse, a


def rope_axes(x, pos, pair_axis, base, weight=None, eps=None):
    """x fp64 [n, heads, d], pos [axes, n]: pair c turned by pos[pair_axis[c]] base^(-2c/d), after an RMS norm where
    eps is given."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    if eps is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x = x * np.asarray(weight, np.float64)
    out = np.empty_like(x)
    for c in range(d // 2):
        angle = np.asarray(pos[pair_axis[c]], np.float64) * base ** (-2.0 * c / d)
        cs, sn = np.cos(angle)[:, None], np.sin(angle)[:, None]
        lo, hi = x[..., c], x[..., c + d // 2]
        out[..., c] = lo * cs - hi * sn
        out[..., c + d // 2] = hi * cs + lo * sn
    return out


def step_maps(req_idx, prefix_len, new_len, rtt, num_slots, max_tokens, pages=None, page_size=0):
    """(qo_indptr, seq_len, pos, slots, rtt after the call, bad length, bad slot); pos and slots as long as the tokens
    that fit."""
    rtt = np.array(rtt)
    limit = rtt.shape[1] if pages is None else min(rtt.shape[1], pages.shape[1] * page_size)
    indptr, seq, pos, slots = [0], [], [], []
    bad_len = bad_slot = False
    for b in range(len(req_idx)):
        P, E, r = int(prefix_len[b]), int(new_len[b]), int(req_idx[b])
        if P < 0 or E < 0 or P + E > limit:
            bad_len = True
            seq.append(0)
            E = 0
        else:
            seq.append(P + E)
        for p in range(P, P + E):
            if len(pos) >= max_tokens:
                bad_len = True
                break
            if pages is None:
                s = int(rtt[r, p])
            else:
                g = int(pages[r, p // page_size])
                s = g * page_size + p % page_size if g >= 0 else -1
            if s < 0 or s >= num_slots:
                bad_slot, s = True, -1
            if pages is not None:
                rtt[r, p] = s
            pos.append(p)
            slots.append(s)
        indptr.append(len(pos))
    return indptr, seq, pos, slots, rtt, bad_len, bad_slot
