"""Thin ctypes binding of librx (``include/rx.h``).

Argument marshalling only: every function here checks the tensors it is
given (device, dtype, contiguity), passes their data pointers and the current
CUDA stream to the library function of the same name, and turns a non-zero
status into ``RxError``.  No step of the path runs in Python, and there is no
fallback: if ``_build/librx.so`` is missing, importing this module raises.

Device tensors come from PyTorch (it owns device memory and streams); host
arrays are numpy.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import List, Optional, Sequence, Tuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "librx.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"librx.so is not built ({LIB_PATH}); run __graft_entry__.build() or "
                      "python -m prefix_shared_kv_radixattention_gb300.build")
_lib = ctypes.CDLL(LIB_PATH)

RX_OK = 0
RX_ERR_INVALID = -1
RX_ERR_CAPACITY = -2
RX_ERR_NOMEM = -3
RX_ERR_NOT_ENOUGH = -4
RX_ERR_CUDA = -5
RX_ERR_UNSUPPORTED = -6
RX_SCHED_FCFS = 0
RX_SCHED_LPM = 1
RX_DEV_BAD_SLOT = 1
RX_DEV_BAD_LEN = 2
RX_DEV_TIMEOUT = 4
RX_DEV_FSM_DONE = 8
RX_DEV_BAD_STATE = 16
RX_DEV_BAD_TOKEN = 32
RX_PLAN_OPEN_END = -1


class RxError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class KVPool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_slots", ctypes.c_int64),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("num_layers", ctypes.c_int32), ("layer", ctypes.c_int32)]


class DecodePlan(ctypes.Structure):
    _fields_ = [("order", ctypes.c_void_p), ("nparts", ctypes.c_void_p), ("items", ctypes.c_void_p),
                ("n_items", ctypes.c_int32), ("max_parts", ctypes.c_int32), ("n_wide", ctypes.c_int32)]


class DecodePlanInfo(ctypes.Structure):
    _fields_ = [("n_items", ctypes.c_int32), ("max_parts", ctypes.c_int32),
                ("n_segments", ctypes.c_int32), ("kv_chunk", ctypes.c_int32),
                ("shared_tokens", ctypes.c_int64), ("tokens_read", ctypes.c_int64),
                ("buf_words", ctypes.c_int64), ("n_wide", ctypes.c_int32)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_PI64 = ctypes.POINTER(ctypes.c_int64)


def _sig(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_sig("rx_last_error", ctypes.c_char_p)
_sig("rx_version", ctypes.c_int)
_sig("rx_tree_create", ctypes.c_int, ctypes.POINTER(_P))
_sig("rx_tree_destroy", None, _P)
_sig("rx_match_prefix", ctypes.c_int, _P, _P, _I64, _P, _I64, _PI64)
_sig("rx_insert", ctypes.c_int, _P, _P, _P, _I64, _PI64)
_sig("rx_evict_lru", ctypes.c_int, _P, _I64, _P, _I64, _PI64)
_sig("rx_lock_prefix", ctypes.c_int, _P, _P, _I64, _I32, _PI64)
_sig("rx_tree_stats", ctypes.c_int, _P, _PI64, _PI64, _PI64)
_sig("rx_tree_dump", ctypes.c_int, _P, _P, _I64, _PI64)
_sig("rx_slot_alloc_create", ctypes.c_int, _P, _I64, _I64, ctypes.POINTER(_P))
_sig("rx_slot_alloc_destroy", None, _P)
_sig("rx_slot_alloc_take", ctypes.c_int, _P, _I64, _P)
_sig("rx_slot_alloc_give", ctypes.c_int, _P, _P, _I64)
_sig("rx_slot_alloc_free_count", _I64, _P)
_sig("rx_admit", ctypes.c_int, _P, _P, _P, _I64, _P, _PI64, _PI64)
_sig("rx_commit", ctypes.c_int, _P, _P, _P, _P, _I64, _I64)
_sig("rx_prefix_len", ctypes.c_int, _P, _P, _I64, _PI64)
_sig("rx_image_keys", ctypes.c_int, _P, _I64, _I64, _P)


class KVPoolFp8(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("num_slots", ctypes.c_int64), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
                ("num_layers", ctypes.c_int32), ("layer", ctypes.c_int32)]


_sig("rx_kv_store_fp8", ctypes.c_int, ctypes.POINTER(KVPoolFp8), _P, _P, _P, _I64, _P, _P)
_sig("rx_attn_decode_fp8", ctypes.c_int, ctypes.POINTER(KVPoolFp8), _P, _P, _P, _I32, _P, _P, _P, _I64, _I32,
     _I32, _P, _P, ctypes.c_size_t, ctypes.c_float, _P, _P)
_sig("rx_attn_extend_fp8", ctypes.c_int, ctypes.POINTER(KVPoolFp8), _P, _P, _P, _I32, _P, _P, _P, _P, _P,
     _I64, _I32, _I32, _P, ctypes.c_size_t, ctypes.c_float, _P, _P)
_sig("rx_kv_store_rope_fp8", ctypes.c_int, ctypes.POINTER(KVPoolFp8), _P, _P, _P, _P, _I64, ctypes.c_double, _P, _P)


class FsmInfo(ctypes.Structure):
    _fields_ = [("n_edges", ctypes.c_int64), ("jump_tokens", ctypes.c_int64), ("n_singular", ctypes.c_int32),
                ("n_looped", ctypes.c_int32), ("longest_jump", ctypes.c_int32)]


class FsmStruct(ctypes.Structure):
    _fields_ = [("row_ptr", _P), ("tok", _P), ("nxt", _P), ("mask", _P), ("rank", _P), ("jump_len", _P),
                ("jump_off", _P), ("jump_end", _P), ("jump_tok", _P), ("n_states", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("max_jump", ctypes.c_int32)]


_sig("rx_fsm_compress", ctypes.c_int, _I32, _I32, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _I64,
     ctypes.POINTER(FsmInfo))
_sig("rx_fsm_step", ctypes.c_int, ctypes.POINTER(FsmStruct), _P, _I64, _I32, _P, _P, _P, _P, _P, _P)
class LogitsRulesStruct(ctypes.Structure):
    _fields_ = [("n_req", ctypes.c_int32), ("vocab", ctypes.c_int32), ("hist", _P), ("hist_ptr", _P),
                ("prompt_len", _P), ("repetition", _P), ("frequency", _P), ("presence", _P), ("bias_ptr", _P),
                ("bias_tok", _P), ("bias_val", _P), ("qo_indptr", _P), ("draft_tok", _P), ("tree_mask", _P),
                ("tree_words", ctypes.c_int32), ("n_allow", ctypes.c_int32), ("allow", _P), ("allow_row", _P)]


_sig("rx_logits_process", ctypes.c_int, ctypes.POINTER(LogitsRulesStruct), _P, _I32, _I64, _P, _I64, _I32, _P, _P)
_sig("rx_qk_norm_rope_store", ctypes.c_int, ctypes.POINTER(KVPool), _P, _I64, _P, _P, _P, _I64, _P, _P, _P, _P, _I64,
     _I32, ctypes.c_double, ctypes.c_float, _P, _P)
_sig("rx_qk_norm_rope_store_fp8", ctypes.c_int, ctypes.POINTER(KVPoolFp8), _P, _I64, _P, _P, _P, _I64, _P, _P, _P, _P,
     _I64, _I32, ctypes.c_double, ctypes.c_float, _P, _P)
_sig("rx_tree_mask_build", ctypes.c_int, _P, _I32, _I32, _P, _P)
_sig("rx_attn_tree", ctypes.c_int, ctypes.POINTER(KVPool), _P, _P, _P, _I32, _P, _P, _P, _P, _I32, _P, _I64, _I32, _I32,
     _P, ctypes.c_size_t, ctypes.c_float, _P, _P)
_sig("rx_attn_tree_fp8", ctypes.c_int, ctypes.POINTER(KVPoolFp8), _P, _P, _P, _I32, _P, _P, _P, _P, _I32, _P, _I64,
     _I32, _I32, _P, ctypes.c_size_t, ctypes.c_float, _P, _P)
_sig("rx_attn_tree_workspace", ctypes.c_size_t, _I32, _I32, _I32, _I32, _I32)
_sig("rx_schedule", ctypes.c_int, _P, _P, _P, _I32, _I32, _P, _P)
_sig("rx_kv_store", ctypes.c_int, ctypes.POINTER(KVPool), _P, _P, _P, _I64, _P, _P)
_sig("rx_rope", ctypes.c_int, _P, _P, _I64, _I32, _I32, ctypes.c_double, _P)
_sig("rx_kv_store_rope", ctypes.c_int, ctypes.POINTER(KVPool), _P, _P, _P, _P, _I64, ctypes.c_double, _P, _P)
_sig("rx_attn_extend", ctypes.c_int, ctypes.POINTER(KVPool), _P, _P, _P, _I32, _P, _P, _P, _P, _P,
     _I64, _I32, _I32, _P, ctypes.c_size_t, ctypes.c_float, _P, _P)
_sig("rx_attn_extend_workspace", ctypes.c_size_t, _I64, _I32, _I32, _I32)
_sig("rx_decode_plan_build", ctypes.c_int, _P, _I64, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _I64,
     ctypes.POINTER(DecodePlanInfo))
_sig("rx_attn_decode_workspace", ctypes.c_size_t, _I32, _I32, _I32, _I32, _I32,
     ctypes.POINTER(DecodePlan))
_sig("rx_attn_decode", ctypes.c_int, ctypes.POINTER(KVPool), _P, _P, _P, _I32, _P, _P, _P, _I64, _I32,
     _I32, ctypes.POINTER(DecodePlan), _P, ctypes.c_size_t, ctypes.c_float, _P, _P)
_sig("rx_attn_decode_static", ctypes.c_int, ctypes.POINTER(KVPool), _P, _P, _P, _I32, _P, _P, _P, _I64,
     _I32, _I32, ctypes.POINTER(DecodePlan), ctypes.c_float, _P, _P)
RX_DECODE_STATIC_SCRATCH_BYTES = 16 << 20
_sig("rx_test_fail_alloc", ctypes.c_int, _I64)
_sig("rx_decode_set_wait_limit", ctypes.c_int, _I64)


def rx_test_fail_alloc(n: int) -> None:
    """The n-th next radix-tree node allocation fails (0: off); see rx.h."""
    _check(_lib.rx_test_fail_alloc(int(n)))


def rx_decode_set_wait_limit(cycles: int) -> None:
    """Bound on each decode pipeline wait, in SM cycles (<= 0: the default)."""
    _check(_lib.rx_decode_set_wait_limit(int(cycles)))


def library():
    """The loaded ctypes.CDLL (for symbol checks)."""
    return _lib


def version() -> int:
    return _lib.rx_version()


def last_error() -> str:
    return _lib.rx_last_error().decode()


def _check(rc: int, allow=()) -> int:
    if rc != RX_OK and rc not in allow:
        raise RxError(rc, last_error())
    return rc


def _np(a, dtype):
    a = np.ascontiguousarray(a, dtype=dtype)
    return a, a.ctypes.data_as(ctypes.c_void_p)


# ---------------------------------------------------------------------------
# radix tree and slot free list (host)
# ---------------------------------------------------------------------------


class RadixTree:
    """rx_tree: prefix match, insert, LRU eviction and locks over token ids."""

    def __init__(self):
        h = _P()
        _check(_lib.rx_tree_create(ctypes.byref(h)))
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _lib.rx_tree_destroy(h)
            self._h = None

    def match_prefix(self, tokens: Sequence[int]) -> Tuple[int, List[int]]:
        t, tp = _np(tokens, np.int64)
        out = np.empty(max(1, len(t)), np.int32)
        k = ctypes.c_int64()
        _check(_lib.rx_match_prefix(self._h, tp, len(t), out.ctypes.data_as(_P), len(t),
                                    ctypes.byref(k)))
        return k.value, out[:k.value].tolist()

    def insert(self, tokens: Sequence[int], slots: Sequence[int]) -> int:
        t, tp = _np(tokens, np.int64)
        s, sp = _np(slots, np.int32)
        assert len(t) == len(s)
        k = ctypes.c_int64()
        _check(_lib.rx_insert(self._h, tp, sp, len(t), ctypes.byref(k)))
        return k.value

    def evict(self, num_tokens: int, cap: Optional[int] = None) -> List[int]:
        """Freed slots; raises RxError(RX_ERR_CAPACITY) if ``cap`` is too small."""
        if cap is None:
            _, _, ev = self.stats()
            cap = max(ev, 1)
        out = np.empty(max(1, cap), np.int32)
        n = ctypes.c_int64()
        rc = _lib.rx_evict_lru(self._h, int(num_tokens), out.ctypes.data_as(_P), cap, ctypes.byref(n))
        _check(rc, allow=(RX_ERR_NOT_ENOUGH,))
        return out[:n.value].tolist()

    def lock(self, tokens: Sequence[int], delta: int) -> int:
        t, tp = _np(tokens, np.int64)
        k = ctypes.c_int64()
        _check(_lib.rx_lock_prefix(self._h, tp, len(t), int(delta), ctypes.byref(k)))
        return k.value

    def prefix_len(self, tokens: Sequence[int]) -> int:
        """Cached prefix length, without touching the LRU clock."""
        t, tp = _np(tokens, np.int64)
        k = ctypes.c_int64()
        _check(_lib.rx_prefix_len(self._h, tp, len(t), ctypes.byref(k)))
        return k.value

    def stats(self) -> Tuple[int, int, int]:
        a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(_lib.rx_tree_stats(self._h, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
        return a.value, b.value, c.value

    def dump(self) -> List[dict]:
        need = ctypes.c_int64()
        _check(_lib.rx_tree_dump(self._h, None, 0, ctypes.byref(need)), allow=(RX_ERR_CAPACITY,))
        buf = np.empty(max(1, need.value), np.int64)
        _check(_lib.rx_tree_dump(self._h, buf.ctypes.data_as(_P), len(buf), ctypes.byref(need)))
        out, i = [], 0
        while i < need.value:
            nid, par, last, n = buf[i:i + 4].tolist()
            i += 4
            toks = buf[i:i + n].tolist()
            slots = buf[i + n:i + 2 * n].tolist()
            locks = buf[i + 2 * n:i + 3 * n].tolist()
            i += 3 * n
            out.append(dict(id=nid, parent=par, last=last, tokens=toks, slots=slots, locks=locks))
        return out

    def nodes(self) -> List[Tuple[Tuple[int, ...], Tuple[int, ...]]]:
        """Every node as (token path before it, its own tokens), sorted."""
        recs = self.dump()
        path = {}
        out = []
        for r in recs:  # depth-first: parents come before children
            before = () if r["parent"] < 0 else path[r["parent"]]
            path[r["id"]] = before + tuple(r["tokens"])
            out.append((before, tuple(r["tokens"])))
        return sorted(out)


class SlotAllocator:
    """rx_slot_alloc: first-in first-out free list of pool slots."""

    def __init__(self, free_order: Sequence[int], num_slots: int):
        o, op = _np(free_order, np.int32)
        h = _P()
        _check(_lib.rx_slot_alloc_create(op, len(o), int(num_slots), ctypes.byref(h)))
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _lib.rx_slot_alloc_destroy(h)
            self._h = None

    def take(self, n: int) -> np.ndarray:
        out = np.empty(max(1, n), np.int32)
        _check(_lib.rx_slot_alloc_take(self._h, int(n), out.ctypes.data_as(_P)))
        return out[:n]

    def give(self, slots: Sequence[int]) -> None:
        s, sp = _np(slots, np.int32)
        _check(_lib.rx_slot_alloc_give(self._h, sp, len(s)))

    def free_count(self) -> int:
        return _lib.rx_slot_alloc_free_count(self._h)


def rx_admit(tree: RadixTree, alloc: SlotAllocator, tokens: Sequence[int]):
    """(slot row int32 [n], prefix_len, evicted tokens)."""
    t, tp = _np(tokens, np.int64)
    row = np.empty(max(1, len(t)), np.int32)
    k, ev = ctypes.c_int64(), ctypes.c_int64()
    _check(_lib.rx_admit(tree._h, alloc._h, tp, len(t), row.ctypes.data_as(_P), ctypes.byref(k),
                         ctypes.byref(ev)))
    return row[:len(t)], k.value, ev.value


def rx_commit(tree: RadixTree, alloc: SlotAllocator, tokens: Sequence[int], row: Sequence[int],
              prefix_len: int) -> None:
    t, tp = _np(tokens, np.int64)
    r, rp = _np(row, np.int32)
    _check(_lib.rx_commit(tree._h, alloc._h, tp, rp, len(t), int(prefix_len)))


def rx_image_keys(data: bytes, n_tokens: int) -> np.ndarray:
    """int64 keys of the n_tokens positions an image (its raw bytes) occupies."""
    buf = np.frombuffer(bytes(data), dtype=np.uint8)
    out = np.empty(max(1, n_tokens), np.int64)
    _check(_lib.rx_image_keys(buf.ctypes.data_as(_P) if len(buf) else None, len(buf), int(n_tokens),
                              out.ctypes.data_as(_P)))
    return out[:n_tokens]


def rx_schedule(tree: RadixTree, requests: Sequence[Sequence[int]], policy: int):
    """(order int32 [n], cached prefix lengths int64 [n]) for waiting requests."""
    n = len(requests)
    offs = np.zeros(n + 1, np.int64)
    for i, r in enumerate(requests):
        offs[i + 1] = offs[i] + len(r)
    toks = np.concatenate([np.asarray(r, np.int64) for r in requests]) if n else np.zeros(0, np.int64)
    toks = np.ascontiguousarray(toks, np.int64)
    order = np.empty(max(1, n), np.int32)
    plen = np.empty(max(1, n), np.int64)
    _check(_lib.rx_schedule(tree._h, toks.ctypes.data_as(_P), offs.ctypes.data_as(_P), n, int(policy),
                            order.ctypes.data_as(_P), plen.ctypes.data_as(_P)))
    return order[:n], plen[:n]


# ---------------------------------------------------------------------------
# device entry points
# ---------------------------------------------------------------------------


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dev(t, dtype, name):
    if t is None:
        return None
    if not isinstance(t, (_torch_module or _torch()).Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    # the current stream's handle without the Python object around it, which
    # takes 3 us to make: a sixth of a call on a small batch
    c = _torch()._C
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


def _pool_dims(k_pool, v_pool, layer: int):
    """(num_slots, kv heads, head_dim, num_layers) of a one-layer pool
    [S, Hkv, d] or a layered one [L, S, Hkv, d]."""
    if k_pool.shape != v_pool.shape or k_pool.dim() not in (3, 4):
        raise ValueError("k_pool and v_pool must both be [num_slots, num_kv_heads, head_dim] or "
                         "[num_layers, num_slots, num_kv_heads, head_dim]")
    if k_pool.dim() == 3:
        return (*k_pool.shape, 0)
    L, S, hkv, d = k_pool.shape
    return S, hkv, d, L


def make_pool(k_pool, v_pool, layer: int = 0) -> KVPool:
    """The C pool of k_pool / v_pool: one layer [S, Hkv, d], or layer `layer`
    of a layered pool [L, S, Hkv, d]."""
    torch = _torch()
    _dev(k_pool, torch.bfloat16, "k_pool")
    _dev(v_pool, torch.bfloat16, "v_pool")
    S, hkv, d, L = _pool_dims(k_pool, v_pool, layer)
    return KVPool(k_pool.data_ptr(), v_pool.data_ptr(), S, hkv, d, L, int(layer))


def rx_kv_store(k_pool, v_pool, k_new, v_new, slots, dev_status=None, stream=None, layer: int = 0) -> None:
    torch = _torch()
    pool = make_pool(k_pool, v_pool, layer)
    _dev(k_new, torch.bfloat16, "k_new")
    _dev(v_new, torch.bfloat16, "v_new")
    _dev(slots, torch.int32, "slots")
    _dev(dev_status, torch.int32, "dev_status")
    n = slots.numel()
    if k_new.numel() != n * pool.num_kv_heads * pool.head_dim or k_new.shape != v_new.shape:
        raise ValueError("k_new/v_new must be [n, num_kv_heads, head_dim]")
    _check(_lib.rx_kv_store(ctypes.byref(pool), _ptr(k_new), _ptr(v_new), _ptr(slots), n,
                            _ptr(dev_status), _stream(stream)))


def rx_rope(x, pos, base: float, stream=None) -> None:
    """In place on x (bf16 [n, heads, head_dim]) at positions pos (int32 [n])."""
    torch = _torch()
    _dev(x, torch.bfloat16, "x")
    _dev(pos, torch.int32, "pos")
    if x.dim() != 3 or pos.numel() != x.shape[0]:
        raise ValueError("x must be [n, heads, head_dim] and pos [n]")
    _check(_lib.rx_rope(_ptr(x), _ptr(pos), x.shape[0], x.shape[1], x.shape[2], float(base), _stream(stream)))


def rx_kv_store_rope(k_pool, v_pool, k_new, v_new, slots, pos, base: float, dev_status=None,
                     stream=None, layer: int = 0) -> None:
    torch = _torch()
    pool = make_pool(k_pool, v_pool, layer)
    _dev(k_new, torch.bfloat16, "k_new")
    _dev(v_new, torch.bfloat16, "v_new")
    _dev(slots, torch.int32, "slots")
    _dev(pos, torch.int32, "pos")
    _dev(dev_status, torch.int32, "dev_status")
    n = slots.numel()
    if k_new.numel() != n * pool.num_kv_heads * pool.head_dim or k_new.shape != v_new.shape or pos.numel() != n:
        raise ValueError("k_new/v_new must be [n, num_kv_heads, head_dim] and pos [n]")
    _check(_lib.rx_kv_store_rope(ctypes.byref(pool), _ptr(k_new), _ptr(v_new), _ptr(slots), _ptr(pos), n,
                                 float(base), _ptr(dev_status), _stream(stream)))


def rx_kv_store_rope_fp8(k_pool, v_pool, k_scale: float, v_scale: float, k_new, v_new, slots, pos, base: float,
                         dev_status=None, stream=None, layer: int = 0) -> None:
    """rx_kv_store_rope into uint8 E4M3 pools ([L,] S, Hkv, d) with per-pool scales."""
    torch = _torch()
    _dev(k_pool, torch.uint8, "k_pool")
    _dev(v_pool, torch.uint8, "v_pool")
    _dev(k_new, torch.bfloat16, "k_new")
    _dev(v_new, torch.bfloat16, "v_new")
    _dev(slots, torch.int32, "slots")
    _dev(pos, torch.int32, "pos")
    _dev(dev_status, torch.int32, "dev_status")
    S, hkv, d, L = _pool_dims(k_pool, v_pool, layer)
    n = slots.numel()
    if k_new.shape != (n, hkv, d) or v_new.shape != k_new.shape or pos.numel() != n:
        raise ValueError("k_new/v_new must be [n, num_kv_heads, head_dim] and pos [n]")
    pool = KVPoolFp8(k_pool.data_ptr(), v_pool.data_ptr(), S, hkv, d, float(k_scale), float(v_scale), L,
                     int(layer))
    _check(_lib.rx_kv_store_rope_fp8(ctypes.byref(pool), _ptr(k_new), _ptr(v_new), _ptr(slots), _ptr(pos), n,
                                     float(base), _ptr(dev_status), _stream(stream)))


def rx_attn_extend_workspace(total_ctx_tokens: int, batch: int, num_kv_heads: int, head_dim: int) -> int:
    """Workspace bytes for rx_attn_extend's staged path (contexts summing to at
    most total_ctx_tokens tokens)."""
    n = _lib.rx_attn_extend_workspace(int(total_ctx_tokens), int(batch), int(num_kv_heads), int(head_dim))
    if n == 0:
        raise RxError(last_error())
    return int(n)


def rx_attn_extend(k_pool, v_pool, q, o, lse, qo_indptr, req_idx, prefix_len, extend_len,
                   req_to_token, max_extend_len: int, sm_scale: float, dev_status=None,
                   stream=None, workspace=None, layer: int = 0) -> None:
    """Extend attention; `workspace` (a device uint8 tensor of at least
    rx_attn_extend_workspace(...) bytes) selects the staged path."""
    torch = _torch()
    pool = make_pool(k_pool, v_pool, layer)
    for t, n in ((q, "q"), (o, "o")):
        _dev(t, torch.bfloat16, n)
    _dev(lse, torch.float32, "lse")
    for t, n in ((qo_indptr, "qo_indptr"), (req_idx, "req_idx"), (prefix_len, "prefix_len"),
                 (extend_len, "extend_len"), (req_to_token, "req_to_token")):
        _dev(t, torch.int32, n)
    _dev(dev_status, torch.int32, "dev_status")
    _dev(workspace, torch.uint8, "workspace")
    if q.dim() != 3 or q.shape != o.shape:
        raise ValueError("q and o must be [tokens, num_q_heads, head_dim]")
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check(_lib.rx_attn_extend(ctypes.byref(pool), _ptr(q), _ptr(o), _ptr(lse), q.shape[1],
                               _ptr(qo_indptr), _ptr(req_idx), _ptr(prefix_len), _ptr(extend_len),
                               _ptr(req_to_token), req_to_token.shape[1], req_idx.numel(),
                               int(max_extend_len), _ptr(workspace), ws_bytes, float(sm_scale),
                               _ptr(dev_status), _stream(stream)))


@dataclass
class DevicePlan:
    """A decode plan copied to the device; keeps its buffer alive."""

    buf: object          # torch int32 tensor on the device
    info: DecodePlanInfo
    batch: int
    struct: DecodePlan


def rx_decode_plan_build(req_to_token_host, req_idx_host, seq_len_host, num_q_heads: int,
                         num_kv_heads: int, kv_chunk: int = 0, min_shared: int = 16):
    """Host plan: (packed int32 numpy buffer, DecodePlanInfo)."""
    rtt, rp = _np(req_to_token_host, np.int32)
    ri, rip = _np(req_idx_host, np.int32)
    sl, slp = _np(seq_len_host, np.int32)
    info = DecodePlanInfo()
    # one call with room for the usual plan sizes; a second one only when the
    # library reports that more words are needed
    buf = np.empty(2 * len(ri) + 8 * max(8192, 64 * len(ri)), np.int32)
    rc = _lib.rx_decode_plan_build(rp, rtt.shape[1], rip, slp, len(ri), num_q_heads, num_kv_heads,
                                   kv_chunk, min_shared, buf.ctypes.data_as(_P), len(buf), ctypes.byref(info))
    if rc == RX_ERR_CAPACITY:
        buf = np.empty(max(1, info.buf_words), np.int32)
        rc = _lib.rx_decode_plan_build(rp, rtt.shape[1], rip, slp, len(ri), num_q_heads, num_kv_heads,
                                       kv_chunk, min_shared, buf.ctypes.data_as(_P), len(buf), ctypes.byref(info))
    _check(rc)
    return buf[:info.buf_words], info


def plan_to_device(buf: np.ndarray, info: DecodePlanInfo, batch: int, device="cuda") -> DevicePlan:
    torch = _torch()
    d = torch.from_numpy(np.ascontiguousarray(buf)).to(device)
    base = d.data_ptr()
    st = DecodePlan(base, base + 4 * batch, base + 8 * batch, info.n_items, info.max_parts, info.n_wide)
    return DevicePlan(d, info, batch, st)


def rx_attn_decode_workspace(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                             max_seq_len: int, plan: Optional[DevicePlan] = None) -> int:
    pp = ctypes.byref(plan.struct) if plan is not None else None
    return _lib.rx_attn_decode_workspace(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, pp)


def rx_attn_decode(k_pool, v_pool, q, o, lse, req_idx, seq_len, req_to_token, max_seq_len: int,
                   sm_scale: float, plan: Optional[DevicePlan] = None, workspace=None,
                   dev_status=None, stream=None, layer: int = 0) -> None:
    torch = _torch()
    pool = make_pool(k_pool, v_pool, layer)
    _dev(q, torch.bfloat16, "q")
    _dev(o, torch.bfloat16, "o")
    _dev(lse, torch.float32, "lse")
    for t, n in ((req_idx, "req_idx"), (seq_len, "seq_len"), (req_to_token, "req_to_token")):
        _dev(t, torch.int32, n)
    _dev(dev_status, torch.int32, "dev_status")
    if workspace is not None:
        _dev(workspace, workspace.dtype, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    pp = ctypes.byref(plan.struct) if plan is not None else None
    _check(_lib.rx_attn_decode(ctypes.byref(pool), _ptr(q), _ptr(o), _ptr(lse), q.shape[1],
                               _ptr(req_idx), _ptr(seq_len), _ptr(req_to_token),
                               req_to_token.shape[1], req_idx.numel(), int(max_seq_len), pp,
                               _ptr(workspace), ws_bytes, float(sm_scale), _ptr(dev_status),
                               _stream(stream)))


def rx_attn_decode_static(k_pool, v_pool, q, o, lse, req_idx, seq_len, req_to_token, max_seq_len: int,
                          sm_scale: float, plan: Optional[DevicePlan] = None, dev_status=None,
                          stream=None, layer: int = 0) -> None:
    """rx_attn_decode with the library's fixed scratch array instead of a
    workspace (for callers that cannot allocate device memory; see rx.h)."""
    torch = _torch()
    pool = make_pool(k_pool, v_pool, layer)
    _dev(q, torch.bfloat16, "q")
    _dev(o, torch.bfloat16, "o")
    _dev(lse, torch.float32, "lse")
    for t, n in ((req_idx, "req_idx"), (seq_len, "seq_len"), (req_to_token, "req_to_token")):
        _dev(t, torch.int32, n)
    _dev(dev_status, torch.int32, "dev_status")
    pp = ctypes.byref(plan.struct) if plan is not None else None
    _check(_lib.rx_attn_decode_static(ctypes.byref(pool), _ptr(q), _ptr(o), _ptr(lse), q.shape[1],
                                      _ptr(req_idx), _ptr(seq_len), _ptr(req_to_token),
                                      req_to_token.shape[1], req_idx.numel(), int(max_seq_len), pp,
                                      float(sm_scale), _ptr(dev_status), _stream(stream)))


# ---------------------------------------------------------------------------
# compressed finite-state machine (constrained decoding)
# ---------------------------------------------------------------------------


def rx_fsm_compress(n_states: int, vocab: int, row_ptr, tok, nxt, max_jump: int):
    """Host compression of a token automaton (CSR).  Returns (mask uint32
    [S, W], rank int32 [S, W] with W = ceil(V / 128) * 4, jump_len int32 [S],
    jump_off int64 [S], jump_end int32 [S], jump_tok int32 [total], info)."""
    rp, rpp = _np(row_ptr, np.int64)
    t, tp = _np(tok, np.int32)
    n, np_ = _np(nxt, np.int32)
    info = FsmInfo()
    _check(_lib.rx_fsm_compress(int(n_states), int(vocab), rpp, tp if len(t) else None, np_ if len(n) else None,
                                int(max_jump), None, None, None, None, None, None, 0, ctypes.byref(info)))
    W = (int(vocab) + 127) // 128 * 4   # mask words per state, rows padded to 16 bytes
    mask = np.empty((int(n_states), W), np.uint32)
    rank = np.empty((int(n_states), W), np.int32)
    jl = np.empty(int(n_states), np.int32)
    jo = np.empty(int(n_states), np.int64)
    je = np.empty(int(n_states), np.int32)
    jt = np.empty(max(1, int(info.jump_tokens)), np.int32)
    _check(_lib.rx_fsm_compress(int(n_states), int(vocab), rpp, tp if len(t) else None, np_ if len(n) else None,
                                int(max_jump), mask.ctypes.data_as(_P), rank.ctypes.data_as(_P),
                                jl.ctypes.data_as(_P), jo.ctypes.data_as(_P), je.ctypes.data_as(_P),
                                jt.ctypes.data_as(_P), len(jt), ctypes.byref(info)))
    return mask, rank, jl, jo, je, jt[:int(info.jump_tokens)], info


class Fsm:
    """A compressed machine resident on the current CUDA device: the
    automaton and its compression (rx_fsm_compress), as torch tensors."""

    def __init__(self, n_states: int, vocab: int, row_ptr, tok, nxt, max_jump: int):
        torch = _torch()
        mask, rank, jl, jo, je, jt, info = rx_fsm_compress(n_states, vocab, row_ptr, tok, nxt, max_jump)
        self.info = info
        self.n_states, self.vocab, self.max_jump = int(n_states), int(vocab), int(max_jump)

        def dev(a, dt):
            a = np.ascontiguousarray(a, dtype=dt)
            if a.size == 0:
                a = np.zeros(1, dt)
            return torch.from_numpy(a).cuda()

        self.row_ptr = dev(row_ptr, np.int64)
        self.tok = dev(tok, np.int32)
        self.nxt = dev(nxt, np.int32)
        self.mask = torch.from_numpy(mask.view(np.int32)).cuda()
        self.rank = torch.from_numpy(rank).cuda()
        self.jump_len, self.jump_off = dev(jl, np.int32), dev(jo, np.int64)
        self.jump_end, self.jump_tok = dev(je, np.int32), dev(jt, np.int32)
        self.struct = FsmStruct(self.row_ptr.data_ptr(), self.tok.data_ptr(), self.nxt.data_ptr(),
                                self.mask.data_ptr(), self.rank.data_ptr(), self.jump_len.data_ptr(),
                                self.jump_off.data_ptr(),
                                self.jump_end.data_ptr(), self.jump_tok.data_ptr(), self.n_states, self.vocab,
                                self.max_jump)


def fsm_workspace(batch: int):
    """The zeroed device workspace rx_fsm_step needs for `batch` requests:
    batch + 1 words (every call leaves it zero, so it can be kept and
    reused)."""
    torch = _torch()
    return torch.zeros(max(1, int(batch)) + 1, dtype=torch.int64, device="cuda")


def rx_fsm_step(fsm: Fsm, logits, state, out_tokens, out_count, workspace, dev_status=None,
                stream=None) -> None:
    """One constrained decoding step: logits fp32 [B, >= V] (rows 16-byte
    aligned), state int32 [B] (updated), out_tokens int32 [B, 1 + max_jump],
    out_count int32 [B], workspace from fsm_workspace(B)."""
    torch = _torch()
    _dev(workspace, torch.int64, "workspace")
    if workspace.numel() < state.numel():
        raise ValueError("rx_fsm_step: workspace smaller than the batch")
    _dev(logits, torch.float32, "logits")
    _dev(state, torch.int32, "state")
    _dev(out_tokens, torch.int32, "out_tokens")
    _dev(out_count, torch.int32, "out_count")
    _dev(dev_status, torch.int32, "dev_status")
    B = state.numel()
    if logits.dim() != 2 or logits.shape[0] != B or out_tokens.shape != (B, 1 + fsm.max_jump) or \
            out_count.numel() != B:
        raise ValueError("rx_fsm_step: logits [B, V], out_tokens [B, 1 + max_jump], out_count [B]")
    _check(_lib.rx_fsm_step(ctypes.byref(fsm.struct), _ptr(logits), logits.shape[1], B, _ptr(state),
                            _ptr(out_tokens), _ptr(out_count), _ptr(workspace), _ptr(dev_status),
                            _stream(stream)))


# ---------------------------------------------------------------------------
# FP8 key/value pools
# ---------------------------------------------------------------------------


def rx_kv_store_fp8(k_pool, v_pool, k_scale: float, v_scale: float, k_new, v_new, slots, dev_status=None,
                    stream=None, layer: int = 0) -> None:
    """Store bf16 rows into uint8 E4M3 pools ([L,] S, Hkv, d) with per-pool scales."""
    torch = _torch()
    _dev(k_pool, torch.uint8, "k_pool")
    _dev(v_pool, torch.uint8, "v_pool")
    _dev(k_new, torch.bfloat16, "k_new")
    _dev(v_new, torch.bfloat16, "v_new")
    _dev(slots, torch.int32, "slots")
    _dev(dev_status, torch.int32, "dev_status")
    S, hkv, d, L = _pool_dims(k_pool, v_pool, layer)
    n = slots.numel()
    if k_new.shape != (n, hkv, d) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [n, num_kv_heads, head_dim]")
    pool = KVPoolFp8(k_pool.data_ptr(), v_pool.data_ptr(), S, hkv, d, float(k_scale), float(v_scale), L,
                     int(layer))
    _check(_lib.rx_kv_store_fp8(ctypes.byref(pool), _ptr(k_new), _ptr(v_new), _ptr(slots), n,
                                _ptr(dev_status), _stream(stream)))


def rx_attn_extend_fp8(k_pool, v_pool, k_scale: float, v_scale: float, q, o, lse, qo_indptr, req_idx,
                       prefix_len, extend_len, req_to_token, max_extend_len: int, sm_scale: float, workspace,
                       dev_status=None, stream=None, layer: int = 0) -> None:
    """Extend attention over uint8 E4M3 pools ([L,] S, Hkv, d) with per-pool
    scales; `workspace` (at least rx_attn_extend_workspace(...) bytes, or
    None for the gather path) as in rx_attn_extend."""
    torch = _torch()
    _dev(k_pool, torch.uint8, "k_pool")
    _dev(v_pool, torch.uint8, "v_pool")
    for t, n in ((q, "q"), (o, "o")):
        _dev(t, torch.bfloat16, n)
    _dev(lse, torch.float32, "lse")
    for t, n in ((qo_indptr, "qo_indptr"), (req_idx, "req_idx"), (prefix_len, "prefix_len"),
                 (extend_len, "extend_len"), (req_to_token, "req_to_token")):
        _dev(t, torch.int32, n)
    _dev(dev_status, torch.int32, "dev_status")
    _dev(workspace, torch.uint8, "workspace")
    if q.dim() != 3 or q.shape != o.shape:
        raise ValueError("q and o must be [tokens, num_q_heads, head_dim]")
    S, hkv, d, L = _pool_dims(k_pool, v_pool, layer)
    pool = KVPoolFp8(k_pool.data_ptr(), v_pool.data_ptr(), S, hkv, d, float(k_scale), float(v_scale), L,
                     int(layer))
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check(_lib.rx_attn_extend_fp8(ctypes.byref(pool), _ptr(q), _ptr(o), _ptr(lse), q.shape[1],
                                   _ptr(qo_indptr), _ptr(req_idx), _ptr(prefix_len), _ptr(extend_len),
                                   _ptr(req_to_token), req_to_token.shape[1], req_idx.numel(),
                                   int(max_extend_len), _ptr(workspace), ws_bytes, float(sm_scale),
                                   _ptr(dev_status), _stream(stream)))


def rx_attn_decode_fp8(k_pool, v_pool, k_scale: float, v_scale: float, q, o, lse, req_idx, seq_len, req_to_token,
                       max_seq_len: int, sm_scale: float, plan: DevicePlan, workspace, dev_status=None, stream=None,
                       layer: int = 0) -> None:
    """Decode attention over uint8 E4M3 pools ([L,] S, Hkv, d) with per-pool
    scales; the plan (or None) and the workspace (rx_attn_decode_workspace
    bytes, or None when no row is split) as in rx_attn_decode."""
    torch = _torch()
    _dev(k_pool, torch.uint8, "k_pool")
    _dev(v_pool, torch.uint8, "v_pool")
    _dev(q, torch.bfloat16, "q")
    _dev(o, torch.bfloat16, "o")
    _dev(lse, torch.float32, "lse")
    for t, n in ((req_idx, "req_idx"), (seq_len, "seq_len"), (req_to_token, "req_to_token")):
        _dev(t, torch.int32, n)
    _dev(dev_status, torch.int32, "dev_status")
    if workspace is not None:
        _dev(workspace, workspace.dtype, "workspace")
    S, hkv, d, L = _pool_dims(k_pool, v_pool, layer)
    pool = KVPoolFp8(k_pool.data_ptr(), v_pool.data_ptr(), S, hkv, d, float(k_scale), float(v_scale), L, int(layer))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    pp = ctypes.byref(plan.struct) if plan is not None else None
    _check(_lib.rx_attn_decode_fp8(ctypes.byref(pool), _ptr(q), _ptr(o), _ptr(lse), q.shape[1], _ptr(req_idx),
                                   _ptr(seq_len), _ptr(req_to_token), req_to_token.shape[1], req_idx.numel(),
                                   int(max_seq_len), pp, _ptr(workspace), ws_bytes, float(sm_scale),
                                   _ptr(dev_status), _stream(stream)))


# ---------------------------------------------------------------------------
# verification of drafted tokens: norm + rotation + store, tree attention,
# logits
# ---------------------------------------------------------------------------


def _head_rows(t, name):
    """A CUDA bf16 [n, heads, d] tensor whose rows (all heads of a token) are
    contiguous; the rows themselves may be strided (a part of a projected
    row).  Returns n, heads, d and the row stride in elements."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name}: must be [n, heads, head_dim] with contiguous rows")
    (n, h, d), (row, head, one) = t.shape, t.stride()
    if n and ((d > 1 and one != 1) or (h > 1 and head != d)):
        raise ValueError(f"{name}: must be [n, heads, head_dim] with contiguous rows")
    return n, h, d, row if n > 1 else h * d


def _norm_args(k_pool, v_pool, q, q_out, k_new, v_new, q_weight, k_weight, slots, pos, dev_status):
    torch = _torch()
    bf16, i32 = torch.bfloat16, torch.int32
    n, hq, d, qs = _head_rows(q, "q")
    new, v_row = _head_rows(k_new, "k_new"), _head_rows(v_new, "v_new")
    _dev(q_out, bf16, "q_out")
    _dev(q_weight, bf16, "q_weight")
    _dev(k_weight, bf16, "k_weight")
    _dev(slots, i32, "slots")
    _dev(pos, i32, "pos")
    _dev(dev_status, i32, "dev_status")
    S, hkv, dim, L = _pool_dims(k_pool, v_pool, 0)
    if new[:3] != (slots.numel(), hkv, dim) or v_row[:3] != new[:3] or pos.numel() != new[0]:
        raise ValueError("k_new/v_new must be [n, num_kv_heads, head_dim] and pos [n]")
    if n != new[0] or d != dim or q_out.shape != q.shape:
        raise ValueError("q and q_out must be [n, num_q_heads, head_dim]")
    if new[3] != v_row[3]:
        raise ValueError("k_new and v_new must have the same row stride")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None and w.numel() != d:
            raise ValueError(f"{name} must be [head_dim]")
    return qs, new[3], n, hq, S, hkv, d, L


def rx_qk_norm_rope_store(k_pool, v_pool, q, q_out, k_new, v_new, q_weight, k_weight, slots, pos, base: float,
                          eps: float, dev_status=None, stream=None, layer: int = 0) -> None:
    """RMS norm of every q and k head (weights bf16 [d] or None), rotation to
    pos, q into q_out, K and V into the pool.  q, k_new, v_new: bf16 [n,
    heads, d], for example the three parts of one projected row."""
    torch = _torch()
    _dev(k_pool, torch.bfloat16, "k_pool")
    _dev(v_pool, torch.bfloat16, "v_pool")
    qs, ks, n, hq, S, hkv, d, L = _norm_args(k_pool, v_pool, q, q_out, k_new, v_new, q_weight, k_weight, slots, pos,
                                             dev_status)
    pool = KVPool(k_pool.data_ptr(), v_pool.data_ptr(), S, hkv, d, L, int(layer))
    _check(_lib.rx_qk_norm_rope_store(ctypes.byref(pool), _ptr(q), qs, _ptr(q_out), _ptr(k_new), _ptr(v_new), ks,
                                      _ptr(q_weight), _ptr(k_weight), _ptr(slots), _ptr(pos), n, hq,
                                      float(base), float(eps), _ptr(dev_status), _stream(stream)))


def rx_qk_norm_rope_store_fp8(k_pool, v_pool, k_scale: float, v_scale: float, q, q_out, k_new, v_new, q_weight,
                              k_weight, slots, pos, base: float, eps: float, dev_status=None, stream=None,
                              layer: int = 0) -> None:
    """rx_qk_norm_rope_store into uint8 E4M3 pools ([L,] S, Hkv, d) with
    per-pool scales."""
    torch = _torch()
    _dev(k_pool, torch.uint8, "k_pool")
    _dev(v_pool, torch.uint8, "v_pool")
    qs, ks, n, hq, S, hkv, d, L = _norm_args(k_pool, v_pool, q, q_out, k_new, v_new, q_weight, k_weight, slots, pos,
                                             dev_status)
    pool = KVPoolFp8(k_pool.data_ptr(), v_pool.data_ptr(), S, hkv, d, float(k_scale), float(v_scale), L, int(layer))
    _check(_lib.rx_qk_norm_rope_store_fp8(ctypes.byref(pool), _ptr(q), qs, _ptr(q_out), _ptr(k_new), _ptr(v_new), ks,
                                          _ptr(q_weight), _ptr(k_weight), _ptr(slots), _ptr(pos), n, hq,
                                          float(base), float(eps), _ptr(dev_status), _stream(stream)))


def rx_tree_mask_build(parent, words: Optional[int] = None):
    """(mask int32 [n, words], depth int32 [n]) of one drafted tree from its
    nodes' parents (-1: the token follows the text so far); host arrays."""
    p, pp = _np(parent, np.int32)
    n = len(p)
    words = (n + 31) // 32 if words is None else int(words)
    mask = np.zeros((n, max(words, 0)), np.uint32)
    depth = np.zeros(n, np.int32)
    _check(_lib.rx_tree_mask_build(pp, n, words, mask.ctypes.data_as(_P), depth.ctypes.data_as(_P)))
    return mask.view(np.int32), depth


def rx_attn_tree_workspace(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_tree_len: int) -> int:
    """Workspace bytes for rx_attn_tree and rx_attn_tree_fp8."""
    n = _lib.rx_attn_tree_workspace(int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim), int(max_tree_len))
    if n == 0:
        raise RxError(RX_ERR_INVALID, last_error())
    return int(n)


def _tree_args(q, o, lse, qo_indptr, req_idx, prefix_len, tree_mask, req_to_token, workspace, dev_status):
    torch = _torch()
    i32 = torch.int32
    _dev(q, torch.bfloat16, "q")
    _dev(o, torch.bfloat16, "o")
    _dev(lse, torch.float32, "lse")
    _dev(qo_indptr, i32, "qo_indptr")
    _dev(req_idx, i32, "req_idx")
    _dev(prefix_len, i32, "prefix_len")
    _dev(tree_mask, i32, "tree_mask")
    _dev(req_to_token, i32, "req_to_token")
    _dev(workspace, torch.uint8, "workspace")
    _dev(dev_status, i32, "dev_status")
    if q.dim() != 3 or q.shape != o.shape:
        raise ValueError("q and o must be [tokens, num_q_heads, head_dim]")
    if lse is not None and lse.shape != q.shape[:2]:
        raise ValueError("lse must be [tokens, num_q_heads]")
    B = req_idx.numel()
    if qo_indptr.numel() != B + 1 or prefix_len.numel() != B or req_to_token.dim() != 2:
        raise ValueError("qo_indptr must be [batch + 1], prefix_len [batch] and req_to_token [requests, stride]")
    # an empty tensor has no address, and without one the call is that of chains
    if tree_mask is not None and (tree_mask.dim() != 2 or tree_mask.shape[0] != q.shape[0] or tree_mask.shape[1] == 0):
        raise ValueError("tree_mask must be [tokens, words], words at least 1")
    words = 0 if tree_mask is None else tree_mask.shape[1]
    # empty tensors have no address; without tokens or requests there is nothing to do
    return words, B, 0 if workspace is None else workspace.numel(), B > 0 and q.shape[0] > 0


def rx_attn_tree(k_pool, v_pool, q, o, lse, qo_indptr, req_idx, prefix_len, tree_mask, req_to_token,
                 max_tree_len: int, sm_scale: float, workspace, dev_status=None, stream=None, layer: int = 0) -> None:
    """Attention of drafted trees: q, o bf16 [tokens, Hq, d], request b's
    drafted tokens at rows qo_indptr[b] .. qo_indptr[b+1]; tree_mask int32
    [tokens, words] (rx_tree_mask_build) or None for chains; workspace uint8
    of rx_attn_tree_workspace(...) bytes.  Without drafted tokens (no rows of q)
    or requests the call does nothing."""
    pool = make_pool(k_pool, v_pool, layer)
    if q.dim() == 3 and q.shape[2] != pool.head_dim:
        raise ValueError("q and the pools must have the same head_dim")
    words, B, ws_bytes, any_work = _tree_args(q, o, lse, qo_indptr, req_idx, prefix_len, tree_mask, req_to_token,
                                              workspace, dev_status)
    if not any_work:
        return
    _check(_lib.rx_attn_tree(ctypes.byref(pool), _ptr(q), _ptr(o), _ptr(lse), q.shape[1], _ptr(qo_indptr),
                             _ptr(req_idx), _ptr(prefix_len), _ptr(tree_mask), words, _ptr(req_to_token),
                             req_to_token.shape[1], B, int(max_tree_len), _ptr(workspace), ws_bytes, float(sm_scale),
                             _ptr(dev_status), _stream(stream)))


def rx_attn_tree_fp8(k_pool, v_pool, k_scale: float, v_scale: float, q, o, lse, qo_indptr, req_idx, prefix_len,
                     tree_mask, req_to_token, max_tree_len: int, sm_scale: float, workspace, dev_status=None,
                     stream=None, layer: int = 0) -> None:
    """rx_attn_tree over uint8 E4M3 pools ([L,] S, Hkv, d) with per-pool scales."""
    torch = _torch()
    _dev(k_pool, torch.uint8, "k_pool")
    _dev(v_pool, torch.uint8, "v_pool")
    S, hkv, d, L = _pool_dims(k_pool, v_pool, layer)
    if q.dim() == 3 and q.shape[2] != d:
        raise ValueError("q and the pools must have the same head_dim")
    words, B, ws_bytes, any_work = _tree_args(q, o, lse, qo_indptr, req_idx, prefix_len, tree_mask, req_to_token,
                                              workspace, dev_status)
    if not any_work:
        return
    pool = KVPoolFp8(k_pool.data_ptr(), v_pool.data_ptr(), S, hkv, d, float(k_scale), float(v_scale), L, int(layer))
    _check(_lib.rx_attn_tree_fp8(ctypes.byref(pool), _ptr(q), _ptr(o), _ptr(lse), q.shape[1], _ptr(qo_indptr),
                                 _ptr(req_idx), _ptr(prefix_len), _ptr(tree_mask), words, _ptr(req_to_token),
                                 req_to_token.shape[1], B, int(max_tree_len), _ptr(workspace), ws_bytes,
                                 float(sm_scale), _ptr(dev_status), _stream(stream)))


class LogitsRules:
    """What rx_logits_process applies to a batch's logits (rx_logits_rules):
    CUDA tensors, each optional, kept alive here.  Their contents may change
    between calls; their sizes may not.  They are checked here, once, not at
    each call.  hist may be longer than its lists, so that they can grow in
    place, but request b's list ends where that of b + 1 starts: a list that
    grows moves those behind it.

    hist int32 [tokens], hist_ptr int64 [n_req + 1], prompt_len int32
    [n_req]; repetition, frequency, presence fp32 [n_req]; bias_tok int32 and
    bias_val fp32 [entries], bias_ptr int64 [n_req + 1]; for drafted trees
    qo_indptr int32 [n_req + 1], draft_tok int32 [rows], tree_mask int32
    [rows, words]; allow int32 [mask rows, ceil(vocab / 128) * 4] (Fsm.mask),
    allow_row int32 [rows]."""

    def __init__(self, n_req: int, vocab: int, hist=None, hist_ptr=None, prompt_len=None, repetition=None,
                 frequency=None, presence=None, bias_tok=None, bias_val=None, bias_ptr=None, qo_indptr=None,
                 draft_tok=None, tree_mask=None, allow=None, allow_row=None):
        torch = _torch()
        self.n_req, self.vocab = int(n_req), int(vocab)
        i32, i64, f32 = torch.int32, torch.int64, torch.float32
        want = (("hist", hist, i32, None), ("hist_ptr", hist_ptr, i64, n_req + 1), ("prompt_len", prompt_len, i32, n_req),
                ("repetition", repetition, f32, n_req), ("frequency", frequency, f32, n_req),
                ("presence", presence, f32, n_req), ("bias_tok", bias_tok, i32, None),
                ("bias_val", bias_val, f32, None), ("bias_ptr", bias_ptr, i64, n_req + 1),
                ("qo_indptr", qo_indptr, i32, n_req + 1), ("draft_tok", draft_tok, i32, None),
                ("tree_mask", tree_mask, i32, None), ("allow", allow, i32, None), ("allow_row", allow_row, i32, None))
        self._keep = []
        for name, t, dt, size in want:
            _dev(t, dt, name)
            if t is not None and size is not None and t.numel() != size:
                raise ValueError(f"LogitsRules: {name} must have {size} entries")
            self._keep.append(t)
        if (hist is None) != (hist_ptr is None):
            raise ValueError("LogitsRules: hist and hist_ptr go together")
        if len({bias_tok is None, bias_val is None, bias_ptr is None}) != 1 or \
                (bias_tok is not None and bias_tok.numel() != bias_val.numel()):
            raise ValueError("LogitsRules: bias_tok, bias_val and bias_ptr go together")
        if (allow is None) != (allow_row is None):
            raise ValueError("LogitsRules: allow and allow_row go together")
        if draft_tok is not None and qo_indptr is None:
            raise ValueError("LogitsRules: draft_tok needs qo_indptr")
        if allow is not None and (allow.dim() != 2 or allow.shape[1] != (self.vocab + 127) // 128 * 4):
            raise ValueError("LogitsRules: allow must be [mask rows, ceil(vocab / 128) * 4]")
        if allow is not None and allow.shape[0] == 0:
            raise ValueError("LogitsRules: allow must have a mask row")
        if tree_mask is not None and (tree_mask.dim() != 2 or tree_mask.shape[1] == 0):
            raise ValueError("LogitsRules: tree_mask must be [rows, words], words at least 1")
        # rows the per-row tensors hold: rx_logits_process checks them against the logits
        self.row_tensors = [t for t in (draft_tok, tree_mask, allow_row) if t is not None]

        def p(t):
            return None if t is None or t.numel() == 0 else t.data_ptr()

        empty = torch.zeros(1, dtype=i32, device="cuda") if any(t is not None and t.numel() == 0
                                                                for t in (hist, bias_tok)) else None
        if empty is not None:  # lists without entries still need an address
            self._keep.append(empty)

        def q(t):
            return None if t is None else (t if t.numel() else empty).data_ptr()

        self.struct = LogitsRulesStruct(self.n_req, self.vocab, q(hist), p(hist_ptr), p(prompt_len), p(repetition),
                                        p(frequency), p(presence), p(bias_ptr), q(bias_tok), q(bias_val),
                                        p(qo_indptr), p(draft_tok), p(tree_mask),
                                        0 if tree_mask is None else tree_mask.shape[1],
                                        0 if allow is None else allow.shape[0], p(allow), p(allow_row))


def _logit_rows(t, name, vocab):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if t.dim() != 2 or t.shape[1] < vocab or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: must be [rows, >= vocab] with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), vocab)


def rx_logits_process(rules: LogitsRules, logits, out, dev_status=None, stream=None) -> None:
    """Penalties, biases and grammar masks: logits fp32 or bf16 [rows, >= V],
    out fp32 [rows, >= V] (may be logits itself)."""
    torch = _torch()
    ls, os_ = _logit_rows(logits, "logits", rules.vocab), _logit_rows(out, "out", rules.vocab)
    if logits.dtype not in (torch.float32, torch.bfloat16) or out.dtype != torch.float32:
        raise TypeError("rx_logits_process: logits must be float32 or bfloat16, out float32")
    _dev(dev_status, torch.int32, "dev_status")
    rows = logits.shape[0]
    if out.shape[0] != rows or any(t.shape[0] < rows for t in rules.row_tensors):
        raise ValueError("rx_logits_process: logits, out, draft_tok, tree_mask and allow_row must have the same rows")
    _check(_lib.rx_logits_process(ctypes.byref(rules.struct), _ptr(logits), int(logits.dtype == torch.bfloat16), ls,
                                  _ptr(out), os_, rows, _ptr(dev_status), _stream(stream)))
