"""Attention over a cache held in 4 bits: rotary positions, the cache's writing
and reading, and the attention of a ragged batch's rows over it.

The same manner as in block.py: every function has the name of the C entry
point it calls and only marshals arguments, runs on the GPU that holds its
tensors, and with `stream` on that stream; what the C side cannot see is
checked here and raises TypeError or ValueError.

    cache = KVCache(n_pages, page, kv_heads, head_dim)
    q, k  = moe_rope(...)                 # or one call over neighbouring heads
    moe_kv_write(cache, k, v, slots)
    out   = moe_attn_cache(attn, cache, q, table, kv_lens)
"""
from __future__ import annotations

import ctypes as C

import torch

from . import block
from .block import (F, I, I64, P, SZ, _MOST, _TYPES, _current_gpu, _fail, _given, _gpu, _int, _kept,
                    _raw_stream, _refuse_gpu, _same_gpu, _vec, _workspace)

EXPORTS = ["moe_rope", "moe_kv_cache_bytes", "moe_kv_write", "moe_kv_read", "moe_attn_cache",
           "moe_attn_cache_workspace_bytes"]

_I32 = torch.int32


class moe_rope_t(C.Structure):
    _fields_ = [("rot_dim", I), ("n_axes", I), ("interleaved", I), ("scale", F), ("steps", P),
                ("axes", P)]


class moe_kv_cache_t(C.Structure):
    _fields_ = [("n_heads", I), ("head_dim", I), ("page", I), ("n_pages", I), ("data", P)]


class moe_attn_t(C.Structure):
    _fields_ = [("n_heads", I), ("window", I), ("scale", F), ("softcap", F), ("slopes", P)]


def declare(L):
    """Argument types of this module's entry points on the loaded library."""
    global _lib
    rope, cache, attn = C.POINTER(moe_rope_t), C.POINTER(moe_kv_cache_t), C.POINTER(moe_attn_t)
    heads = [P, I64, I64]
    L.moe_rope.argtypes = [rope, P, I, I64, I64, I, I, I, P, I64] + heads + [P]
    L.moe_kv_cache_bytes.argtypes = [cache]
    L.moe_kv_write.argtypes = [cache] + heads + heads + [I, I, P, P]
    L.moe_kv_read.argtypes = [cache, P, I] + heads + heads + [I, P]
    L.moe_attn_cache_workspace_bytes.argtypes = [attn, cache, I, I]
    L.moe_attn_cache.argtypes = ([attn, cache, P, I, I64, I64, I, P, I, P, P, I64, I, P] + heads
                                 + [P, SZ, P])
    for f in EXPORTS:
        getattr(L, f).restype = SZ if f.endswith("_bytes") else I
    _lib = L


_lib = None  # set by declare()


def _load():
    block._load()
    return _lib


def _heads(name, t, gpu, shape=None):
    """(pointer, type, row stride, head stride) of [rows][heads][head_dim] on a GPU, the channels
    of a head contiguous; `shape` is one that has been checked."""
    kind, sh, st = _TYPES.get(t.dtype), t.shape, t.stride()
    if (kind is None or len(st) != 3 or (st[2] != 1 and sh[2] > 1) or t.get_device() != gpu
            or gpu < 0 or (sh != shape if shape else max(sh) > _MOST)):
        _refuse_heads(name, t, gpu, shape)
    return t.data_ptr(), kind, st[0], st[1]


def _refuse_heads(name, t, gpu, shape):
    if t.dtype not in _TYPES:
        raise TypeError(f"{name}: {t.dtype} is not one of {[str(d) for d in _TYPES]}")
    if t.get_device() != gpu or gpu < 0:
        _refuse_gpu(name, t, gpu)
    if max(t.shape, default=0) > _MOST:
        raise ValueError(f"{name}: {list(t.shape)} is more than {_MOST} rows, heads or channels")
    raise ValueError(f"{name}: need {list(shape) if shape else '[rows][heads][head_dim]'} with the "
                     f"channels of a head contiguous, got {list(t.shape)} with strides {t.stride()}")


# ---------------------------------------------------------- rotary positions
# round(2^192 / (2 pi)), from the first 70 digits of pi
_PI_70 = 31415926535897932384626433832795028841971693993751058209749445923078164
_TURN = ((10**70 << 192) + _PI_70) // (2 * _PI_70)


def _step(frequency):
    """Turns per position in units of 2^-64 of a frequency in radians per position, rounded once
    and modulo a turn."""
    num, den = float(frequency).as_integer_ratio()  # (den is a power of two)
    return ((num * _TURN >> den.bit_length() + 126) + 1 >> 1) % 2**64


class Rope:
    """moe_rope_t: inv_freq, the pairs' frequencies in radians per position (numbers or a float
    tensor, rot_dim/2 of them); axes, each pair's axis (None: all 0, or whole numbers below 8);
    interleaved, pairs (2i, 2i+1) instead of (i, i + rot_dim/2); scale, a factor on the rotated
    channels."""

    def __init__(self, inv_freq, axes=None, interleaved=False, scale=1.0, device="cuda"):
        freq = inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else list(inv_freq)
        steps = [_step(f) for f in freq]
        signed = torch.tensor([s - 2**64 if s >= 2**63 else s for s in steps], dtype=torch.int64)
        axes = axes.tolist() if isinstance(axes, torch.Tensor) else axes
        if axes is not None:
            axes = [int(a) for a in axes]
            if len(axes) != len(freq) or not all(0 <= a < 8 for a in axes):
                raise ValueError(f"axes: need {len(freq)} of 0..7, got {axes}")
        self.n_axes = 1 if not axes else 1 + max(axes)
        self.rot_dim = 2 * len(freq)
        self.tensors = (signed.to(device),
                        None if axes is None else torch.tensor(axes, dtype=torch.uint8).to(device))
        self.gpu = gpu = self.tensors[0].get_device()
        n = len(freq)
        self.c = moe_rope_t(self.rot_dim, self.n_axes, int(interleaved), scale,
                            _vec("inv_freq", self.tensors[0], n, gpu, torch.int64),
                            _vec("axes", self.tensors[1], n, gpu, torch.uint8))
        self.ref = C.byref(self.c)


def _positions(positions, rope, rows, gpu):
    sh, st = positions.shape, positions.stride()
    if (st == (1,) and sh[0] == rows and rope.n_axes == 1 and positions.dtype == _I32
            and positions.get_device() == gpu):
        return positions.data_ptr(), 0
    if positions.dtype != _I32:
        raise TypeError(f"positions: {positions.dtype}, need {_I32}")
    if positions.get_device() != gpu:
        _refuse_gpu("positions", positions, gpu)
    if len(sh) == 1 and rope.n_axes == 1:
        sh, st = (1,) + tuple(sh), (0,) + tuple(st)
    if len(sh) != 2 or sh[0] != rope.n_axes or sh[1] != rows or (rows > 1 and st[1] != 1):
        raise ValueError(f"positions: need contiguous [{rope.n_axes}][{rows}], got "
                         f"{list(positions.shape)} with strides {positions.stride()}")
    return positions.data_ptr(), st[0] if rows > 1 or rope.n_axes == 1 else max(st[0], 1)


def moe_rope(rope, x, positions, out=None, stream=None):
    """Rotary positions of x [rows][heads][head_dim] (f32 or bf16): neighbouring query and key
    heads of a fused projection take one call.  positions: int32 [rows], or [n_axes][rows].  out is
    of x's type and may be x itself."""
    gpu = x.get_device()
    if stream is not None and out is None:
        _given(stream, gpu)
        with torch.cuda.stream(stream):
            return moe_rope(rope, x, positions)
    if gpu >= 0 and gpu != _current_gpu():
        with torch.cuda.device(gpu):
            return moe_rope(rope, x, positions, out, stream)
    xp, kind, ld_x, hs_x = _heads("x", x, gpu)
    rows, heads, dim = shape = x.shape
    _same_gpu("rope", rope.gpu, gpu)
    pp, ld_pos = _positions(positions, rope, rows, gpu)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    op, out_kind, ld_out, hs_out = _heads("out", out, gpu, shape)
    if out_kind != kind:
        raise TypeError(f"out: {out.dtype}, x is {x.dtype}")
    rc = (_lib or _load()).moe_rope(
        rope.ref, xp, kind, ld_x, hs_x, rows, heads, dim, pp, ld_pos, op, ld_out, hs_out,
        _given(stream, gpu) if stream else _raw_stream(gpu))
    if rc:
        _fail("moe_rope", rc)
    return out


# ----------------------------------------------------------------- the cache
class KVCache:
    """moe_kv_cache_t with its memory: n_pages pages of `page` tokens, n_heads key heads of
    head_dim channels, 4.25 bits a channel.  data: a uint8 tensor of moe_kv_cache_bytes() to use,
    or None (allocated, zero)."""

    def __init__(self, n_pages, page, n_heads, head_dim, device="cuda", data=None):
        self.n_pages, self.page = n_pages, page
        self.n_heads, self.head_dim = n_heads, head_dim
        self.c = moe_kv_cache_t(_int("n_heads", n_heads), _int("head_dim", head_dim),
                                _int("page", page), _int("n_pages", n_pages), None)
        n = int((_lib or _load()).moe_kv_cache_bytes(C.byref(self.c)))
        if n == 0:
            raise ValueError(f"{n_pages} pages of {page} tokens, {n_heads} heads of {head_dim}: not "
                             "sizes of a cache")
        if data is None:
            data = torch.zeros(n, dtype=torch.uint8, device=device)
        self.tensors = _kept(data)
        self.gpu = data.get_device()
        self.c.data = _vec("data", data, n, self.gpu, torch.uint8)
        self.ref = C.byref(self.c)


def _slots(slots, rows, gpu):
    return _vec("slots", slots, rows, gpu, _I32)


def moe_kv_write(cache, k, v, slots, stream=None):
    """Keys and values k, v [rows][n_heads][head_dim] (f32 or bf16) into slots int32 [rows]: slot
    s is token s % page of page s // page, and a row without one (negative) is skipped."""
    gpu = k.get_device()
    if gpu >= 0 and gpu != _current_gpu():
        with torch.cuda.device(gpu):
            return moe_kv_write(cache, k, v, slots, stream)
    rows = k.shape[0]
    if rows > _MOST:
        raise ValueError(f"k: {rows} is more than {_MOST} rows")
    shape = (rows, cache.n_heads, cache.head_dim)
    kp, kind, ld_k, hs_k = _heads("k", k, gpu, shape)
    vp, v_kind, ld_v, hs_v = _heads("v", v, gpu, shape)
    if v_kind != kind:
        raise TypeError(f"v: {v.dtype}, k is {k.dtype}")
    _same_gpu("cache", cache.gpu, gpu)
    rc = (_lib or _load()).moe_kv_write(
        cache.ref, kp, ld_k, hs_k, vp, ld_v, hs_v, kind, rows, _slots(slots, rows, gpu),
        _given(stream, gpu) if stream else _raw_stream(gpu))
    if rc:
        _fail("moe_kv_write", rc)


def moe_kv_read(cache, slots, k=None, v=None, dtype=torch.bfloat16, stream=None):
    """Keys and values of slots int32 [rows], [rows][n_heads][head_dim] each; a row without a slot
    (negative) is 0.  k, v: the tensors to fill, or None (allocated with `dtype`)."""
    gpu = slots.get_device()
    if stream is not None and (k is None or v is None):
        _given(stream, gpu)
        with torch.cuda.stream(stream):
            return moe_kv_read(cache, slots, k, v, dtype)
    if gpu >= 0 and gpu != _current_gpu():
        with torch.cuda.device(gpu):
            return moe_kv_read(cache, slots, k, v, dtype, stream)
    rows = slots.numel()
    if rows > _MOST:
        raise ValueError(f"slots: {rows} is more than {_MOST}")
    shape = (rows, cache.n_heads, cache.head_dim)
    if k is None:
        k = torch.empty(shape, dtype=dtype if v is None else v.dtype, device=slots.device)
    if v is None:
        v = torch.empty(shape, dtype=k.dtype, device=slots.device)
    kp, kind, ld_k, hs_k = _heads("k", k, gpu, shape)
    vp, v_kind, ld_v, hs_v = _heads("v", v, gpu, shape)
    if v_kind != kind:
        raise TypeError(f"v: {v.dtype}, k is {k.dtype}")
    _same_gpu("cache", cache.gpu, gpu)
    rc = (_lib or _load()).moe_kv_read(
        cache.ref, _slots(slots, rows, gpu), rows, kp, ld_k, hs_k, vp, ld_v, hs_v, kind,
        _given(stream, gpu) if stream else _raw_stream(gpu))
    if rc:
        _fail("moe_kv_read", rc)
    return k, v


# -------------------------------------------------------------- the attention
class Attention:
    """moe_attn_t: n_heads query heads, scale of the scores, softcap (0: none) their bound by a
    tanh, window (0: none) the tokens up to and with its own that a row sees, slopes f32 [n_heads]
    or None a bias of -slope per token of distance."""

    def __init__(self, n_heads, scale, softcap=0.0, window=0, slopes=None):
        self.tensors = _kept(slopes)
        self.n_heads, self.gpu = n_heads, _gpu(slopes)
        self.c = moe_attn_t(_int("n_heads", n_heads), _int("window", window), scale, softcap,
                            _vec("slopes", slopes, n_heads, self.gpu))
        self.ref = C.byref(self.c)


def moe_attn_cache_workspace_bytes(attn, cache, rows, n_seqs):
    """Bytes that serve moe_attn_cache for up to `rows` rows of up to `n_seqs` sequences."""
    gpu = cache.gpu
    if gpu != _current_gpu():
        with torch.cuda.device(gpu):
            return moe_attn_cache_workspace_bytes(attn, cache, rows, n_seqs)
    return int((_lib or _load()).moe_attn_cache_workspace_bytes(
        attn.ref, cache.ref, _int("rows", rows), _int("n_seqs", n_seqs)))


def _table(table, gpu):
    sh, st = table.shape, table.stride()
    if table.dtype != _I32:
        raise TypeError(f"table: {table.dtype}, need {_I32}")
    if table.get_device() != gpu:
        _refuse_gpu("table", table, gpu)
    if len(sh) != 2 or (st[1] != 1 and sh[1] > 1) or max(sh) > _MOST:
        raise ValueError(f"table: need contiguous rows [n_seqs][pages], got {list(sh)} with strides "
                         f"{st}")
    return table.data_ptr(), st[0] if sh[0] > 1 else sh[1], sh[1]


def moe_attn_cache(attn, cache, q, table, kv_lens, q_offsets=None, prefix=None, out=None, ws=None,
                   stream=None):
    """Attention of q [rows][n_heads][head_dim] (f32 or bf16) over the cached tokens of their
    sequences, whose own rows are in the cache already.
      table     int32 [n_seqs][pages]: each sequence's pages in order
      kv_lens   int32 [n_seqs]: its cached tokens
      q_offsets int32 [n_seqs + 1]: its rows, q_offsets[s] .. q_offsets[s+1] - 1; None: one each
      prefix    int32 [n_seqs] or None: so many first tokens are seen by all of its rows
    Chunks of a prompt and single tokens are faster in calls of their own, and with a table of no
    more columns than the longest text needs.  Returns out, of q's type."""
    gpu = q.get_device()
    if stream is not None and (out is None or ws is None):
        _given(stream, gpu)
        with torch.cuda.stream(stream):
            return moe_attn_cache(attn, cache, q, table, kv_lens, q_offsets, prefix, out, ws)
    if gpu >= 0 and gpu != _current_gpu():
        with torch.cuda.device(gpu):
            return moe_attn_cache(attn, cache, q, table, kv_lens, q_offsets, prefix, out, ws,
                                  stream)
    rows = q.shape[0]
    if rows > _MOST:
        raise ValueError(f"q: {rows} is more than {_MOST} rows")
    shape = (rows, attn.n_heads, cache.head_dim)
    qp, kind, ld_q, hs_q = _heads("q", q, gpu, shape)
    _same_gpu("cache", cache.gpu, gpu)
    _same_gpu("attn", attn.gpu, gpu)
    tp, ld_table, pages = _table(table, gpu)
    n_seqs = table.shape[0]
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    op, out_kind, ld_out, hs_out = _heads("out", out, gpu, shape)
    if out_kind != kind:
        raise TypeError(f"out: {out.dtype}, q is {q.dtype}")
    if ws is None:
        ws = torch.empty(moe_attn_cache_workspace_bytes(attn, cache, rows, n_seqs),
                         dtype=torch.uint8, device=q.device)
    rc = (_lib or _load()).moe_attn_cache(
        attn.ref, cache.ref, qp, kind, ld_q, hs_q, rows,
        _vec("q_offsets", q_offsets, n_seqs + 1, gpu, _I32), n_seqs,
        _vec("kv_lens", kv_lens, n_seqs, gpu, _I32), tp, ld_table, pages,
        _vec("prefix", prefix, n_seqs, gpu, _I32), op, ld_out, hs_out, *_workspace(ws, gpu),
        _given(stream, gpu) if stream else _raw_stream(gpu))
    if rc:
        _fail("moe_attn_cache", rc)
    return out
