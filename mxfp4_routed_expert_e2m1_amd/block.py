"""The operators around the routed experts: block norms with gate and
residual, scored routing, int8 linear layers.

Like the rest of the binding, every function has the name of the C entry point
it calls and only marshals arguments; a non-zero status raises MoeError.
Element types and devices, which the C side cannot see, are checked here and
raise TypeError or ValueError.  A call runs on the GPU that holds its tensors,
all on the same one, also where another is current.  A call with `stream` (of
that GPU) runs on it, and what it was not given (outputs, workspaces) it
allocates as under torch.cuda.stream(stream).
"""
from __future__ import annotations

import ctypes as C

import torch

P, I, I64, SZ, F = C.c_void_p, C.c_int, C.c_int64, C.c_size_t, C.c_float

EXPORTS = ["moe_norm_pre", "moe_norm_post", "moe_route_scored",
           "moe_route_scored_workspace_bytes", "moe_quant_row_q8", "moe_linear_q8",
           "moe_linear_q8_workspace_bytes"]

MOE_TYPE_F32, MOE_TYPE_BF16 = 0, 1
MOE_QUANT_NONE, MOE_QUANT_BLOCK, MOE_QUANT_ROW = 0, 1, 2
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2 = 0, 1

_TYPES = {torch.float32: MOE_TYPE_F32, torch.bfloat16: MOE_TYPE_BF16}
_F32, _INT8 = {torch.float32: MOE_TYPE_F32}, {torch.int8: 0}
_QUANT = {None: MOE_QUANT_NONE, "block": MOE_QUANT_BLOCK, "row": MOE_QUANT_ROW}
_SCORE = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
_GROUP = {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP2}


_MOST = 2**31 - 1  # of a C int, which ctypes would cut larger numbers to without an error


class moe_norm_t(C.Structure):
    _fields_ = [("d_model", I), ("post_norm", I), ("eps", F), ("residual_scale", F),
                ("pre_w", P), ("post_w", P)]


class moe_router_rule_t(C.Structure):
    _fields_ = [("n_experts", I), ("top_k", I), ("n_groups", I), ("top_groups", I),
                ("score", I), ("group_score", I), ("renorm", I), ("scale", F), ("bias", P)]


class moe_linear_t(C.Structure):
    _fields_ = [("n_out", I), ("d_in", I), ("w", P), ("ld_w", I64), ("w_scales", P),
                ("bias", P)]


def declare(L):
    """Argument types of this module's entry points on the loaded library."""
    global _lib
    norm, rule, lin = C.POINTER(moe_norm_t), C.POINTER(moe_router_rule_t), C.POINTER(moe_linear_t)
    out = [P, I, I64, I, P, I64, P, I64]
    L.moe_norm_pre.argtypes = [norm, P, I, I64, I] + out + [P]
    L.moe_norm_post.argtypes = ([norm, P, I, I64, P, I, I64, P, I, I64, I64, I, P, I64, norm]
                                + out + [P])
    L.moe_route_scored_workspace_bytes.argtypes = [rule, I]
    L.moe_route_scored.argtypes = [rule, P, I, I64, I, P, P, P, P, P, P, SZ, P]
    L.moe_quant_row_q8.argtypes = [P, I, I64, I, I, P, I64, P, P]
    L.moe_linear_q8_workspace_bytes.argtypes = [lin, I]
    L.moe_linear_q8.argtypes = [lin, P, I64, P, I, P, I, I64, P, SZ, P]
    for f in EXPORTS:
        getattr(L, f).restype = SZ if f.endswith("_bytes") else I
    _lib = L


_lib = None  # set by declare()


def _load():
    import mxfp4_routed_expert_e2m1_amd as m
    m.lib()
    return _lib


def _fail(fn, rc):
    import mxfp4_routed_expert_e2m1_amd as m
    raise m.MoeError(fn, rc)


# The raw handle of torch's current stream on a GPU, and the current GPU.  Making the stream
# object costs 2 us, about what the launch does, so torch's own shortcuts are taken where it has
# them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda gpu: torch.cuda.current_stream(gpu).cuda_stream)
_current_gpu = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _given(stream, gpu):
    """Handle of a caller's stream for work on a GPU."""
    if gpu >= 0 and getattr(stream, "device_index", gpu) != gpu:
        raise ValueError(f"stream: of GPU {stream.device_index}, the tensors are on GPU {gpu}")
    return stream.cuda_stream


def _gpu(*tensors):
    """The first tensor's GPU (-1: host memory; None without a tensor)."""
    for t in tensors:
        if t is not None:
            return t.get_device()
    return None


def _refuse_gpu(name, t, gpu):
    if not t.is_cuda:
        raise ValueError(f"{name}: not a GPU tensor")
    raise ValueError(f"{name}: on GPU {t.get_device()}, need GPU {gpu} as the other tensors")


def _same_gpu(name, have, gpu):
    """A descriptor's tensors are on the call's GPU."""
    if have != gpu and have is not None:
        raise ValueError(f"{name}: its tensors are on GPU {have}, the call's on GPU {gpu}")


def _rows(name, t, gpu, shape=None, types=_TYPES):
    """(pointer, type, leading dimension) of a 2-d tensor of contiguous rows on a GPU
    (row-strided views are fine).  A single row needs no leading dimension: any aligned one."""
    kind, sh, st = types.get(t.dtype), t.shape, t.stride()
    if (kind is None or len(st) != 2 or (st[1] != 1 and sh[1] > 1) or t.get_device() != gpu
            or gpu < 0 or sh[0] > _MOST or sh[1] > _MOST
            or (shape is not None and sh != shape)):
        _refuse_rows(name, t, gpu, shape, types)
    return t.data_ptr(), kind, st[0] if sh[0] > 1 else (sh[1] + 15) // 16 * 16


def _refuse_rows(name, t, gpu, shape, types):
    if t.dtype not in types:
        raise TypeError(f"{name}: {t.dtype} is not one of {[str(d) for d in types]}")
    if t.get_device() != gpu or gpu < 0:
        _refuse_gpu(name, t, gpu)
    if max(t.shape, default=0) > _MOST:
        raise ValueError(f"{name}: {list(t.shape)} is more than {_MOST} rows or columns")
    raise ValueError(f"{name}: need contiguous rows {list(shape) if shape else '[rows][cols]'}, "
                     f"got {list(t.shape)} with strides {t.stride()}")


def _vec(name, t, n, gpu, dtype=torch.float32, least=False):
    """Pointer of a contiguous tensor of n (or, with `least`, at least n) elements, or None."""
    if t is None:
        return None
    have = t.numel()
    if (t.dtype != dtype or (have != n and not (least and have > n)) or t.get_device() != gpu
            or gpu < 0 or not t.is_contiguous()):
        if t.dtype != dtype:
            raise TypeError(f"{name}: {t.dtype}, need {dtype}")
        if t.is_cuda and t.get_device() != gpu:
            _refuse_gpu(name, t, gpu)
        raise ValueError(f"{name}: need {n} contiguous elements on the GPU")
    return t.data_ptr()


def _int(name, v):
    if not -_MOST <= v <= _MOST:
        raise ValueError(f"{name}: {v} is more than {_MOST}")
    return v


def _workspace(ws, gpu):
    """Pointer and bytes of a workspace, which the kernels fill from its first byte to its last."""
    n = ws.nbytes
    if n and (ws.get_device() != gpu or not ws.is_contiguous()):
        raise ValueError(f"ws: need a contiguous tensor on GPU {gpu}")
    return ws.data_ptr(), n


def _kept(*tensors):
    """The tensors' memory as it is now, kept alive (assigning to a tensor's .data leaves it)."""
    return tuple(None if t is None else t.detach() for t in tensors)


# --------------------------------------------------------------------- norms
class Norm:
    """moe_norm_t with its weights (f32 [d_model] or None): pre_w of the norm
    before a block, post_w and post_norm of the norm after one.  Like the
    other descriptors it reads its tensors' memory as it was given."""

    def __init__(self, d_model, pre_w=None, post_w=None, post_norm=True, eps=1e-6,
                 residual_scale=1.0):
        self.tensors = _kept(pre_w, post_w)
        self.d_model = d_model
        self.gpu = gpu = _gpu(pre_w, post_w)
        self.c = moe_norm_t(_int("d_model", d_model), int(post_norm), eps, residual_scale,
                            _vec("pre_w", pre_w, d_model, gpu),
                            _vec("post_w", post_w, d_model, gpu))
        self.ref = C.byref(self.c)


def _norm_out(like, gpu, h, h_dtype, quant, q, qs):
    """Output buffers of a norm and their C arguments."""
    shape = like.shape
    if h is None:
        h = torch.empty(shape, dtype=h_dtype or like.dtype, device=like.device)
    if h is False:
        h, ha = None, (None, 0, 0)
    else:
        ha = _rows("h", h, gpu, shape)
    if quant is None:
        return h, None, None, ha + (0, None, 0, None, 0)
    if quant not in _QUANT:
        raise ValueError(f"quant: {quant!r} is not one of {list(_QUANT)}")
    rows, cols = shape
    if q is None:
        q = codes_buffer(rows, cols, like.device)
    n = cols // 32 if quant == "block" else 1
    if qs is None:
        qs = torch.empty((rows, n) if quant == "block" else rows, device=like.device)
    qp, _, ld_q = _rows("q", q, gpu, shape, _INT8)
    if quant == "block":
        qsp, _, ld_qs = _rows("qs", qs, gpu, (rows, n), _F32)
    else:
        qsp, ld_qs = _vec("qs", qs, rows, gpu), 1
    return h, q, qs, ha + (_QUANT[quant], qp, ld_q, qsp, ld_qs)


def _codes_missing(quant, q, qs):
    return quant is not None and (q is None or qs is None)


def moe_norm_pre(norm, x, h=None, h_dtype=None, quant=None, q=None, qs=None, stream=None):
    """h = rms(x) * pre_w of x [rows][d_model] (f32 or bf16).  h: the tensor to
    fill, None (allocated; h_dtype, by default x's type) or False (codes
    only).  quant: None, "block" (codes as moe_quant_act_q8's, for the routed
    experts) or "row" (as moe_quant_row_q8's, for moe_linear_q8).  Returns h,
    or (h, q, qs) with quant."""
    gpu = x.get_device()
    if stream is not None and (h is None or _codes_missing(quant, q, qs)):
        _given(stream, gpu)
        with torch.cuda.stream(stream):
            return moe_norm_pre(norm, x, h, h_dtype, quant, q, qs)
    if gpu >= 0 and gpu != _current_gpu():
        with torch.cuda.device(gpu):
            return moe_norm_pre(norm, x, h, h_dtype, quant, q, qs, stream)
    xa = _rows("x", x, gpu)
    rows, cols = x.shape
    if cols != norm.d_model:
        raise ValueError(f"x: {cols} columns, the norm has d_model {norm.d_model}")
    _same_gpu("norm", norm.gpu, gpu)
    h, q, qs, out = _norm_out(x, gpu, h, h_dtype, quant, q, qs)
    rc = (_lib or _load()).moe_norm_pre(
        norm.ref, *xa, rows, *out, _given(stream, gpu) if stream else _raw_stream(gpu))
    if rc:
        _fail("moe_norm_pre", rc)
    return h if quant is None else (h, q, qs)


_NO_GATE = (None, 0, 0, 0)


def _gate_args(gate, gpu, shape):
    kind, sh, st = _TYPES.get(gate.dtype), gate.shape, gate.stride()
    if kind is None:
        raise TypeError(f"gate: {gate.dtype} is not one of {[str(d) for d in _TYPES]}")
    if gate.get_device() != gpu:
        _refuse_gpu("gate", gate, gpu)
    if len(sh) < 2:
        sh, st = (1,) * (2 - len(sh)) + tuple(sh), (0,) * (2 - len(st)) + tuple(st)
    if len(sh) != 2 or sh[0] not in (1, shape[0]) or sh[1] not in (1, shape[1]):
        raise ValueError(f"gate: {tuple(gate.shape)} does not broadcast to {tuple(shape)}")
    return gate.data_ptr(), kind, st[0] if sh[0] > 1 else 0, st[1] if sh[1] > 1 else 0


def moe_norm_post(norm, y, residual, gate=None, out=None, next_norm=None, h=None, h_dtype=None,
                  quant=None, q=None, qs=None, stream=None):
    """out = residual_scale * residual + gate * b, b = rms(y) * post_w (or y
    without post_norm).  gate: None or f32/bf16 that broadcasts to
    [rows][d_model] (a number, per channel, per token or per element).  out is
    of residual's type and may be residual itself.  With next_norm, also the
    next block's h = rms(out) * pre_w in the same pass; h, h_dtype (default:
    residual's type), quant, q, qs as for moe_norm_pre.  Returns out, (out, h)
    with next_norm, (out, h, q, qs) with quant too."""
    gpu = y.get_device()
    if stream is not None and (out is None or next_norm is not None and (
            h is None or _codes_missing(quant, q, qs))):
        _given(stream, gpu)
        with torch.cuda.stream(stream):
            return moe_norm_post(norm, y, residual, gate, out, next_norm, h, h_dtype, quant, q,
                                 qs)
    if gpu >= 0 and gpu != _current_gpu():
        with torch.cuda.device(gpu):
            return moe_norm_post(norm, y, residual, gate, out, next_norm, h, h_dtype, quant, q,
                                 qs, stream)
    shape = y.shape
    ya, ra = _rows("y", y, gpu), _rows("residual", residual, gpu, shape)
    if shape[1] != norm.d_model:
        raise ValueError(f"y: {shape[1]} columns, the norm has d_model {norm.d_model}")
    _same_gpu("norm", norm.gpu, gpu)
    if out is None:
        out = torch.empty(shape, dtype=residual.dtype, device=y.device)
    op, ot, ld_out = _rows("out", out, gpu, shape)
    if ot != ra[1]:
        raise TypeError(f"out: {out.dtype}, the residual is {residual.dtype}")
    if next_norm is None:
        if quant is not None or (h is not None and h is not False):
            raise ValueError("h and codes belong to next_norm, which is None")
        nx, nargs = None, (None, 0, 0, 0, None, 0, None, 0)
    else:
        _same_gpu("next_norm", next_norm.gpu, gpu)
        h, q, qs, nargs = _norm_out(residual, gpu, h, h_dtype, quant, q, qs)
        nx = next_norm.ref
    rc = (_lib or _load()).moe_norm_post(
        norm.ref, *ya, *ra, *(_NO_GATE if gate is None else _gate_args(gate, gpu, shape)),
        shape[0], op, ld_out, nx, *nargs, _given(stream, gpu) if stream else _raw_stream(gpu))
    if rc:
        _fail("moe_norm_post", rc)
    if next_norm is None:
        return out
    return (out, h) if quant is None else (out, h, q, qs)


# ------------------------------------------------------------------- routing
class RouterRule:
    """moe_router_rule_t: score "softmax" or "sigmoid", bias f32 [n_experts]
    or None (added for the choice, not in the weights), group_score "max" or
    "top2", renorm and scale of the weights."""

    def __init__(self, n_experts, top_k, score="sigmoid", bias=None, n_groups=1, top_groups=None,
                 group_score="top2", renorm=True, scale=1.0):
        if score not in _SCORE or group_score not in _GROUP:
            raise ValueError(f"score {score!r} / group_score {group_score!r}: need one of "
                             f"{list(_SCORE)} / {list(_GROUP)}")
        self.tensors = _kept(bias)
        self.n_experts, self.top_k, self.gpu = n_experts, top_k, _gpu(bias)
        top_groups = n_groups if top_groups is None else top_groups
        self.c = moe_router_rule_t(_int("n_experts", n_experts), _int("top_k", top_k),
                                   _int("n_groups", n_groups), _int("top_groups", top_groups),
                                   _SCORE[score], _GROUP[group_score], int(renorm), scale,
                                   _vec("bias", bias, n_experts, self.gpu))
        self.ref = C.byref(self.c)


class RouteOutputs(tuple):
    """Buffers (ids, w, counts, offsets, sorted) of a routing call, checked when they are made, for
    callers that keep them: all the checks of five tensors are a fifth of a decode call's host
    time.  A call looks whether they are still where they were and of the size they were, and
    otherwise checks them again."""

    def __new__(cls, ids, w, counts, offsets, srt):
        self = super().__new__(cls, (ids, w, counts, offsets, srt))
        rows, k = self.shape = ids.shape
        E, gpu, i32 = counts.numel(), ids.get_device(), torch.int32
        self.key = (rows, E, k, gpu)
        self.ptrs = (_vec("ids", ids, rows * k, gpu, i32), _vec("w", w, rows * k, gpu),
                     _vec("counts", counts, E, gpu, i32),
                     _vec("offsets", offsets, E + 1, gpu, i32),
                     _vec("sorted", srt, rows * k, gpu, i32, least=True))
        self.sizes = (w.numel(), E, E + 1, srt.numel())
        return self

    def __reduce__(self):  # (a copy of the buffers has addresses of its own)
        return RouteOutputs, tuple(self)

    def unchanged(self):
        ids, w, counts, offsets, srt = self
        return (ids.shape == self.shape
                and (w.numel(), counts.numel(), offsets.numel(), srt.numel()) == self.sizes
                and (ids.data_ptr(), w.data_ptr(), counts.data_ptr(), offsets.data_ptr(),
                     srt.data_ptr()) == self.ptrs)


def route_outputs(rows, n_experts, top_k, device="cuda"):
    """New buffers for a routing call."""
    i32 = torch.int32
    return RouteOutputs(torch.empty((rows, top_k), dtype=i32, device=device),
                        torch.empty((rows, top_k), dtype=torch.float32, device=device),
                        torch.empty(n_experts, dtype=i32, device=device),
                        torch.empty(n_experts + 1, dtype=i32, device=device),
                        torch.empty(rows * top_k, dtype=i32, device=device))


def moe_route_scored_workspace_bytes(rule, rows):
    """Bytes that serve moe_route_scored for any number of rows up to `rows`."""
    return int((_lib or _load()).moe_route_scored_workspace_bytes(rule.ref, _int("rows", rows)))


def moe_route_scored(rule, logits, out=None, ws=None, stream=None):
    """Picks, weights and grouping of logits [rows][n_experts] (f32 or bf16)
    under a RouterRule.  Returns (ids, w, counts, offsets, sorted), as
    moe_route_group does; a slot without an expert holds id -1 and weight 0."""
    gpu = logits.get_device()
    if stream is not None and (out is None or ws is None):
        _given(stream, gpu)
        with torch.cuda.stream(stream):
            return moe_route_scored(rule, logits, out, ws)
    if gpu >= 0 and gpu != _current_gpu():
        with torch.cuda.device(gpu):
            return moe_route_scored(rule, logits, out, ws, stream)
    la = _rows("logits", logits, gpu)
    rows, E, k = logits.shape[0], rule.n_experts, rule.top_k
    if logits.shape[1] != E:
        raise ValueError(f"logits: {logits.shape[1]} columns, the rule has {E} experts")
    _same_gpu("rule", rule.gpu, gpu)
    if out is None:
        out = route_outputs(rows, E, k, logits.device)
    elif type(out) is not RouteOutputs or not out.unchanged():
        out = RouteOutputs(*out)
    if out.key != (rows, E, k, gpu):
        raise ValueError(f"out: buffers of {out.key} rows, experts, picks and GPU, need "
                         f"{(rows, E, k, gpu)}")
    if ws is None:
        ws = torch.empty(moe_route_scored_workspace_bytes(rule, rows), dtype=torch.uint8,
                         device=logits.device)
    rc = (_lib or _load()).moe_route_scored(
        rule.ref, *la, rows, *out.ptrs, *_workspace(ws, gpu),
        _given(stream, gpu) if stream else _raw_stream(gpu))
    if rc:
        _fail("moe_route_scored", rc)
    return out


# ------------------------------------------------------------- linear layers
def codes_buffer(rows, cols, device="cuda"):
    """int8 [rows][cols] with rows a multiple of 128 bytes apart: the int8 calls need 16, and
    rows that start a cache line are read fastest."""
    return torch.empty((rows, (cols + 127) // 128 * 128), dtype=torch.int8,
                       device=device)[:, :cols]


def moe_quant_row_q8(x, q=None, scales=None, stream=None):
    """int8 codes and one scale per row of x [rows][cols] (f32 or bf16): of
    activations per token, or of weights [n_out][d_in] per channel.  Returns
    (q, scales); a q allocated here has 16-byte-aligned rows."""
    gpu = x.get_device()
    if stream is not None and (q is None or scales is None):
        _given(stream, gpu)
        with torch.cuda.stream(stream):
            return moe_quant_row_q8(x, q, scales)
    if gpu >= 0 and gpu != _current_gpu():
        with torch.cuda.device(gpu):
            return moe_quant_row_q8(x, q, scales, stream)
    xa = _rows("x", x, gpu)
    rows, cols = shape = x.shape
    if q is None:
        q = codes_buffer(rows, cols, x.device)
    if scales is None:
        scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    qp, _, ld_q = _rows("q", q, gpu, shape, _INT8)
    rc = (_lib or _load()).moe_quant_row_q8(
        *xa, rows, cols, qp, ld_q, _vec("scales", scales, rows, gpu),
        _given(stream, gpu) if stream else _raw_stream(gpu))
    if rc:
        _fail("moe_quant_row_q8", rc)
    return q, scales


def _codes(name, t, gpu):
    """int8 rows that are readable up to the next multiple of 16 codes."""
    ptr, _, ld = _rows(name, t, gpu, None, _INT8)
    rows, cols = t.shape
    if cols % 16 and rows:
        end = t.storage_offset() + (rows - 1) * t.stride(0) + (cols + 15) // 16 * 16
        if end > t.untyped_storage().nbytes():
            raise ValueError(f"{name}: the last row has to be readable up to a multiple of 16 "
                             "codes (codes_buffer allocates such rows)")
    return ptr, ld


class Linear:
    """moe_linear_t: int8 codes w [n_out][d_in] (16-byte-aligned rows, e.g.
    from moe_quant_row_q8 of the weights), w_scales f32 [n_out], bias f32
    [n_out] or None."""

    def __init__(self, w, w_scales, bias=None):
        self.tensors = _kept(w, w_scales, bias)
        self.n_out, self.d_in = w.shape
        self.gpu = gpu = w.get_device()
        self.c = moe_linear_t(self.n_out, self.d_in, *_codes("w", w, gpu),
                              _vec("w_scales", w_scales, self.n_out, gpu),
                              _vec("bias", bias, self.n_out, gpu))
        self.ref = C.byref(self.c)


def moe_linear_q8_workspace_bytes(linear, rows):
    """Bytes that serve moe_linear_q8 for any number of rows up to `rows`."""
    return int((_lib or _load()).moe_linear_q8_workspace_bytes(linear.ref, _int("rows", rows)))


def moe_linear_q8(linear, q, qs, y=None, dtype=torch.bfloat16, ws=None, stream=None):
    """y[t][n] = qs[t] w_scales[n] sum_k q[t][k] w[n][k] (+ bias[n]) of int8
    codes q [rows][d_in] (16-byte-aligned rows) and their row scales.  y: the
    f32 or bf16 tensor to fill, or None (allocated with `dtype`)."""
    gpu = q.get_device()
    if stream is not None and (y is None or ws is None):
        _given(stream, gpu)
        with torch.cuda.stream(stream):
            return moe_linear_q8(linear, q, qs, y, dtype, ws)
    if gpu >= 0 and gpu != _current_gpu():
        with torch.cuda.device(gpu):
            return moe_linear_q8(linear, q, qs, y, dtype, ws, stream)
    qp, ld_q = _codes("q", q, gpu)
    rows, cols = q.shape
    if cols != linear.d_in:
        raise ValueError(f"q: {cols} columns, the layer has d_in {linear.d_in}")
    _same_gpu("linear", linear.gpu, gpu)
    if y is None:
        y = torch.empty((rows, linear.n_out), dtype=dtype, device=q.device)
    if ws is None:
        ws = torch.empty(moe_linear_q8_workspace_bytes(linear, rows), dtype=torch.uint8,
                         device=q.device)
    rc = (_lib or _load()).moe_linear_q8(
        linear.ref, qp, ld_q, _vec("qs", qs, rows, gpu), rows,
        *_rows("y", y, gpu, (rows, linear.n_out)), *_workspace(ws, gpu),
        _given(stream, gpu) if stream else _raw_stream(gpu))
    if rc:
        _fail("moe_linear_q8", rc)
    return y
