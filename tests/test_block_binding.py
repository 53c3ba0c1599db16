"""What the binding of the block operators refuses or hands on, with CPU tensors
that say they are on a GPU and a library that only records its calls."""
import contextlib
import copy
import subprocess
import sys
import types

import pytest
import torch

import mxfp4_routed_expert_e2m1_amd as m
from conftest import ROOT
from mxfp4_routed_expert_e2m1_amd import block as b

F32, I8, U8 = torch.float32, torch.int8, torch.uint8


class OnGpu(torch.Tensor):
    """A tensor in host memory that gives itself out as one of GPU `gpu`."""
    gpu = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.gpu

    def __deepcopy__(self, memo):
        t = self.clone()
        t.gpu = self.gpu
        return t


def on(gpu, *shape, dtype=F32):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)
    t.gpu = gpu
    return t


class Recorder:
    """Stands for the loaded library: every entry point succeeds and is noted down, with the
    GPU that was current then."""

    def __init__(self):
        self.calls, self.gpu, self.gpus = [], 0, []

    def __getattr__(self, fn):
        def call(*args):
            if fn.endswith("_bytes"):
                return 64
            self.calls.append((fn, args))
            self.gpus.append(self.gpu)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(b, "_lib", r)
    monkeypatch.setattr(b, "_raw_stream", lambda gpu: 1000 + gpu)
    monkeypatch.setattr(b, "_current_gpu", lambda: r.gpu, raising=False)

    @contextlib.contextmanager
    def device(gpu):
        r.gpu, was = gpu, r.gpu
        yield
        r.gpu = was
    monkeypatch.setattr(torch.cuda, "device", device)
    return r


def a_route(gpu=0, **kw):
    i32 = torch.int32
    out = (on(gpu, 20, 4, dtype=i32), on(gpu, 20, 4), on(gpu, 64, dtype=i32),
           on(gpu, 65, dtype=i32), on(gpu, 80, dtype=i32))
    return m.moe_route_scored(m.RouterRule(64, 4), on(gpu, 20, 64),
                              **{"out": out, "ws": on(gpu, 64, dtype=U8), **kw})


def a_linear(gpu=0, **kw):
    lay = m.Linear(on(gpu, 8, 32, dtype=I8), on(gpu, 8))
    return m.moe_linear_q8(lay, on(gpu, 20, 32, dtype=I8), on(gpu, 20),
                           **{"y": on(gpu, 20, 8), "ws": on(gpu, 64, dtype=U8), **kw})


# ---------------------------------------------------------------- workspaces
@pytest.mark.parametrize("call", [a_route, a_linear])
def test_a_workspace_in_host_memory_is_refused(lib, call):
    with pytest.raises(ValueError):
        call(ws=torch.zeros(64, dtype=U8))
    assert not lib.calls
    call(ws=torch.empty(0, dtype=U8))  # (nothing in it that could be read)
    assert len(lib.calls) == 1


@pytest.mark.parametrize("call", [a_route, a_linear])
def test_a_workspace_with_gaps_is_refused(lib, call):
    with pytest.raises(ValueError):
        call(ws=on(0, 128, dtype=U8)[::2])
    one = on(0, 1, dtype=U8).expand(64)
    one.gpu = 0
    with pytest.raises(ValueError):
        call(ws=one)
    assert not lib.calls


@pytest.mark.parametrize("call,at", [(a_route, -2), (a_linear, -2)])
def test_a_workspace_counts_in_bytes(lib, call, at):
    call(ws=on(0, 16))
    assert lib.calls[0][1][at] == 64


# ------------------------------------------------- buffers that a caller keeps
def addresses(out):
    return tuple(t.data_ptr() for t in out)


def kept(lib):
    return m.RouteOutputs(*a_route())


def test_kept_outputs_that_moved_are_written_where_they_are(lib):
    out = kept(lib)
    out[0].set_(torch.zeros(20, 4, dtype=torch.int32))
    out[1].data = torch.zeros(20, 4)
    a_route(out=out)
    assert lib.calls[-1][1][5:10] == addresses(out)


@pytest.mark.parametrize("i", range(5))
def test_kept_outputs_of_another_size_are_refused(lib, i):
    out = kept(lib)
    n = len(lib.calls)
    out[i].resize_(3, 1)        # in place: the address stays
    with pytest.raises(ValueError):
        a_route(out=out)
    assert len(lib.calls) == n


def test_kept_outputs_that_grow_serve_the_larger_call(lib):
    out = kept(lib)
    for i, shape in ((0, (21, 4)), (1, (21, 4)), (4, (84,))):
        out[i].resize_(shape)
    m.moe_route_scored(m.RouterRule(64, 4), on(0, 21, 64), out=out, ws=on(0, 64, dtype=U8))
    assert lib.calls[-1][1][5:10] == addresses(out)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy])
def test_kept_outputs_can_be_copied(lib, how):
    out = kept(lib)
    other = how(out)
    assert type(other) is m.RouteOutputs
    assert (addresses(other) == addresses(out)) == (how is copy.copy)
    a_route(out=other)
    assert lib.calls[-1][1][5:10] == addresses(other)


# ------------------------------------------------------------------- devices
def a_norm_pre(gpu=0, w=None, **kw):
    return m.moe_norm_pre(m.Norm(64, pre_w=w), on(gpu, 5, 64),
                          **{"h": on(gpu, 5, 64), "quant": "row", "q": on(gpu, 5, 64, dtype=I8),
                             "qs": on(gpu, 5), **kw})


def a_norm_post(gpu=0, w=None, w2=None, **kw):
    kw = {"residual": on(gpu, 5, 64), "out": on(gpu, 5, 64), "h": on(gpu, 5, 64),
          "quant": "block", "q": on(gpu, 5, 64, dtype=I8), "qs": on(gpu, 5, 2), **kw}
    return m.moe_norm_post(m.Norm(64, post_w=w), on(gpu, 5, 64),
                           next_norm=m.Norm(64, pre_w=w2), **kw)


def a_quant(gpu=0, **kw):
    return m.moe_quant_row_q8(on(gpu, 5, 64), **{"q": on(gpu, 5, 64, dtype=I8),
                                                "scales": on(gpu, 5), **kw})


NEW = {a_norm_pre: "h", a_norm_post: "out", a_quant: "q", a_route: "ws", a_linear: "ws"}
CALLS = [a_norm_pre, a_norm_post, a_quant, a_route, a_linear]


@pytest.mark.parametrize("call", CALLS)
def test_the_tensors_gpu_is_current_during_the_call(lib, call):
    call(1)
    call(0)
    assert lib.gpus == [1, 0] and lib.gpu == 0
    assert [args[-1] for _, args in lib.calls] == [1001, 1000]


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_gpu_is_refused(lib, call):
    stream = lambda gpu: types.SimpleNamespace(device_index=gpu, cuda_stream=77)  # noqa: E731
    with pytest.raises(ValueError):
        call(0, stream=stream(1))
    with pytest.raises(ValueError):  # (with a buffer that would be allocated under it)
        call(0, stream=stream(1), **{NEW[call]: None})
    assert not lib.calls
    call(1, stream=stream(1))
    assert lib.gpus == [1] and lib.calls[0][1][-1] == 77


F, R = (on(1, 5, 64), on(1, 5))
Q = on(1, 5, 64, dtype=I8)


@pytest.mark.parametrize("call,kw", [
    (a_norm_pre, {"w": on(1, 64)}), (a_norm_pre, {"h": F}), (a_norm_pre, {"q": Q}),
    (a_norm_pre, {"qs": R}),
    (a_norm_post, {"w": on(1, 64)}), (a_norm_post, {"w2": on(1, 64)}),
    (a_norm_post, {"residual": F}), (a_norm_post, {"gate": on(1, 64)}), (a_norm_post, {"out": F}),
    (a_norm_post, {"h": F}), (a_norm_post, {"q": Q}), (a_norm_post, {"qs": on(1, 5, 2)}),
    (a_quant, {"q": Q}), (a_quant, {"scales": R}),
    (a_route, {"ws": on(1, 64, dtype=U8)}), (a_linear, {"ws": on(1, 64, dtype=U8)}),
    (a_linear, {"y": on(1, 20, 8)})])
def test_tensors_of_two_gpus_are_refused(lib, call, kw):
    with pytest.raises(ValueError):
        call(**kw)
    assert not lib.calls


def test_descriptors_and_kept_outputs_of_another_gpu_are_refused(lib):
    out, ws = m.RouteOutputs(*a_route(1)), on(0, 64, dtype=U8)
    lib.calls.clear()
    z, q, s = on(0, 20, 64), on(0, 20, 32, dtype=I8), on(0, 20)
    lay = m.Linear(on(1, 8, 32, dtype=I8), on(1, 8))
    for f in (lambda: m.moe_route_scored(m.RouterRule(64, 4), z, out=out, ws=ws),
              lambda: m.moe_route_scored(m.RouterRule(64, 4, bias=on(1, 64)), z, ws=ws,
                                         out=a_route()),
              lambda: m.moe_linear_q8(lay, q, s, y=on(0, 20, 8), ws=ws),
              lambda: m.Linear(on(0, 8, 32, dtype=I8), on(1, 8)),
              lambda: m.Linear(on(0, 8, 32, dtype=I8), on(0, 8), on(1, 8)),
              lambda: m.Norm(64, pre_w=on(0, 64), post_w=on(1, 64)),
              lambda: m.RouteOutputs(*[t for t in out[:4]], on(0, 80, dtype=torch.int32))):
        with pytest.raises(ValueError):
            f()
    assert [fn for fn, args in lib.calls] == ["moe_route_scored"]  # a_route()'s own


def test_the_package_needs_no_private_names_of_torch():
    """Without torch's quick ways to the current stream and GPU the package still imports, and
    asks the public ones."""
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from mxfp4_routed_expert_e2m1_amd import block
class Stream:
    cuda_stream = 77
torch.cuda.current_stream = lambda gpu: Stream
assert block._raw_stream(1) == 77 and block._current_gpu is torch.cuda.current_device
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


# ------------------------------------------------------ sizes past 32 bits
BIG = 2**32 + 20  # (its low 32 bits are an ordinary size)


class Says(OnGpu):
    """One that gives itself another shape, its rows without gaps."""
    shape = property(lambda self: torch.Size(self.says))

    def stride(self):
        return (self.says[1], 1)

    def numel(self):
        return self.says[0] * self.says[-1]


def says(*shape, dtype=F32):
    t = torch.zeros(1, dtype=dtype).as_subclass(Says)
    t.says = shape
    return t


def test_sizes_that_c_would_cut_are_refused(lib):
    tall, wide, codes = says(BIG, 64), says(20, BIG), says(BIG, 64, dtype=I8)
    many = on(0, 1).expand(BIG)
    norm = m.Norm(64)
    norm.d_model = BIG
    for f in (lambda: m.moe_norm_pre(m.Norm(64), tall, h=tall),
              lambda: m.moe_norm_pre(norm, wide, h=wide),
              lambda: m.moe_norm_post(m.Norm(64), tall, tall, out=tall),
              lambda: m.moe_quant_row_q8(tall, q=codes, scales=many),
              lambda: m.moe_quant_row_q8(wide, q=says(20, BIG, dtype=I8), scales=on(0, 20)),
              lambda: m.moe_route_scored(m.RouterRule(64, 4), tall),
              lambda: m.moe_linear_q8(m.Linear(on(0, 8, 64, dtype=I8), on(0, 8)), codes, many),
              lambda: m.Linear(codes, many),
              lambda: m.moe_route_scored_workspace_bytes(m.RouterRule(64, 4), BIG),
              lambda: m.moe_linear_q8_workspace_bytes(
                  m.Linear(on(0, 8, 64, dtype=I8), on(0, 8)), BIG)):
        with pytest.raises(ValueError, match="2147483647"):
            f()
    assert not lib.calls


@pytest.mark.parametrize("kw", [{"n_experts": BIG}, {"top_k": BIG}, {"n_groups": BIG},
                                {"top_groups": BIG}, {"n_experts": -BIG}])
def test_rules_that_c_would_cut_are_refused(kw):
    with pytest.raises(ValueError):
        m.RouterRule(**{"n_experts": 64, "top_k": 4, **kw})
    with pytest.raises(ValueError):
        m.Norm(BIG)


# ------------------------------------------------------------- descriptors
def test_descriptors_keep_the_memory_they_were_made_from(lib):
    """A weight whose data is replaced afterwards leaves the descriptor on live memory."""
    w, w2, bias, q, s, y = (on(0, 64), on(0, 64), on(0, 64), on(0, 64, 64, dtype=I8), on(0, 64),
                            on(0, 64))
    made = [m.Norm(64, pre_w=w, post_w=w2), m.RouterRule(64, 4, bias=bias), m.Linear(q, s, y)]
    for t in (w, w2, bias, s, y):
        t.data = torch.ones(64)
    q.data = torch.ones(64, 64, dtype=I8)
    fields = [("pre_w", "post_w"), ("bias",), ("w", "w_scales", "bias")]
    for d, names in zip(made, fields):
        assert [t.data_ptr() for t in d.tensors] == [getattr(d.c, n) for n in names]
        assert all((t == 0).all() for t in d.tensors)


def test_linear_rows_whose_last_tile_passes_31_bits_are_refused():
    """The library itself: a tile's rows are numbered past the last one, up to 255 further."""
    A, SHAPE = 0x100000, -2
    lay = b.moe_linear_t(1, 16, A, 16, A, None)
    for rows in (2**31 - 255, 2**31 - 100, 2**31 - 1):
        # (y is misaligned, so that no call gets further than the checks)
        assert m.lib().moe_linear_q8(lay, A, 16, A, rows, A + 1, 0, 1, A, 1 << 30, None) == SHAPE
