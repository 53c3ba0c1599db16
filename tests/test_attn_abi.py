"""The calls around the 4-bit cache reject bad arguments before touching the GPU (CPU only: every
call here fails validation or has nothing to do), and what their binding refuses or hands on."""
import contextlib
import ctypes as C

import pytest
import torch

import mxfp4_routed_expert_e2m1_amd as m
from mxfp4_routed_expert_e2m1_amd import attention as at
from mxfp4_routed_expert_e2m1_amd import block as b
from test_block_binding import Recorder, on

OK, INVALID, SHAPE, STRIDE, WORKSPACE, ALIGN = 0, -1, -2, -3, -4, -5
A = C.c_void_p(0x100000)     # fake device address, never dereferenced
ODD = C.c_void_p(0x100001)
MIS4 = C.c_void_p(0x100002)  # not 4-byte aligned
INF, NAN = float("inf"), float("nan")
I32, U8 = torch.int32, torch.uint8


def rope(rot=64, axes=1, inter=0, scale=1.0, steps=0x100000, ax=0):
    return C.byref(at.moe_rope_t(rot, axes, inter, scale, steps, ax))


def test_rope_validation():
    f = m.lib().moe_rope

    def call(R=None, x=A, t=0, ld=256, hs=64, rows=4, heads=4, dim=64, pos=A, ldp=4, out=A, ldo=256,
             hso=64):
        return f(R or rope(), x, t, ld, hs, rows, heads, dim, pos, ldp, out, ldo, hso, None)
    assert f(None, A, 0, 256, 64, 4, 4, 64, A, 4, A, 256, 64, None) == INVALID
    assert call(rows=0, x=None, pos=None, out=None) == OK
    assert call(heads=0, x=None, pos=None, out=None) == OK
    for R in (rope(rot=0), rope(rot=63), rope(rot=66), rope(axes=0), rope(axes=9)):
        assert call(R=R) == SHAPE
    assert call(dim=1026, hs=1026, ld=1 << 14) == SHAPE
    for R in (rope(inter=2), rope(scale=INF), rope(scale=NAN), rope(steps=0)):
        assert call(R=R) == INVALID
    assert call(rows=-1) == INVALID
    assert call(heads=-1) == INVALID
    assert call(t=2) == INVALID
    for k in ("x", "pos", "out"):
        assert call(**{k: None}) == INVALID
        assert call(**{k: ODD}) == ALIGN
    assert call(R=rope(steps=0x100004)) == ALIGN
    for kw in (dict(hs=63), dict(ld=63), dict(ld=255), dict(hso=63), dict(ldo=255)):
        assert call(**kw) == STRIDE, kw
    assert call(R=rope(axes=3), ldp=3) == STRIDE
    # in place, with other strides
    assert call(ldo=512) == INVALID
    assert call(hs=256, ld=64, hso=64, ldo=256) == INVALID
    assert call(rows=2**31 - 1, heads=2**20, hs=64, ld=64 * 2**20, ldo=64 * 2**20) == SHAPE
    # 32 pairs in 4 threads of one head, 2^32 of them
    assert call(rows=2**30, heads=1, ld=64, ldo=64) == SHAPE


def cache(heads=4, dim=64, page=16, pages=8, data=0x100000):
    return C.byref(at.moe_kv_cache_t(heads, dim, page, pages, data))


BAD_CACHES = [dict(heads=0), dict(heads=1025), dict(dim=32), dict(dim=96), dict(dim=0), dict(page=8),
              dict(page=24), dict(page=512), dict(page=0), dict(page=-16), dict(pages=0),
              dict(pages=2**27)]


def test_cache_bytes():
    f = m.lib().moe_kv_cache_bytes
    assert f(cache()) == 8 * 16 * 4 * 2 * (32 + 2)
    assert f(cache(heads=8, dim=128, page=64, pages=2**25 - 1)) == (2**25 - 1) * 64 * 8 * 136
    assert f(cache(data=0)) == f(cache())
    assert f(None) == 0
    for kw in BAD_CACHES:
        assert f(cache(**kw)) == 0, kw


@pytest.mark.parametrize("write", [True, False])
def test_write_and_read_validation(write):
    L = m.lib()

    def call(K=None, k=A, ldk=256, hsk=64, v=A, ldv=256, hsv=64, t=0, rows=4, slots=A):
        K = K or cache()
        if write:
            return L.moe_kv_write(K, k, ldk, hsk, v, ldv, hsv, t, rows, slots, None)
        return L.moe_kv_read(K, slots, rows, k, ldk, hsk, v, ldv, hsv, t, None)
    assert call(rows=0, k=None, v=None, slots=None) == OK
    for kw in BAD_CACHES:
        assert call(K=cache(**kw)) == SHAPE, kw
    assert call(K=cache(data=0)) == INVALID
    assert call(K=cache(data=0x100008)) == ALIGN
    assert call(rows=-1) == INVALID
    assert call(t=2) == INVALID
    for k in ("k", "v", "slots"):
        assert call(**{k: None}) == INVALID
        assert call(**{k: MIS4}) == ALIGN
    for kw in (dict(ldk=63), dict(ldk=255), dict(hsk=63), dict(ldv=255), dict(hsv=63)):
        assert call(**kw) == STRIDE, kw
    assert call(rows=2**27) == SHAPE
    assert call(rows=2**31 - 1) == SHAPE


def attn(heads=8, window=0, scale=1.0, softcap=0.0, slopes=0):
    return C.byref(at.moe_attn_t(heads, window, scale, softcap, slopes))


def test_attn_validation():
    L = m.lib()

    def call(T=None, K=None, q=A, t=0, ld=512, hs=64, rows=4, off=A, seqs=2, lens=A, table=A, ldt=8,
             pages=8, prefix=None, out=C.c_void_p(0x200000), ldo=512, hso=64, ws=A, wsb=1 << 30):
        return L.moe_attn_cache(T or attn(), K or cache(), q, t, ld, hs, rows, off, seqs, lens, table,
                                ldt, pages, prefix, out, ldo, hso, ws, wsb, None)
    assert L.moe_attn_cache(None, cache(), A, 0, 512, 64, 4, A, 2, A, A, 8, 8, None, A, 512, 64, A, 0,
                            None) == INVALID
    assert L.moe_attn_cache(attn(), None, A, 0, 512, 64, 4, A, 2, A, A, 8, 8, None, A, 512, 64, A, 0,
                            None) == INVALID
    assert call(rows=0, q=None, out=None, lens=None, table=None) == OK
    assert call(seqs=0, q=None, out=None, lens=None, table=None) == OK
    for kw in BAD_CACHES:
        assert call(K=cache(**kw)) == SHAPE, kw
    assert call(K=cache(data=0)) == INVALID
    for heads in (0, 7, -8, 16388):
        assert call(T=attn(heads=heads)) == SHAPE
    for T in (attn(window=-1), attn(scale=NAN), attn(scale=INF), attn(softcap=-1.0), attn(softcap=NAN),
              attn(softcap=INF)):
        assert call(T=T) == INVALID
    for kw in (dict(rows=-1), dict(seqs=-1), dict(pages=-1), dict(t=2)):
        assert call(**kw) == INVALID, kw
    for k in ("q", "out", "lens", "table"):
        assert call(**{k: None}) == INVALID
        assert call(**{k: ODD}) == ALIGN
    assert call(off=MIS4) == ALIGN
    assert call(prefix=MIS4) == ALIGN
    assert call(T=attn(slopes=0x100002)) == ALIGN
    assert call(out=A) == INVALID                       # in place
    assert call(off=None) == INVALID                    # 4 rows for 2 sequences
    for kw in (dict(ld=63), dict(ld=511), dict(hs=63), dict(ldo=511), dict(hso=63), dict(ldt=7)):
        assert call(**kw) == STRIDE, kw
    assert call(pages=2**26, ldt=2**26) == SHAPE
    assert call(rows=2**28, ld=512, ldo=512) == SHAPE
    assert call(seqs=2**25, ldt=8) == SHAPE
    big = dict(pages=1000, ldt=1000)
    assert call(ws=None, **big) == INVALID
    assert call(wsb=16, **big) == WORKSPACE
    assert call(ws=C.c_void_p(0x100008), **big) == ALIGN


def test_attn_workspace_bytes():
    f = m.lib().moe_attn_cache_workspace_bytes
    assert f(None, cache(), 4, 1) == 0 and f(attn(), None, 4, 1) == 0
    assert f(attn(), cache(dim=96), 4, 1) == 0 and f(attn(heads=7), cache(), 4, 1) == 0
    assert f(attn(), cache(), 0, 1) == 0 and f(attn(), cache(), 4, 0) == 0
    for K, heads in ((cache(), 8), (cache(heads=1, dim=256), 40), (cache(heads=8, dim=128), 32)):
        last = 0
        for rows in list(range(1, 200)) + [500, 1000, 4096, 2**20]:
            n = f(attn(heads=heads), K, rows, 1)
            assert n >= last
            last = n
        for seqs in (1, 2, 3, 10, 100, 1000, 10**6):
            n = f(attn(heads=heads), K, 2**20, seqs)
            assert n >= last
            last = n
        assert last < 2**30


# ------------------------------------------------------------------- the binding
@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(at, "_lib", r)
    monkeypatch.setattr(b, "_lib", r)
    monkeypatch.setattr(at, "_raw_stream", lambda gpu: 1000 + gpu)
    monkeypatch.setattr(at, "_current_gpu", lambda: r.gpu, raising=False)

    @contextlib.contextmanager
    def device(gpu):
        r.gpu, was = gpu, r.gpu
        yield
        r.gpu = was
    monkeypatch.setattr(torch.cuda, "device", device)
    return r


def a_cache(gpu=0):
    return m.KVCache(4, 16, 2, 64, data=on(gpu, 64, dtype=U8))


def a_rope(gpu=0):
    r = m.Rope.__new__(m.Rope)
    r.gpu, r.n_axes, r.rot_dim, r.ref = gpu, 1, 64, None
    return r


def do_rope(gpu=0, **kw):
    kw = {"rope": a_rope(gpu), "x": on(gpu, 5, 2, 64), "positions": on(gpu, 5, dtype=I32),
          "out": on(gpu, 5, 2, 64), **kw}
    return m.moe_rope(kw.pop("rope"), kw.pop("x"), kw.pop("positions"), **kw)


def do_write(gpu=0, **kw):
    kw = {"cache": a_cache(gpu), "k": on(gpu, 5, 2, 64), "v": on(gpu, 5, 2, 64),
          "slots": on(gpu, 5, dtype=I32), **kw}
    return m.moe_kv_write(**kw)


def do_read(gpu=0, **kw):
    kw = {"cache": a_cache(gpu), "slots": on(gpu, 5, dtype=I32), "k": on(gpu, 5, 2, 64),
          "v": on(gpu, 5, 2, 64), **kw}
    return m.moe_kv_read(**kw)


def do_attn(gpu=0, **kw):
    kw = {"attn": m.Attention(4, 0.125), "cache": a_cache(gpu), "q": on(gpu, 5, 4, 64),
          "table": on(gpu, 2, 3, dtype=I32), "kv_lens": on(gpu, 2, dtype=I32),
          "q_offsets": on(gpu, 3, dtype=I32), "out": on(gpu, 5, 4, 64), "ws": on(gpu, 64, dtype=U8),
          **kw}
    return m.moe_attn_cache(**kw)


CALLS = [do_rope, do_write, do_read, do_attn]


@pytest.mark.parametrize("call", CALLS)
def test_calls_run_on_their_tensors_gpu(lib, call):
    call()
    call(gpu=1)
    assert lib.gpus == [0, 1] and lib.gpu == 0
    assert [c[1][-1] for c in lib.calls] == [1000, 1001]


@pytest.mark.parametrize("call,names", [(do_rope, ["rope", "positions", "out"]),
                                        (do_write, ["cache", "v", "slots"]),
                                        (do_read, ["cache", "k", "v"]),
                                        (do_attn, ["cache", "table", "kv_lens", "q_offsets", "out",
                                                   "ws", "attn", "prefix"])])
def test_tensors_of_another_gpu_or_of_the_host_are_refused(lib, call, names):
    other = {"rope": lambda g: a_rope(g), "cache": lambda g: a_cache(g),
             "attn": lambda g: m.Attention(4, 0.125, slopes=on(g, 4)),
             "positions": lambda g: on(g, 5, dtype=I32), "slots": lambda g: on(g, 5, dtype=I32),
             "table": lambda g: on(g, 2, 3, dtype=I32), "kv_lens": lambda g: on(g, 2, dtype=I32),
             "prefix": lambda g: on(g, 2, dtype=I32), "q_offsets": lambda g: on(g, 3, dtype=I32),
             "ws": lambda g: on(g, 64, dtype=U8),
             "out": lambda g: on(g, 5, 4 if call is do_attn else 2, 64),
             "k": lambda g: on(g, 5, 2, 64), "v": lambda g: on(g, 5, 2, 64)}
    for name in names:
        with pytest.raises(ValueError):
            call(**{name: other[name](1)})
        if name not in ("rope", "cache", "attn"):
            like = other[name](0)
            with pytest.raises(ValueError):
                call(**{name: torch.zeros(tuple(like.shape), dtype=like.dtype)})
    assert not lib.calls


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_gpu_is_refused(lib, call):
    class Stream:
        device_index, cuda_stream = 1, 77
    with pytest.raises(ValueError):
        call(stream=Stream())
    assert not lib.calls
    call(gpu=1, stream=Stream())
    assert lib.calls[0][1][-1] == 77


@pytest.mark.parametrize("call,kw", [
    (do_rope, dict(x=on(0, 5, 2, 64, dtype=torch.float16))), (do_rope, dict(positions=on(0, 5))),
    (do_rope, dict(out=on(0, 5, 2, 64, dtype=torch.bfloat16))),
    (do_write, dict(k=on(0, 5, 2, 64, dtype=torch.float16))),
    (do_write, dict(v=on(0, 5, 2, 64, dtype=torch.bfloat16))), (do_write, dict(slots=on(0, 5))),
    (do_read, dict(k=on(0, 5, 2, 64, dtype=torch.bfloat16))),
    (do_attn, dict(q=on(0, 5, 4, 64, dtype=torch.float64))), (do_attn, dict(table=on(0, 2, 3))),
    (do_attn, dict(kv_lens=on(0, 2, dtype=torch.int64))),
    (do_attn, dict(out=on(0, 5, 4, 64, dtype=torch.bfloat16)))])
def test_other_types_are_refused(lib, call, kw):
    with pytest.raises(TypeError):
        call(**kw)
    assert not lib.calls


@pytest.mark.parametrize("call,kw", [
    (do_rope, dict(x=on(0, 5, 128))), (do_rope, dict(positions=on(0, 4, dtype=I32))),
    (do_rope, dict(positions=on(0, 3, 5, dtype=I32))), (do_rope, dict(out=on(0, 5, 1, 64))),
    (do_rope, dict(positions=on(0, 10, dtype=I32)[::2])),
    (do_write, dict(k=on(0, 5, 3, 64))), (do_write, dict(v=on(0, 4, 2, 64))),
    (do_write, dict(slots=on(0, 4, dtype=I32))), (do_read, dict(v=on(0, 5, 2, 128))),
    (do_attn, dict(q=on(0, 5, 2, 64))), (do_attn, dict(q=on(0, 5, 4, 128)[:, :, ::2])),
    (do_attn, dict(table=on(0, 6, dtype=I32))), (do_attn, dict(kv_lens=on(0, 3, dtype=I32))),
    (do_attn, dict(q_offsets=on(0, 2, dtype=I32))), (do_attn, dict(prefix=on(0, 3, dtype=I32))),
    (do_attn, dict(out=on(0, 4, 4, 64))), (do_attn, dict(ws=on(0, 128, dtype=U8)[::2]))])
def test_other_shapes_are_refused(lib, call, kw):
    with pytest.raises(ValueError):
        call(**kw)
    assert not lib.calls


def test_descriptors_refuse():
    with pytest.raises(ValueError):
        m.KVCache(4, 16, 2, 96)
    with pytest.raises(ValueError):
        m.KVCache(4, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        m.KVCache(4, 16, 2, 64, data=torch.zeros(5, dtype=U8))
    with pytest.raises(ValueError):
        m.KVCache(2**31, 16, 2, 64)
    with pytest.raises(ValueError):
        m.Rope([1.0, 0.5], device="cpu")
    with pytest.raises(ValueError):
        m.Rope([1.0, 0.5], axes=[0], device="cpu")
    with pytest.raises(ValueError):
        m.Rope([1.0, 0.5], axes=[0, 8], device="cpu")
    with pytest.raises(ValueError):
        m.Attention(4, 0.1, slopes=torch.zeros(4))
    with pytest.raises(TypeError):
        m.Attention(4, 0.1, slopes=on(0, 4, dtype=torch.bfloat16))


def test_steps_are_turns_to_the_last_bit():
    """The frequency over 2 pi, rounded once, against exact fractions."""
    from fractions import Fraction
    two_pi = 2 * Fraction(31415926535897932384626433832795028841971693993751, 10**49)
    for f in (1.0, 0.1, 10000.0 ** -0.73, 3.0, 1e-12, 6.283185307179586, 100.0, -1.0, 0.0):
        want = Fraction(f) / two_pi * 2**64
        got = at._step(f)
        near = round(want) % 2**64
        assert got == near, f
