"""Attention over a cache held in 4 bits, as cases to measure.

Four operators, in the order in which a served block uses them:

  rope   rotary positions with one or several axes (text; time, height, width)
         over query and key heads
  write  keys and values quantised into the pages of the cache: E2M1 codes, one
         power-of-two scale for 32 channels (a pass writes rows and reads them
         back, so that its outputs are the values that the cache then holds)
  read   keys and values of given slots, back from the cache
  attn   attention of a ragged batch's new rows over their sequences' cached
         tokens: drafted or single tokens, prefill chunks; causal, with a
         window, a prefix that all rows see, capped scores, a bias by distance

`run` computes a case in elementary torch operations (own = False) or through
this package's entry points (own = True); `exact` is the definition in 64
bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token far into a long text: 32 query and 8 key heads
        rope("rope_1", 1, 40, 128, 128, 1, False, "bf16", 1000003),
        # a chunk of image tokens: three axes, pairs side by side, part of a
        # head rotated
        rope("rope_777", 777, 20, 64, 48, 3, True, "f32", 5000),
        # a prefill chunk of text
        rope("rope_4096", 4096, 40, 128, 128, 1, False, "bf16", 131072),
        # the new tokens of a decode batch, two of its requests idle
        write("write_16", 16, 8, 128, 16, "bf16", 2),
        # a prefill chunk's keys and values
        write("write_4096", 4096, 8, 128, 64, "bf16", 0),
        # a short ragged piece for a caller that computes in f32
        read("read_777", 777, 5, 64, 16, "f32"),
        # a whole context, back in bf16
        read("read_65536", 65536, 8, 128, 64, "bf16"),
        # one decoded token over a short context
        attn("attn_1", 1, 1003, 0.0, 1, 32, 8, 128, 16, "bf16"),
        # a decode batch of uneven contexts, one request idle
        attn("attn_16", 16, 8192, 0.75, 1, 32, 8, 128, 64, "bf16", idle=1),
        # five drafted tokens of three long texts, scores capped, f32, three
        # query heads to a key head
        attn("attn_long", 3, 100001, 0.3, 5, 24, 8, 128, 64, "f32", softcap=30.0),
        # a few short prompts with a common prefix that all rows see, a window,
        # a bias by distance
        attn("attn_prefix", 4, 901, 0.5, 700, 12, 4, 64, 16, "bf16", window=256, slopes=True,
             prefix=100),
        # a prefill chunk over a context of its own size and itself
        attn("attn_4096", 1, 8192, 0.0, 4096, 32, 8, 128, 64, "bf16"),
    ]


def rope(name, rows, heads, dim, rot, axes, interleaved, kind, far):
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "dim": dim, "rot": rot,
            "axes": axes, "interleaved": interleaved, "type": kind, "far": far}


def write(name, rows, heads, dim, page, kind, idle):
    return {"name": name, "op": "write", "rows": rows, "heads": heads, "dim": dim, "page": page,
            "type": kind, "idle": idle}


def read(name, rows, heads, dim, page, kind):
    return {"name": name, "op": "read", "rows": rows, "heads": heads, "dim": dim, "page": page,
            "type": kind}


def attn(name, seqs, ctx, ragged, new, heads, kv, dim, page, kind, softcap=0.0, window=0,
         slopes=False, prefix=0, idle=0):
    """seqs requests with up to ctx cached tokens, of which the last (up to)
    `new` are the rows; `idle` more requests with one row and no tokens."""
    return {"name": name, "op": "attn", "seqs": seqs, "ctx": ctx, "ragged": ragged, "new": new,
            "heads": heads, "kv": kv, "dim": dim, "page": page, "type": kind, "softcap": softcap,
            "window": window, "slopes": slopes, "prefix": prefix, "idle": idle}


def spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn", "attn"])
    kind, dim = rng.choice(["f32", "bf16", "bf16"]), rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        heads = spread(rng, 1, 64)
        rows = spread(rng, 1, max(1, min(8192, 4096 * 40 * 128 // (heads * dim))))
        c = rope("", rows, heads, dim, rng.choice([dim, dim, dim // 2, dim // 4 * 3]),
                 rng.choice([1, 1, 3]), rng.random() < 0.3, kind, spread(rng, 100, 1 << 20))
    elif op == "write":
        heads = spread(rng, 1, 16)
        rows = spread(rng, 1, max(1, min(8192, 4096 * 8 * 128 // (heads * dim))))
        c = write("", rows, heads, dim, page, kind, rng.randint(0, rows // 8))
    elif op == "read":
        heads = spread(rng, 1, 16)
        rows = spread(rng, 1, max(1, min(65536, 65536 * 8 * 128 // (heads * dim))))
        c = read("", rows, heads, dim, page, kind)
    else:
        kv, seqs = rng.choice([1, 2, 4, 8]), spread(rng, 1, 32)
        heads = kv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        new = rng.choice([1, 1, rng.randint(2, 8), spread(rng, 16, 4096)])
        # what the plain form holds stays within the largest listed cases'
        most = min(3 * 100001 * 8 * 128 // (seqs * kv * dim),
                   4096 * 32 * 8192 // (seqs * new * heads),
                   4096 * 32 * 8192 * 128 // (seqs * new * heads * dim), 131072)
        if kind == "f32":  # (the largest products are listed in bf16)
            most = min(most, 512 * 32 * 8192 * 128 // (seqs * new * heads * dim))
        ctx = spread(rng, 1, max(1, most))
        new = min(new, ctx)
        c = attn("", seqs, ctx, rng.choice([0.0, 0.5, 0.9]), new, heads, kv, dim, page, kind,
                 rng.choice([0.0, 0.0, 30.0]), rng.choice([0, 0, spread(rng, 1, 4096)]),
                 rng.random() < 0.25, rng.choice([0, 0, 0, spread(rng, 1, ctx)]),
                 rng.choice([0, 0, 1]))
    del c["name"]
    return c


def lengths(c):
    """(cached tokens, rows) of each request: set by the case."""
    rng = random.Random("%d %d %s %d" % (c["seqs"], c["ctx"], c["ragged"], c["new"]))
    lens = [c["ctx"]] + [rng.randint(max(1, int(c["ctx"] * (1 - c["ragged"]))), c["ctx"])
                         for _ in range(c["seqs"] - 1)]
    new = [min(c["new"], n) if c["new"] <= 8 or i == 0 else min(rng.randint(1, c["new"]), n)
           for i, n in enumerate(lens)]
    return lens + [0] * c["idle"], new + [1] * c["idle"]


def work(c):
    H, D = c["heads"], c["dim"]
    if c["op"] == "rope":
        n = c["rows"] * H
        return {"bytes": 2 * n * D * SIZE[c["type"]] + 4 * c["axes"] * c["rows"],
                "flops": 3 * n * c["rot"]}
    if c["op"] == "write":
        n = c["rows"] * H * D * 2
        return {"bytes": n * SIZE[c["type"]] + 2 * n * 17 // 32 + 2 * n + 8 * c["rows"],
                "flops": 8 * n}
    if c["op"] == "read":
        n = c["rows"] * H * D * 2
        return {"bytes": n * SIZE[c["type"]] + n * 17 // 32 + 4 * c["rows"], "flops": 2 * n}
    lens, new = lengths(c)
    pairs = cached = 0
    for n, m in zip(lens, new):
        if n == 0:
            continue
        i = np.arange(n - m, n, dtype=np.int64)
        first = np.maximum(0, i - c["window"] + 1) if c["window"] else 0 * i
        last = np.maximum(i + 1, min(c["prefix"], n))
        pairs += int((last - first).sum())
        cached += int(last.max() - first.min())
    return {"bytes": cached * c["kv"] * D * 2 * 17 // 32 + 2 * sum(new) * H * D * SIZE[c["type"]],
            "flops": 4 * pairs * H * D}


# ---------------------------------------------------------------- the inputs
def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"rope": rope_inputs, "write": write_inputs, "read": read_inputs,
         "attn": attn_inputs}[c["op"]](c, g)
    s["case"] = c
    return s


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32, device=DEV)


def heads_of(g, rows, heads, dim):
    """Rows of keys or queries: channels of different sizes, the same ones in
    every row, as projections have them."""
    return randn(g, rows, heads, dim) * torch.exp(0.4 * randn(g, heads, dim))


def rope_inputs(c, g):
    T, n = c["rows"], c["rot"] // 2
    inv = [10000.0 ** (-i / n) for i in range(n)]
    axes = [i % c["axes"] for i in range(n)]
    x = heads_of(g, T, c["heads"], c["dim"]).to(TYPES[c["type"]])
    first = int(torch.randint(0, 50, (1,), generator=g, device=DEV))
    t = max(0, c["far"] - T - first) + torch.arange(T, device=DEV)
    pos = t if c["axes"] == 1 else torch.stack([t // 256 + first, t // 16 % 16, t % 16])
    s = {"x": x, "pos": i32(pos), "inv": inv, "axes": axes, "scale": 1.0}
    if own:
        import mxfp4_routed_expert_e2m1_amd as m
        s["rope"] = m.Rope(inv, axes=axes, interleaved=c["interleaved"], scale=s["scale"])
        s["out"] = torch.empty_like(x)
    else:
        s["inv_gpu"] = torch.tensor(inv, dtype=torch.float64, device=DEV)
        s["axes_gpu"] = torch.tensor(axes, device=DEV)
    return s


def quantise(x):
    """E2M1 codes (two to a byte, the even channel low) and scale bytes of
    x [...][D]: per 32 channels a scale 2^(u - 127), such that the largest
    value rounds to 4 or 6."""
    b = x.float().unflatten(-1, (-1, 32))
    bits = b.abs().amax(-1).view(torch.int32)
    u = (((bits + 0x200000) >> 23) - 2).clamp(2, 252)
    a = b.abs() * torch.exp2((127 - u).float())[..., None]
    q = (a > 0.25).to(torch.uint8)
    for over in (a >= 0.75, a > 1.25, a >= 1.75, a > 2.5, a >= 3.5, a > 5.0):
        q += over
    q = (q + 8 * torch.signbit(b)).to(torch.uint8).flatten(-2)
    return q[..., 0::2] | q[..., 1::2] << 4, u.to(torch.uint8)


def values(s, name, at):
    """What the codes and scale bytes of slots `at` stand for, f32 [...][D]."""
    codes, u = s[name + "c"][at], s[name + "u"][at]
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    x = s["e2m1"][q]
    return (x.unflatten(-1, (-1, 32)) * torch.exp2(u.float() - 127)[..., None]).flatten(-2)


def pool(c, g, n_pages, heads, filled):
    """The cache's pages: for the plain form packed rows of codes and of scale
    bytes by slot (one more than there are, for rows without a slot)."""
    D, page = c["dim"], c["page"]
    n = n_pages * page
    if own:
        import mxfp4_routed_expert_e2m1_amd as m
        cache = m.KVCache(n_pages, page, heads, D)
        if filled:
            k, v = keys_values(c, g, n, heads)
            m.moe_kv_write(cache, k, v, i32(torch.arange(n)))
        return {"cache": cache}
    byte = {"dtype": torch.uint8, "device": DEV}
    s = {"e2m1": torch.tensor(E2M1 + [-v for v in E2M1], device=DEV)}
    kv = keys_values(c, g, n, heads) if filled else (None, None)
    for name, x in zip("kv", kv):
        s[name + "c"] = torch.zeros((n + 1, heads, D // 2), **byte)
        s[name + "u"] = torch.zeros((n + 1, heads, D // 32), **byte)
        if filled:
            s[name + "c"][:n], s[name + "u"][:n] = quantise(x)
    return s


def keys_values(c, g, n, heads):
    k = heads_of(g, n, heads, c["dim"])
    return k, randn(g, n, heads, c["dim"]) + 0.5 * randn(g, heads, c["dim"])


def slots_of(c, g, rows, n_pages):
    """Slots of `rows` tokens in a row, over pages in no order."""
    page = c["page"]
    order = torch.randperm(n_pages, generator=g, device=DEV)
    t = torch.arange(rows, device=DEV)
    return i32(order[t // page] * page + t % page)


def write_inputs(c, g):
    T, H, D = c["rows"], c["heads"], c["dim"]
    n_pages = T + 1 if T <= 64 else 2 * (T // c["page"]) + 2
    if T <= 64:  # a request each, at some place of a page of its own
        at = torch.randint(0, c["page"], (T,), generator=g, device=DEV)
        slots = i32(torch.randperm(n_pages, generator=g, device=DEV)[:T] * c["page"] + at)
    else:
        slots = slots_of(c, g, T, n_pages)
    slots[torch.randperm(T, generator=g, device=DEV)[: c["idle"]]] = -1
    k, v = keys_values(c, g, T, H)
    kind = TYPES[c["type"]]
    s = {"k": k.to(kind), "v": v.to(kind), "slots": slots}
    s.update(pool(c, g, n_pages, H, False))
    if own:
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    return s


def read_inputs(c, g):
    T, H = c["rows"], c["heads"]
    n_pages = T // c["page"] + 3
    s = {"slots": slots_of(c, g, T, n_pages)}
    s.update(pool(c, g, n_pages, H, True))
    if own:
        shape, kind = (T, H, c["dim"]), TYPES[c["type"]]
        s["k_out"] = torch.empty(shape, dtype=kind, device=DEV)
        s["v_out"] = torch.empty(shape, dtype=kind, device=DEV)
    return s


def attn_inputs(c, g):
    lens, new = lengths(c)
    page, D = c["page"], c["dim"]
    wide = max(1, -(-c["ctx"] // page))
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 2
    order = torch.randperm(n_pages, generator=g, device=DEV)
    table = torch.full((len(lens), wide), 0, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at: at + n]
        at += n
    T = sum(new)
    s = {"q": heads_of(g, T, c["heads"], D).to(TYPES[c["type"]]), "table": table,
         "lens": i32(lens), "offsets": i32(np.concatenate([[0], np.cumsum(new)])),
         "scale": D ** -0.5, "longest": max(lens), "most": max(new),
         "prefix": i32([min(c["prefix"], n) for n in lens]) if c["prefix"] else None,
         "slopes": 0.5 ** (1 + 7 * torch.rand(c["heads"], generator=g, device=DEV))
         if c["slopes"] else None}
    s.update(pool(c, g, n_pages, c["kv"], True))
    if own:
        import mxfp4_routed_expert_e2m1_amd as m
        s["attn"] = m.Attention(c["heads"], scale=s["scale"], softcap=c["softcap"],
                                window=c["window"], slopes=s["slopes"])
        s["out"] = torch.empty_like(s["q"])
        s["ws"] = torch.empty(m.moe_attn_cache_workspace_bytes(s["attn"], s["cache"], T,
                                                               len(lens)),
                              dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        import mxfp4_routed_expert_e2m1_amd as m
        return {"rope": own_rope, "write": own_write, "read": own_read, "attn": own_attn}[op](m, s)
    return {"rope": plain_rope, "write": plain_write, "read": plain_read,
            "attn": plain_attn}[op](s)


def own_rope(m, s):
    return m.moe_rope(s["rope"], s["x"], s["pos"], out=s["out"])


def own_write(m, s):
    m.moe_kv_write(s["cache"], s["k"], s["v"], s["slots"])
    return m.moe_kv_read(s["cache"], s["slots"], k=s["k_out"], v=s["v_out"])


def own_read(m, s):
    return m.moe_kv_read(s["cache"], s["slots"], k=s["k_out"], v=s["v_out"])


def own_attn(m, s):
    single = s["most"] == 1
    return m.moe_attn_cache(s["attn"], s["cache"], s["q"], s["table"], s["lens"],
                            q_offsets=None if single else s["offsets"], prefix=s["prefix"],
                            out=s["out"], ws=s["ws"])


def plain_rope(s):
    c, n = s["case"], s["case"]["rot"] // 2
    x, pos = s["x"].float(), s["pos"].double()
    pos = pos[:, None] if c["axes"] == 1 else pos[s["axes_gpu"]].t()
    angle = pos * s["inv_gpu"]
    cos = (s["scale"] * torch.cos(angle)).float()[:, None]
    sin = (s["scale"] * torch.sin(angle)).float()[:, None]
    r = x[..., : c["rot"]]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :n], r[..., n:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((r, x[..., c["rot"]:]), -1).to(TYPES[c["type"]])


def plain_write(s):
    spare = s["kc"].shape[0] - 1
    at = torch.where(s["slots"] < 0, spare, s["slots"]).long()
    for name in "kv":
        s[name + "c"][at], s[name + "u"][at] = quantise(s[name])
    return plain_read(s)


def plain_read(s):
    at, kind = s["slots"].long(), TYPES[s["case"]["type"]]
    on = (at >= 0)[:, None, None]
    return tuple(torch.where(on, values(s, n, at), 0.0).to(kind)
                 for n in "kv")


def plain_attn(s):
    c = s["case"]
    H, KV, D, page, L, Q = c["heads"], c["kv"], c["dim"], c["page"], s["longest"], s["most"]
    S, G, off, lens = len(s["lens"]), H // KV, s["offsets"].long(), s["lens"].long()
    j = torch.arange(L, device=DEV)
    slots = s["table"].long()[:, j // page] * page + j % page
    get = lambda n: values(s, n, slots).transpose(1, 2).contiguous()  # noqa: E731
    k, v = get("k"), get("v")                                    # [S][KV][L][D]
    new = off[1:] - off[:-1]
    i = torch.arange(Q, device=DEV)
    rows = (off[:-1, None] + i).clamp_max(off[-1] - 1)           # [S][Q]
    q = s["q"].float()[rows].view(S, Q, KV, G, D).permute(0, 2, 3, 1, 4).reshape(S, KV, G * Q, D)
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).view(S, KV, G, Q, L)
    p *= s["scale"]
    if c["softcap"]:
        p = torch.tanh(p.div_(c["softcap"])).mul_(c["softcap"])
    at = (lens - new)[:, None] + i                               # a row's place in its text
    far = at[:, :, None] - j                                     # [S][Q][L]
    if s["slopes"] is not None:
        p -= s["slopes"].view(KV, G, 1, 1) * far.abs().float()[:, None, None]
    see = far >= 0
    if s["prefix"] is not None:
        see = see | (j < s["prefix"][:, None])[:, None]
    if c["window"]:
        see = see & (far < c["window"])
    see = see & (j < lens[:, None])[:, None]
    p.masked_fill_(~see[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, KV, G * Q, L), v).view(S, KV, G, Q, D)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(S, Q, H, D)
    which = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(off[1:], which, right=True)
    return o[seq, which - off[seq]].to(TYPES[c["type"]])


# ------------------------------------------------------- the definition, 64 bits
def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    return {"rope": exact_rope, "write": exact_write, "read": exact_read,
            "attn": exact_attn}[c["op"]](c, s)


def exact_rope(c, s):
    x = s["x"].double().cpu().numpy()
    pos = s["pos"].cpu().numpy().astype(np.float64).reshape(c["axes"], c["rows"])
    out, n = x.copy(), c["rot"] // 2
    for i in range(n):
        turn = np.exp(1j * pos[s["axes"][i]] * s["inv"][i]) * s["scale"]
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, n + i)
        z = (x[:, :, a] + 1j * x[:, :, b]) * turn[:, None]
        out[:, :, a], out[:, :, b] = z.real, z.imag
    return out


def exact_write(c, s):
    """The nearest E2M1 multiple of the block's scale, ties to the even code."""
    grid = np.array(E2M1)
    gone = s["slots"].cpu().numpy() < 0

    def stored(t):
        x = t.double().cpu().numpy()
        b = x.reshape(-1, 32)
        out = np.zeros_like(b)
        for lo in range(0, len(b), 1 << 16):
            v = b[lo: lo + (1 << 16)]
            most = np.abs(v).max(1)
            m, e = np.frexp(np.where(most > 0, most, 1.0))       # most = m 2^e, 0.5 <= m < 1
            e = np.where(most > 0, e - 3 + (m >= 0.875), -125)   # 4..7 times the scale
            e = np.clip(e, -125, 125)
            a = np.abs(v) / np.exp2(e)[:, None]
            far = np.abs(a[:, :, None] - grid)
            near = far == far.min(2, keepdims=True)
            # (of two as near, which are neighbours, the even code)
            pick = np.argmax(2 * near - near * (np.arange(8) % 2), axis=2)
            out[lo: lo + (1 << 16)] = grid[pick] * np.exp2(e)[:, None] * np.sign(v)
        out = out.reshape(x.shape)
        out[gone] = 0.0
        return out

    return stored(s["k"]), stored(s["v"])


def decoded(codes, u):
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    e, m = (q >> 1) & 3, (q & 1).double()
    x = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    x = torch.where(q >= 8, -x, x) * torch.exp2(u.double() - 127).repeat_interleave(32, -1)
    return x


def exact_read(c, s):
    at = s["slots"].long()
    return decoded(s["kc"][at], s["ku"][at]), decoded(s["vc"][at], s["vu"][at])


def exact_attn(c, s):
    H, KV, D, page = c["heads"], c["kv"], c["dim"], c["page"]
    G = H // KV
    lens, new = lengths(c)
    out = torch.zeros((sum(new), H, D), dtype=torch.float64, device=DEV)
    row = 0
    for r, (n, m) in enumerate(zip(lens, new)):
        if n:
            j = torch.arange(n, device=DEV)
            at = s["table"][r].long()[j // page] * page + j % page
            i = torch.arange(n - m, n, device=DEV)
            hidden = (j > i[:, None])
            if c["prefix"]:
                hidden &= j >= min(c["prefix"], n)
            if c["window"]:
                hidden |= j <= i[:, None] - c["window"]
            for h in range(KV):
                k = decoded(s["kc"][at, h], s["ku"][at, h])
                v = decoded(s["vc"][at, h], s["vu"][at, h])
                for g in range(h * G, h * G + G):
                    z = s["scale"] * (s["q"][row: row + m, g].double() @ k.t())
                    if c["softcap"]:
                        z = c["softcap"] * torch.tanh(z / c["softcap"])
                    if s["slopes"] is not None:
                        z = z - s["slopes"][g].double() * (i[:, None] - j).abs()
                    w = torch.softmax(z.masked_fill(hidden, -math.inf), 1)
                    out[row: row + m, g] = w @ v
        row += m
    return out
