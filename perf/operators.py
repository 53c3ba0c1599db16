"""The operators around the routed experts, as cases to measure.

Four operators frame the expert layer of a decoder block:

  norm      RMS norm before a block, or after it together with the gate, the
            scaled residual and the next block's RMS norm
  route     scores of the router's logits (softmax or sigmoid), balance bias,
            expert groups, top-k, weights, and the grouping by expert
  linear    product of int8 codes [rows][d_in] with int8 weights
            [n_out][d_in], a scale per row and per channel (and a bias)
  quantised linear  the same from f32 or bf16 rows: a scale and int8 codes per
            row, then the product

`run` computes a case in elementary torch operations (own = False) or through
this package's entry points (own = True); `exact` is the definition in 64
bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token entering the expert layer: f32 residual stream,
        # f32 rows for the router and the quantiser
        norm("norm_pre_1", "pre", 1, 4096, "f32", "f32", "f32", "none", False, False),
        # a decode batch leaving the layer: norm of its output, per-channel
        # residual gate, the next block's norm
        norm("norm_post_16", "post", 16, 4096, "f32", "f32", "bf16", "channel", True, True),
        # rows of an odd width, a gate of its own for each element
        norm("norm_post_odd", "post", 1000, 2049, "bf16", "f32", "f32", "full", True, False),
        # a prefill chunk: bf16 residual stream, f32 layer output, a gate per
        # token, the next block's norm in bf16
        norm("norm_post_4096", "post", 4096, 4096, "f32", "bf16", "bf16", "token", True, True),
        # one decoded token: sigmoid scores, balance bias, 4 of 8 groups
        route("route_1", 1, 256, 6, "f32", "sigmoid", True, 8, 4, "top2", True, 2.5, 0.0),
        # a ragged chunk, bf16 softmax scores, no bias, some experts out of service
        route("route_777", 777, 160, 6, "bf16", "softmax", False, 8, 3, "max", False, 16.0, 0.1),
        # a prefill chunk: sigmoid scores, balance bias, 4 of 8 groups
        route("route_4096", 4096, 256, 8, "f32", "sigmoid", True, 8, 4, "top2", True, 2.5, 0.0),
        # one decoded token through a wide dense projection
        linear("linear_1", 1, 14336, 4096, "codes", "bf16", False),
        # a decode batch through a narrow one over a long row
        linear("linear_16", 16, 4096, 14336, "codes", "f32", False),
        # a short ragged chunk, odd channels and row length, with a bias
        linear("linear_100", 100, 4001, 2050, "codes", "f32", True),
        # bf16 rows quantised on the way, one short chunk
        linear("linear_512", 512, 4096, 4096, "bf16", "bf16", False),
        # a prefill chunk through the wide projection
        linear("linear_4096", 4096, 14336, 4096, "codes", "bf16", False),
    ]


def norm(name, kind, rows, cols, x, res, h, gate, post, nxt):
    return {"name": name, "op": "norm", "kind": kind, "rows": rows, "cols": cols, "x": x,
            "res": res, "h": h, "gate": gate, "post": post, "next": nxt}


def route(name, rows, experts, top_k, logits, score, bias, groups, top_groups, group_score,
          renorm, scale, off):
    return {"name": name, "op": "route", "rows": rows, "experts": experts, "top_k": top_k,
            "logits": logits, "score": score, "bias": bias, "groups": groups,
            "top_groups": top_groups, "group_score": group_score, "renorm": renorm,
            "scale": scale, "off": off}


def linear(name, rows, n_out, d_in, x, y, bias):
    return {"name": name, "op": "linear", "rows": rows, "n_out": n_out, "d_in": d_in, "x": x,
            "y": y, "bias": bias}


def spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = max(lo, min(hi, n))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["norm", "route", "linear"])
    if op == "norm":
        cols = spread(rng, 64, 8192)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
            cols = cols + 64 if cols == 3072 else cols
        rows = spread(rng, 1, max(1, min(8192, (4096 * 4096) // cols)))
        kind = rng.choice(["pre", "post", "post"])
        c = norm("", kind, rows, cols, rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"]),
                 rng.choice(["f32", "bf16"]), rng.choice(["none", "channel", "token", "full"]),
                 rng.random() < 0.7, rng.random() < 0.7)
        if kind == "pre":
            c.update(res="f32", gate="none", post=False, next=False)
    elif op == "route":
        groups = rng.choice([1, 2, 4, 8])
        experts = groups * max(2, spread(rng, 8, 512) // groups)
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, top_groups * (experts // groups)))
        c = route("", spread(rng, 1, 4096), experts, top_k, rng.choice(["f32", "bf16"]),
                  rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups, top_groups,
                  rng.choice(["max", "top2"]), rng.random() < 0.5, rng.choice([1.0, 2.5, 16.0]),
                  rng.choice([0.0, 0.1]))
    else:
        most = 4096 * 14336 * 4096
        d_in, n_out = spread(rng, 64, 14336), spread(rng, 64, 14336)
        if rng.random() < 0.6:
            d_in, n_out = max(64, d_in // 64 * 64), max(64, n_out // 64 * 64)
            d_in = d_in + 64 if d_in == 3072 else d_in
            n_out = n_out + 64 if n_out == 3072 else n_out
        rows = spread(rng, 1, max(1, min(4096, most // (d_in * n_out))))
        c = linear("", rows, n_out, d_in, rng.choice(["codes", "codes", "f32", "bf16"]),
                   rng.choice(["f32", "bf16"]), rng.random() < 0.3)
    del c["name"]
    return c


def work(c):
    if c["op"] == "norm":
        n = c["rows"] * c["cols"]
        if c["kind"] == "pre":
            return {"bytes": n * (SIZE[c["x"]] + SIZE[c["h"]]) + 4 * c["cols"], "flops": 4 * n}
        gate = {"none": 0, "channel": c["cols"], "token": c["rows"], "full": n}[c["gate"]]
        b = n * (SIZE[c["x"]] + 2 * SIZE[c["res"]]) + 4 * gate + (4 * c["cols"] if c["post"] else 0)
        if c["next"]:
            b += n * SIZE[c["h"]] + 4 * c["cols"]
        return {"bytes": b, "flops": n * (3 + 4 * c["post"] + 4 * c["next"])}
    if c["op"] == "route":
        T, E, k = c["rows"], c["experts"], c["top_k"]
        b = T * E * SIZE[c["logits"]] + 12 * T * k + 8 * E + 4 + (4 * E if c["bias"] else 0)
        return {"bytes": b, "flops": T * E * (4 + k)}
    T, N, K = c["rows"], c["n_out"], c["d_in"]
    x = T * K + 4 * T if c["x"] == "codes" else T * K * SIZE[c["x"]]
    b = x + N * K + 4 * N * (2 if c["bias"] else 1) + T * N * SIZE[c["y"]]
    return {"bytes": b, "flops": 2 * T * N * K}


# ---------------------------------------------------------------- the inputs
def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"norm": norm_inputs, "route": route_inputs, "linear": linear_inputs}[c["op"]](c, g)
    s["case"] = c
    if own:
        import mxfp4_routed_expert_e2m1_amd as m
        handles(m, c, s)
    return s


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def hidden(g, rows, cols):
    """Rows as a residual stream holds them: each of its own size, a few
    channels far larger than the rest."""
    channel = torch.exp(0.4 * randn(g, cols))
    channel[torch.randint(cols, (max(1, cols // 256),), generator=g, device=DEV)] *= 12.0
    return randn(g, rows, cols) * channel * torch.exp(0.5 * randn(g, rows, 1))


def norm_inputs(c, g):
    T, D = c["rows"], c["cols"]
    s = {"x": hidden(g, T, D).to(TYPES[c["x"]]), "w": 1.0 + 0.2 * randn(g, D), "eps": 1e-6}
    if c["kind"] == "post":
        s["res"] = (2.0 * hidden(g, T, D)).to(TYPES[c["res"]])
        s["res_scale"] = 0.875
        shape = {"none": None, "channel": (1, D), "token": (T, 1), "full": (T, D)}[c["gate"]]
        s["gate"] = None if shape is None else 0.5 + 0.3 * randn(g, *shape)
        s["next_w"] = 1.0 + 0.2 * randn(g, D)
    return s


def route_inputs(c, g):
    T, E = c["rows"], c["experts"]
    s = {"bias": 0.1 * randn(g, E) if c["bias"] else None}
    # some experts out of service: their logits are -infinity in every row
    off = torch.rand(E, generator=g, device=DEV) < c["off"]
    off[torch.randperm(E, generator=g, device=DEV)[: max(E // 2, c["top_k"])]] = False
    tilt = 0.5 * randn(g, E)
    make = lambda: (1.5 * randn(g, T, E) + tilt).to(TYPES[c["logits"]])  # noqa: E731
    logits = make()
    for _ in range(8):
        # whole numbers have one right value: a row whose picks hang on less
        # than 32-bit arithmetic resolves is drawn again
        bad = hangs(c, logits.masked_fill(off, -math.inf), s["bias"])
        logits = torch.where(bad[:, None], make(), logits)
    s["logits"] = logits.masked_fill(off, -math.inf)
    return s


def hangs(c, logits, bias):
    """Rows in which two different scores that an order decides by lie closer
    than 2e-6 of the row's largest."""
    T, E = logits.shape
    z = logits.double()
    p = torch.softmax(z, 1) if c["score"] == "softmax" else torch.sigmoid(z)
    p = p + (bias.double() if bias is not None else 0.0)
    p = p.masked_fill(z == -math.inf, -math.inf)
    near = lambda v, n: close(torch.sort(v, dim=1, descending=True).values[:, : n + 1])  # noqa: E731
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    if c["groups"] > 1:
        by = torch.sort(p.view(T, c["groups"], -1), dim=2, descending=True).values
        if c["group_score"] == "top2":
            two = by[:, :, :2]
            v = torch.where(two == -math.inf, 0.0, two).sum(2)
            v = v.masked_fill(by[:, :, 0] == -math.inf, -math.inf)
        else:
            v = by[:, :, 0]
        bad |= near(v, c["groups"] - 1)
        kept = torch.zeros_like(v).scatter_(
            1, torch.sort(v, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]], 1.0)
        p = p.masked_fill(kept.repeat_interleave(E // c["groups"], 1) == 0, -math.inf)
    return bad | near(p, c["top_k"])


def close(v):
    gap = v[:, :-1] - v[:, 1:]  # NaN where both are -infinity
    lim = 2e-6 * v[:, :1].abs().clamp_min(1e-30)
    return ((gap > 0) & (gap < lim)).any(1)


def linear_inputs(c, g):
    T, N, K = c["rows"], c["n_out"], c["d_in"]
    w, ws = codes(randn(g, N, K) * torch.exp(0.3 * randn(g, N, 1)))
    s = {"w": w, "ws": ws * (K ** -0.5), "bias": randn(g, N) if c["bias"] else None}
    x = hidden(g, T, K)
    if c["x"] == "codes":
        s["x"], s["xs"] = codes(x)
    else:
        s["x"] = x.to(TYPES[c["x"]])
    return s


def codes(v):
    """int8 codes and a scale for each row, in rows that start 16 bytes apart
    or a multiple of it (what lies between the rows is no part of them)."""
    rows, cols = v.shape
    d = v.abs().amax(1) / 127.0
    buf = torch.full((rows, (cols + 15) // 16 * 16), 77, dtype=torch.int8, device=DEV)
    q = buf[:, :cols]
    q.copy_(torch.clamp(torch.round(v / d[:, None]), -127, 127))
    return q, d


def handles(m, c, s):
    """What a program keeps beside its weights: descriptors, output buffers
    and workspaces."""
    T = c["rows"]
    if c["op"] == "norm":
        D = c["cols"]
        h = torch.empty((T, D), dtype=TYPES[c["h"]], device=DEV)
        if c["kind"] == "pre":
            s["norm"], s["out"] = m.Norm(D, pre_w=s["w"], eps=s["eps"]), h
            return
        s["norm"] = m.Norm(D, post_w=s["w"], post_norm=c["post"], eps=s["eps"],
                           residual_scale=s["res_scale"])
        s["next"] = m.Norm(D, pre_w=s["next_w"], eps=s["eps"]) if c["next"] else None
        s["out"] = torch.empty_like(s["res"])
        s["h"] = h if c["next"] else None
    elif c["op"] == "route":
        s["rule"] = m.RouterRule(c["experts"], c["top_k"], score=c["score"], bias=s["bias"],
                                 n_groups=c["groups"], top_groups=c["top_groups"],
                                 group_score=c["group_score"], renorm=c["renorm"],
                                 scale=c["scale"])
        s["out"] = m.route_outputs(T, c["experts"], c["top_k"], device=DEV)
        s["ws"] = torch.empty(m.moe_route_scored_workspace_bytes(s["rule"], T),
                              dtype=torch.uint8, device=DEV)
    else:
        s["lin"] = m.Linear(s["w"], s["ws"], s["bias"])
        s["out"] = torch.empty((T, c["n_out"]), dtype=TYPES[c["y"]], device=DEV)
        s["ws_buf"] = torch.empty(m.moe_linear_q8_workspace_bytes(s["lin"], T),
                                  dtype=torch.uint8, device=DEV)
        if c["x"] != "codes":
            K16 = (c["d_in"] + 15) // 16 * 16
            s["q"] = torch.empty((T, K16), dtype=torch.int8, device=DEV)[:, : c["d_in"]]
            s["qs"] = torch.empty(T, device=DEV)


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        import mxfp4_routed_expert_e2m1_amd as m
        return {"norm": own_norm, "route": own_route, "linear": own_linear}[op](m, s)
    return {"norm": plain_norm, "route": plain_route, "linear": plain_linear}[op](s)


def own_norm(m, s):
    c = s["case"]
    if c["kind"] == "pre":
        return m.moe_norm_pre(s["norm"], s["x"], h=s["out"])
    return m.moe_norm_post(s["norm"], s["x"], s["res"], gate=s["gate"], out=s["out"],
                           next_norm=s["next"], h=s["h"])


def own_route(m, s):
    return m.moe_route_scored(s["rule"], s["logits"], out=s["out"], ws=s["ws"])


def own_linear(m, s):
    q, qs = s["x"], s.get("xs")
    if s["case"]["x"] != "codes":
        q, qs = m.moe_quant_row_q8(s["x"], q=s["q"], scales=s["qs"])
    return m.moe_linear_q8(s["lin"], q, qs, y=s["out"], ws=s["ws_buf"])


def plain_norm(s):
    c = s["case"]
    rms = lambda v, w: v * torch.rsqrt((v * v).mean(1, keepdim=True) + s["eps"]) * w  # noqa: E731
    x = s["x"].float()
    if c["kind"] == "pre":
        return rms(x, s["w"]).to(TYPES[c["h"]])
    b = rms(x, s["w"]) if c["post"] else x
    if s["gate"] is not None:
        b = s["gate"] * b
    out = (s["res_scale"] * s["res"].float() + b).to(TYPES[c["res"]])
    if not c["next"]:
        return out
    # the next block reads the residual as it is stored
    return out, rms(out.float(), s["next_w"]).to(TYPES[c["h"]])


def plain_route(s):
    c, logits = s["case"], s["logits"].float()
    T, E = logits.shape
    k, G = c["top_k"], c["groups"]
    if c["score"] == "softmax":
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-logits))
    key = p if s["bias"] is None else p + s["bias"]
    key = key.masked_fill(logits == -math.inf, -math.inf)
    if G > 1:
        by = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
        v = by[:, :, 0]
        if c["group_score"] == "top2":
            v = torch.where(by[:, :, 1] == -math.inf, v, v + by[:, :, 1])
        first = torch.sort(v, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=DEV).scatter_(1, first, True)
        key = key.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    ids = torch.where(order.values[:, :k] == -math.inf, -1, order.indices[:, :k])
    w = torch.where(ids < 0, 0.0, torch.gather(p, 1, order.indices[:, :k]))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    w = w * c["scale"]
    flat = ids.reshape(-1)
    at = torch.where(flat < 0, E, flat)
    by = torch.sort(at, stable=True)
    srt = torch.where(by.values == E, -1, by.indices)
    offsets = torch.searchsorted(by.values, torch.arange(E + 1, device=DEV))
    counts = offsets[1:] - offsets[:-1]
    i32 = torch.int32
    return ids.to(i32), w, counts.to(i32), offsets.to(i32), srt.to(i32)


def plain_linear(s):
    c, x, xs = s["case"], s["x"], s.get("xs")
    if c["x"] != "codes":
        x = x.float()
        # (a tensor's quotient is rounded once; by a number, torch multiplies)
        most = x.abs().amax(1)
        xs = most / torch.full_like(most, 127.0)
        x = torch.clamp(torch.round(x / torch.where(xs > 0, xs, 1.0)[:, None]), -127, 127)
    y = x.float() @ s["w"].float().t() * xs[:, None] * s["ws"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(TYPES[c["y"]])


# ------------------------------------------------------- the definition, 64 bits
def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    return {"norm": exact_norm, "route": exact_route, "linear": exact_linear}[c["op"]](c, s)


def exact_norm(c, s):
    def rms(v, w):
        mean = np.einsum("td,td->t", v, v) / v.shape[1]
        return v / np.sqrt(mean + s["eps"])[:, None] * w

    get = lambda t: t.detach().to(torch.float64).cpu().numpy()  # noqa: E731
    x, w = get(s["x"]), get(s["w"])
    if c["kind"] == "pre":
        return rms(x, w)
    b = rms(x, w) if c["post"] else x
    if s["gate"] is not None:
        b = b * get(s["gate"])
    out = s["res_scale"] * get(s["res"]) + b
    if not c["next"]:
        return out
    # the next norm's input is the residual as stored: rounded to its type
    kept = get(torch.from_numpy(out).to(TYPES[c["res"]]))
    return out, rms(kept, get(s["next_w"]))


def exact_route(c, s):
    z = s["logits"].to(torch.float64).cpu().numpy()
    bias = np.zeros(c["experts"]) if s["bias"] is None else s["bias"].double().cpu().numpy()
    T, E = z.shape
    k, size = c["top_k"], E // c["groups"]
    ids = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        on = [e for e in range(E) if z[t, e] != -math.inf]
        top = max((z[t, e] for e in on), default=0.0)
        p = np.exp(z[t] - top) if c["score"] == "softmax" else 1.0 / (1.0 + np.exp(-z[t]))
        if c["score"] == "softmax":
            p = p / math.fsum(p[on])
        key = p + bias
        if c["groups"] > 1:
            value = {}
            for e in on:
                value.setdefault(e // size, []).append(key[e])
            most = 2 if c["group_score"] == "top2" else 1
            value = {g: math.fsum(sorted(v)[-most:]) for g, v in value.items()}
            best = sorted(value, key=lambda g: (-value[g], g))[: c["top_groups"]]
            on = [e for e in on if e // size in best]
        picks = sorted(on, key=lambda e: (-key[e], e))[:k]
        ids[t, : len(picks)] = picks
        v = p[picks]
        total = math.fsum(v)
        w[t, : len(picks)] = (v / total if c["renorm"] and total > 0 else v) * c["scale"]
    flat = [(int(e), a) for a, e in enumerate(ids.reshape(-1)) if e >= 0]
    counts = np.bincount([e for e, _ in flat], minlength=E).astype(np.int64)
    srt = np.full(T * k, -1, dtype=np.int64)
    srt[: len(flat)] = [a for _, a in sorted(flat)]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    return ids, w, counts, offsets, srt


def exact_linear(c, s):
    x, w, ws = s["x"].double(), s["w"].double(), s["ws"].double()
    if c["x"] == "codes":
        xs = s["xs"].double()
    else:
        # the codes are whole numbers by the quantiser's rule in 32 bits
        v = s["x"].float().cpu().numpy()
        d = np.abs(v).max(1) / np.float32(127.0)
        q = np.clip(np.rint(v / np.where(d > 0, d, np.float32(1.0))[:, None]), -127, 127)
        x, xs = torch.from_numpy(q).to(DEV).double(), torch.from_numpy(d).to(DEV).double()
    y = torch.matmul(x, w.t()) * (xs[:, None] * ws[None, :])
    if s["bias"] is not None:
        y = y + s["bias"].double()
    return y
