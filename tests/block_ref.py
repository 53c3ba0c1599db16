"""Plain 64-bit forms of the operators around the routed experts (block norms,
scored routing, row quantiser, int8 linear layer), written from their formulas
and used by the tests alone."""
import numpy as np
import torch


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def rms(v, w, eps):
    r = 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    return v * r * (1.0 if w is None else w)


def bf16(v):
    """float64 -> nearest bf16 value (through the float32 it is rounded from)."""
    return torch.from_numpy(np.asarray(v, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def quant_rows(x):
    """float32 rows -> (codes, scales): every step is one rounded fp32 operation."""
    x = np.asarray(x, dtype=np.float32)
    d = np.abs(x).max(axis=1) / np.float32(127)
    safe = np.where(d > 0, d, np.float32(1))[:, None]
    q = np.where(d[:, None] > 0, np.clip(np.rint(x / safe), -127, 127), 0)
    return q.astype(np.int8), d


def linear(q, w, qs, ws, bias=None, dtype=torch.float32):
    """The layer's value with its own roundings: exact whole sum, then fp32
    steps one at a time, then the output's type."""
    s = q.astype(np.int64) @ w.astype(np.int64).T if q.shape[0] * w.shape[0] < 1 << 16 else \
        np.rint(q.astype(np.float64) @ w.astype(np.float64).T).astype(np.int64)
    assert np.abs(s).max(initial=0) < 2**31
    v = s.astype(np.int32).astype(np.float32) * qs[:, None].astype(np.float32)
    v = v * ws[None, :].astype(np.float32)
    if bias is not None:
        v = v + bias[None, :].astype(np.float32)
    return torch.from_numpy(v).to(dtype)


def scores(z, kind):
    on = z > -np.inf  # NaN is out as well
    p = np.zeros_like(z)
    for t in range(z.shape[0]):
        v = z[t, on[t]]
        if v.size == 0:
            continue
        if kind == "softmax":
            with np.errstate(invalid="ignore"):
                e = np.where(v == v.max(), 1.0, np.exp(v - v.max()))
            p[t, on[t]] = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                p[t, on[t]] = 1.0 / (1.0 + np.exp(-v))
    return p, on


def route(z, top_k, score, bias=None, n_groups=1, top_groups=1, group_score="top2", renorm=True,
          scale=1.0):
    """(ids, w, counts, offsets, sorted, margin): margin[t] is the smallest
    difference between unequal values that an order in row t was decided by."""
    T, E = z.shape
    size = E // n_groups
    p, on = scores(z, score)
    key = p + (0.0 if bias is None else bias)
    ids = np.full((T, top_k), -1, dtype=np.int64)
    w = np.zeros((T, top_k))
    margin = np.full(T, np.inf)

    def gaps(t, values):
        d = np.abs(np.diff(values))
        d = d[d > 0]
        if d.size:
            margin[t] = min(margin[t], d.min())

    for t in range(T):
        left = [e for e in range(E) if on[t, e]]
        if n_groups > 1 and top_groups < n_groups:
            val = {}
            for e in left:
                val.setdefault(e // size, []).append(key[t, e])
            val = {g: sum(sorted(v)[-(2 if group_score == "top2" else 1):])
                   for g, v in val.items()}
            order = sorted(val, key=lambda g: (-val[g], g))
            gaps(t, [val[g] for g in order[:top_groups + 1]])
            left = [e for e in left if e // size in order[:top_groups]]
        order = sorted(left, key=lambda e: (-key[t, e], e))
        gaps(t, key[t, order[:top_k + 1]])
        pick = order[:top_k]
        ids[t, :len(pick)] = pick
        v = p[t, pick]
        if renorm and v.sum() > 0:
            v = v / v.sum()
        w[t, :len(pick)] = v * scale
    counts, offsets, srt = group(ids, E)
    return ids, w, counts, offsets, srt, margin


def group(ids, E):
    flat = np.asarray(ids).reshape(-1)
    own = np.nonzero(flat >= 0)[0]
    counts = np.bincount(flat[own], minlength=E)
    srt = np.full(flat.size, -1, dtype=np.int64)
    srt[:own.size] = own[np.argsort(flat[own], kind="stable")]
    return counts, np.concatenate([[0], np.cumsum(counts)]), srt
