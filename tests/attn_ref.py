"""Plain 64-bit forms of rotary positions, the 4-bit cache and the attention over it, written from
their formulas and used by the tests alone."""
import math

import numpy as np
import torch

import mxfp4_routed_expert_e2m1_amd as m

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def half_step(dtype):
    """The largest relative error of a rounding to a type."""
    return torch.finfo(dtype).eps / 2


def rope(x, pos, freq, axes=None, interleaved=False, scale=1.0):
    """x [rows][heads][dim], pos [axes][rows], both float64."""
    out, n = x.copy(), len(freq)
    for i in range(n):
        angle = pos[axes[i] if axes is not None else 0] * freq[i]
        c, s = scale * np.cos(angle)[:, None], scale * np.sin(angle)[:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
        out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        out[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return out


def rope_error(x, freq, interleaved, scale):
    """What fp32 may be off by: the sines and cosines (3 steps of 2^-24: the reduced angle, the
    series' last operations), their scaling, two products and a sum, each half a step of a value of
    at most scale (|a| + |b|): 8 in all."""
    n, bound = len(freq), np.zeros_like(x)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
        size = abs(scale) * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
        bound[:, :, a] = bound[:, :, b] = 8 * 2.0**-24 * size
    return bound


def stored(x):
    """What the cache holds of rows of channels (float64 in, float64 out)."""
    b = np.asarray(x, dtype=np.float64).reshape(-1, 32)
    most = np.abs(b).max(axis=1)
    fine = np.isfinite(most)
    size = np.where(fine & (most > 0), most, 1.0)
    m, e = np.frexp(size)                       # size = m 2^e, 1/2 <= m < 1
    e = np.where(most > 0, e - 3 + (m >= 0.875), -125)
    e = np.clip(e, -125, 125)
    a = np.abs(np.where(fine[:, None], b, 0.0)) * np.exp2(-e.astype(np.float64))[:, None]
    far = np.abs(a[:, :, None] - GRID)
    least = far.min(axis=2, keepdims=True)
    # of two as near the even code
    code = np.where(far == least, 10 - (np.arange(8) % 2), 0).argmax(axis=2)
    out = np.copysign(GRID[code] * np.exp2(e.astype(np.float64))[:, None], b)
    out[~fine] = np.nan
    return out.reshape(np.shape(x))


def sees(n, m, prefix=0, window=0):
    """[m][n] truth values: what the rows of a sequence see of its tokens."""
    i = np.arange(n - m, n)[:, None]
    j = np.arange(n)[None, :]
    ok = (j <= i) | (j < prefix)
    if window:
        ok = ok & (i - j < window)
    return ok


def attention(q, k, v, scale, softcap=0.0, slopes=None, prefix=0, window=0, capped=np.tanh):
    """One sequence: q [m][H][D], k and v [n][KV][D] (float64) -> (out, bound), bound[i][h][d] the
    sum of weight times |v| that errors are counted in, and the scores' own error."""
    m, H, D = q.shape
    n, KV = k.shape[0], k.shape[1]
    out, size, ds = np.zeros_like(q), np.zeros_like(q), np.zeros((m, H))
    ok = sees(n, m, prefix, window)
    dist = np.abs(np.arange(n - m, n)[:, None] - np.arange(n)[None, :])
    for h in range(H):
        kk, vv = k[:, h // (H // KV)], v[:, h // (H // KV)]
        with np.errstate(invalid="ignore", over="ignore"):
            s = scale * (q[:, h] @ kk.T)
            mag = abs(scale) * (np.abs(q[:, h]) @ np.abs(kk).T)
            if softcap:
                s = softcap * capped(s / softcap)
            if slopes is not None:
                s = s - slopes[h] * dist
                mag = mag + np.abs(slopes[h]) * dist * 2.0**-6
        for r in range(m):
            on = ok[r]
            if not on.any():
                continue
            with np.errstate(invalid="ignore", over="ignore"):
                w = np.exp(s[r, on] - s[r, on].max())
                w = w / w.sum()
                out[r, h] = w @ vv[on]
                size[r, h] = w @ np.abs(vv[on])
                # the D products are exact and added in fp32: within D + 16 half steps of their
                # magnitudes' sum, the scale, cap, bias and base of the exponential among the 16
                ds[r, h] = (D + 16) * 2.0**-24 * (mag[r, on].max() + np.abs(s[r, on]).max())
    return out, size, ds


def attention_error(size, ds, n, dtype):
    """What the kernel may be off by before its last rounding.  A score that is off by d changes a
    weight by a factor within e^(2d) (its own, and the sum's); the exponentials and sums are fp32:
    a wave adds a row's weights one after the other, every fourth of at most n / 4, and the
    products by the matrix core, 32 at a time: n / 8 + 128 half steps for all; weights are rounded
    to bf16 (half a step) for the product in bf16 calls, not in f32 ones."""
    weights = half_step(dtype) if dtype == torch.bfloat16 else 0.0
    rel = np.expm1(2 * ds)[:, :, None] + weights + (n / 8 + 128) * 2.0**-24
    return rel * size


class Paged:
    """A batch in pages: sequences' tokens in pages of a random order, each page whole."""

    def __init__(self, lens, heads, dim, page, seed, spare=3, wide=None, dtype=torch.float32,
                 grow=1.0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.lens, self.page = lens, page
        n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=g)
        wide = max(need + [1]) if wide is None else wide
        # (entries past a sequence's last page are not to be looked at)
        self.table = torch.full((len(lens), wide), 0x7FFFFFF0, dtype=torch.int32)
        at, self.slots, self.k, self.v = 0, [], [], []
        for i, n in enumerate(need):
            self.table[i, :n] = order[at: at + n].int()
            at += n
            t = torch.arange(lens[i])
            self.slots.append((self.table[i].long()[t // page] * page + t % page).int())
            shape = (lens[i], heads, dim)
            self.k.append(grow * torch.randn(shape, generator=g).to(dtype))
            self.v.append((torch.randn(shape, generator=g) + 0.3).to(dtype))
        self.cache = m.KVCache(n_pages, page, heads, dim)
        # what no token was written to holds any bytes
        self.cache.tensors[0].copy_(torch.randint(0, 256, self.cache.tensors[0].shape, generator=g,
                                                  dtype=torch.uint8))
        if sum(lens):
            m.moe_kv_write(self.cache, torch.cat(self.k).cuda(), torch.cat(self.v).cuda(),
                           torch.cat(self.slots).cuda())

    def values(self, s):
        return stored(f64(self.k[s])), stored(f64(self.v[s]))


def check(got, want, err, dtype):
    """got within err and a last rounding of want; NaN where want has it."""
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN in other places"
    off = np.abs(got - want)
    allowed = err + half_step(dtype) * (np.abs(want) + err) + 1e-37
    bad = ~(off <= allowed) & ~np.isnan(want)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} off, worst {np.nanmax(off / allowed):.2f} times the "
                           f"bound at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}")


def check_batch(got, paged, q, new, dtype, scale, softcap=0.0, slopes=None, prefix=None, window=0):
    at = 0
    for s, m in enumerate(new):
        n = paged.lens[s]
        k, v = paged.values(s)
        rows = f64(q[at: at + m])
        want, size, ds = attention(rows, k, v, scale, softcap,
                                   None if slopes is None else f64(slopes),
                                   0 if prefix is None else prefix[s], window)
        check(got[at: at + m], want, attention_error(size, ds, n, dtype), dtype)
        at += m


def frequencies(n, base=10000.0):
    return [math.pow(base, -i / n) for i in range(n)]
