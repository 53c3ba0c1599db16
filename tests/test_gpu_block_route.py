"""Scored routing against a 64-bit form.

Scores are fp32 (about 3 2^-24 relative, absolute below 1e-6 with the bias
added), so picks and grouping must be equal wherever no order hangs on less;
the random cases draw such rows again, the tie cases use equal values.
Weights: a score's few roundings, the sum's 16 and two more: 32 2^-24
relative (softmax: its sum over 512 experts, 8 per lane and 6 over the wave,
adds 14 to both numerator and sum, and the exponent's argument, up to 20 in
size here, half a step of its own, 20 2^-24)."""
import numpy as np
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")
DEV = "cuda"
U = 2.0**-24


def run(z, rule, dtype=torch.float32, pad=0):
    rows, E = z.shape
    buf = torch.full((rows, E + pad), 100.0, dtype=dtype, device=DEV)
    buf[:, :E] = torch.from_numpy(z).to(dtype)
    out = m.route_outputs(rows, rule.n_experts, rule.top_k)
    for t in out:
        t.fill_(77)
    got = m.moe_route_scored(rule, buf[:, :E], out=out)
    return [t.cpu().numpy() for t in got]


def check(z, kw, bias=None, dtype=torch.float32, pad=0, rule_bias=None):
    rule = m.RouterRule(z.shape[1], bias=None if bias is None else
                        torch.from_numpy(bias.astype(np.float32)).to(DEV), **kw)
    ids, w, counts, offsets, srt = run(z, rule, dtype, pad)
    kw = dict(kw)
    kw.setdefault("score", "sigmoid")
    kw.setdefault("top_groups", kw.get("n_groups", 1))
    R = ref.route(z.astype(np.float64), bias=bias, **kw)
    assert R[5].min() > 1e-6, "the case hangs on less than fp32 resolves"
    assert np.array_equal(ids, R[0])
    for a, b in zip((counts, offsets, srt), R[2:5]):
        assert np.array_equal(a, b)
    units = 32 if kw["score"] == "sigmoid" else 32 + 28 + 40
    assert (np.abs(w - R[1]) <= units * U * np.abs(R[1]) + 1e-37).all()
    return ids


def logits(rng, rows, E, kw, bias, dtype, spread=1.5):
    """Random rows whose orders fp32 resolves."""
    cast = lambda v: torch.from_numpy(v).to(dtype).float().numpy()  # noqa: E731
    z = cast(rng.standard_normal((rows, E)) * spread)
    for _ in range(20):
        mg = ref.route(z.astype(np.float64), bias=bias, **kw)[5]
        bad = np.nonzero(mg <= 2e-6)[0]
        if bad.size == 0:
            return z
        z[bad] = cast(rng.standard_normal((bad.size, E)) * spread)
    raise AssertionError("no such rows found")


CASES = [
    dict(E=256, top_k=6, score="sigmoid", n_groups=8, top_groups=4, group_score="top2"),
    dict(E=256, top_k=8, score="softmax", n_groups=8, top_groups=3, group_score="max",
         renorm=False, scale=16.0),
    dict(E=160, top_k=6, score="softmax", n_groups=8, top_groups=3, group_score="top2"),
    dict(E=64, top_k=1, score="sigmoid"),
    dict(E=65, top_k=16, score="softmax", scale=2.5),
    dict(E=512, top_k=16, score="sigmoid", n_groups=64, top_groups=7, group_score="max"),
    dict(E=510, top_k=5, score="softmax", n_groups=3, top_groups=1, group_score="top2"),
    dict(E=8, top_k=8, score="softmax", n_groups=4, top_groups=4, group_score="max"),
    dict(E=2, top_k=1, score="sigmoid", n_groups=2, top_groups=1, group_score="top2"),
    dict(E=1, top_k=1, score="softmax"),
]


@pytest.mark.parametrize("rows", [1, 2, 16, 17, 64, 100, 333])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_formula(i, rows):
    kw = dict(CASES[i])
    E = kw.pop("E")
    rng = np.random.default_rng(1000 * i + rows)
    bias = 0.1 * rng.standard_normal(E).astype(np.float32).astype(np.float64) if rows % 2 else None
    dtype = torch.bfloat16 if rows in (2, 100) else torch.float32
    z = logits(rng, rows, E, dict(kw, top_groups=kw.get("top_groups", 1)), bias, dtype)
    check(z, kw, bias, dtype, pad=rows % 5)


@pytest.mark.parametrize("rows", [4096, 8200, 20000])
def test_many_rows_group_stably(rows):
    """Past 8192 rows a run is more than one pass; ids themselves are checked on
    a sample, the grouping of all of them against a stable sort."""
    E, k = 128, 8
    rng = np.random.default_rng(rows)
    z = rng.standard_normal((rows, E)).astype(np.float32)
    z[:, :3] += 3.0  # crowded experts
    rule = m.RouterRule(E, k, n_groups=4, top_groups=2)
    ids, w, counts, offsets, srt = run(z, rule)
    for a, b in zip((counts, offsets, srt), ref.group(ids, E)):
        assert np.array_equal(a, b)
    at = rng.choice(rows, 200, replace=False)
    R = ref.route(z[at].astype(np.float64), k, "sigmoid", None, 4, 2)
    ok = R[5] > 1e-6
    assert ok.sum() > 150 and np.array_equal(ids[at][ok], R[0][ok])
    one = run(z[:5], rule)
    assert np.array_equal(one[0], ids[:5]) and np.array_equal(one[1], w[:5])


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_index(rows, score):
    E = 96
    z = np.zeros((rows, E), dtype=np.float32)
    z[1:, 10::7] = 1.0
    z[2:, 95] = 1.0
    ids = check(z, dict(top_k=12, score=score, n_groups=6, top_groups=2, group_score="max"))
    assert list(ids[0]) == list(range(12))
    check(z, dict(top_k=12, score=score, n_groups=6, top_groups=2, group_score="top2"))
    check(z, dict(top_k=16, score=score))


@pytest.mark.parametrize("rows", [5, 50])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_experts_out_of_reach(rows, score, group_score):
    """-infinity and NaN take an expert out, bias or not; rows with fewer
    experts than slots, and with none, hold -1 and 0 in what is left."""
    E = 64
    rng = np.random.default_rng(rows)
    z = (rng.permutation(E * rows).reshape(rows, E) / (8.0 * rows)).astype(np.float32) - 4
    z[0] = -np.inf
    z[1] = np.nan
    z[2, 3:] = -np.inf
    z[3, :60] = np.nan
    z[4, ::2] = -np.inf
    # (steps no sum of logits' scores comes near)
    bias = np.where(np.arange(E) % 2 == 0, 50.0, 0.0)
    kw = dict(top_k=6, score=score, n_groups=8, top_groups=5, group_score=group_score)
    for b in (None, bias):
        rule = m.RouterRule(E, bias=None if b is None else
                            torch.from_numpy(b.astype(np.float32)).to(DEV), **kw)
        ids, w, counts, offsets, srt = run(z, rule)
        assert (ids[0] == -1).all() and (ids[1] == -1).all() and (w[:2] == 0).all()
        assert sorted(ids[2][:3]) == [0, 1, 2] and (ids[2][3:] == -1).all()
        assert (w[2][3:] == 0).all() and abs(w[2].sum() - 1) < 1e-6
        assert sorted(ids[3][:4]) == [60, 61, 62, 63] and (ids[3][4:] == -1).all()
        assert (ids[4] % 2 == 1).all()
        for a, r in zip((counts, offsets, srt), ref.group(ids, E)):
            assert np.array_equal(a, r)
        reach = np.isfinite(z)
        t, s = np.nonzero(ids >= 0)
        assert reach[t, ids[t, s]].all()


@pytest.mark.parametrize("rows", [2, 20])
def test_extreme_logits(rows):
    E = 32
    low = np.finfo(np.float32).min
    z = np.zeros((rows, E), dtype=np.float32)
    z[0] = low                       # every logit the type's lowest value
    z[1] = low
    z[1, 5], z[1, 9] = np.inf, np.inf
    soft = m.RouterRule(E, 4, score="softmax")
    ids, w, *_ = run(z, soft)
    assert list(ids[0]) == [0, 1, 2, 3] and (w[0] == 0.25).all()
    assert list(ids[1]) == [5, 9, 0, 1] and list(w[1]) == [0.5, 0.5, 0, 0]
    sig = m.RouterRule(E, 4, score="sigmoid")
    ids, w, *_ = run(z, sig)
    assert list(ids[0]) == [0, 1, 2, 3] and (w[0] == 0).all()  # a sum of 0 divides nothing
    assert list(ids[1]) == [5, 9, 0, 1] and list(w[1]) == [0.5, 0.5, 0, 0]


def test_zero_rows():
    rule = m.RouterRule(40, 3)
    out = m.route_outputs(0, 40, 3)
    for t in out:
        t.fill_(7)
    m.moe_route_scored(rule, torch.empty((0, 40), device=DEV), out=out)
    assert (out[2] == 0).all() and (out[3] == 0).all()


def test_feeds_the_plain_rule():
    """Sigmoid scores, one group, no bias: moe_route_group's picks, weights
    and grouping."""
    rng = np.random.default_rng(5)
    for rows in (4, 200):
        z = rng.standard_normal((rows, 256)).astype(np.float32)
        got = run(z, m.RouterRule(256, 6))
        want = [t.cpu().numpy() for t in m.moe_route_group(torch.from_numpy(z).to(DEV), 6)]
        for a, b in zip(got, want):
            assert np.array_equal(a, b)


def test_refusals():
    z = torch.zeros((20, 64), device=DEV)
    rule = m.RouterRule(64, 4)
    with pytest.raises(ValueError):
        m.moe_route_scored(m.RouterRule(32, 4), z)
    with pytest.raises(m.MoeError):
        m.moe_route_scored(m.RouterRule(64, 17), z)
    with pytest.raises(m.MoeError):
        m.moe_route_scored(m.RouterRule(64, 4, n_groups=7), z)
    with pytest.raises(m.MoeError):
        m.moe_route_scored(rule, z, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    out = m.route_outputs(20, 64, 4)
    with pytest.raises(TypeError):
        m.moe_route_scored(rule, z, out=(out[0].long(),) + out[1:])
    with pytest.raises(ValueError):
        m.moe_route_scored(rule, z, out=m.route_outputs(19, 64, 4))
