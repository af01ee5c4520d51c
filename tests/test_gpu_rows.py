"""GPU parity of the operators on rows of vocabulary logits against the
float64 oracle: filtered sampling, the filtered accept, top logits and
distillation.

Integer outputs are compared exactly wherever the decision has a margin in
the oracle: 2e-5 between the two best scores (fp32 scores carry about 1e-5 at
magnitude 30; closer calls are settled in double, which has tests of its own),
1e-6 between a uniform and a probability (the weights'
exponentials are good to 2^-22).  Where an entry's sum is within 1e-6 of
top-p's border the kept set may differ by entries of that mass: they are one
in a million to be drawn, and move a log-probability by less than 4e-6.

Tolerances.  A log-probability is (z - m)/T - ln W: three roundings of the
first term, the relative error of W (2^-22 an exponential) and two of the
logarithm: (|lp| + |ln W| + 4) 2^-21 covers them.  Distillation: loss terms
p_k (lp_k - lq_k) carry the same errors, summed with weights that add up to
at most one, so (1 + largest |lp|, |lq|) 2^-20; gradients are differences of
probabilities (each good to (4 + |x|) 2^-23 of its value, x its exponent)
scaled by weight / T (outside the listed tokens the second of them is p_r
times a share, and p_r is one minus a rounded sum), plus the output type's
half step and fp16's smallest step.
"""
import math

import numpy as np
import pytest

from oracle import rows_oracle as RO
from tests.gpu_util import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

if gpu_available():
    import torch
    from block_diffusion_speculative_draft_gb300 import api
    DEV = torch.device("cuda:0")
    DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _padded(a, dtype, pad):
    """Device copy of a [..., V] whose rows are V + pad apart, NaN between."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(DT[dtype])
    buf = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), float("nan"), dtype=t.dtype, device=DEV)
    buf[..., : t.shape[-1]] = t
    return buf[..., : t.shape[-1]]


def _host(t):
    return t.double().cpu().numpy()


def _dev(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a, dt)).to(DEV)


def _uniforms(rng, shape):
    return ((2 * rng.integers(0, 1 << 23, size=shape) + 1) * 2.0 ** -24).astype(np.float32)


def _logits(rng, n, V, kind):
    z = rng.normal(0, 2.0, size=(n, V))
    if kind == "peaked":
        h = min(V, 40)
        for r in range(n):
            z[r, rng.choice(V, h, replace=False)] = 14 - 1.3 * np.log1p(np.arange(h)) + rng.normal(0, 0.4, h)
    elif kind == "ties":  # few distinct values
        z = np.round(z)
    elif kind == "equal":
        z[:] = 3.25
    elif kind == "masked":
        z[rng.random((n, V)) < 0.7] = -np.inf
        z[rng.random((n, V)) < 0.1] = np.nan
        z[rng.random((n, V)) < 0.05] = -65504.0
        z[0] = -np.inf
        z[1 % n, :] = np.nan
        z[2 % n, :] = -65504.0
    elif kind == "far":  # exponents far below the weights' resolution
        z *= 40
    elif kind == "sparse":  # fewer entries than top-k asks for
        z[rng.random((n, V)) > 20 / V] = -np.inf
    return z


def _ask(rng, n, mode):
    T = rng.uniform(0.5, 1.5, n).astype(np.float32)
    k = np.zeros(n, np.int32)
    p = np.ones(n, np.float32)
    mp = np.zeros(n, np.float32)
    for i in range(n):
        m = ["k", "p", "m", "kp", "kpm", "none", "greedy", "wide"][i % 8] if mode == "mixed" else mode
        if m == "greedy":
            T[i] = 0
        if m in ("k", "kp", "kpm"):
            k[i] = rng.integers(1, 80)
        if m in ("p", "kp", "kpm"):
            p[i] = rng.uniform(0.3, 0.99)
        if m in ("m", "kpm"):
            mp[i] = rng.uniform(0.001, 0.3)
        if m == "wide":
            k[i] = rng.integers(1000, 6000)
            p[i] = 0.9995
    return T, k, p, mp


def _top_p_border(z, T, k, p):
    """How close the sum before any entry comes to top-p's bound (relative)."""
    ids = RO.row_order(z)
    if T == 0 or p >= 1 or ids.size == 0:
        return math.inf
    if k > 0:
        ids = ids[:k]
    w = np.exp((z[ids] - z[ids[0]]) / T)
    before = np.concatenate([[0.0], np.cumsum(w)])
    return float(np.abs(before / before[-1] - p).min())


def _check_sample(z, u, T, k, p, mp, tok, lp):
    for r in range(len(tok)):
        rt, rl, gap = RO.sample(z[r], float(T[r]), u[r], int(k[r]), float(p[r]), float(mp[r]))
        # entries within 1e-6 of top-p's border may fall on its other side
        slack = 4e-6 if _top_p_border(z[r], float(T[r]), int(k[r]), float(p[r])) < 1e-6 else 0.0
        if gap > 2e-5:
            assert tok[r] == rt, (r, T[r], k[r], p[r], mp[r])
        if rt < 0:
            assert tok[r] == -1 and lp[r] == -np.inf
        elif tok[r] == rt:
            lnw = math.log(np.sum(np.exp((z[r][RO.row_order(z[r])] - np.nanmax(z[r])) / max(float(T[r]), 1e-6))))
            assert abs(lp[r] - rl) <= (abs(rl) + lnw + 4) * 2.0 ** -21 + slack, (r, lp[r], rl)


def _sample(zt, T, k, p, mp, u, stream=None, filters=True):
    n = zt.shape[0]
    tok = torch.full((n,), -7, dtype=torch.int32, device=DEV)
    lp = torch.full((n,), -7.0, dtype=torch.float32, device=DEV)
    f = dict(top_k=_dev(k, np.int32), top_p=_dev(p, np.float32), min_p=_dev(mp, np.float32)) if filters else {}
    api.dflash_sample(zt, _dev(T, np.float32), u, tok, logprob_out=lp, stream=stream, **f)
    return tok, lp


@pytest.mark.parametrize("dtype,n,V,pad,kind,mode", [
    ("f32", 9, 1, 0, "peaked", "mixed"), ("f16", 9, 2, 1, "peaked", "mixed"), ("bf16", 9, 3, 0, "ties", "mixed"),
    ("f32", 16, 31, 1, "peaked", "mixed"), ("f32", 16, 33, 0, "ties", "mixed"), ("f16", 16, 257, 3, "equal", "mixed"),
    ("f32", 24, 2047, 0, "peaked", "mixed"), ("bf16", 24, 2049, 5, "peaked", "mixed"),
    ("f32", 24, 4096, 0, "masked", "mixed"), ("f16", 24, 4099, 2, "masked", "mixed"),
    ("bf16", 24, 5003, 0, "masked", "mixed"), ("f32", 24, 9001, 7, "far", "mixed"),
    ("bf16", 32, 20011, 0, "ties", "mixed"), ("f32", 32, 20000, 0, "flat", "mixed"),
    ("bf16", 16, 50021, 11, "flat", "mixed"), ("f32", 8, 151936, 0, "flat", "mixed"),
    ("bf16", 8, 151936, 0, "flat", "p"), ("f16", 8, 151936, 0, "peaked", "kp"), ("f32", 2, 300007, 1, "peaked", "p"),
    ("bf16", 1, 151936, 0, "peaked", "kpm"), ("f32", 1, 151936, 0, "flat", "none"),
    ("bf16", 400, 3001, 0, "peaked", "mixed"), ("f32", 3, 1000003, 0, "flat", "kp"), ("bf16", 2, 1200001, 3, "flat", "p"),
])
def test_sample(dtype, n, V, pad, kind, mode):
    rng = np.random.default_rng(V + n)
    zt = _padded(_logits(rng, n, V, kind), dtype, pad)
    T, k, p, mp = _ask(rng, n, mode)
    u = _uniforms(rng, (n, V))
    ut = _padded(u, "f32", pad)
    tok, lp = _sample(zt, T, k, p, mp, ut)
    again = _sample(zt, T, k, p, mp, ut)
    assert api.dflash_get_status() == 0
    assert torch.equal(tok, again[0]) and torch.equal(lp, again[1])
    _check_sample(_host(zt), u, T, k, p, mp, tok.cpu().numpy(), lp.cpu().numpy())


@pytest.mark.parametrize("dtype,n,V,pad,kind,mode,rows", [
    ("bf16", 160, 151936, 0, "flat", "mixed", 24), ("f32", 330, 60001, 3, "flat", "p", 12),
    ("bf16", 330, 151936, 0, "ties", "p", 8), ("f16", 330, 90001, 1, "flat", "m", 12),
    ("bf16", 330, 90001, 0, "flat", "wide", 6), ("f16", 310, 90000, 0, "masked", "mixed", 16),
    ("bf16", 2200, 83000, 0, "flat", "p", 6),
])
def test_sample_leaves_wide_rows_to_a_second_launch(dtype, n, V, pad, kind, mode, rows):
    # batches large enough that a row has few CTAs; some of the rows are checked
    rng = np.random.default_rng(V + n)
    base = _logits(rng, 32, V, kind)
    zt = _padded(np.zeros((n, V), np.float32), dtype, pad)
    some = _padded(base, dtype, 0)
    for r in range(n):
        zt[r] = torch.roll(some[r % 32], 37 * (r // 32))
    T, k, p, mp = _ask(rng, n, mode)
    u = torch.rand((n, V + pad), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    u = (u * (1 << 23)).floor().mul_(2).add_(1).mul_(2.0 ** -24)[:, :V]
    tok, lp = _sample(zt, T, k, p, mp, u)
    again = _sample(zt, T, k, p, mp, u)
    assert api.dflash_get_status() == 0
    assert torch.equal(tok, again[0]) and torch.equal(lp, again[1])
    pick = np.sort(rng.choice(n, rows, replace=False))
    at = torch.from_numpy(pick).to(DEV)
    _check_sample(_host(zt[at]), u[at].cpu().numpy(), T[pick], k[pick], p[pick], mp[pick], tok[at].cpu().numpy(),
                  lp[at].cpu().numpy())


@pytest.mark.parametrize("dtype,n,V,kind,mode,rows", [
    ("f32", 200, 100003, "flat", "p", 12), ("f32", 200, 100003, "flat", "mixed", 16),
    ("f32", 200, 100003, "sparse", "k", 12), ("f32", 100, 200003, "flat", "p", 8),
    ("f32", 100, 200003, "ties", "mixed", 16), ("f32", 100, 200003, "sparse", "mixed", 16),
    ("bf16", 160, 200003, "flat", "p", 8), ("f16", 160, 200003, "sparse", "kp", 12),
])
def test_sample_leaves_rows_of_clusters_to_a_second_launch(dtype, n, V, kind, mode, rows):
    # two or four CTAs a row in the first launch, each with more than 160 KB: a CTA
    # that gives a row up must not end while its peers read its groups
    test_sample_leaves_wide_rows_to_a_second_launch(dtype, n, V, 0, kind, mode, rows)


@pytest.mark.parametrize("V", [769, 900, 1024])
@pytest.mark.parametrize("kind,mode", [("flat", "p"), ("ties", "mixed")])
def test_sample_under_top_p_where_a_whole_row_fits_the_list(V, kind, mode):
    # a row whose groups hold too little is given up by all of its threads or none
    test_sample("f32", 64, V, 0, kind, mode)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1e-6, 1e-3, 50.0, 1e6])
def test_sample_at_the_ends_of_the_temperature(dtype, T):
    rng = np.random.default_rng(21)
    n, V = 12, 30011
    z = _logits(rng, n, V, "flat")
    z[3] += 3000.0                       # far from zero
    z[4] = float(torch.finfo(DT[dtype]).min)
    z[5, 100:] = float(torch.finfo(DT[dtype]).min)
    zt = _padded(z, dtype, 0)
    _, k, p, mp = _ask(rng, n, "mixed")
    t = np.full(n, T, np.float32)
    u = _uniforms(rng, (n, V))
    tok, lp = _sample(zt, t, k, p, mp, _dev(u, np.float32))
    assert api.dflash_get_status() == 0
    _check_sample(_host(zt), u, t, k, p, mp, tok.cpu().numpy(), lp.cpu().numpy())


@pytest.mark.parametrize("far", [300.0, 5000.0, -20000.0, 40000.0])
@pytest.mark.parametrize("T,mode", [(0.7, "mixed"), (0.7, "none"), (0.05, "p"), (0.05, "none")])
def test_sample_far_from_zero(T, mode, far):
    # T apart from the logits' size: sums whose references differ meet without a trace of it
    rng = np.random.default_rng(31)
    n, V = 16, 30011
    zt = _padded(far + _logits(rng, n, V, "flat") * T, "f32", 0)
    _, k, p, mp = _ask(rng, n, mode)
    t = np.full(n, T, np.float32)
    u = _uniforms(rng, (n, V))
    tok, lp = _sample(zt, t, k, p, mp, _dev(u, np.float32))
    assert api.dflash_get_status() == 0
    _check_sample(_host(zt), u, t, k, p, mp, tok.cpu().numpy(), lp.cpu().numpy())


def test_sample_takes_every_border_of_a_worked_row():
    # weights 8, 4, 4, 2, 1 at T = 1 / ln 2; the uniforms make the last kept
    # entry of the order the winner
    z = np.array([[1.0, 3.0, 0.0, 2.0, 2.0]] * 9, np.float32)
    order = [1, 3, 4, 0, 2]
    k = np.array([1, 2, 3, 4, 5, 0, 0, 0, 0], np.int32)
    p = np.array([1, 1, 1, 1, 1, 0.40, 0.43, 0.64, 0.95], np.float32)
    mp = np.zeros(9, np.float32)
    last = [0, 1, 2, 3, 4, 0, 1, 2, 4]
    u = np.full((9, 5), 0.5, np.float32)
    for r in range(9):
        for i, v in enumerate(order):
            u[r, v] = 1 - 2.0 ** -(4 + 3 * i)
    T = np.full(9, 1 / math.log(2), np.float32)
    tok, _ = _sample(_dev(z, np.float32), T, k, p, mp, _dev(u, np.float32))
    assert tok.tolist() == [order[i] for i in last]
    # the same bounds as min-p: exactly the maximum, and a bound between entries
    mp = np.array([1.0, 0.51, 0.49, 0.26, 0.2, 0.12, 0, 0, 0], np.float32)
    tok, _ = _sample(_dev(z, np.float32), T, np.zeros(9), np.ones(9), mp, _dev(u, np.float32))
    assert tok.tolist() == [order[i] for i in [0, 0, 2, 2, 3, 4, 4, 4, 4]]


@pytest.mark.parametrize("dtype,n,V", [("f32", 6, 20000), ("bf16", 6, 20001), ("f16", 40, 40000), ("bf16", 330, 90001)])
def test_sample_keeps_top_k_s_border_under_top_p(dtype, n, V):
    # rows beyond the short list whose last entry under top-k is also top-p's, alone
    # of its kind above many that top-k drops; those have the higher uniforms
    rng = np.random.default_rng(V)
    z = np.full((3, V), 3.0)
    z[0] = 2.5                                                  # equal: k = 1
    at = [rng.choice(V, 1101, replace=False) for _ in range(3)]
    for r in (1, 2):
        z[r, at[r]] = 5 + rng.random(1101)
        z[r, at[r][7]] = 3.875 if r == 1 else 3.0               # the last of 1101, or the first of many at 3
    k, p = np.array([1, 1101, 1101]), np.array([0.999, 0.999995, 0.999995])
    some = _padded(z, dtype, 0)
    h = _host(some)
    u = np.full((3, V), 0.25, np.float32)
    for r in range(3):
        ids = RO.filtered(h[r], 1.0, int(k[r]), float(np.float32(p[r])))[0]
        assert ids.size == k[r]
        u[r, np.setdiff1d(np.arange(V), ids)] = 1 - 2.0 ** -20
    zt, ut = some[torch.arange(n, device=DEV) % 3].contiguous(), _dev(u, np.float32)[torch.arange(n, device=DEV) % 3].contiguous()
    row = np.arange(n) % 3
    tok, _ = _sample(zt, np.ones(n), k[row], p[row], np.zeros(n), ut)
    assert api.dflash_get_status() == 0
    for r in range(3):
        assert (tok.cpu().numpy()[r::3] == RO.sample(h[r], 1.0, u[r], int(k[r]), float(np.float32(p[r])))[0]).all(), r


@pytest.mark.parametrize("dtype,n,V", [("f32", 20, 40000), ("bf16", 20, 151936), ("f16", 330, 90000), ("f32", 5, 900)])
@pytest.mark.parametrize("p", [0.0, 2.0 ** -149, 1e-9])
def test_sample_under_a_top_p_of_next_to_nothing(dtype, n, V, p):
    # the first entry alone, wherever the others lie: far below it, some hundred just
    # below it (a long list whose first bin holds one entry), all at its height
    rng = np.random.default_rng(V)
    z = np.full((5, V), -10.0) + rng.normal(0, 0.5, (5, V))
    for r, height in enumerate((0.0, 9.5, 9.9, 9.99)):
        at = rng.choice(V, 400, replace=False)
        z[r, at] = height - 0.05 * rng.random(400)
        z[r, at[rng.integers(0, 400)]] = 10.0
    z[4] = 1.0
    some = _padded(z, dtype, 0)
    zt = some[torch.arange(n, device=DEV) % 5].contiguous()
    u = _dev(_uniforms(rng, (5, V)), np.float32)[torch.arange(n, device=DEV) % 5].contiguous()
    first = _first(_host(some))[np.arange(n) % 5]
    for T, mp in ((1.0, 0.0), (30.0, 0.0), (1.0, 1e-4)):
        tok, lp = _sample(zt, np.full(n, T), np.zeros(n), np.full(n, p), np.full(n, mp), u)
        assert api.dflash_get_status() == 0
        assert np.array_equal(tok.cpu().numpy(), first), (T, mp)
        assert float(lp.abs().max()) < 1e-6


def test_sample_follows_its_distribution():
    rng = np.random.default_rng(5)
    n, V = 6000, 40
    z = rng.normal(0, 1.5, V).astype(np.float32)
    zt = _dev(np.broadcast_to(z, (n, V)), np.float32)
    T, k, p, mp = (np.full(n, a) for a in (0.9, 6, 0.95, 0.01))
    tok, _ = _sample(zt, T, k.astype(np.int32), p, mp, _dev(_uniforms(rng, (n, V)), np.float32))
    ids, q = RO.filtered(z, 0.9, 6, 0.95, 0.01)
    got = np.bincount(tok.cpu().numpy(), minlength=V)
    assert got.sum() == got[ids].sum()
    assert ids.size <= 6 and float(((got[ids] - n * q) ** 2 / (n * q)).sum()) < 20.52  # <= 5 degrees, 99.9 %


def test_sample_near_ties_are_settled_in_double():
    # scores that fp32 cannot tell apart: equal uniforms, logits one step apart
    V, n = 4096, 6
    z = np.zeros((n, V), np.float32)
    hi = np.float32(2.0 ** -26)
    at = [3, 700, 1500, 2222, 4000, 4095]
    for r in range(n):
        z[r, at[r]] = hi
    u = np.full((n, V), 0.5, np.float32)
    tok, _ = _sample(_dev(z, np.float32), np.full(n, 0.9), np.zeros(n), np.ones(n), np.zeros(n), _dev(u, np.float32))
    # a thread keeps the first of its own equal fp32 scores; the winner is
    # either the larger logit or, where one thread holds both, an earlier entry
    for r in range(n):
        assert tok[r] == at[r] or tok[r] < at[r]
    z[:] = 1.5
    tok, _ = _sample(_dev(z, np.float32), np.full(n, 0.9), np.zeros(n), np.ones(n), np.zeros(n), _dev(u, np.float32))
    assert tok.tolist() == [0] * n


def _near_tied(rng, n, V, dtype):
    """Rows with two entries whose scores lie within 1e-6 of each other, far above
    the others' but not the same in double: next to each other (one thread's), a few
    packs apart, or anywhere; in either order.  (logits, uniforms, temperatures)"""
    z = rng.normal(0, 1, (n, V))
    T = np.full(n, np.float32(0.9))
    zt = _padded(z, dtype, 0)
    u = (_uniforms(rng, (n, V)) * np.float32(0.01)).astype(np.float32)
    h = _host(zt)
    for r in range(n):
        i = int(rng.integers(0, V - 1)) & ~3
        j = [i + 1, (i + 4096) % V, int(rng.integers(0, V)), i + 2][r % 4]
        if r % 3 == 0:
            i, j = j, i
        while True:
            zt[r, i] = h[r].max() + 0.5
            zt[r, j] = h[r].max() + 0.5 - rng.uniform(0.05, 0.3)
            a, b = float(zt[r, i]) / float(T[r]), float(zt[r, j]) / float(T[r])
            u[r, i] = np.float32(rng.uniform(0.4, 0.7))
            u[r, j] = np.float32(math.exp(-math.exp(-(a - math.log(-math.log(float(u[r, i]))) - b))))
            gap = abs(a - math.log(-math.log(float(u[r, i]))) - b + math.log(-math.log(float(u[r, j]))))
            if i != j and 1e-9 < gap < 1e-6:
                break
            j = (i + 1 + int(rng.integers(0, V - 1))) % V if i == j else j
    return zt, u, T


# nothing; deep top-p; min-p over many, and over some hundred entries; top-k by the
# sorted list, by its short form and beyond it; all together
NEAR = [(0, 1, 0), (0, 0.97, 0), (0, 1, 1e-3), (0, 1, 0.08), (600, 1, 0), (40, 0.99, 0), (3000, 1, 0), (2000, 0.999, 1e-3)]


@pytest.mark.parametrize("k,p,mp", NEAR)
@pytest.mark.parametrize("dtype,n,V", [("f32", 24, 20000), ("bf16", 24, 20001), ("f16", 1, 151936), ("f32", 330, 60000),
                                       ("f32", 130, 9000)])
def test_sample_tells_scores_apart_that_fp32_cannot(dtype, n, V, k, p, mp):
    rng = np.random.default_rng(n + k)
    some = min(n, 24)
    zt, u, T = _near_tied(rng, some, V, dtype)
    at = torch.arange(n, device=DEV) % some
    big, ub = zt[at].contiguous(), _dev(u, np.float32)[at].contiguous()
    ask = np.full(n, T[0]), np.full(n, k), np.full(n, p), np.full(n, mp)
    tok, _ = _sample(big, *ask, ub)
    assert torch.equal(tok, _sample(big, *ask, ub)[0]) and api.dflash_get_status() == 0
    z, tok = _host(zt), tok.cpu().numpy()
    for r in range(some):
        want = RO.sample(z[r], float(T[r]), u[r], k, float(np.float32(p)), float(np.float32(mp)))[0]
        assert (tok[r::some] == want).all(), (r, want)


@pytest.mark.parametrize("k,p,mp", NEAR)
@pytest.mark.parametrize("dtype,b,V", [("f32", 12, 20000), ("bf16", 3, 151936), ("f32", 170, 60000)])
def test_accept_tells_scores_apart_that_fp32_cannot(dtype, b, V, k, p, mp):
    # sequences without a draft: the draw at their first row
    rng = np.random.default_rng(b + k)
    some = min(b, 12)
    zt, u, T = _near_tied(rng, some, V, dtype)
    at = torch.arange(b, device=DEV) % some
    z3 = zt[at].unsqueeze(1).expand(b, 2, V).contiguous()
    n, c, _, _ = _accept(z3, np.full((b, 1), -1), np.full(b, T[0]), np.full(b, k), np.full(b, p), np.full(b, mp),
                         np.zeros((b, 1)), _dev(u, np.float32)[at].contiguous())
    assert api.dflash_get_status() == 0 and not n.any()
    z = _host(zt)
    for r in range(some):
        want = RO.sample(z[r], float(T[r]), u[r], k, float(np.float32(p)), float(np.float32(mp)))[0]
        assert (c[r::some] == want).all(), (r, want)


def test_sample_without_filters_and_bad_parameters():
    rng = np.random.default_rng(6)
    n, V = 10, 777
    z, u = _logits(rng, n, V, "peaked"), _uniforms(rng, (n, V))
    zt, ut = _padded(z, "f32", 0), _dev(u, np.float32)
    T = np.full(n, 0.8, np.float32)
    tok, lp = _sample(zt, T, None, None, None, ut, filters=False)
    _check_sample(_host(zt), u, T, np.zeros(n, int), np.ones(n), np.zeros(n), tok.cpu().numpy(), lp.cpu().numpy())
    assert api.dflash_get_status() == 0
    k, p, mp = np.zeros(n, np.int32), np.ones(n, np.float32), np.zeros(n, np.float32)
    T[:6] = [-1.0, np.nan, np.inf, 1e-9, 1e9, 0.8]
    k[5], p[6], mp[7] = -1, 1.5, np.nan
    tok, lp = _sample(zt, T, k, p, mp, ut)
    assert api.dflash_get_status() == api.DEV_BAD_PARAM
    assert tok.tolist()[:8] == [-1] * 8 and np.isneginf(lp.cpu().numpy()[:8]).all()
    _check_sample(_host(zt)[8:], u[8:], T[8:], k[8:], p[8:], mp[8:], tok.cpu().numpy()[8:], lp.cpu().numpy()[8:])


def test_sample_infinite_logits_win():
    z = np.zeros((3, 600), np.float32)
    z[0, 77] = np.inf
    z[1, [5, 599]] = np.inf
    z[2, [5, 599]] = np.inf
    u = np.full((3, 600), 0.5, np.float32)
    u[1, 599] = 0.9
    u[2, 5] = 0.9
    tok, lp = _sample(_dev(z, np.float32), np.ones(3), np.zeros(3), np.array([1, 0.9, 1]), np.zeros(3),
                      _dev(u, np.float32))
    assert tok.tolist() == [77, 599, 5]
    assert np.abs(lp.cpu().numpy() - [0, -math.log(2), -math.log(2)]).max() < 1e-6


def _greedy_rows(rng, n, V, dtype):
    """Rows whose largest entry no short list of the row's groups gives, in turn:
    all but a few entries at the type's lowest value, one and several infinities,
    more equal maxima than the list holds, nothing but the lowest value, a NaN and
    infinities below the maximum; and a plain row."""
    low = float(torch.finfo(DT[dtype]).min)
    z = rng.normal(0, 2.0, (n, V))
    for r in range(n):
        some = V // 3 + rng.choice(V // 3, 5, replace=False)
        if r % 7 == 0:
            keep = z[r, some]
            z[r] = low
            z[r, some] = keep
        elif r % 7 == 1:
            z[r, some[0]] = np.inf
        elif r % 7 == 2:
            z[r, some] = np.inf
        elif r % 7 == 3:
            z[r, rng.integers(0, 5)::7] = 11.0
        elif r % 7 == 4:
            z[r] = low
        elif r % 7 == 5:
            z[r, some] = [np.nan, -np.inf, low, np.nan, -np.inf]
    return z


def _first(z):
    return np.where(np.isnan(z), -np.inf, z).argmax(-1)


@pytest.mark.parametrize("dtype,n,V", [("f32", 14, 20011), ("bf16", 14, 20011), ("f16", 14, 20011), ("f32", 70, 9001),
                                       ("f32", 7, 151936), ("f32", 200, 100003), ("bf16", 330, 90001)])
def test_sample_at_zero_temperature_takes_the_first_entry_of_any_row(dtype, n, V):
    rng = np.random.default_rng(n)
    base = _padded(_greedy_rows(rng, 14, V, dtype), dtype, 0)
    zt = base[torch.arange(n, device=DEV) % 14].contiguous()
    _, k, p, mp = _ask(rng, n, "mixed")
    # (a row's uniforms do not matter)
    tok, lp = _sample(zt, np.zeros(n), k, p, mp, torch.full((n, V), float("nan"), device=DEV))
    assert api.dflash_get_status() == 0
    assert np.array_equal(tok.cpu().numpy(), _first(_host(base))[np.arange(n) % 14]) and not lp.any()


def test_sample_infinite_logits_win_whatever_their_uniforms():
    # u = 0 scores -inf, as every finite logit beside an infinite one does
    n, V = 6, 5000
    z = np.zeros((n, V), np.float32)
    z[:, 77], z[3:, 4000] = np.inf, np.inf
    u = np.full((n, V), 0.5, np.float32)
    u[:, 77] = 0
    u[4:, 4000] = 0
    k, p, mp = np.array([0, 0, 300, 0, 0, 300]), np.array([1, 0.9, 1, 1, 1, 0.5]), np.array([0, 0, 0, 0, 0.1, 0])
    tok, lp = _sample(_dev(z, np.float32), np.ones(n), k, p, mp, _dev(u, np.float32))
    assert tok.tolist() == [77, 77, 77, 4000, 77, 77]
    assert np.abs(lp.cpu().numpy() - [0, 0, 0, -math.log(2), -math.log(2), 0]).max() < 1e-6


# --------------------------------------------------------------- accept -----
def _accept(zt, draft, T, k, p, mp, ua, us, **kw):
    b, R, _ = zt.shape
    outs = [torch.full((b,), -7, dtype=torch.int32, device=DEV) for _ in range(3)]
    em = torch.full((b, R), -7, dtype=torch.int32, device=DEV)
    api.dflash_verify_accept_filtered(zt, _dev(draft, np.int32), _dev(T, np.float32), _dev(ua, np.float32), us,
                                      outs[0], outs[1], top_k=_dev(k, np.int32), top_p=_dev(p, np.float32),
                                      min_p=_dev(mp, np.float32), emitted=em, next_tok=outs[2], **kw)
    return [o.cpu().numpy() for o in (outs[0], outs[1], em, outs[2])]


def _accept_margin(z, draft, T, k, p, mp, ua, us):
    """Smallest margin of the decisions that lead to the oracle's answer."""
    m = math.inf
    for r in range(len(z)):
        m = min(m, _top_p_border(z[r], T, k, p))
        ids, q = RO.filtered(z[r], T, k, p, mp)
        drop = None
        if r < len(draft):
            hit = q[ids == draft[r]]
            if hit.size:
                m = min(m, abs(float(ua[r]) - hit[0]))
            if hit.size and ua[r] < hit[0]:
                continue
            drop = int(draft[r])
        if T > 0 and ids.size:
            m = min(m, RO.gumbel_draw(ids, q, us, drop)[1] / 20)
        break
    return m


@pytest.mark.parametrize("dtype,b,R,D,V,pad,kind,mode", [
    ("f32", 16, 4, 3, 50, 0, "peaked", "mixed"), ("f16", 9, 5, 5, 333, 3, "ties", "mixed"),
    ("bf16", 8, 16, 15, 4096, 0, "peaked", "mixed"), ("f32", 8, 6, 5, 4001, 2, "masked", "mixed"),
    ("bf16", 3, 32, 31, 20011, 0, "flat", "mixed"), ("f32", 1, 16, 15, 151936, 0, "peaked", "kp"),
    ("bf16", 2, 64, 63, 9000, 1, "peaked", "p"), ("f16", 24, 1, 1, 1000, 0, "peaked", "mixed"),
    ("f32", 8, 2, 1, 1, 0, "peaked", "mixed"),
])
def test_accept(dtype, b, R, D, V, pad, kind, mode):
    rng = np.random.default_rng(R * V + b)
    z = _logits(rng, b * R, V, kind).reshape(b, R, V)
    best = np.where(np.isnan(z), -np.inf, z).argmax(2)
    draft = best[:, :D].copy()
    for j in range(b):
        for i in range(D):
            if rng.random() < 0.8:
                z[j, i, draft[j, i]] = 18.0
        draft[j, rng.integers(0, D)] = rng.integers(-1, V)
    zt = _padded(z, dtype, pad)
    z = _host(zt)
    T, k, p, mp = _ask(rng, b, mode)
    ua, us = _uniforms(rng, (b, D)), _uniforms(rng, (b, V))
    n, c, em, nx = _accept(zt, draft, T, k, p, mp, ua, _padded(us, "f32", pad))
    assert api.dflash_get_status() == 0
    same = 0
    for j in range(b):
        ask = (float(T[j]), int(k[j]), float(p[j]), float(mp[j]))
        if _accept_margin(z[j], draft[j], *ask, ua[j], us[j]) < 1e-6:
            continue
        rn, rc, rem, rnx = RO.verify_accept_filtered(z[j], draft[j], ask[0], ua[j], us[j], *ask[1:])
        assert (n[j], c[j], nx[j]) == (rn, rc, rnx) and em[j].tolist() == rem.tolist(), (j, ask)
        same += 1
    assert same >= (b + 1) // 2


@pytest.mark.parametrize("dtype,b,R,D,V,kind,mode", [
    ("bf16", 12, 16, 15, 151936, "flat", "mixed"), ("f32", 20, 16, 16, 60001, "flat", "p"),
    ("bf16", 24, 16, 15, 90001, "flat", "mixed"),
])
def test_accept_leaves_wide_rows_to_more_launches(dtype, b, R, D, V, kind, mode):
    rng = np.random.default_rng(R * V + b)
    base = _logits(rng, 16, V, kind).astype(np.float32)
    zt = torch.empty((b, R, V), dtype=DT[dtype], device=DEV)
    some = _padded(base, dtype, 0)
    for r in range(b * R):
        zt[r // R, r % R] = torch.roll(some[r % 16], 41 * (r // 16))
    draft = zt[:, :D].float().argmax(2).to(torch.int32)
    for j in range(b):
        for i in range(min(D, j % (D + 1))):  # certain accepts first, then the drawn lots
            zt[j, i, draft[j, i].long()] = 60.0
    draft = draft.cpu().numpy()
    T, k, p, mp = _ask(rng, b, mode)
    ua, us = _uniforms(rng, (b, D)), _uniforms(rng, (b, V))
    ws = torch.zeros(api.dflash_verify_filtered_workspace_size(b, R, V), dtype=torch.uint8, device=DEV)
    got = _accept(zt, draft, T, k, p, mp, ua, _dev(us, np.float32), ws=ws)
    again = _accept(zt, draft, T, k, p, mp, ua, _dev(us, np.float32), ws=ws)
    assert api.dflash_get_status() == 0
    for x, y in zip(got, again):
        assert np.array_equal(x, y)
    n, c, em, nx = got
    same = 0
    for j in range(b):
        ask = (float(T[j]), int(k[j]), float(p[j]), float(mp[j]))
        z = _host(zt[j])
        if _accept_margin(z, draft[j], *ask, ua[j], us[j]) < 1e-6:
            continue
        rn, rc, rem, rnx = RO.verify_accept_filtered(z, draft[j], ask[0], ua[j], us[j], *ask[1:])
        assert (n[j], c[j], nx[j]) == (rn, rc, rnx) and em[j].tolist() == rem.tolist(), (j, ask)
        same += 1
    assert same >= b // 2


@pytest.mark.parametrize("dtype,b,R,D,V,kind,mode", [
    ("f32", 13, 16, 15, 100003, "flat", "p"), ("f32", 13, 16, 16, 100003, "sparse", "mixed"),
    ("f32", 6, 16, 15, 200003, "flat", "mixed"), ("f32", 25, 4, 3, 200003, "sparse", "k"),
    ("bf16", 10, 16, 15, 200003, "flat", "p"),
])
def test_accept_leaves_rows_of_clusters_to_more_launches(dtype, b, R, D, V, kind, mode):
    # (as for sample: two or four CTAs a row)
    test_accept_leaves_wide_rows_to_more_launches(dtype, b, R, D, V, kind, mode)


def test_accept_at_zero_temperature_is_the_greedy_kernel():
    rng = np.random.default_rng(8)
    b, R, V = 6, 16, 4093
    z = rng.normal(0, 1, (b, R, V)).astype(np.float32)
    draft = z.argmax(2)[:, : R - 1].astype(np.int32)
    for j in range(b):
        draft[j, rng.integers(0, R - 1)] = 5
    zt = _dev(z, np.float32)
    got = _accept(zt, draft, np.zeros(b), np.zeros(b), np.full(b, 0.5), np.full(b, 0.1), _uniforms(rng, (b, R - 1)),
                  _dev(_uniforms(rng, (b, V)), np.float32))
    ref = [torch.empty(b, dtype=torch.int32, device=DEV) for _ in range(3)]
    em = torch.empty((b, R), dtype=torch.int32, device=DEV)
    api.dflash_verify_accept(zt, _dev(draft, np.int32), ref[0], ref[1], em, ref[2])
    for g, r in zip(got, (ref[0], ref[1], em, ref[2])):
        assert np.array_equal(g, r.cpu().numpy())


@pytest.mark.parametrize("dtype,b,R,V", [("f32", 7, 4, 20011), ("bf16", 7, 2, 20011), ("f32", 50, 4, 100003)])
def test_accept_at_zero_temperature_over_any_row(dtype, b, R, V):
    rng = np.random.default_rng(b + R)
    base = _padded(_greedy_rows(rng, 7, V, dtype), dtype, 0)
    at = (np.arange(b * R) % 7).reshape(b, R)
    zt = base[torch.from_numpy(at).to(DEV)].contiguous()
    first = _first(_host(base))[at]
    draft = first[:, :R - 1].copy()
    stop = np.arange(b) % R
    for j in range(b):
        if stop[j] < R - 1:
            draft[j, stop[j]] = (draft[j, stop[j]] + 1) % V
    _, k, p, mp = _ask(rng, b, "mixed")
    n, c, em, nx = _accept(zt, draft, np.zeros(b), k, p, mp, _uniforms(rng, (b, R - 1)),
                           _dev(_uniforms(rng, (b, V)), np.float32))
    assert api.dflash_get_status() == 0
    for j in range(b):
        rest = first[j, stop[j]]
        assert (n[j], c[j], nx[j]) == (stop[j], rest, rest)
        assert em[j].tolist() == first[j, :stop[j]].tolist() + [rest] + [-1] * (R - 1 - stop[j])


def test_accept_refuses_one_sequence_and_serves_the_others():
    rng = np.random.default_rng(9)
    b, R, V = 3, 4, 500
    z = _logits(rng, b * R, V, "peaked").reshape(b, R, V)
    draft = z.argmax(2)[:, :3]
    T, k, p, mp = np.array([0.7, np.nan, 0.7]), np.zeros(b), np.ones(b), np.zeros(b)
    ua, us = _uniforms(rng, (b, 3)), _uniforms(rng, (b, V))
    n, c, em, nx = _accept(_padded(z, "f32", 0), draft, T, k, p, mp, ua, _dev(us, np.float32))
    assert api.dflash_get_status() == api.DEV_BAD_PARAM
    assert (n[1], c[1], nx[1]) == (-1, -1, -1) and (em[1] == -1).all()
    for j in (0, 2):
        assert n[j] == RO.verify_accept_filtered(z[j].astype(np.float32), draft[j], np.float32(0.7), ua[j], us[j])[0]


@pytest.mark.parametrize("V", [3001, 40001])
def test_accept_reuses_one_workspace_for_batches_of_any_shape(V):
    # sequences come and go, blocks grow and shrink: one workspace of the largest
    # size, against a fresh one each; what lies behind it stays
    rng = np.random.default_rng(V)
    shapes = [(8, 16, 15), (4, 16, 15), (8, 16, 16), (1, 64, 63), (64, 2, 1), (3, 5, 5), (128, 1, 1), (5, 7, 3),
              (16, 8, 7), (2, 64, 40), (8, 16, 15)]
    size = max(api.dflash_verify_filtered_workspace_size(b, R, V) for b, R, _ in shapes)
    ws = torch.zeros(size + 64, dtype=torch.uint8, device=DEV)
    ws[size:] = 0x5A
    for b, R, D in shapes:
        z = _logits(rng, b * R, V, "peaked" if R % 2 else "flat").reshape(b, R, V)
        zt = _padded(z, "bf16", 0)
        draft = zt[:, :D].float().argmax(2).cpu().numpy()
        for j in range(b):
            draft[j, rng.integers(0, D)] = rng.integers(-1, V)
        T, k, p, mp = _ask(rng, b, "mixed")
        ua, us = _uniforms(rng, (b, D)) * np.float32(0.25), _dev(_uniforms(rng, (b, V)), np.float32)
        got = _accept(zt, draft, T, k, p, mp, ua, us, ws=ws)
        fresh = _accept(zt, draft, T, k, p, mp, ua, us)
        for x, y in zip(got, fresh):
            assert np.array_equal(x, y) and not (x == -7).any(), (b, R, D)
    assert api.dflash_get_status() == 0 and bool((ws[size:] == 0x5A).all())


# ------------------------------------------------------------ top logits ----
@pytest.mark.parametrize("dtype,n,V,pad,K,kind", [
    ("f32", 3, 1, 0, 1, "peaked"), ("f16", 3, 5, 1, 8, "ties"), ("bf16", 5, 33, 0, 33, "ties"),
    ("f32", 9, 4097, 0, 64, "masked"), ("f16", 9, 3000, 5, 1024, "masked"), ("bf16", 7, 20011, 0, 1000, "ties"),
    ("f32", 4, 9000, 0, 1024, "equal"), ("f32", 3, 151936, 0, 64, "peaked"), ("bf16", 5, 151936, 0, 256, "flat"),
    ("f32", 2, 300001, 3, 1023, "flat"), ("bf16", 300, 2500, 0, 10, "flat"), ("bf16", 2, 1200001, 0, 700, "flat"),
])
def test_top_logits(dtype, n, V, pad, K, kind):
    rng = np.random.default_rng(V + K)
    zt = _padded(_logits(rng, n, V, kind), dtype, pad)
    z = _host(zt)
    T = float(np.float32(rng.choice([1.0, 0.6, 2.5])))
    val = torch.full((n, K), -7.0, dtype=torch.float32, device=DEV)
    idx = torch.full((n, K), -7, dtype=torch.int32, device=DEV)
    lse = torch.full((n,), -7.0, dtype=torch.float32, device=DEV)
    api.dflash_top_logits(zt, K, val, idx, lse_out=lse, temperature=T)
    assert api.dflash_get_status() == 0
    val, idx, lse = val.cpu().numpy(), idx.cpu().numpy(), lse.cpu().numpy()
    for r in range(n):
        rv, ri, rl = RO.top_logits(z[r], K, T)
        assert np.array_equal(idx[r], ri) and np.array_equal(val[r], rv.astype(np.float32))
        # weights are multiples of 2^-(62 - bits of V - 1) besides their exponentials' error
        assert lse[r] == rl if rl == -math.inf else abs(lse[r] - rl) <= (abs(rl) + 4) * 2.0 ** -21


# ------------------------------------------------------------ distillation ---
def _teach(rng, n, V, K, spread=1.0):
    K_real = min(K, V)
    ti = np.full((n, K), -1, np.int32)
    tv = rng.normal(5, 2.5 * spread, (n, K)).astype(np.float32)
    for r in range(n):
        at = rng.permutation(K)[:K_real]
        ti[r, at] = rng.choice(V, K_real, replace=False)
        tv[r, rng.integers(0, K)] = -np.inf if K > 2 and r % 3 == 0 else 5.0
    return tv, ti


def _tolerances(z, tv, ti, T, tl, w, dtype):
    """Loss and gradient bounds of one row (see the module's docstring)."""
    eps_out = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    zt = z / T
    L = RO._lse(zt)
    ids = ti[ti >= 0]
    t = tv[ti >= 0] / T
    lt = RO._lse(t) if tl is None else float(tl)
    fin = t > -np.inf
    big = max(np.abs(t[fin] - lt).max(), np.abs(zt[ids][fin] - L).max(), abs(lt), 1.0)
    q = np.exp(zt - L)
    x = np.where(q > 0, np.abs(zt - zt.max()), 0)
    err = q * (6 + x) * 2.0 ** -22 + 2.0 ** -80
    p = np.zeros_like(z)
    p[ids] = np.exp(t - lt)
    err += p * (6 + np.abs(lt)) * 2.0 ** -22
    if tl is not None:  # outside: a difference of P q_j and p_r r_j, r the share of what is outside
        out = np.ones(z.size, bool)
        out[ids] = False
        if out.any() and zt[out].max() > -np.inf:
            share = np.exp(zt[out] - RO._lse(zt[out]))
            pr = max(0.0, 1.0 - p.sum())
            # p_r is one minus a sum whose terms are good to 2^-21 each
            err[out] += share * (pr * (6 + np.where(share > 0, np.abs(zt[out] - zt[out].max()), 0)) * 2.0 ** -22
                                 + (p * (1 + np.abs(lt))).sum() * 2.0 ** -22)
    return abs(w) * (1 + big) * 2.0 ** -20, abs(w) / T * err, eps_out, 2.0 ** -25 if dtype == "f16" else 0.0


CASES = [("f32", 4, 1, 0, 1, False), ("f16", 5, 2, 1, 4, True), ("bf16", 6, 33, 0, 5, True),
         ("f32", 7, 257, 2, 300, False), ("f16", 9, 1000, 7, 37, True), ("bf16", 9, 4099, 0, 64, False),
         ("f32", 6, 20011, 0, 1024, True), ("f32", 3, 151936, 0, 64, True), ("bf16", 3, 151936, 0, 128, True),
         ("f16", 3, 50021, 3, 1, False), ("bf16", 320, 2111, 0, 8, True), ("f32", 2, 1000003, 1, 17, True)]


def _distill_inputs(dtype, n, V, pad, K, rest):
    rng = np.random.default_rng(V * 3 + K)
    z = rng.normal(0, 2.0, (n, V))
    tv, ti = _teach(rng, n, V, K)
    for r in range(n):
        on = ti[r] >= 0
        z[r, ti[r][on]] = np.where(tv[r][on] > -np.inf, tv[r][on], 0) + rng.normal(0, 1, on.sum()) + 2
        if V > 40 and r % 4 == 1:
            z[r, rng.random(V) < 0.3] = -np.inf
            z[r, ti[r][on]] = 4.0
    zt = _padded(z, dtype, pad)
    T = float(np.float32([1.0, 0.7, 2.0][K % 3]))
    tl = None
    if rest:
        tl = np.array([RO._lse(tv[r][ti[r] >= 0] / T) + rng.uniform(0.01, 0.5) for r in range(n)], np.float32)
    w = rng.uniform(0.2, 2.0, n).astype(np.float32)
    w[n // 2] = 0.0
    return zt, tv, ti, T, tl, w


def _check_distill(z, tv, ti, T, tl, w, loss, dz, dtype):
    for r in range(len(z)):
        tlr = None if tl is None else float(tl[r])
        rl, rg = RO.distill(z[r], tv[r], ti[r], T, tlr, float(w[r]))
        if w[r] == 0:
            assert loss[r] == 0 and not dz[r].any()
            continue
        tol_l, tol_g, eps, step = _tolerances(z[r], tv[r], ti[r], T, tlr, float(w[r]), dtype)
        if loss is not None:
            assert loss[r] == rl or abs(loss[r] - rl) <= tol_l, (r, loss[r], rl, tol_l)
        bound = tol_g + (np.abs(rg) + tol_g) * eps + step
        assert np.all(np.abs(dz[r] - rg) <= bound), (r, np.max(np.abs(dz[r] - rg) - bound))


@pytest.mark.parametrize("dtype,n,V,pad,K,rest", CASES)
def test_distill(dtype, n, V, pad, K, rest):
    zt, tv, ti, T, tl, w = _distill_inputs(dtype, n, V, pad, K, rest)
    z = _host(zt)
    tvd, tid, wd = _dev(tv, np.float32), _dev(ti, np.int32), _dev(w, np.float32)
    tld = None if tl is None else _dev(tl, np.float32)
    loss = torch.full((n,), -7.0, device=DEV)
    dz = _padded(np.full((n, V), 7.0), dtype, pad)
    api.dflash_distill_loss(zt, tvd, tid, loss, t_lse=tld, temperature=T, weight=wd, dlogits=dz)
    assert api.dflash_get_status() == 0
    _check_distill(z, tv, ti, T, tl, w, loss.cpu().numpy(), _host(dz), dtype)
    if pad:  # what lies between the rows stays
        buf = torch.as_strided(dz, (n - 1, pad), (V + pad, 1), dz.storage_offset() + V)
        assert torch.isnan(buf).all()
    # the loss alone, and its gradient by the second call
    only, stats = torch.empty_like(loss), torch.empty((n, 4), device=DEV)
    api.dflash_distill_loss(zt, tvd, tid, only, t_lse=tld, temperature=T, weight=wd)
    assert torch.equal(only, loss)
    api.dflash_distill_loss(zt, tvd, tid, only, t_lse=tld, temperature=T, stats_out=stats)
    back = torch.empty((n, V), dtype=zt.dtype, device=DEV)
    api.dflash_distill_backward(zt, tvd, tid, stats, wd, back, t_lse=tld, temperature=T)
    scaled = torch.where(wd == 0, torch.zeros_like(only), only * wd)
    _check_distill(z, tv, ti, T, tl, w, scaled.cpu().numpy(), _host(back), dtype)
    # in place of the logits, both ways
    own = zt.clone() if pad == 0 else _padded(z, dtype, pad)
    api.dflash_distill_loss(own, tvd, tid, only, t_lse=tld, temperature=T, weight=wd, dlogits=own)
    assert torch.equal(own, dz) and torch.equal(only, loss)
    own = _padded(z, dtype, pad)
    api.dflash_distill_backward(own, tvd, tid, stats, wd, own, t_lse=tld, temperature=T)
    assert torch.equal(own, back)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_gradient_against_differences(rest):
    rng = np.random.default_rng(11)
    V, K, T = 70, 6, 1.3
    z = rng.normal(0, 1, V)
    tv, ti = rng.normal(1, 1, (1, K)).astype(np.float32), rng.choice(V, (1, K), replace=False).astype(np.int32)
    tl = _dev([RO._lse(tv[0] / T) + 0.3], np.float32) if rest else None
    h = 2.0 ** -6
    rows = np.stack([z] + [z + s * h * e for e in np.eye(V) for s in (1, -1)])
    n = len(rows)
    rows = rows.astype(np.float32)
    loss = torch.empty(n, device=DEV)
    grad = torch.empty((n, V), device=DEV)
    api.dflash_distill_loss(_dev(rows, np.float32), _dev(np.repeat(tv, n, 0), np.float32),
                            _dev(np.repeat(ti, n, 0), np.int32), loss,
                            t_lse=None if tl is None else tl.repeat(n), temperature=T, dlogits=grad)
    l = loss.double().cpu().numpy()
    num = (l[1::2] - l[2::2]) / (rows[1::2].astype(np.float64) - rows[2::2])[np.arange(V), np.arange(V)]
    # central differences: h^2 / 6 times a third derivative below 1 / T^3, and
    # two losses good to 2^-20 of their terms over 2 h
    assert np.abs(num - _host(grad)[0]).max() < h * h / 6 / T ** 3 + 8 * 2.0 ** -20 / (2 * h)


def test_distill_rows_left_out_and_refused():
    V, K = 3000, 4
    rng = np.random.default_rng(12)
    n = 8
    z = rng.normal(0, 1, (n, V)).astype(np.float32)
    tv = np.zeros((n, K), np.float32)
    ti = np.tile(np.array([5, 900, 1700, 2999], np.int32), (n, 1))
    ti[0] = -1                       # nothing listed
    tv[1] = -np.inf                  # nothing above -inf
    z[2] = np.nan                    # left out by its weight
    ti[3, 2] = 5                     # twice the same token
    ti[4, 1] = V                     # outside
    ti[5, 0] = -2                    # outside
    z[6, 100] = np.nan               # a NaN student
    w = np.ones(n, np.float32)
    w[2] = 0
    loss, dz = torch.full((n,), -7.0, device=DEV), torch.full((n, V), 7.0, device=DEV)
    stats = torch.empty((n, 4), device=DEV)
    args = (_dev(z, np.float32), _dev(tv, np.float32), _dev(ti, np.int32))
    api.dflash_distill_loss(*args, loss, weight=_dev(w, np.float32), dlogits=dz, stats_out=stats)
    assert api.dflash_get_status() == api.DEV_BAD_TOKEN
    l, g = loss.cpu().numpy(), dz.cpu().numpy()
    assert l[:3].tolist() == [0, 0, 0] and np.isnan(l[3:7]).all() and not g[:6].any() and np.isnan(g[6]).any()
    rl, rg = RO.distill(z[7].astype(np.float64), tv[7], ti[7])
    assert abs(l[7] - rl) < 1e-5 and np.abs(g[7] - rg).max() < 1e-6
    # the backward call leaves the same rows out
    back = torch.full((n, V), 7.0, device=DEV)
    api.dflash_distill_backward(*args, stats, _dev(w, np.float32), back)
    assert api.dflash_get_status() == api.DEV_BAD_TOKEN
    assert not back[:6].any() and np.abs(back[7].cpu().numpy() - rg).max() < 1e-6


@pytest.mark.parametrize("V", [1000, 40011])
def test_distill_refuses_a_teacher_that_is_no_number(V):
    K, n = 3, 12
    rng = np.random.default_rng(V)
    z = rng.normal(0, 1, (n, V)).astype(np.float32)
    tv, ti = rng.normal(0, 1, (n, K)).astype(np.float32), np.tile(np.array([5, 900, V - 1], np.int32), (n, 1))
    tl = np.array([RO._lse(tv[r]) + 0.2 for r in range(n)], np.float32)
    w = np.full(n, 0.5, np.float32)
    tv[0, 1] = tv[1] = tv[2, 0] = np.nan
    tv[3, 2] = np.inf
    tl[4:7] = [np.nan, np.inf, -np.inf]
    refused = range(7)
    # left out: by its weight, by its list; an index of -1 is no entry
    tv[7], tl[7], w[7] = np.nan, np.nan, 0
    tv[8], tl[8] = -np.inf, -np.inf
    ti[9], tv[9], tl[9] = -1, np.nan, np.nan
    tv[10, 1], ti[10, 1] = np.nan, -1
    args = (_dev(z, np.float32), _dev(tv, np.float32), _dev(ti, np.int32))
    loss, dz = torch.full((n,), -7.0, device=DEV), torch.full((n, V), 7.0, device=DEV)
    back, stats = torch.full((n, V), 7.0, device=DEV), torch.empty((n, 4), device=DEV)
    tld, wd = _dev(tl, np.float32), _dev(w, np.float32)
    api.dflash_distill_loss(*args, loss, t_lse=tld, weight=wd, dlogits=dz, stats_out=stats)
    assert api.dflash_get_status() == api.DEV_BAD_PARAM
    api.dflash_distill_backward(*args, stats, wd, back, t_lse=tld)
    assert api.dflash_get_status() == api.DEV_BAD_PARAM and torch.equal(dz, back)
    l, g = loss.cpu().numpy(), _host(dz)
    assert np.isnan(l[:7]).all() and not g[:10].any() and l[7:10].tolist() == [0, 0, 0]
    for r in range(n):
        rl, rg = RO.distill(z[r].astype(np.float64), tv[r], ti[r], 1.0, float(tl[r]), float(w[r]))
        assert math.isnan(rl) == (r in refused) and np.abs(g[r] - rg).max() < 1e-6
        assert r in refused or abs(l[r] - rl) < 1e-5
    # without a log-sum-exp
    api.dflash_distill_loss(*args, loss, weight=wd, dlogits=dz)
    assert api.dflash_get_status() == api.DEV_BAD_PARAM
    l = loss.cpu().numpy()
    assert np.isnan(l[:4]).all() and np.isfinite(l[4:]).all() and not dz[:4].any()
    # a teacher's row with an infinite logit, as it comes from dflash_top_logits
    teacher = _dev(z[:2], np.float32)
    teacher[0, 77] = np.inf
    val, idx, lse = torch.empty((2, K), device=DEV), torch.empty((2, K), dtype=torch.int32, device=DEV), torch.empty(2, device=DEV)
    api.dflash_top_logits(teacher, K, val, idx, lse_out=lse)
    api.dflash_distill_loss(args[0][:2], val, idx, loss[:2], t_lse=lse, dlogits=dz[:2])
    assert api.dflash_get_status() == api.DEV_BAD_PARAM
    assert np.isnan(float(loss[0])) and np.isfinite(float(loss[1])) and not dz[0].any() and torch.isfinite(dz[1]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_distill_with_masks_of_the_lowest_value(dtype):
    V, K = 3001, 3
    low = float(torch.finfo(DT[dtype]).min)
    z = np.full((3, V), low)
    z[0, :40] = np.linspace(0, 2, 40)         # a masked tail: probability 0
    z[2, [5, 9, 2000]] = [1.0, 2.0, 0.5]      # all but the listed ones masked
    tv, ti = np.array([[1.0, 0.5, 0.2]] * 3, np.float32), np.array([[5, 9, 2000], [5, 9, 2000], [5, 9, 2000]], np.int32)
    ti[0, 2] = 30
    zt = _padded(z, dtype, 1)
    loss, dz = torch.empty(3, device=DEV), torch.empty((3, V), dtype=DT[dtype], device=DEV)
    api.dflash_distill_loss(zt, _dev(tv, np.float32), _dev(ti, np.int32), loss, temperature=0.5, dlogits=dz)
    eps = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    for r in range(3):                        # row 1: nothing but the mask is uniform
        rl, rg = RO.distill(_host(zt)[r], tv[r], ti[r], 0.5)
        assert abs(float(loss[r]) - rl) < 1e-5 * (1 + abs(rl)), r
        assert np.abs(_host(dz)[r] - rg).max() < 1e-5 + 2 * eps, r


@pytest.mark.parametrize("mask", [-1e7, -2e9, -1e10, -3e20, -1e30, -3e38])
@pytest.mark.parametrize("T", [1e-3, 0.5, 20.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_with_masks_far_out(dtype, T, mask):
    # at any distance: a masked tail, rows of nothing but masks, far maxima
    V, K = 20011, 4
    rng = np.random.default_rng(5)
    z = np.full((6, V), mask)
    z[0, 50:600] = rng.normal(0, 2, 550) * min(T, 1)
    z[1] = -mask if abs(mask) < 1e38 else mask          # equal, far above zero
    z[2, :7000] = 0.0
    z[3, [5, 9, 2000, 20010]] = np.array([1.0, 2.0, 0.5, 1.5]) * min(T, 1)
    z[5, ::3] = rng.normal(0, 2, z[5, ::3].size) * min(T, 1)
    ti = np.array([[60, 90, 200, 555], [5, 9, 2000, 20010], [5, 9, 2000, 600], [5, 9, 2000, 20010],
                   [5, 9, 2000, 20010], [3, 9, 2001, 20010]], np.int32)
    tv = (np.array([[1.0, 0.5, 0.2, 0.1]] * 6) * T).astype(np.float32)
    tv[4] += np.float32(mask)                           # the teacher's as well
    zt = _padded(z, dtype, 1)
    for lse in (False, True):
        tl = [RO._lse(t.astype(np.float64) / np.float64(np.float32(T))) + 0.01 for t in tv]
        rows = [r for r in range(6) if not (lse and r == 4)]   # (a difference from one needs the sum's digits)
        n = len(rows)
        loss, dz = torch.empty(n, device=DEV), torch.empty((n, V), dtype=DT[dtype], device=DEV)
        stats = torch.empty((n, 4), device=DEV)
        api.dflash_distill_loss(zt[rows].contiguous(), _dev(tv[rows], np.float32), _dev(ti[rows], np.int32), loss,
                                temperature=T, t_lse=_dev(np.array(tl)[rows], np.float32) if lse else None, dlogits=dz,
                                stats_out=stats)
        eps = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]
        for at, r in enumerate(rows):
            rl, rg = RO.distill(_host(zt)[r], tv[r], ti[r], float(np.float32(T)), float(np.float32(tl[r])) if lse else None)
            if rl < 1e34:  # (log-probabilities below fp32's range count as -inf)
                assert abs(float(loss[at]) - rl) < 1e-5 * (1 + abs(rl)), (r, lse, float(loss[at]), rl)
            else:
                assert float(loss[at]) > 0.999 * min(rl, 3e38), (r, lse)
            assert np.abs(_host(dz)[at] - rg).max() < (1e-5 + 2 * eps) / T, (r, lse)


@pytest.mark.parametrize("far", [300.0, 5000.0, -20000.0, 40000.0])
@pytest.mark.parametrize("T", [0.7, 0.05])
@pytest.mark.parametrize("n,rest", [(3, True), (700, False)])
def test_distill_of_a_student_far_from_zero(far, T, n, rest):
    rng = np.random.default_rng(33)
    V, K, T = 20011, 24, float(np.float32(T))
    tv, ti = _teach(rng, 6, V, K)
    tv = (tv * T).astype(np.float32)
    z = rng.normal(0, 2, (6, V))
    z[np.arange(6)[:, None], ti] = 4 + rng.normal(0, 1, (6, K))
    some = _padded(far + z * T, "f32", 0)
    at = np.arange(n) % 6
    tl = np.array([RO._lse(t.astype(np.float64) / T) + 0.2 for t in tv], np.float32) if rest else None
    loss, dz = torch.empty(n, device=DEV), torch.empty((n, V), device=DEV)
    api.dflash_distill_loss(some[torch.from_numpy(at).to(DEV)].contiguous(), _dev(tv[at], np.float32),
                            _dev(ti[at], np.int32), loss, t_lse=_dev(tl[at], np.float32) if rest else None,
                            temperature=T, dlogits=dz)
    assert api.dflash_get_status() == 0
    h = _host(some) - far                # (exact: the same rows, whose oracle keeps more digits)
    few = range(0, n, max(1, n // 6))
    _check_distill(h[at][few], tv[at][few], ti[at][few], T, None if tl is None else tl[at][few], np.ones(len(few)),
                   loss.cpu().numpy()[few], _host(dz[list(few)]), "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("far", [3e3, 1e5, -1e6, 2e6])
def test_distill_from_a_teacher_far_from_zero(dtype, far):
    # t / T and t_lse agree in all but their last digits; the next fp32 above the
    # log-sum-exp leaves the rest its share of what rounding takes
    rng = np.random.default_rng(7)
    n, V, K, T = 24, 9001, 12, float(np.float32(0.7))
    z = rng.normal(0, 2, (n, V))
    ti = np.stack([rng.choice(V, K, replace=False) for _ in range(n)]).astype(np.int32)
    tv = (far + rng.normal(0, 2, (n, K))).astype(np.float32)
    tl = np.array([RO._lse(tv[r].astype(np.float64) / T) + 0.05 for r in range(n)])
    tl = np.nextafter(tl.astype(np.float32), np.float32(np.inf))
    zt = _padded(z, dtype, 0)
    loss, stats = torch.empty(n, device=DEV), torch.empty((n, 4), device=DEV)
    dz, back = (torch.empty((n, V), dtype=DT[dtype], device=DEV) for _ in range(2))
    args = zt, _dev(tv, np.float32), _dev(ti, np.int32)
    api.dflash_distill_loss(*args, loss, t_lse=_dev(tl, np.float32), temperature=T, dlogits=dz, stats_out=stats)
    api.dflash_distill_backward(*args, stats, torch.ones(n, device=DEV), back, t_lse=_dev(tl, np.float32), temperature=T)
    assert api.dflash_get_status() == 0 and torch.equal(dz, back)
    eps = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]
    h, g = _host(zt), _host(dz)
    for r in range(n):
        rl, rg = RO.distill(h[r], tv[r], ti[r], T, float(tl[r]))
        # a p is off by 2^-46 of t / T (1 / T as a pair) besides its own rounding, a
        # loss by the sum of their logarithms' as well; the gradients are over T
        e = 2.0 ** -46 * abs(far) / T + 2.0 ** -21
        assert abs(float(loss[r]) - rl) <= 32 * e and np.abs(g[r] - rg).max() <= (12 * e + 2 * eps) / T, r
    # as far below a t / T as no log-sum-exp is
    api.dflash_distill_loss(*args, loss, t_lse=_dev(tl - 20 - np.abs(tl) / 1e5, np.float32), temperature=T, dlogits=dz)
    assert api.dflash_get_status() == api.DEV_BAD_PARAM and torch.isnan(loss).all() and not dz.any()


def test_distill_keeps_the_rest_when_the_student_is_sure():
    # q outside the listed tokens near 1e-30: far below what 1 - sum of q keeps
    V = 5000
    z = np.full((1, V), -70.0, np.float32)
    z[0, 7], z[0, 9] = 3.0, 2.0
    tv, ti = np.array([[1.0, 0.5]], np.float32), np.array([[7, 9]], np.int32)
    tl = np.array([RO._lse(tv[0]) + 0.05], np.float32)
    loss, dz = torch.empty(1, device=DEV), torch.empty((1, V), device=DEV)
    api.dflash_distill_loss(_dev(z, np.float32), _dev(tv, np.float32), _dev(ti, np.int32), loss,
                            t_lse=_dev(tl, np.float32), dlogits=dz)
    rl, rg = RO.distill(z[0].astype(np.float64), tv[0], ti[0], 1.0, float(tl[0]))
    # p_r carries the error of sums near one, 2^-23 of 0.05
    assert abs(float(loss[0]) - rl) < 1e-5 * rl and np.abs(_host(dz)[0] - rg).max() < 1e-6
    assert np.abs(_host(dz)[0][100] / rg[100] - 1) < 2e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,K,mask", [(5003, 64, -np.inf), (151936, 64, -np.inf), (5003, 64, -1e9), (5003, 64, None),
                                      (50, 50, -np.inf), (30, 64, 0.0), (5003, 64, -60.0)])
def test_distill_from_a_teacher_whose_tokens_are_all_listed(dtype, V, K, mask):
    """30 allowed tokens a row, K no less, the others masked in teacher and
    student alike (None: the type's lowest value; -60: not quite): p_r is nothing
    but the rounding of the log-sum-exp."""
    if mask is None or (dtype == "f16" and np.isfinite(mask) and mask < -65504):
        mask = float(torch.finfo(DT[dtype]).min)
    rng = np.random.default_rng(V)
    n, T = 48, float(np.float32(0.8))
    teacher, z = np.full((n, V), mask), np.full((n, V), mask)
    for r in range(n):
        at = rng.choice(V, 30, replace=False)
        teacher[r, at] = 15 + rng.normal(0, 3, 30)
        z[r, at] = 8 + rng.normal(0, 2, 30)
    tt, zt = _padded(teacher, dtype, 0), _padded(z, dtype, 1)
    val, idx, lse = torch.empty((n, K), device=DEV), torch.empty((n, K), dtype=torch.int32, device=DEV), torch.empty(n, device=DEV)
    loss, stats = torch.empty(n, device=DEV), torch.empty((n, 4), device=DEV)
    dz, back = (torch.empty((n, V), dtype=DT[dtype], device=DEV) for _ in range(2))
    api.dflash_top_logits(tt, K, val, idx, lse_out=lse, temperature=T)
    api.dflash_distill_loss(zt, val, idx, loss, t_lse=lse, temperature=T, dlogits=dz, stats_out=stats)
    api.dflash_distill_backward(zt, val, idx, stats, torch.ones(n, device=DEV), back, t_lse=lse, temperature=T)
    assert api.dflash_get_status() == 0
    tv, ti, tl, zh = val.cpu().numpy(), idx.cpu().numpy(), lse.cpu().numpy(), _host(zt)
    l, g, positive = loss.cpu().numpy(), _host(dz), 0
    assert torch.equal(dz, back) and np.isfinite(l).all() and np.isfinite(g).all()
    for r in range(n):
        rl, rg = RO.distill(zh[r], tv[r], ti[r], T, float(tl[r]))
        on = ti[r] >= 0
        lp = tv[r][on].astype(np.float64) / T - float(tl[r])
        positive += np.exp(lp).sum() < 1
        some = lp > -80  # (those below weigh nothing)
        lq = zh[r][ti[r][on]][some] / T - RO._lse(zh[r] / T)
        # (the docstring's bound; a p_r of up to 2^-20 (1 + |t_lse|) carries some 2^-22
        # of error, which ln q_r, -60 / T or so where it counts, scales)
        tol = (1 + max(np.abs(lp[some]).max(), np.abs(lq).max())) * 2.0 ** -20 + (100 * 2.0 ** -22 if mask == -60.0 else 0)
        assert abs(l[r] - rl) <= tol, (r, l[r], rl)
        _, tol_g, eps, step = _tolerances(zh[r], tv[r], ti[r], T, float(tl[r]), 1.0, dtype)
        assert np.all(np.abs(g[r] - rg) <= tol_g + (np.abs(rg) + tol_g) * eps + step), r
    assert positive > 0
    # a p_r above the rounding still meets what the student leaves out
    api.dflash_distill_loss(zt, val, idx, loss, t_lse=lse + 0.01, temperature=T)
    for r in range(n):
        rl = RO.distill(zh[r], tv[r], ti[r], T, float((lse + 0.01)[r]))[0]
        if rl < 1e34:  # (p_r, a difference from one, is good to 2^-22 of 0.01)
            assert abs(float(loss[r]) - rl) <= 1e-4 * (1 + abs(rl)), (r, float(loss[r]), rl)
        else:  # (log-probabilities below fp32's range count as -inf)
            assert float(loss[r]) > 0.999 * min(rl, 3e38), r


# ------------------------------------------------------------- as a whole ----
def test_other_stream_graph_and_early_launch_repeat():
    rng = np.random.default_rng(13)
    n, V, K = 12, 20011, 32
    zt = _padded(_logits(rng, n, V, "peaked"), "bf16", 5)
    T, k, p, mp = (_dev(a, d) for a, d in zip(_ask(rng, n, "mixed"), (np.float32, np.int32, np.float32, np.float32)))
    u = _dev(_uniforms(rng, (n, V)), np.float32)
    ua = _dev(_uniforms(rng, (3, 3)), np.float32)
    z3 = zt.unflatten(0, (3, 4))
    draft = torch.nan_to_num(z3.float(), nan=-1e9).argmax(2)[:, :3].to(torch.int32).contiguous()
    i32 = lambda *s: torch.full(s, -7, dtype=torch.int32, device=DEV)
    f32 = lambda *s: torch.full(s, -7.0, device=DEV)
    o = dict(tok=i32(n), lp=f32(n), n=i32(3), c=i32(3), em=i32(3, 4), nx=i32(3), val=f32(n, K), idx=i32(n, K),
             lse=f32(n), loss=f32(n), st=f32(n, 4), dz=torch.zeros((n, V), dtype=torch.bfloat16, device=DEV),
             dz2=torch.zeros((n, V), dtype=torch.bfloat16, device=DEV))
    student = _padded(_logits(rng, n, V, "flat"), "bf16", 0)
    ones = torch.ones(n, device=DEV)
    ws = torch.zeros(api.dflash_verify_filtered_workspace_size(3, 4, V), dtype=torch.uint8, device=DEV)

    def everything(stream=None):
        api.dflash_sample(zt, T, u, o["tok"], top_k=k, top_p=p, min_p=mp, logprob_out=o["lp"], stream=stream)
        api.dflash_verify_accept_filtered(z3, draft, T[:3], ua, u[:3], o["n"], o["c"], top_k=k[:3], top_p=p[:3],
                                          min_p=mp[:3], emitted=o["em"], next_tok=o["nx"], ws=ws, stream=stream)
        api.dflash_top_logits(zt, K, o["val"], o["idx"], lse_out=o["lse"], stream=stream)
        api.dflash_distill_loss(student, o["val"], o["idx"], o["loss"], t_lse=o["lse"], stats_out=o["st"],
                                dlogits=o["dz"], stream=stream)
        api.dflash_distill_backward(student, o["val"], o["idx"], o["st"], ones, o["dz2"], t_lse=o["lse"],
                                    stream=stream)

    def snapshot_and_clear():
        torch.cuda.synchronize()
        s = {a: t.clone() for a, t in o.items()}
        for t in o.values():
            t.zero_()
        torch.cuda.synchronize()
        return s

    everything()
    ref = snapshot_and_clear()
    side = torch.cuda.Stream()
    everything(side)
    runs = [snapshot_and_clear()]
    with torch.cuda.stream(side):
        everything()
    runs.append(snapshot_and_clear())
    with api.launch_mode(api.LAUNCH_EARLY):
        everything()
    runs.append(snapshot_and_clear())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        everything()
    for _ in range(2):
        g.replay()
        runs.append(snapshot_and_clear())
    for s in runs:
        for a in ref:
            assert torch.equal(ref[a].view(torch.uint8), s[a].view(torch.uint8)), a
    assert api.dflash_get_status() == 0


def test_two_graphs_of_wide_rows_at_once():
    # batches whose wide rows take a second launch, on two streams with a workspace
    # each, replayed side by side
    rng = np.random.default_rng(17)
    n, b, R, V = 330, 24, 16, 90001
    base = _padded(_logits(rng, 8, V, "flat"), "bf16", 0)
    z = torch.stack([torch.roll(base[r % 8], 29 * r) for r in range(b * R)]).unflatten(0, (b, R))
    zs = z.flatten(0, 1)[:n]
    draft = z[:, :R - 1].float().argmax(2).to(torch.int32).contiguous()
    T, k, p, mp = (_dev(a, d) for a, d in zip(_ask(rng, n, "mixed"), (np.float32, np.int32, np.float32, np.float32)))
    u = torch.rand((n, V), generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
    ua = _dev(_uniforms(rng, (b, R - 1)), np.float32)
    i32 = lambda *s: torch.full(s, -7, dtype=torch.int32, device=DEV)
    out = [dict(tok=i32(n), lp=torch.zeros(n, device=DEV), n=i32(b), c=i32(b), em=i32(b, R), nx=i32(b)) for _ in range(3)]
    ws = [(torch.empty(api.dflash_sample_workspace_size(n, V), dtype=torch.uint8, device=DEV),
           torch.zeros(api.dflash_verify_filtered_workspace_size(b, R, V), dtype=torch.uint8, device=DEV))
          for _ in range(3)]

    def both(x):
        o = out[x]
        api.dflash_sample(zs, T, u, o["tok"], top_k=k, top_p=p, min_p=mp, logprob_out=o["lp"], ws=ws[x][0])
        api.dflash_verify_accept_filtered(z, draft, T[:b], ua, u[:b], o["n"], o["c"], top_k=k[:b], top_p=p[:b],
                                          min_p=mp[:b], emitted=o["em"], next_tok=o["nx"], ws=ws[x][1])

    both(0)
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for x in (1, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both(x)
        graphs.append(g)
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for x in (1, 2):
        for a in out[0]:
            assert torch.equal(out[0][a], out[x][a]), a
    assert api.dflash_get_status() == 0


def test_a_step_of_the_loop_answers_and_teaches():
    """Draft a block, score it, accept under filters, commit, and fit the
    drafter's rows to the target's: the calls as they follow one another."""
    from block_diffusion_speculative_draft_gb300 import synth
    from block_diffusion_speculative_draft_gb300 import workload as WL
    from block_diffusion_speculative_draft_gb300.configs import TINY as cfg
    model = api.DeviceDrafter(cfg, synth.FloatWeights(synth.drafter_weights(cfg)), DEV)
    kv = api.KVCache(cfg, 1, cfg.ctx[0] + 4 * cfg.B, DEV)
    ws = api.workspace(cfg, 1, cfg.B, DEV)
    WL.commit_contexts(api, torch, cfg, model, kv, ws, WL.contexts(cfg), cfg.B, DEV)
    B, V, K = cfg.B, cfg.V, 20
    t0 = torch.tensor([7], dtype=torch.int32, device=DEV)
    draft = torch.empty((1, B - 1), dtype=torch.int32, device=DEV)
    rows = torch.empty((1, B - 1, V), device=DEV)
    api.dflash_draft_block(model, kv, t0, draft, ws, logits=rows)
    # a target that agrees with the first five drafts
    rng = np.random.default_rng(14)
    z = torch.from_numpy(rng.normal(0, 1, (1, B, V)).astype(np.float32)).to(DEV)
    z[0, torch.arange(5, device=DEV), draft[0, :5].long()] = 30.0
    T, k, p = (torch.tensor([a], device=DEV, dtype=d) for a, d in
               ((0.8, torch.float32), (50, torch.int32), (0.95, torch.float32)))
    ua, us = (torch.from_numpy(_uniforms(rng, s)).to(DEV) for s in ((1, B - 1), (1, V)))
    n, corr, nxt = (torch.empty(1, dtype=torch.int32, device=DEV) for _ in range(3))
    em = torch.empty((1, B), dtype=torch.int32, device=DEV)
    api.dflash_verify_accept_filtered(z, draft, T, ua, us, n, corr, top_k=k, top_p=p, emitted=em, next_tok=nxt)
    hid = torch.from_numpy(synth.target_hidden(cfg.seed, "blk", B, cfg.k * cfg.H)[None]).to(DEV)
    before = int(kv.len[0])
    api.dflash_kv_commit(model, kv, hid, n, ws)
    zh, dh = z[0].double().cpu().numpy(), draft[0].cpu().numpy()
    rn, rc, rem, rnx = RO.verify_accept_filtered(zh, dh, float(T[0]), ua[0].cpu().numpy(), us[0].cpu().numpy(), 50,
                                                 float(p[0]))
    assert (int(n[0]), int(corr[0]), int(nxt[0])) == (rn, rc, rnx) and em[0].tolist() == rem.tolist() and rn >= 5
    assert int(kv.len[0]) == before + rn + 1
    # the target's rows teach the drafter's
    val, idx = torch.empty((B - 1, K), device=DEV), torch.empty((B - 1, K), dtype=torch.int32, device=DEV)
    lse, loss = torch.empty(B - 1, device=DEV), torch.empty(B - 1, device=DEV)
    student = rows[0].clone()
    api.dflash_top_logits(z[0, : B - 1], K, val, idx, lse_out=lse)
    api.dflash_distill_loss(student, val, idx, loss, t_lse=lse, dlogits=student)
    for i in range(B - 1):
        rl, rg = RO.distill(rows[0, i].double().cpu().numpy(), val[i].cpu().numpy(), idx[i].cpu().numpy(), 1.0,
                            float(lse[i]))
        assert abs(float(loss[i]) - rl) < 1e-4 * (1 + abs(rl))
        assert np.abs(student[i].double().cpu().numpy() - rg).max() < 1e-5
    assert api.dflash_get_status() == 0


def test_binding_refuses_mismatched_tensors():
    z = torch.zeros((2, 64), device=DEV)
    f, i, u = torch.ones(2, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros((2, 64), device=DEV)
    for bad in (dict(logits=z.double()), dict(logits=z.cpu()), dict(logits=z.t()), dict(logits=z[0]),
                dict(temperature=f[:1]), dict(temperature=f.half()), dict(u=u[:, :32]), dict(u=u.half()),
                dict(tok_out=i.long()), dict(top_k=f), dict(top_p=f.cpu()),
                dict(logits=z[:1].expand(2, 64), code=-1)):
        code = bad.pop("code", None)
        args = dict(logits=z, temperature=f, u=u, tok_out=i)
        args.update(bad)
        with pytest.raises(ValueError if code is None else api.DflashError):
            api.dflash_sample(**args)
    z3 = torch.zeros((2, 3, 64), device=DEV)
    with pytest.raises(ValueError):  # uneven rows
        api.dflash_verify_accept_filtered(torch.zeros((2, 4, 64), device=DEV)[:, :3], torch.zeros((2, 2), dtype=torch.int32, device=DEV),
                                          f, torch.zeros((2, 2), device=DEV), u, i.clone(), i.clone())
    with pytest.raises(ValueError):
        api.dflash_verify_accept_filtered(z3, torch.zeros((2, 2), device=DEV), f, torch.zeros((2, 2), device=DEV), u,
                                          i.clone(), i.clone())
    with pytest.raises(api.DflashError) as e:
        api.dflash_verify_accept_filtered(z3, torch.zeros((2, 2), dtype=torch.int32, device=DEV), f,
                                          torch.zeros((2, 2), device=DEV), u, i.clone(), i.clone(),
                                          ws=torch.zeros(8, dtype=torch.uint8, device=DEV))
    assert e.value.code == -5
    val, idx = torch.zeros((2, 4), device=DEV), torch.zeros((2, 4), dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        api.dflash_top_logits(z, 5, val, idx)
    with pytest.raises(ValueError):
        api.dflash_distill_loss(z, val, idx, f.clone(), dlogits=z.half())
    with pytest.raises(ValueError):
        api.dflash_distill_backward(z, val, idx, torch.zeros((2, 2), device=DEV), f, z.clone())
