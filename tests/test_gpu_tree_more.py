"""More of the calls on trees: workspaces as they are found, work cut in many
places, and keys whose loss shows wherever they lie."""
import types

import numpy as np
import pytest

from oracle import tree_oracle as TO
from tests.gpu_util import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

if gpu_available():
    import torch
    from block_diffusion_speculative_draft_gb300 import api
    from tests.test_gpu_tree import DEV, _attend, _attention_case, _check_attention, _i32, _trees


# -------------------------------------------------------------- workspaces ---
@pytest.mark.parametrize("N,nq,nkv,cap", [(1, 8, 2, 900), (9, 8, 2, 700), (40, 4, 2, 3000), (64, 8, 2, 2000)])
def test_attention_takes_its_workspace_as_it_finds_it(N, nq, nkv, cap, monkeypatch):
    """A workspace of any bits gives the same results, bit for bit, and one that
    the call allocates itself is not filled first."""
    rng = np.random.default_rng(N)
    lens, nodes = [cap, cap // 3], [N, max(1, N - 2)]
    kv, q, kt, vt = _attention_case(rng, "f16", 2, N, nq, nkv, 128, cap, lens, nodes, L=1)
    mask, n = _i32(TO.pack_bits(np.stack([TO.tree_mask(p)[0] for p in _trees(rng, 2, N)]))), _i32(nodes)
    size = api.dflash_tree_attention_workspace_size(2, N, nq, nkv, 128)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    api.dflash_get_status()
    out, lse = _attend(kv, 0, q, kt, vt, mask, n, ws=ws)
    for byte in (0xff, 0x7f):
        ws.fill_(byte)
        got, l = _attend(kv, 0, q, kt, vt, mask, n, ws=ws)
        assert torch.equal(got, out) and torch.equal(l, lse)

    def filled(*a, **k):
        raise AssertionError("the workspace is filled")

    monkeypatch.setattr(torch, "zeros", filled)
    got, l = _attend(kv, 0, q, kt, vt, mask, n)
    assert torch.equal(got, out) and torch.equal(l, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out2, lse2 = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    api.dflash_tree_attention(q, kv, 0, kt, vt, mask, out2, n_nodes=n, lse_out=lse2, stream=side)
    side.synchronize()
    assert torch.equal(out2, out) and torch.equal(lse2, lse) and api.dflash_get_status() == 0


# ----------------------------------------------- every key of a long run ---
LONG = [
    ("f16", 3, 32, 8, 2, 128, 30011),    # 128 rows: the streams take tiles in turn
    ("bf16", 2, 20, 10, 2, 64, 60000),   # 100 rows
    ("bf16", 2, 32, 10, 2, 128, 20011),  # 160 rows: a stream has its own
    ("f16", 2, 64, 8, 2, 64, 40001),     # 256 rows
    ("bf16", 1, 70, 8, 1, 128, 30000),   # 560 rows: three query tiles
    ("f16", 5, 12, 4, 1, 128, 50000),    # 48 rows
    ("f16", 6, 1, 16, 4, 128, 30000),    # one token
    ("bf16", 2, 4, 8, 2, 64, 40000),     # 16 rows
]


def _long(dtype, b, N, nq, nkv, d, cap, turned=False):
    """Keys of zeros, so that every score is 0, over caches of unequal lengths."""
    rng = np.random.default_rng(cap + N)
    lens, nodes = [cap - 77 * j for j in range(b)], [N - j % 2 * (N // 3) for j in range(b)]
    kv, q, kt, vt = _attention_case(rng, dtype, b, N, nq, nkv, d, cap, lens, nodes, L=1)
    kv.k.zero_()
    for j in range(b):
        kv.k[0, j, :, lens[j]:] = float("nan")
        kt[j, :nodes[j]] = 0
    if turned:
        kt, vt = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (kt, vt))
    sees = np.stack([TO.tree_mask(p)[0] for p in _trees(rng, b, N)])
    for j in range(b):
        sees[j, :, nodes[j]:] = False
    return kv, q, kt, vt, sees, lens, nodes


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("dtype,b,N,nq,nkv,d,cap", LONG)
@pytest.mark.parametrize("share", ["key", "block"])
def test_equal_weights_count_every_key_once(dtype, b, N, nq, nkv, d, cap, share, turned):
    """Key t (or its block of 64) has a 1 in one column of V: with weights of 1
    the output is the share of keys that have one in that column, and e^lse
    their number.  Weights and products are whole numbers below 2^24, so nothing
    is rounded before the division, whatever the number of keys: the output is
    off by the reciprocal's and the product's roundings (2^-23) and its own.  A
    block that is lost or counted twice changes it by 64 d / T >= 6.8 %, a single
    key, by its column, by d / T (0.2 % in fp16, which 2^-11 shows)."""
    kv, q, kt, vt, sees, lens, nodes = _long(dtype, b, N, nq, nkv, d, cap, turned)
    unit = 1 if share == "key" else 64
    t = torch.arange(cap, device=DEV)
    one = torch.nn.functional.one_hot(t // unit % d, d).to(kv.v.dtype)
    for j in range(b):
        kv.v[0, j, :, :lens[j]] = one[:lens[j]]
        vt[j, :nodes[j]] = 0
        vt[j, :nodes[j], :, 3] = 1
    api.dflash_get_status()
    out, lse = _attend(kv, 0, q, kt, vt, _i32(TO.pack_bits(sees)), _i32(nodes))
    assert api.dflash_get_status() == 0
    half = 2.0 ** -11 if dtype == "f16" else 2.0 ** -8
    for j in range(b):
        n = nodes[j]
        seen = sees[j, :n].sum(1)  # nodes that each node sees
        count = np.bincount(np.arange(lens[j]) // unit % d, minlength=d)[None] + np.eye(d)[3] * seen[:, None]
        total = lens[j] + seen
        want = (count / total[:, None])[:, None]
        got, gl = out[j, :n].double().cpu().numpy(), lse[j, :n].double().cpu().numpy()
        assert (np.abs(got - want) <= (half + 2.0 ** -22) * want + 2.0 ** -25).all(), j
        # ln of a whole number, on numbers below 2^4: the logarithm's last place (2^-20), half
        # of one for the product, and 2^-24 of 11 for the constant; a key more is 2^-16
        assert (np.abs(gl - np.log(total)[:, None]) <= 2.0 ** -18).all(), j
        assert (out[j, n:] == 7).all() and (lse[j, n:] == 7).all()


@pytest.mark.parametrize("dtype,b,N,nq,nkv,d,cap", LONG)
def test_a_heavy_key_is_found_wherever_it_lies(dtype, b, N, nq, nkv, d, cap):
    """One key of each cache and kv head scores 24, all others 0: with T e^-24
    below 2.4e-6 the output is that key's V, off by its weight's rounding, its own
    and the others' part, and lse is 24.  The key goes to the first and the last
    place of every 64: the edges of all tiles, runs and turns of the ring."""
    kv, q, kt, vt, sees, lens, nodes = _long(dtype, b, N, nq, nkv, d, cap)
    q[...] = 0
    q[..., 0] = 4
    mask, n = _i32(TO.pack_bits(sees)), _i32(nodes)
    out = torch.zeros((b, N, nq, d), dtype=q.dtype, device=DEV)
    lse = torch.zeros((b, N, nq), dtype=torch.float32, device=DEV)
    ws = torch.empty(api.dflash_tree_attention_workspace_size(b, N, nq, nkv, d), dtype=torch.uint8, device=DEV)
    there = (torch.arange(N, device=DEV)[None] < n[:, None])[:, :, None]
    half = 2.0 ** -11 if dtype == "f16" else 2.0 ** -8
    vmax = 10.0  # of 1.3 times a normal number
    assert float(kv.v.nan_to_num(0.0).abs().max()) < vmax
    lengths = torch.tensor(lens, device=DEV)[:, None]
    jj, hh = torch.arange(b, device=DEV)[:, None], torch.arange(nkv, device=DEV)[None]
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    api.dflash_get_status()
    places = [p for x in range(0, cap, 64) for p in (x, x + 63)]
    for p in places:
        # kv heads and sequences a block apart, so that a launch has several places
        t = (p + 64 * (3 * jj + hh)) % lengths
        kv.k[0, jj, hh, t, 0] = 6
        api.dflash_tree_attention(q, kv, 0, kt, vt, mask, out, n_nodes=n, lse_out=lse, scale=1.0, ws=ws)
        kv.k[0, jj, hh, t, 0] = 0
        want = kv.v[0, jj, hh, t].float().repeat_interleave(nq // nkv, 1)[:, None]  # [b][1][nq][d]
        bad = (out.float() - want).abs() > (2 * half + 2.0 ** -20) * want.abs() + 2.4e-6 * 2 * vmax
        # 24 + ln(1 + T e^-24), the exponent's roundings at 35 log2 units
        off = (lse - 24).abs() > 2.4e-6 + 24 * 2.0 ** -20
        wrong += ((bad.any(-1) | off | ~torch.isfinite(lse)) & there).sum()
    assert int(wrong) == 0 and api.dflash_get_status() == 0


# --------------------------------------------- several items in one run ---
@pytest.mark.parametrize("dtype,b,N,nq,nkv,d,hi", [
    ("f16", 300, 64, 4, 2, 64, 200),   # 128 rows, streams in turn: about eight items a run
    ("bf16", 400, 9, 4, 2, 128, 300),  # 18 rows
    ("f16", 260, 40, 8, 2, 128, 150),  # 160 rows, a stream's own
    ("bf16", 240, 64, 8, 2, 64, 300),  # 256 rows
    ("f16", 90, 128, 8, 2, 64, 200),   # 512 rows: two query tiles of a head
])
def test_runs_of_several_items(dtype, b, N, nq, nkv, d, hi):
    rng = np.random.default_rng(b + N)
    lens = [int(x) for x in rng.integers(0, hi + 1, b)]
    nodes = rng.integers(0, N + 1, b)
    nodes[rng.random(b) < 0.5] = N
    kv, q, kt, vt = _attention_case(rng, dtype, b, N, nq, nkv, d, hi, lens, nodes, L=1)
    sees = np.stack([TO.tree_mask(p)[0] for p in _trees(rng, b, N)])
    mask, n = _i32(TO.pack_bits(sees)), _i32(nodes)
    api.dflash_get_status()
    out, lse = _attend(kv, 0, q, kt, vt, mask, n)
    _check_attention(dtype, kv, 0, q, kt, vt, sees, lens, nodes, d ** -0.5, out, lse, 7.0)
    for _ in range(10):
        again, lse2 = _attend(kv, 0, q, kt, vt, mask, n)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert api.dflash_get_status() == 0
