"""GPU parity of the operators on a tree of drafts and of the adjustments of
logits against the float64 oracle.

Tolerances of the attention.  With A = sum p |v| / sum p, T keys and u the half
step of the type (2^-11 fp16, 2^-8 bf16): the output's rounding u |o|; each p
enters its product rounded, u A (fp16: at least half of its smallest step, 2^-25
of the largest p, a key); a score is a sum of d products in fp32, off by at most
d 2^-24 scale sum |q k|, its place in the exponent by 2^-23 of the largest
|score| log2(e), the exponential by 2^-22, each once for p and once for the sum:
2 e_s A; sums over keys in fp32: T 2^-24 A.  lse: e_s, the sum's T 2^-24, and
2^-22 (1 + |lse|) for the logarithm and the units' products.

Tolerance of the adjustments: at most 4 + (biases of the entry) fp32 operations
on numbers no larger than `size`, each half a step of 2^-23, then the type's
half step (and fp16's smallest one).
"""
import types

import numpy as np
import pytest

from oracle import tree_oracle as TO
from tests.gpu_util import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

if gpu_available():
    import torch
    from block_diffusion_speculative_draft_gb300 import api
    DEV = torch.device("cuda:0")
    DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def _f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV)


def _host(t):
    return t.double().cpu().numpy()


def _trees(rng, b, N):
    parent = np.full((b, N), -1)
    for i in range(1, N):
        parent[:, i] = rng.integers(max(0, i - 1 - int(rng.integers(0, 8))), i, b)
    return parent


# ------------------------------------------------------------------- masks ---
@pytest.mark.parametrize("b,N", [(1, 1), (3, 2), (2, 31), (2, 32), (5, 33), (3, 64), (2, 100), (4, 256)])
def test_mask(b, N):
    rng = np.random.default_rng(N)
    W = (N + 31) // 32
    parent = _trees(rng, b, N)
    if N > 4:
        parent[0, 1:] = np.arange(N - 1)  # a chain: the deepest tree
        parent[-1, N // 2] = -1           # a second root
    n = rng.integers(0, N + 1, b)
    n[0] = N
    mask = torch.full((b, N, W), 77, dtype=torch.int32, device=DEV)
    depth = torch.full((b, N), 77, dtype=torch.int32, device=DEV)
    api.dflash_get_status()
    api.dflash_tree_mask(_i32(parent), mask, n_nodes=_i32(n), depth_out=depth)
    for j in range(b):
        sees, d = TO.tree_mask(parent[j], int(n[j]))
        assert np.array_equal(mask[j].cpu().numpy(), TO.pack_bits(sees))
        assert np.array_equal(depth[j].cpu().numpy(), d)
    assert api.dflash_get_status() == 0
    api.dflash_tree_mask(_i32(parent), mask)  # all nodes, no depths
    assert np.array_equal(mask[0].cpu().numpy(), TO.pack_bits(TO.tree_mask(parent[0])[0]))


def test_mask_of_bad_trees():
    parent = np.array([[-1, 1, 1, 0, 2, 7, -2, 3], [0, 0, 1, 2, 3, 4, 5, 6], [-1] * 8, [-1] * 8])
    n = np.array([8, 8, 9, -1])
    mask = torch.full((4, 8, 1), 77, dtype=torch.int32, device=DEV)
    depth = torch.full((4, 8), 77, dtype=torch.int32, device=DEV)
    api.dflash_get_status()
    api.dflash_tree_mask(_i32(parent), mask, n_nodes=_i32(n), depth_out=depth)
    assert api.dflash_get_status() == api.DEV_BAD_TREE | api.DEV_BAD_LENGTH
    for j, cnt in enumerate([8, 8, 0, 0]):
        sees, d = TO.tree_mask(parent[j], cnt)
        assert np.array_equal(mask[j].cpu().numpy(), TO.pack_bits(sees)) and np.array_equal(depth[j].cpu().numpy(), d)


# --------------------------------------------------------------- attention ---
def _attention_case(rng, dtype, b, N, nq, nkv, d, cap, lens, nodes, L=2):
    """A cache whose rows past the lengths, and trees whose nodes past the
    counts, hold NaN; queries, keys and values of the nodes in one buffer."""
    t = lambda *s: torch.from_numpy(rng.normal(0, 1.3, size=s).astype(np.float32)).to(DEV).to(DT[dtype])
    k, v = t(L, b, nkv, cap, d), t(L, b, nkv, cap, d)
    qkv = t(b, N, nq + 2 * nkv, d)
    for j in range(b):
        k[:, j, :, max(0, lens[j]):] = float("nan")
        v[:, j, :, max(0, lens[j]):] = float("nan")
        qkv[j, max(0, nodes[j]):] = float("nan")
    kv = api.KVCache(types.SimpleNamespace(L=L, nkv=nkv, d=d), b, cap, k=k, v=v, len=_i32(lens))
    return kv, qkv[:, :, :nq], qkv[:, :, nq:nq + nkv], qkv[:, :, nq + nkv:]


def _check_attention(dtype, kv, layer, q, kt, vt, sees, lens, nodes, scale, out, lse, keep):
    b, N, nq, d = q.shape
    for j in range(b):
        n, C = nodes[j], lens[j]
        # rows of nodes that are not there are left as they were
        assert (out[j, n:] == keep).all() and (lse[j, n:] == keep).all()
        if not n:
            continue
        Q, K, V = _host(q[j, :n]), _host(kv.k[layer, j, :, :C]).transpose(1, 0, 2), _host(kv.v[layer, j, :, :C]).transpose(1, 0, 2)
        KT, VT = _host(kt[j, :n]), _host(vt[j, :n])
        o, l, spread = TO.tree_attention(Q, K, V, KT, VT, sees[j][:n, :n], scale)
        g = nq // kt.shape[2]
        big = scale * max(np.abs(Q[:, h]).max(0) @ np.concatenate([np.abs(K[:, h // g]), np.abs(KT[:, h // g])]).max(0)
                          for h in range(nq))
        T = C + n
        es = d * 2.0 ** -24 * big + 2.0 ** -22 * (1 + big)
        vmax = max(np.abs(V).max(initial=0), np.abs(VT).max(initial=0))
        tol = U[dtype] * (np.abs(o) + spread) + (2 * es + T * 2.0 ** -24) * spread + 2.0 ** -25
        if dtype == "f16":
            tol = tol + T * 2.0 ** -25 * vmax
        got, gl = _host(out[j, :n]), _host(lse[j, :n])
        assert (np.abs(got - o) <= tol).all(), (j, np.abs(got - o).max(), (np.abs(got - o) / tol).max())
        none = np.isneginf(l)
        assert np.array_equal(none, np.isneginf(gl))
        ll = np.where(none, 0, l)
        assert (np.abs(np.where(none, 0, gl) - ll) <= es + T * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(ll))).all()


def _attend(kv, layer, q, kt, vt, mask, n, **kw):
    b, N, nq, d = q.shape
    out = torch.full((b, N, nq, d), 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full((b, N, nq), 7.0, dtype=torch.float32, device=DEV)
    api.dflash_tree_attention(q, kv, layer, kt, vt, mask, out, n_nodes=n, lse_out=lse, **kw)
    return out, lse


@pytest.mark.parametrize("dtype,d,nq,nkv,N,cap,lens", [
    ("f16", 128, 8, 2, 1, 70, [0, 1, 63, 64, 70]),          # one token's step
    ("bf16", 64, 1, 1, 1, 9, [9]),
    ("f16", 64, 6, 2, 5, 200, [0, 1, 59, 60, 64, 128, 200]),  # 15 rows; the tree ends at, before, past a tile's end
    ("bf16", 128, 4, 4, 17, 130, [130, 47, 48]),            # no sharing: 17 rows
    ("f16", 128, 8, 2, 8, 300, [255, 256, 257]),            # 32 rows
    ("bf16", 64, 6, 2, 13, 1000, [1000, 3, 700]),           # 39 rows
    ("f16", 128, 5, 1, 12, 900, [900, 0]),                  # 60 rows
    ("f16", 128, 8, 2, 16, 1500, [1500, 400, 1]),           # 64 rows
    ("bf16", 128, 8, 2, 17, 500, [500, 77]),                # 68 rows
    ("bf16", 128, 10, 2, 32, 700, [700, 64]),               # 160 rows
    ("f16", 64, 16, 2, 32, 600, [600, 1, 0]),               # 256 rows
    ("f16", 128, 8, 1, 33, 400, [400, 200]),                # 264 rows
    ("bf16", 128, 4, 2, 64, 321, [321, 0]),                 # 128 rows
    ("f16", 64, 40, 1, 7, 250, [250, 13]),                  # 280 rows of few nodes
    ("bf16", 64, 3, 3, 256, 300, [300, 5]),                 # the largest tree
    ("f16", 128, 4, 1, 256, 200, [200]),                    # 1024 rows
])
def test_attention(dtype, d, nq, nkv, N, cap, lens):
    rng = np.random.default_rng(N * 1000 + cap)
    b = len(lens)
    nodes = rng.integers((N + 1) // 2, N + 1, b)
    nodes[0] = N
    if b > 2:
        nodes[-1] = 0
    parent = _trees(rng, b, N)
    sees = np.stack([TO.tree_mask(p)[0] for p in parent])
    if N > 2 and b > 1:
        sees[1, 1] = False  # a node that sees no node
    kv, q, kt, vt = _attention_case(rng, dtype, b, N, nq, nkv, d, cap, lens, nodes)
    mask = _i32(TO.pack_bits(sees))
    api.dflash_get_status()
    out, lse = _attend(kv, 1, q, kt, vt, mask, _i32(nodes))
    assert api.dflash_get_status() == 0
    _check_attention(dtype, kv, 1, q, kt, vt, sees, lens, nodes, d ** -0.5, out, lse, 7.0)
    again, lse2 = _attend(kv, 1, q, kt, vt, mask, _i32(nodes))
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # bit for bit


@pytest.mark.parametrize("N,cap", [(1, 33), (16, 400), (70, 150)])
def test_attention_of_a_chain_needs_no_mask(N, cap):
    rng = np.random.default_rng(N)
    lens, nodes = [cap, 2], np.array([N, (N + 1) // 2])
    kv, q, kt, vt = _attention_case(rng, "bf16", 2, N, 8, 2, 128, cap, lens, nodes, L=1)
    sees = np.broadcast_to(np.tril(np.ones((N, N), bool)), (2, N, N))
    out, lse = _attend(kv, 0, q, kt, vt, None, _i32(nodes), scale=0.05)
    _check_attention("bf16", kv, 0, q, kt, vt, sees, lens, nodes, 0.05, out, lse, 7.0)


@pytest.mark.parametrize("b,N,lo,hi", [(300, 3, 0, 90), (40, 16, 0, 2000), (700, 1, 0, 40)])
def test_attention_of_many_sequences(b, N, lo, hi):
    """More items than resident CTAs: runs that hold several whole items, and
    sequences without nodes between them."""
    rng = np.random.default_rng(b)
    lens = [int(x) for x in rng.integers(lo, hi + 1, b)]
    nodes = rng.integers(0, N + 1, b)
    kv, q, kt, vt = _attention_case(rng, "f16", b, N, 4, 2, 64, hi, lens, nodes, L=1)
    sees = np.stack([TO.tree_mask(p)[0] for p in _trees(rng, b, N)])
    out, lse = _attend(kv, 0, q, kt, vt, _i32(TO.pack_bits(sees)), _i32(nodes))
    _check_attention("f16", kv, 0, q, kt, vt, sees, lens, nodes, 0.125, out, lse, 7.0)


@pytest.mark.parametrize("dtype,b,N,nq,nkv,d,cap", [
    ("f16", 3, 32, 8, 2, 128, 30011),    # 128 rows: both streams walk the tiles of long runs
    ("bf16", 2, 20, 10, 2, 64, 60000),   # 100 rows
    ("bf16", 2, 64, 8, 2, 128, 40001),   # 256 rows
    ("f16", 5, 12, 4, 1, 128, 50000),    # 48 rows
    ("f16", 6, 1, 16, 4, 128, 30000)])   # one token
def test_attention_over_long_runs(dtype, b, N, nq, nkv, d, cap):
    rng = np.random.default_rng(cap)
    lens, nodes = [cap - 7 * j for j in range(b)], np.array([N - j % 2 * (N // 3) for j in range(b)])
    kv, q, kt, vt = _attention_case(rng, dtype, b, N, nq, nkv, d, cap, lens, nodes, L=1)
    sees = np.stack([TO.tree_mask(p)[0] for p in _trees(rng, b, N)])
    mask = _i32(TO.pack_bits(sees))
    api.dflash_get_status()
    out, lse = _attend(kv, 0, q, kt, vt, mask, _i32(nodes))
    _check_attention(dtype, kv, 0, q, kt, vt, sees, lens, nodes, d ** -0.5, out, lse, 7.0)
    for _ in range(20):
        again, lse2 = _attend(kv, 0, q, kt, vt, mask, _i32(nodes))
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert api.dflash_get_status() == 0


@pytest.mark.parametrize("dtype,N,nq,nkv,d,cap", [
    ("f16", 9, 2, 1, 64, 100), ("bf16", 40, 4, 2, 128, 333), ("f16", 130, 2, 1, 64, 70), ("bf16", 200, 4, 1, 128, 260)])
def test_attention_with_any_bits(dtype, N, nq, nkv, d, cap):
    """Masks that are no tree's: nodes see later ones, not themselves, or bits of
    nodes that are not there; and no log-sum-exp asked for."""
    rng = np.random.default_rng(N + 1)
    lens, nodes = [cap, 0, 65], np.array([N - 3, N, N // 2 + 1])
    kv, q, kt, vt = _attention_case(rng, dtype, 3, N, nq, nkv, d, cap, lens, nodes, L=1)
    sees = rng.random((3, N, N)) < 0.3
    sees[1, 0] = False   # with no cached key either: nothing
    sees[1, 1] = False
    sees[1, 1, N - 1] = True
    mask = _i32(TO.pack_bits(sees))
    out, lse = _attend(kv, 0, q, kt, vt, mask, _i32(nodes))
    _check_attention(dtype, kv, 0, q, kt, vt, sees, lens, nodes, d ** -0.5, out, lse, 7.0)
    alone = torch.full_like(out, 7.0)
    api.dflash_tree_attention(q, kv, 0, kt, vt, mask, alone, n_nodes=_i32(nodes))
    assert torch.equal(out, alone)


@pytest.mark.parametrize("N,nq,nkv", [(5, 4, 2), (20, 8, 2), (70, 10, 2)])
def test_attention_in_other_orders(N, nq, nkv):
    """Trees kept node by node (a sequence's nodes apart), one sequence's keys
    given to all, and one token's to all nodes."""
    rng = np.random.default_rng(N + 2)
    b, d, cap = 3, 64, 90
    lens, nodes = [90, 31, 0], [N] * 3
    kv, q, kt, vt = _attention_case(rng, "bf16", b, N, nq, nkv, d, cap, lens, nodes, L=1)
    sees = np.stack([TO.tree_mask(p)[0] for p in _trees(rng, b, N)])
    mask = _i32(TO.pack_bits(sees))
    turned = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
    for kk, vv in ((turned(kt), turned(vt)), (kt[:1].expand(b, -1, -1, -1), vt[:1].expand(b, -1, -1, -1)),
                   (kt[:, :1].expand(-1, N, -1, -1), vt[:, :1].expand(-1, N, -1, -1))):
        out, lse = _attend(kv, 0, turned(q), kk, vv, mask, None)
        _check_attention("bf16", kv, 0, q, kk, vv, sees, lens, nodes, d ** -0.5, out, lse, 7.0)


@pytest.mark.parametrize("N", [6, 40, 128])
def test_attention_values_that_a_node_does_not_see_do_not_matter(N):
    rng = np.random.default_rng(N)
    kv, q, kt, vt = _attention_case(rng, "f16", 1, N, 4, 2, 64, 50, [50], [N], L=1)
    parent = np.full((1, N), -1)
    parent[0, 1:] = 0
    sees = TO.tree_mask(parent[0])[0][None]
    mask = _i32(TO.pack_bits(sees))
    vt[0, 2, 0, 5], vt[0, 3, 1, 6], vt[0, 4, 0, 7], kt[0, 5, :, 3] = float("inf"), float("nan"), float("-inf"), float("nan")
    out, lse = _attend(kv, 0, q, kt, vt, mask, None)
    clean = vt.clone()
    clean[~torch.isfinite(clean)] = 0
    kc = torch.where(torch.isnan(kt), torch.zeros_like(kt), kt)
    qkv = torch.cat([q, kc, clean], 2)
    want, _ = _attend(kv, 0, qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:], mask, None)
    rest = [i for i in range(N) if i not in (2, 3, 4, 5)]
    assert torch.equal(out[0, rest], want[0, rest]) and torch.isfinite(out[0, rest]).all()
    assert (out[0, 2, :2, 5] == float("inf")).all() and (out[0, 4, :2, 7] == float("-inf")).all()
    assert torch.isnan(out[0, 3, 2:, 6]).all() and torch.isnan(out[0, 5]).all() and torch.isnan(lse[0, 5]).all()
    assert torch.equal(out[0, 2, 2:], want[0, 2, 2:]) and torch.isfinite(out[0, 3, :2]).all()


def test_attention_without_any_key():
    rng = np.random.default_rng(1)
    kv, q, kt, vt = _attention_case(rng, "bf16", 2, 4, 4, 2, 64, 30, [0, 30], [4, 4], L=1)
    out, lse = _attend(kv, 0, q, kt, vt, torch.zeros((2, 4, 1), dtype=torch.int32, device=DEV), None)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all() and torch.isfinite(lse[1]).all()


def test_attention_bad_lengths_leave_sequences_out():
    rng = np.random.default_rng(2)
    kv, q, kt, vt = _attention_case(rng, "f16", 5, 3, 4, 2, 64, 30, [10] * 5, [3] * 5, L=1)
    mask = _i32(TO.pack_bits(np.broadcast_to(np.tril(np.ones((3, 3), bool)), (5, 3, 3))))
    want, _ = _attend(kv, 0, q, kt, vt, mask, None)
    api.dflash_get_status()
    kv.len.copy_(_i32([-1, 10, 31, 10, 10]))
    out, lse = _attend(kv, 0, q, kt, vt, mask, _i32([3, 3, 3, 4, -1]))
    assert api.dflash_get_status() == api.DEV_BAD_LENGTH
    assert torch.equal(out[1], want[1]) and (out[[0, 2, 3, 4]] == 7).all() and (lse[[0, 2, 3, 4]] == 7).all()


def test_attention_of_a_cache_past_32_bits():
    """16 million keys of 128 dimensions: rows past 2^31 elements.  All keys are
    zero but the last 64, which outweigh the others' 2^24 by e^(8 - ln 2^24)."""
    cap, d = (1 << 24) - 64, 128
    k = torch.zeros((1, 2, 1, cap, d), dtype=torch.float16, device=DEV)
    v = torch.zeros((1, 2, 1, cap, d), dtype=torch.float16, device=DEV)
    g = torch.Generator(device="cuda").manual_seed(3)
    last = torch.randn((64, d), device=DEV, generator=g).half()
    k[0, 1, 0, -64:, 0] = 8.0
    v[0, 1, 0, -64:] = last
    kv = api.KVCache(types.SimpleNamespace(L=1, nkv=1, d=d), 2, cap, k=k, v=v, len=_i32([0, cap]))
    q = torch.zeros((2, 1, 4, d), dtype=torch.float16, device=DEV)
    q[..., 0] = 2.0
    z = torch.zeros((2, 1, 1, d), dtype=torch.float16, device=DEV)
    out, lse = _attend(kv, 0, q, z, z, None, None, scale=1.0)
    e = np.exp(16.0)
    total = 64 * e + (cap - 64) + 1
    want = last.double().sum(0).cpu().numpy() * e / total
    # as at the top of the file, but keys of no value add nothing; 64 terms carry the sum
    A = last.double().abs().sum(0).cpu().numpy() * e / total
    assert (np.abs(_host(out[1, 0, 2]) - want) <= U["f16"] * (np.abs(want) + A) + 2.0 ** -16 * A + 2.0 ** -25).all()
    assert abs(float(lse[1, 0, 2]) - np.log(total)) <= 2.0 ** -16
    assert (out[0] == 0).all() and (lse[0] == 0).all()


# ------------------------------------------------------------------ accept ---
@pytest.mark.parametrize("b,N,R", [(1, 1, 1), (4, 8, 8), (7, 33, 5), (3, 64, 64), (50, 100, 20), (2, 256, 256)])
def test_accept(b, N, R):
    rng = np.random.default_rng(N + R)
    parent, tree, tok = _trees(rng, b, N), rng.integers(0, 6, (b, N)), rng.integers(-1, 6, (b, N))
    if N > 4:  # a chain that is all accepted, but for the path's room
        parent[0, 1:] = np.arange(N - 1)
        tok[0, :-1] = tree[0, 1:]
    n = rng.integers(0, N + 1, b)
    n[0] = N
    mk = lambda *s: torch.full(s, 77, dtype=torch.int32, device=DEV)
    outs = [mk(b), mk(b), mk(b, R), mk(b, R), mk(b)]
    api.dflash_get_status()
    api.dflash_tree_accept(_i32(tok), _i32(tree), _i32(parent), outs[0], outs[1], outs[2], n_nodes=_i32(n),
                           emitted=outs[3], next_tok=outs[4])
    assert api.dflash_get_status() == 0
    for j in range(b):
        want = TO.tree_accept(tok[j], tree[j], parent[j], R, int(n[j]))
        for got, w in zip(outs, want):
            assert np.array_equal(got[j].cpu().numpy(), w), (j, want)
    again = [mk(b), mk(b), mk(b, R)]
    api.dflash_tree_accept(_i32(tok), _i32(tree), _i32(parent), *again)  # all nodes, optional outputs left out
    assert again[2][0].cpu().tolist() == TO.tree_accept(tok[0], tree[0], parent[0], R)[2]


def test_accept_of_bad_trees():
    mk = lambda *s: torch.full(s, 77, dtype=torch.int32, device=DEV)
    n, corr, path = mk(3), mk(3), mk(3, 3)
    api.dflash_get_status()
    # node 1 is its own parent: no child; a count out of range: no nodes
    api.dflash_tree_accept(_i32([[5, 5, 5]] * 3), _i32([[5, 5, 5]] * 3), _i32([[-1, 1, 0], [-1, 0, 1], [-1, 0, 1]]), n, corr,
                           path, n_nodes=_i32([3, 4, 3]))
    assert api.dflash_get_status() == api.DEV_BAD_TREE | api.DEV_BAD_LENGTH
    assert n.tolist() == [1, -1, 2] and corr.tolist() == [5, -1, 5]
    assert path.tolist() == [[0, 2, -1], [-1, -1, -1], [0, 1, 2]]


# ------------------------------------------------------------------ commit ---
@pytest.mark.parametrize("b,N,R,L,nkv,d,cap,cols,in_place,dtype", [
    (1, 1, 1, 1, 1, 64, 1, 8, True, "f16"), (3, 16, 7, 5, 2, 128, 40, 1536, True, "bf16"),
    (9, 40, 40, 3, 3, 64, 100, 1032, False, "f16"), (2, 256, 256, 2, 1, 8, 300, 24, True, "f16"),
    (70, 8, 5, 2, 8, 128, 33, 0, True, "f16")])
def test_commit(b, N, R, L, nkv, d, cap, cols, in_place, dtype):
    rng = np.random.default_rng(b * N)
    t = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).to(DEV).to(DT[dtype])
    k, v, tree = t(L, b, nkv, cap, d), t(L, b, nkv, cap, d), t(L, b, N, 2 * nkv + 1, d)
    kt, vt = tree[:, :, :, :nkv], tree[:, :, :, nkv:2 * nkv]
    hid = t(b, N, cols) if cols else None
    hid_out = torch.full((b, R, cols), 7.0, dtype=DT[dtype], device=DEV) if cols else None
    n = rng.integers(-1, R, b)
    n[0] = R - 1
    lens = rng.integers(0, cap - R + 1, b)
    path = np.full((b, R), -1)
    for j in range(b):
        path[j, :n[j] + 1] = rng.integers(0, N, n[j] + 1)  # (any nodes, some twice)
    wk, wv, wl = k.clone(), v.clone(), lens.copy()
    wh = hid_out.clone() if cols else None
    for j in range(b):
        for i in range(n[j] + 1):
            wk[:, j, :, lens[j] + i], wv[:, j, :, lens[j] + i] = kt[:, j, path[j, i]], vt[:, j, path[j, i]]
            if cols:
                wh[j, i] = hid[j, path[j, i]]
        wl[j] += n[j] + 1
    kv = api.KVCache(types.SimpleNamespace(L=L, nkv=nkv, d=d), b, cap, k=k, v=v, len=_i32(lens))
    ws = torch.zeros(api.dflash_tree_commit_workspace_size(b), dtype=torch.uint8, device=DEV)
    len_out = None if in_place else torch.full((b,), 77, dtype=torch.int32, device=DEV)
    api.dflash_get_status()
    api.dflash_tree_commit(kv, kt, vt, _i32(path), _i32(n), hid=hid, hid_out=hid_out, len_out=len_out, ws=ws)
    assert api.dflash_get_status() == 0
    assert torch.equal(kv.k, wk) and torch.equal(kv.v, wv)
    assert np.array_equal((kv.len if in_place else len_out).cpu().numpy(), wl)
    assert in_place or np.array_equal(kv.len.cpu().numpy(), lens)
    if cols:
        assert torch.equal(hid_out, wh)
    assert not ws.any()


def test_commit_leaves_faulty_sequences():
    L, b, N, R, nkv, d, cap = 2, 6, 4, 3, 2, 64, 10
    tree = torch.randn((L, b, N, 2 * nkv, d), device=DEV).half()
    lens = [8, 7, 0, 0, -1, 0]
    kv = api.KVCache(types.SimpleNamespace(L=L, nkv=nkv, d=d), b, cap, len=_i32(lens))
    path = _i32([[0, 1, 2], [0, 1, 2], [0, 4, 1], [0, 1, 2], [0, 1, 2], [0, -1, 2]])
    n = _i32([2, 2, 1, 3, 1, 0])
    hid, hid_out = torch.randn((b, N, 16), device=DEV).half(), torch.full((b, R, 16), 7.0, dtype=torch.float16, device=DEV)
    seen = []
    for j in range(b):
        one = torch.full((b,), -1, dtype=torch.int32, device=DEV)
        one[j] = n[j]
        api.dflash_get_status()
        api.dflash_tree_commit(kv, tree[:, :, :, :nkv], tree[:, :, :, nkv:], path, one, hid=hid, hid_out=hid_out)
        seen.append(api.dflash_get_status())
    # sequence 4's length is out of range for every call
    L4 = api.DEV_BAD_LENGTH
    assert seen == [api.DEV_KV_CAPACITY | L4, L4, api.DEV_BAD_TREE | L4, L4, L4, L4]
    assert kv.len.tolist() == [8, 10, 0, 0, -1, 1]
    assert not kv.k[:, [0, 2, 3, 4]].any() and (hid_out[[0, 2, 3, 4]] == 7).all()
    assert torch.equal(kv.k[:, 1, :, 7:], tree[:, 1, :3, :nkv].transpose(1, 2))
    assert torch.equal(kv.v[:, 5, :, 0], tree[:, 5, 0, nkv:]) and not kv.v[:, 5, :, 1:].any()


# ------------------------------------------------------------- adjustments ---
def _request(rng, b, R, V, H, tree, D=None):
    """Tokens near one another, so that histories repeat themselves."""
    near = lambda s: np.minimum(V - 1, (rng.random(s) ** 3 * V).astype(np.int64))
    n = rng.integers(0, H + 1, b)
    D = (R if tree else max(1, R - 1)) if D is None else D
    q = dict(hist=near((b, H)), n_hist=n, n_prompt=(n * rng.random(b)).astype(np.int64), draft=near((b, D)),
             repetition=rng.uniform(0.7, 1.6, b), frequency=rng.uniform(-0.5, 1, b), presence=rng.uniform(-0.5, 1, b),
             bias_idx=near((b, 20)), bias_val=rng.normal(0, 3, (b, 20)))
    q["hist"][rng.random((b, H)) < 0.1] = -1
    q["hist"][rng.random((b, H)) < 0.05] = V + 3
    q["draft"][rng.random((b, D)) < 0.2] = q["hist"][:, :1].max()
    q["bias_idx"][:, 3:6] = q["bias_idx"][:, :1]  # the same token again
    q["bias_idx"][:, 7] = -1
    q["bias_val"][:, 8] = -np.inf
    q["path"] = rng.random((b, R, D)) < 0.4 if tree else None
    q["allow"] = rng.random((3, V)) < np.array([0.9, 0.02, 0.5])[:, None]
    q["allow_row"] = rng.integers(-1, 3, (b, R))
    return q


def _to_device(q):
    bits = ("path", "allow")
    ints = ("hist", "n_hist", "n_prompt", "draft", "bias_idx", "allow_row")
    return {k: None if a is None else _i32(TO.pack_bits(a)) if k in bits else _i32(a) if k in ints else _f32(a)
            for k, a in q.items()}


def _padded(z, dtype, pad):
    t = torch.from_numpy(np.ascontiguousarray(z, np.float32)).to(DEV).to(DT[dtype])
    buf = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), float("nan"), dtype=t.dtype, device=DEV)
    buf[..., :t.shape[-1]] = t
    return buf[..., :t.shape[-1]]


def _check_adjust(dtype, zt, q, out):
    b, R, V = zt.shape
    f = lambda name, j, other: other if q.get(name) is None else np.float32(q[name][j]).astype(np.float64)
    for j in range(b):
        bias = [] if q.get("bias_idx") is None else list(zip(q["bias_idx"][j], np.float32(q["bias_val"][j]).astype(np.float64)))
        prompt = made = []
        if q.get("hist") is not None:
            a = 0 if q.get("n_prompt") is None else q["n_prompt"][j]
            prompt, made = list(q["hist"][j][:a]), list(q["hist"][j][a:q["n_hist"][j]])
        for r in range(R):
            mine = []
            if q.get("draft") is not None:
                mine = list(q["draft"][j][q["path"][j, r]] if q.get("path") is not None else q["draft"][j][:r])
            ok = None
            if q.get("allow") is not None:
                ar = q["allow_row"][j, r] if q.get("allow_row") is not None else j * R + r
                ok = q["allow"][ar] if ar >= 0 else None
            z = _host(zt[j, r])
            x, size = TO.adjust_row(z, prompt, made + mine, f("repetition", j, 1.0), f("frequency", j, 0.0),
                                    f("presence", j, 0.0), bias, ok)
            got = _host(out[j, r])
            with np.errstate(invalid="ignore"):
                tol = 10 * 2.0 ** -24 * size + U[dtype] * np.abs(x) + (2.0 ** -25 if dtype == "f16" else 0)
                near = np.abs(got - x) <= tol
            same = (got == x) | (np.isnan(got) & np.isnan(x))
            assert (near | same).all(), (j, r, np.flatnonzero(~(near | same))[:5])
            kept = np.ones(V, bool) if ok is None else ok
            free = kept & ~np.isin(np.arange(V), np.array(prompt + made + mine + [t for t, _ in bias] + [-1], np.int64))
            assert ((got == z) | (np.isnan(got) & np.isnan(z)))[free].all()  # untouched: the bits themselves


@pytest.mark.parametrize("dtype,b,R,V,H,tree,pad,pad_out", [
    ("f32", 1, 1, 1, 1, False, 0, 0), ("f16", 3, 2, 2, 5, True, 1, 0), ("bf16", 2, 3, 31, 40, False, 0, 3),
    ("f32", 2, 5, 33, 64, True, 1, 1), ("f16", 4, 1, 1023, 300, False, 0, 0), ("bf16", 3, 4, 1025, 900, True, 7, 7),
    ("f32", 2, 16, 4099, 2000, False, 0, 0), ("f16", 2, 13, 8191, 700, True, 3, 5), ("bf16", 5, 33, 8193, 100, True, 0, 8),
    ("f32", 3, 7, 20000, 5000, True, 0, 4), ("bf16", 2, 2, 151936, 4000, False, 0, 0), ("f16", 40, 3, 9001, 50, True, 2, 2),
    ("f32", 1, 256, 700, 30, True, 0, 0), ("bf16", 330, 1, 50021, 600, False, 11, 11)])
def test_adjust(dtype, b, R, V, H, tree, pad, pad_out):
    rng = np.random.default_rng(V + H)
    z = rng.normal(0, 4, (b, R, V))
    if V > 30:
        z[..., 3], z[..., 4], z[..., 5], z[..., 6] = np.nan, np.inf, -np.inf, 0.0
    zt = _padded(z, dtype, pad)
    q = _request(rng, b, R, V, H, tree)
    out = torch.full((b, R, V + pad_out), 7.0, dtype=zt.dtype, device=DEV)
    api.dflash_get_status()
    api.dflash_adjust_logits(zt, out[..., :V], **_to_device(q))
    assert api.dflash_get_status() == 0
    _check_adjust(dtype, zt, q, out[..., :V])
    assert (out[..., V:] == 7).all()
    # in place, the same bits
    same = zt._base.clone()[..., :V] if zt._base is not None else zt.clone()
    api.dflash_adjust_logits(same, same, **_to_device(q))
    assert torch.equal(torch.nan_to_num(same.float(), nan=1e30), torch.nan_to_num(out[..., :V].float(), nan=1e30))


@pytest.mark.parametrize("parts", [(), ("hist",), ("repetition",), ("bias",), ("allow",), ("draft",), ("hist", "draft", "allow"),
                                   ("hist", "frequency"), ("draft", "presence", "bias")])
def test_adjust_parts(parts):
    """Each part of a request may be left out."""
    rng = np.random.default_rng(len(parts) + 5)
    b, R, V = 3, 4, 3001
    q = _request(rng, b, R, V, 200, False)
    group = dict(hist=("hist", "n_hist", "n_prompt"), bias=("bias_idx", "bias_val"), allow=("allow", "allow_row"))
    keep = [n for p in parts for n in group.get(p, (p,))]
    if "frequency" in parts:
        keep = [n for n in keep if n != "n_prompt"]
    q = {n: a if n in keep else None for n, a in q.items()}
    zt = _padded(rng.normal(0, 4, (b, R, V)), "f32", 0)
    out = torch.empty_like(zt)
    api.dflash_adjust_logits(zt, out, **_to_device(q))
    _check_adjust("f32", zt, q, out)


def test_adjust_mask_a_row_and_two_dimensions():
    rng = np.random.default_rng(8)
    b, V = 6, 777
    zt = _padded(rng.normal(0, 4, (b, V)), "bf16", 5)
    allow = rng.random((b, V)) < 0.3
    wide = torch.zeros((b, 40), dtype=torch.int32, device=DEV)
    wide[:, :(V + 31) // 32] = _i32(TO.pack_bits(allow))
    out = torch.empty((b, V), dtype=torch.bfloat16, device=DEV)
    api.dflash_adjust_logits(zt, out, allow=wide[:, :30])
    assert torch.equal(out, torch.where(torch.from_numpy(allow).to(DEV), zt, torch.full_like(zt, float("-inf"))))


def test_adjust_counts_a_token_a_million_times():
    b, V, H = 2, 500, (1 << 20) - 257
    hist = torch.full((b, H), 7, dtype=torch.int32, device=DEV)
    z = torch.zeros((b, 1, V), device=DEV)
    api.dflash_adjust_logits(z, z, hist=hist, n_hist=_i32([H, 3]), frequency=_f32([0.5, 0.5]), presence=_f32([1.0, 1.0]))
    assert z[0, 0, 7] == -(0.5 * H + 1) and z[1, 0, 7] == -2.5 and z.count_nonzero() == 2


def test_adjust_refuses_a_sequence_or_a_row():
    V, R = 100, 2
    z = torch.randn((9, R, V), device=DEV)
    one = dict(hist=_i32(np.zeros((9, 4))), n_hist=_i32([4, 5, 4, 4, 4, 4, 4, 4, 4]), n_prompt=_i32([0, 0, -1, 0, 0, 0, 0, 0, 0]),
               repetition=_f32([1, 1, 1, 0, np.inf, 1, 1, 1, 1]), frequency=_f32([0, 0, 0, 0, 0, np.nan, 0, 0, 0]),
               presence=_f32([0, 0, 0, 0, 0, 0, np.inf, 0, 0]), bias_idx=_i32([[-1, 3]] * 8 + [[200, 3]]),
               bias_val=_f32([[np.nan, 1]] * 7 + [[0, np.inf]] + [[np.nan, 1]]),
               allow=torch.full((2, 4), -1, dtype=torch.int32, device=DEV), allow_row=_i32([[2, -1]] + [[0, 1]] * 7 + [[-2, 0]]))
    out = torch.empty_like(z)
    api.dflash_get_status()
    api.dflash_adjust_logits(z, out, **one)
    assert api.dflash_get_status() == api.DEV_BAD_PARAM | api.DEV_BAD_LENGTH
    nan = torch.isnan(out).all(2)
    assert nan.tolist() == [[True, False], *[[True, True]] * 7, [True, False]]
    assert torch.isfinite(out[0, 1]).all() and torch.isfinite(out[8, 1]).all()
    # such rows give no token
    tok = torch.empty(9 * R, dtype=torch.int32, device=DEV)
    api.dflash_sample(out.flatten(0, 1), torch.zeros(9 * R, device=DEV), torch.rand((9 * R, V), device=DEV), tok)
    assert ((tok == -1) == nan.flatten()).all()


# --------------------------------------------------------------- refusals ---
def test_python_refusals():
    z = torch.zeros((2, 3, 50), device=DEV)
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    for kw in (dict(hist=i(3, 4), n_hist=i(2)), dict(n_hist=i(2)), dict(hist=i(2, 4), n_hist=i(3)), dict(hist=i(2, 4).float(), n_hist=i(2)),
               dict(draft=i(2, 3), path=i(2, 3, 2)), dict(draft=i(3, 3)), dict(repetition=i(2)), dict(bias_idx=i(2, 3), bias_val=z[:, 0, :2]),
               dict(allow=i(6, 1)), dict(allow=i(5, 2)), dict(allow=i(6, 2), allow_row=i(6)), dict(allow=i(6, 4)[:, ::2])):
        with pytest.raises(ValueError):
            api.dflash_adjust_logits(z, torch.empty_like(z), **kw)
    for bad in (torch.empty((2, 3, 50), dtype=torch.float16, device=DEV), torch.empty((2, 3, 51), device=DEV),
                torch.empty((2, 3, 100), device=DEV)[..., ::2], torch.empty((2, 3, 50))):
        with pytest.raises(ValueError):
            api.dflash_adjust_logits(z, bad)
    with pytest.raises(ValueError):
        api.dflash_adjust_logits(z, torch.empty_like(z), path=i(2, 3, 0))
    shape = types.SimpleNamespace(L=1, nkv=2, d=64)
    kv = api.KVCache(shape, 2, 16)
    h = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt, device=DEV)
    good = dict(q=h(2, 3, 4, 64), kv=kv, layer=0, k_tree=h(2, 3, 2, 64), v_tree=h(2, 3, 2, 64), mask=i(2, 3, 1),
                out=h(2, 3, 4, 64))
    api.dflash_tree_attention(**good)
    for kw in (dict(q=h(2, 3, 4, 64, dt=torch.bfloat16)), dict(q=h(2, 3, 4, 64).float()), dict(layer=1), dict(layer=-1),
               dict(q=h(3, 3, 4, 64)), dict(k_tree=h(2, 3, 4, 64)), dict(k_tree=h(2, 3, 4, 64)[:, :, ::2]),
               dict(k_tree=h(2, 4, 2, 64)[:, :3]), dict(mask=i(2, 3, 2)), dict(out=h(2, 3, 64, 4).transpose(2, 3)),
               dict(lse_out=h(2, 3, 4)), dict(n_nodes=i(3)), dict(q=h(2, 3, 4, 128)), dict(ws=torch.zeros(9))):
        with pytest.raises(ValueError):
            api.dflash_tree_attention(**{**good, **kw})
    for kw in (dict(scale=0.0), dict(ws=torch.zeros(16, dtype=torch.uint8, device=DEV)), dict(q=h(2 * 3 * 4 * 64 + 1)[1:].view(2, 3, 4, 64))):
        with pytest.raises(api.DflashError):
            api.dflash_tree_attention(**{**good, **kw})
    with pytest.raises(ValueError):
        api.dflash_tree_mask(i(2, 3), i(2, 3, 2))
    with pytest.raises(ValueError):
        api.dflash_tree_accept(i(2, 3), i(2, 3), i(2, 3), i(2), i(3), i(2, 2))
    with pytest.raises(api.DflashError):
        api.dflash_tree_accept(i(2, 3), i(2, 3), i(2, 3), i(2), i(2), i(2, 4))
    with pytest.raises(ValueError):
        api.dflash_tree_commit(kv, h(1, 2, 3, 2, 64), h(1, 2, 3, 2, 64), i(2, 2), i(2), hid=h(2, 3, 8))
    with pytest.raises(ValueError):
        api.dflash_tree_commit(kv, h(2, 2, 3, 2, 64), h(2, 2, 3, 2, 64), i(2, 2), i(2))
    for kw in (dict(k=h(1, 2, 2, 16, 64)), dict(k=h(1, 2, 2, 15, 64), v=h(1, 2, 2, 15, 64)), dict(dtype=torch.float32),
               dict(len=torch.zeros(2, dtype=torch.int64, device=DEV))):
        with pytest.raises(ValueError):
            api.KVCache(shape, 2, 16, **kw)


def test_a_drafter_refuses_a_bf16_cache():
    from block_diffusion_speculative_draft_gb300 import synth
    from block_diffusion_speculative_draft_gb300.configs import TINY as cfg
    model = api.DeviceDrafter(cfg, synth.FloatWeights(synth.drafter_weights(cfg)), DEV)
    kv, ws = api.KVCache(cfg, 1, 64, DEV, dtype=torch.bfloat16), api.workspace(cfg, 1, cfg.B, DEV)
    one, hid = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros((1, 4, cfg.k * cfg.H), dtype=torch.float16, device=DEV)
    draft = torch.zeros((1, cfg.B - 1), dtype=torch.int32, device=DEV)
    for call in (lambda: api.dflash_draft_block(model, kv, one, draft, ws), lambda: api.dflash_kv_commit(model, kv, hid, one, ws),
                 lambda: api.dflash_commit_draft_block(model, kv, hid, one, one, draft, ws)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------ streams and graphs ---
def test_calls_on_another_stream_and_in_graphs():
    """All calls of one block on a side stream, captured twice over one
    workspace, and replayed with other inputs in the same buffers."""
    rng = np.random.default_rng(11)
    b, N, nq, nkv, d, cap, V, L, R = 2, 20, 8, 2, 128, 300, 999, 2, 9
    parent = _trees(rng, b, N)
    lens = [200, 33]
    kv, q, kt, vt = _attention_case(rng, "f16", b, N, nq, nkv, d, cap, [cap, cap], [N, N], L=L)
    kv.len.copy_(_i32(lens))
    tree_kv = torch.randn((L, b, N, 2 * nkv, d), device=DEV).half()
    z = torch.randn((b, N, V), device=DEV)
    buf = dict(parent=_i32(parent), tree=_i32(rng.integers(0, 4, (b, N))), hist=_i32(rng.integers(0, V, (b, 30))), nh=_i32([30, 9]),
               rho=_f32([1.5, 1.1]), u=torch.rand((b * N, V), device=DEV), T=torch.full((b * N,), 0.0, device=DEV))
    z[..., :4] += 4
    ws = torch.zeros(api.dflash_tree_attention_workspace_size(b, N, nq, nkv, d), dtype=torch.uint8, device=DEV)
    wc = torch.zeros(api.dflash_tree_commit_workspace_size(b), dtype=torch.uint8, device=DEV)

    def outputs():
        i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
        return dict(mask=i(b, N, 1), depth=i(b, N), out=torch.zeros((b, N, nq, d), dtype=torch.float16, device=DEV),
                    adj=torch.zeros_like(z), tok=i(b * N), n=i(b), corr=i(b), path=i(b, R), len=i(b))

    def block(o, stream=None):
        kw = dict(stream=stream)
        api.dflash_tree_mask(buf["parent"], o["mask"], depth_out=o["depth"], **kw)
        api.dflash_tree_attention(q, kv, 1, kt, vt, o["mask"], o["out"], ws=ws, **kw)
        api.dflash_adjust_logits(z, o["adj"], hist=buf["hist"], n_hist=buf["nh"], draft=buf["tree"], path=o["mask"],
                                 repetition=buf["rho"], **kw)
        api.dflash_sample(o["adj"].flatten(0, 1), buf["T"], buf["u"], o["tok"], ws=ws, **kw)
        api.dflash_tree_accept(o["tok"].view(b, N), buf["tree"], buf["parent"], o["n"], o["corr"], o["path"], **kw)
        api.dflash_tree_commit(kv, tree_kv[:, :, :, :nkv], tree_kv[:, :, :, nkv:], o["path"], o["n"], len_out=o["len"], ws=wc,
                               **kw)
    want = outputs()
    block(want)
    torch.cuda.synchronize()
    k1 = kv.k.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = outputs()
    block(other, stream=side)
    side.synchronize()
    assert all(torch.equal(want[x], other[x]) for x in want)
    graphs, outs = [], []
    for _ in range(2):
        g, o = torch.cuda.CUDAGraph(), outputs()
        with torch.cuda.graph(g):
            block(o)
        graphs.append(g)
        outs.append(o)
    for g in graphs + graphs[:1]:
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(want[x], o[x]) for x in want)
    assert torch.equal(kv.k, k1)
    # other inputs in the same buffers
    z.copy_(torch.randn((b, N, V), device=DEV))
    z[..., :4] += 4
    kv.len.copy_(_i32([17, 256]))
    buf["parent"].copy_(_i32(_trees(rng, b, N)))
    graphs[1].replay()
    torch.cuda.synchronize()
    fresh = outputs()
    block(fresh)
    torch.cuda.synchronize()
    assert all(torch.equal(fresh[x], outs[1][x]) for x in want) and not torch.equal(fresh["out"], want["out"])


def test_early_launches_give_the_same():
    rng = np.random.default_rng(4)
    b, N = 3, 24
    kv, q, kt, vt = _attention_case(rng, "bf16", b, N, 8, 2, 128, 900, [900, 5, 333], [N] * 3, L=1)
    parent = _i32(_trees(rng, b, N))
    mask = torch.zeros((b, N, 1), dtype=torch.int32, device=DEV)
    api.dflash_tree_mask(parent, mask)
    want, lw = _attend(kv, 0, q, kt, vt, mask, None)
    torch.cuda.synchronize()
    with api.launch_mode(api.LAUNCH_EARLY):
        for _ in range(5):
            m2 = torch.zeros_like(mask)
            api.dflash_tree_mask(parent, m2)
            out, lse = _attend(kv, 0, q, kt, vt, m2, None)
            assert torch.equal(out, want) and torch.equal(lse, lw)


# ------------------------------------------------------------------ a loop ---
def test_tree_speculation_follows_the_target():
    """A small target decodes greedily under a repetition penalty and a grammar
    by whole trees: attention over its cache and the trees, adjusted logits,
    draw, accept, commit.  Each token has to be the 64-bit target's choice on the
    tokens before it, up to the logits' rounding (fp16 products: 0.03)."""
    rng = np.random.default_rng(21)
    b, L, nq, nkv, d, V, N, R = 2, 2, 4, 2, 64, 320, 24, 6
    H, prompt, steps = nq * d, 12, 9
    f = lambda *s: rng.normal(0, 1, s)
    E, P = f(V, H) * 0.7, f(200, H) * 0.4
    Wqkv, Wo, Wl = f(L, H, (nq + 2 * nkv) * d) / np.sqrt(H), f(L, H, H) / np.sqrt(H), f(H, V) / np.sqrt(H) * 2
    rho = 1.3
    allowed = rng.random(V) < 0.8

    def target(ids):  # the last row's logits, in 64 bits
        x = E[ids] + P[:len(ids)]
        for l in range(L):
            qkv = (x @ Wqkv[l]).reshape(len(ids), nq + 2 * nkv, d)
            sees = np.tril(np.ones((len(ids),) * 2, bool))
            o, _, _ = TO.tree_attention(qkv[:, :nq], np.zeros((0, nkv, d)), np.zeros((0, nkv, d)), qkv[:, nq:nq + nkv],
                                        qkv[:, nq + nkv:], sees, d ** -0.5)
            x = x + o.reshape(len(ids), H) @ Wo[l]
        return x[-1] @ Wl

    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV)
    e, p, wq, wo, wl = dev(E), dev(P), dev(Wqkv), dev(Wo), dev(Wl)
    kv = api.KVCache(types.SimpleNamespace(L=L, nkv=nkv, d=d), b, 160)
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    rho_t, grammar = torch.full((b,), rho, device=DEV), _i32(TO.pack_bits(allowed[None]))

    def nodes(tree, parent, n, hist, nh):
        """One target pass over a tree: tokens drawn and the layers' K, V."""
        n_nodes = tree.shape[1]
        mask, depth = i(b, n_nodes, (n_nodes + 31) // 32), i(b, n_nodes)
        api.dflash_tree_mask(parent, mask, n_nodes=n, depth_out=depth)
        x = e[tree.long()] + p[(kv.len[:, None] + depth.clamp(min=0)).long()]
        new = torch.zeros((L, b, n_nodes, nq + 2 * nkv, d), dtype=torch.float16, device=DEV)
        for l in range(L):
            new[l] = (x @ wq[l]).half().view(b, n_nodes, nq + 2 * nkv, d)
            o = torch.zeros((b, n_nodes, nq, d), dtype=torch.float16, device=DEV)
            api.dflash_tree_attention(new[l][:, :, :nq], kv, l, new[l][:, :, nq:nq + nkv], new[l][:, :, nq + nkv:], mask, o,
                                      n_nodes=n)
            x = x + o.float().view(b, n_nodes, H) @ wo[l]
        z = (x @ wl).view(b, n_nodes, V)
        api.dflash_adjust_logits(z, z, hist=hist, n_hist=nh, draft=tree, path=mask, repetition=rho_t, allow=grammar,
                                 allow_row=i(b, n_nodes))
        tok = i(b * n_nodes)
        api.dflash_sample(z.flatten(0, 1), torch.zeros(b * n_nodes, device=DEV), torch.rand((b * n_nodes, V), device=DEV), tok)
        return tok.view(b, n_nodes), new

    ids = [list(rng.integers(0, V, prompt)) for _ in range(b)]
    # the prompt but its last token, as one chain
    chain = _i32([s[:-1] for s in ids])
    up = _i32(np.tile(np.arange(-1, prompt - 2), (b, 1)))
    _, new = nodes(chain, up, None, i(b, 1), i(b))
    api.dflash_tree_commit(kv, new[:, :, :, nq:nq + nkv], new[:, :, :, nq + nkv:],
                           _i32(np.tile(np.arange(prompt - 1), (b, 1))), torch.full((b,), prompt - 2, dtype=torch.int32, device=DEV))
    assert kv.len.tolist() == [prompt - 1] * b
    taken = 0
    for step in range(steps):
        parent, tree, count = _trees(rng, b, N), rng.integers(0, V, (b, N)), rng.integers(N // 2, N + 1, b)
        for j in range(b):
            # drafts: the target's own choices along one path of three nodes, chance elsewhere
            tree[j, 0], parent[j, 1:4] = ids[j][-1], [0, 1, 2]
            s = list(ids[j])
            for c in (1, 2, 3):
                z, _ = TO.adjust_row(target(s), made=s, repetition=rho, allowed=allowed)
                tree[j, c] = int(z.argmax())
                s.append(tree[j, c])
            if step % 3 == 2:
                tree[j, 2] = (tree[j, 2] + 1) % V
        hist = _i32([s[:-1] + [-1] * (200 - len(s)) for s in ids])
        tok, new = nodes(_i32(tree), _i32(parent), _i32(count), hist, _i32([len(s) - 1 for s in ids]))
        n, corr, path, emitted, nxt = i(b), i(b), i(b, R), i(b, R), i(b)
        api.dflash_tree_accept(tok, _i32(tree), _i32(parent), n, corr, path, n_nodes=_i32(count), emitted=emitted, next_tok=nxt)
        api.dflash_tree_commit(kv, new[:, :, :, nq:nq + nkv], new[:, :, :, nq + nkv:], path, n)
        for j in range(b):
            out = [t for t in emitted[j].tolist() if t >= 0]
            assert len(out) == int(n[j]) + 1 and out[-1] == int(nxt[j])
            taken += len(out) - 1
            for t in out:
                z, _ = TO.adjust_row(target(ids[j]), made=ids[j], repetition=rho, allowed=allowed)
                assert z[t] >= z.max() - 0.03, (step, j, t)
                ids[j].append(t)
        assert kv.len.tolist() == [len(s) - 1 for s in ids]
    assert taken >= steps * b  # the planted paths are accepted
    assert api.dflash_get_status() == 0
