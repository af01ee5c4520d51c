"""Measured cases of a verified tree of drafts: attention of the tree's nodes
over a cache, penalties / biases / grammar masks on the rows of logits, the
tree's masks and the accepted path, and the path's commit to the cache.

`run` computes an operator either in its plain form (elementary torch
operations in 32 bits) or, with `own` set, through the library's entry
points.  All inputs follow from the seed.
"""
import math
import types

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token of one sequence over a short context: latency
        dict(name="attend-1", op="attend", b=1, N=1, nq=32, nkv=8, d=128, ctx=1024, ragged=False, dtype="f16"),
        # odd everything: three sequences, 13-node trees, three query heads a kv head
        dict(name="attend-3x13-odd", op="attend", b=3, N=13, nq=6, nkv=2, d=64, ctx=2999, ragged=True, dtype="bf16"),
        # a batch of 32-node trees over ragged contexts
        dict(name="attend-8x32", op="attend", b=8, N=32, nq=40, nkv=8, d=128, ctx=8192, ragged=True, dtype="bf16"),
        # 64-node trees over long contexts
        dict(name="attend-4x64-long", op="attend", b=4, N=64, nq=32, nkv=8, d=128, ctx=65536, ragged=False,
             dtype="f16"),
        # one decoded token of one request, every adjustment
        dict(name="adjust-1", op="adjust", b=1, R=1, V=151936, pad=0, dtype="bf16", hist=1024, tree=False, kind="all"),
        # odd vocabulary and stride, 13-node trees
        dict(name="adjust-5x13-odd", op="adjust", b=5, R=13, V=50021, pad=11, dtype="f16", hist=700, tree=True,
             kind="all"),
        # a batch of blocks on fp32 logits, penalties and biases without a grammar
        dict(name="adjust-8x16", op="adjust", b=8, R=16, V=151936, pad=0, dtype="f32", hist=4096, tree=False,
             kind="penalties"),
        # a large batch of trees, every adjustment, long histories
        dict(name="adjust-32x32", op="adjust", b=32, R=32, V=151936, pad=0, dtype="bf16", hist=8192, tree=True,
             kind="all"),
        # one small tree: its masks and its accepted path
        dict(name="walk-1x16", op="walk", b=1, N=16, R=16),
        # a large batch of large trees
        dict(name="walk-64x256", op="walk", b=64, N=256, R=33),
        # a drafter-sized cache of one sequence
        dict(name="commit-1x16", op="commit", b=1, N=16, R=16, L=5, nkv=8, d=128, cap=640, hid=3 * 2560),
        # a batch in a target-sized cache
        dict(name="commit-16x64", op="commit", b=16, N=64, R=24, L=36, nkv=8, d=128, cap=320, hid=5 * 4096),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "adjust", "adjust", "walk", "commit"])
    if op == "attend":
        nkv, g, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([64, 128])
        b, N = _log_int(rng, 1, 16), _log_int(rng, 1, 128)
        # keys that keep a case below the largest listed one, in bytes and in products
        room = min(4 * 65536 * 8 * 128 // (b * nkv * d), 4 * 65536 * 32 * 64 * 128 // (b * nkv * g * N * d))
        return dict(op=op, b=b, N=N, nq=nkv * g, nkv=nkv, d=d, ctx=_log_int(rng, 1, min(65536, room)),
                    ragged=rng.random() < 0.6, dtype=rng.choice(["f16", "bf16"]))
    if op == "adjust":
        V = rng.choice([151936, _log_int(rng, 1000, 260000), _log_int(rng, 1000, 260000)])
        dtype, R = rng.choice(["f32", "f16", "bf16"]), _log_int(rng, 1, 64)
        pad = rng.choice([0, 0, rng.randrange(1, 40)])
        room = 1024 * 151936 * 2 // ((V + pad) * R * ESIZE[dtype])
        return dict(op=op, b=_log_int(rng, 1, max(1, min(64, room))), R=R, V=V, pad=pad, dtype=dtype,
                    hist=_log_int(rng, 1, 16384), tree=rng.random() < 0.5,
                    kind=rng.choice(["all", "all", "penalties", "grammar"]))
    if op == "walk":
        N = _log_int(rng, 1, 256)
        return dict(op=op, b=_log_int(rng, 1, 64), N=N, R=rng.randrange(1, N + 1))
    N = _log_int(rng, 1, 64)
    R = rng.randrange(1, min(N, 24) + 1)
    return dict(op=op, b=_log_int(rng, 1, 16), N=N, R=R, L=_log_int(rng, 1, 36), nkv=rng.choice([1, 2, 4, 8]),
                d=rng.choice([64, 128]), cap=rng.randrange(R, 321), hid=8 * rng.randrange(1, 2561))


# ------------------------------------------------------------------ inputs ---
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def _trees(rs, b, N):
    """Parents of b trees of N nodes: most nodes hang from one of the last few,
    as a drafter's likely continuations do, some from any earlier node."""
    parent = np.full((b, N), -1, np.int64)
    for i in range(1, N):
        near = np.maximum(0, i - 1 - rs.integers(0, 6, b))
        parent[:, i] = np.where(rs.random(b) < 0.7, near, rs.integers(0, i, b))
    return parent


def _seen(parent):
    """[b][N][N] truth values: node i sees node t (itself and its ancestors)."""
    b, N = parent.shape
    seen = np.zeros((b, N, N), bool)
    rows = np.arange(b)
    for i in range(N):
        up = parent[:, i]
        seen[:, i] = np.where((up >= 0)[:, None], seen[rows, np.maximum(up, 0)], False)
        seen[:, i, i] = True
    return seen


def _bits(seen):
    """Truth values along the last axis as 32-bit words, lowest bit first."""
    W = (seen.shape[-1] + 31) // 32
    full = np.zeros(seen.shape[:-1] + (W * 32,), np.uint8)
    full[..., :seen.shape[-1]] = seen
    return np.packbits(full, axis=-1, bitorder="little").view(np.uint32).view(np.int32)


def _tree_tokens(rs, parent, V):
    """A token for each node; a node's children have unlike tokens, but for a
    few that repeat one."""
    b, N = parent.shape
    tok = np.empty((b, N), np.int64)
    tok[:, 0] = rs.integers(0, V, b)
    for i in range(1, N):
        tok[:, i] = (tok[np.arange(b), parent[:, i]] * 31 + 7 + i * 13 * (rs.random(b) < 0.95)) % V
    return tok


def _prepare_attend(case, seed, rs, g):
    b, N, nq, nkv, d, dt = case["b"], case["N"], case["nq"], case["nkv"], case["d"], DTYPES[case["dtype"]]
    # the layer worked on is the second of a two-layer cache with room to grow
    cap = case["ctx"] + 37
    k = torch.empty((2, b, nkv, cap, d), dtype=dt, device="cuda")
    v = torch.empty_like(k)
    for j in range(b):
        for l in (0, 1):
            k[l, j] = torch.randn((nkv, cap, d), device="cuda", generator=g).mul_(1.5).to(dt)
            v[l, j] = torch.randn((nkv, cap, d), device="cuda", generator=g).to(dt)
    if case["ragged"]:
        lens = np.exp(rs.uniform(0, math.log(case["ctx"] + 1), b)).astype(np.int64).clip(1, case["ctx"])
        lens = np.maximum(lens, rs.integers(0, 2, b) * (case["ctx"] // 2))
        lens[rs.integers(b)] = case["ctx"]
        nodes = rs.integers(max(1, N // 2), N + 1, b)
    else:
        lens, nodes = np.full(b, case["ctx"]), np.full(b, N)
    # queries, keys and values of the nodes lie side by side, as one projection leaves them
    qkv = torch.randn((b, N, nq + 2 * nkv, d), device="cuda", generator=g)
    qkv[:, :, :nq + nkv] *= 1.2
    qkv = qkv.to(dt)
    st = dict(k=k, v=v, len=_dev(lens), nodes=_dev(nodes), q=qkv[:, :, :nq], kt=qkv[:, :, nq:nq + nkv],
              vt=qkv[:, :, nq + nkv:], mask=_dev(_bits(_seen(_trees(rs, b, N)))),
              out=torch.zeros((b, N, nq, d), dtype=dt, device="cuda"),
              lse=torch.zeros((b, N, nq), dtype=torch.float32, device="cuda"))
    if own:
        from block_diffusion_speculative_draft_gb300 import api
        shape = types.SimpleNamespace(L=2, nkv=nkv, d=d)
        st["kv"] = api.KVCache(shape, b, cap, k=k, v=v, len=st["len"])
        st["ws"] = torch.zeros(max(16, api.dflash_tree_attention_workspace_size(b, N, nq, nkv, d)), dtype=torch.uint8,
                               device="cuda")
    return st


def _prepare_adjust(case, seed, rs, g):
    b, R, V, ld = case["b"], case["R"], case["V"], case["V"] + case["pad"]
    buf = torch.empty((b, R, ld), dtype=DTYPES[case["dtype"]], device="cuda")
    for j in range(b):
        buf[j] = torch.randn((R, ld), device="cuda", generator=g).mul_(3.0)
    st = dict(z=buf[:, :, :V], out=torch.zeros((b, R, ld), dtype=buf.dtype, device="cuda")[:, :, :V])
    pen = case["kind"] != "grammar"
    # histories as text has them: few tokens often, many once
    H = case["hist"]
    zipf = torch.rand((b, H), device="cuda", generator=g).double()
    st["hist"] = (torch.exp(zipf * math.log(V)) - 1).long().mul_(7919).remainder_(V).to(torch.int32) if pen else None
    n = rs.integers((H + 1) // 2, H + 1, b)
    st["n_hist"] = _dev(n) if pen else None
    st["n_prompt"] = _dev((n * rs.uniform(0.2, 0.9, b)).astype(np.int64)) if pen else None
    for name, lo, hi in (("rep", 1.0, 1.4), ("freq", 0.0, 0.8), ("pres", -0.2, 0.8)):
        st[name] = _dev(rs.uniform(lo, hi, b), torch.float32) if pen else None
    # the drafts of a block (row r follows drafts 0..r-1) or of a tree (row i follows its path)
    st["draft"] = st["path"] = None
    if pen and (case["tree"] or R > 1):
        parent = _trees(rs, b, R) if case["tree"] else None
        draft = rs.integers(0, V, (b, R if case["tree"] else R - 1))
        took = st["hist"].cpu().numpy()[:, rs.integers(0, H, draft.shape[1])]
        draft = np.where(rs.random(draft.shape) < 0.6, took, draft)
        st["draft"] = _dev(draft)
        if case["tree"]:
            st["path"] = _dev(_bits(_seen(parent)))
    st["bi"] = st["bv"] = None
    if pen:
        st["bi"] = _dev(np.where(rs.random((b, 64)) < 0.3, -1, rs.integers(0, V, (b, 64))))
        st["bv"] = torch.randn((b, 64), device="cuda", generator=g).mul_(4.0)
        st["bv"][:, ::9] = -math.inf  # banned tokens
    st["allow"] = st["allow_row"] = None
    if case["kind"] != "penalties":
        # a grammar's states: a few tokens, a share of them, nearly all; rows without a grammar
        G, W = max(1, min(64, b * R)), (V + 31) // 32
        keep = _dev(np.array([0.0003, 0.02, 0.5, 0.999])[np.arange(G) % 4], torch.float32)
        allow = torch.zeros((G, W), dtype=torch.int64, device="cuda")
        for k in range(32):
            allow |= (torch.rand((G, W), device="cuda", generator=g) < keep[:, None]).long() << k
        st["allow"] = allow.to(torch.int32)
        row = rs.integers(0, G, (b, R))
        st["allow_row"] = _dev(np.where(rs.random((b, R)) < 0.25, -1, row))
    return st


def _prepare_walk(case, seed, rs, g):
    b, N = case["b"], case["N"]
    parent = _trees(rs, b, N)
    tok = _tree_tokens(rs, parent, 151936)
    nodes = rs.integers((N + 1) // 2, N + 1, b)
    want = rs.integers(0, 151936, (b, N))  # the target's token at each node: mostly one of its children's
    for i in range(N - 1, 0, -1):
        at = (np.arange(b), parent[:, i])
        want[at] = np.where(rs.random(b) < 0.75, tok[:, i], want[at])
    W = (N + 31) // 32
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
    return dict(parent=_dev(parent), tree=_dev(tok), want=_dev(want), nodes=_dev(nodes), mask=i32(b, N, W),
                depth=i32(b, N), n=i32(b), corr=i32(b), path=i32(b, case["R"]), emitted=i32(b, case["R"]), next=i32(b))


def _prepare_commit(case, seed, rs, g):
    b, N, R, L, nkv, d, cap = (case[x] for x in ("b", "N", "R", "L", "nkv", "d", "cap"))
    k = torch.empty((L, b, nkv, cap, d), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    for l in range(L):
        k[l] = torch.randn(k[l].shape, device="cuda", generator=g).half()
        v[l] = torch.randn(k[l].shape, device="cuda", generator=g).half()
    kv = torch.randn((L, b, N, 2 * nkv, d), device="cuda", generator=g).half()
    # paths of nodes from the root down; n = -1 is a sequence that commits nothing
    path, n = np.full((b, R), -1), rs.integers(-1, R, b)
    n[0] = R - 1
    for j in range(b):
        m = int(n[j]) + 1
        path[j, :m] = np.sort(rs.permutation(N)[:m])
    st = dict(k=k, v=v, len=_dev(rs.integers(0, cap - R + 1, b)), kt=kv[:, :, :, :nkv], vt=kv[:, :, :, nkv:],
              path=_dev(path), n=_dev(n), hid=torch.randn((b, N, case["hid"]), device="cuda", generator=g).half(),
              hid_out=torch.zeros((b, R, case["hid"]), dtype=torch.float16, device="cuda"),
              len_out=torch.zeros(b, dtype=torch.int32, device="cuda"))
    if own:
        from block_diffusion_speculative_draft_gb300 import api
        st["kv"] = api.KVCache(types.SimpleNamespace(L=L, nkv=nkv, d=d), b, cap, k=k, v=v, len=st["len"])
        st["ws"] = torch.zeros(api.dflash_tree_commit_workspace_size(b), dtype=torch.uint8, device="cuda")
    return st


PREPARE = dict(attend=_prepare_attend, adjust=_prepare_adjust, walk=_prepare_walk, commit=_prepare_commit)


def prepare(case, seed):
    st = PREPARE[case["op"]](case, seed, np.random.default_rng(seed * 7919 + 11), _gen(seed, 23))
    st["case"] = case
    return st


# --------------------------------------------------------------- plain forms ---
def _unpack(words, n):
    """32-bit words to truth values [..., n]."""
    sh = torch.arange(32, device=words.device, dtype=torch.int32)
    return ((words[..., None] >> sh) & 1).bool().flatten(-2)[..., :n]


def _plain_attend(st):
    c = st["case"]
    b, N, nq, nkv, d = c["b"], c["N"], c["nq"], c["nkv"], c["d"]
    g, T = nq // nkv, st["k"].shape[3]
    sees = _unpack(st["mask"], N)
    real = torch.arange(N, device="cuda")[None] < st["nodes"][:, None]
    old = torch.arange(T, device="cuda")[None] < st["len"][:, None]
    for j in range(b):
        ok = torch.cat([old[j][None].expand(N, T), sees[j] & real[j][None]], 1)[None, :, None]  # [1][N][1][T + N]
        q = st["q"][j].float().view(N, nkv, g, d).transpose(0, 1)                               # [nkv][N][g][d]
        k = torch.cat([st["k"][1, j].float(), st["kt"][j].float().transpose(0, 1)], 1)
        v = torch.cat([st["v"][1, j].float(), st["vt"][j].float().transpose(0, 1)], 1)
        s = torch.matmul(q.reshape(nkv, N * g, d), k.transpose(1, 2)).view(nkv, N, g, T + N)
        s = (s * (1 / math.sqrt(d))).masked_fill(~ok, -math.inf)
        m = s.amax(3, keepdim=True)
        p = torch.exp(s - m)
        total = p.sum(3, keepdim=True)
        o = torch.matmul(p.view(nkv, N * g, T + N), v).view(nkv, N, g, d) / total
        keep = real[j][:, None, None]
        st["out"][j] = torch.where(keep, o.transpose(0, 1).reshape(N, nq, d).to(st["out"].dtype), st["out"][j])
        lse = (m + torch.log(total))[..., 0].transpose(0, 1).reshape(N, nq)
        st["lse"][j] = torch.where(keep[..., 0], lse, st["lse"][j])
    return st["out"], st["lse"]


def _plain_adjust(st):
    c = st["case"]
    b, R, V = c["b"], c["R"], c["V"]
    for j in range(b):
        x = st["z"][j].float()
        if st["hist"] is not None:
            H = st["hist"].shape[1]
            at = torch.arange(H, device="cuda")
            ids = st["hist"][j].long()
            prompt = (at < st["n_prompt"][j]).float()
            made = ((at < st["n_hist"][j]) & (at >= st["n_prompt"][j])).float()
            there = torch.zeros(V, device="cuda").index_add_(0, ids, prompt) > 0
            count = torch.zeros(V, device="cuda").index_add_(0, ids, made)[None].expand(R, V)
            if st["draft"] is not None:
                D = st["draft"].shape[1]
                follows = (_unpack(st["path"][j], R) if st["path"] is not None else
                           torch.arange(R, device="cuda")[:, None] > torch.arange(D, device="cuda")[None])
                count = count.contiguous().scatter_add_(1, st["draft"][j].long()[None].expand(R, D), follows.float())
            seen = there[None] | (count > 0)
            x = torch.where(seen, torch.where(x > 0, x / st["rep"][j], x * st["rep"][j]), x)
            x = x - st["freq"][j] * count - st["pres"][j] * (count > 0).float()
        if st["bi"] is not None:
            bi = st["bi"][j].long()
            add = torch.zeros(V + 1, device="cuda").index_add_(0, torch.where(bi < 0, V, bi), st["bv"][j])
            x = x + add[:V]
        if st["allow"] is not None:
            row = st["allow_row"][j].long()
            ok = _unpack(st["allow"][row.clamp(min=0)], V) | (row < 0)[:, None]
            x = torch.where(ok, x, torch.full_like(x, -math.inf))
        st["out"][j] = x.to(st["out"].dtype)
    return st["out"]


def _plain_walk(st):
    parent, nodes, tree, want = st["parent"].long(), st["nodes"].long(), st["tree"].long(), st["want"].long()
    b, N = parent.shape
    R = st["case"]["R"]
    at = torch.arange(N, device="cuda")
    real = at[None] < nodes[:, None]
    up = (parent[:, :, None] == at) | torch.eye(N, dtype=torch.bool, device="cuda")
    sees = up.float()
    for _ in range(max(1, (N - 1).bit_length())):  # paths of doubling length
        sees = (torch.matmul(sees, sees) > 0).float()
    sees = (sees > 0) & real[:, :, None]
    depth = torch.where(real, sees.sum(2) - 1, -1)
    W = (N + 31) // 32
    words = torch.nn.functional.pad(sees, (0, W * 32 - N)).view(b, N, W, 32).long()
    mask = (words << torch.arange(32, device="cuda")).sum(3)
    cur, live = torch.zeros(b, dtype=torch.long, device="cuda"), torch.ones(b, dtype=torch.bool, device="cuda")
    n = torch.zeros(b, dtype=torch.long, device="cuda")
    path = torch.full((b, R), -1, dtype=torch.long, device="cuda")
    emitted = path.clone()
    path[:, 0] = 0
    for i in range(1, R):
        t = want.gather(1, cur[:, None])
        match = (parent == cur[:, None]) & (tree == t) & real
        step = torch.where(match, at, N).amin(1)
        live = live & (step < N)
        cur = torch.where(live, step, cur)
        n = n + live.long()
        path[:, i] = torch.where(live, cur, -1)
        emitted[:, i - 1] = torch.where(live, t[:, 0], -1)
    corr = want.gather(1, cur[:, None])
    emitted.scatter_(1, n[:, None], corr)
    i32 = lambda x: x.to(torch.int32)
    return i32(mask), i32(depth), i32(n), i32(corr[:, 0]), i32(path), i32(emitted), i32(corr[:, 0])


def _plain_commit(st):
    c = st["case"]
    b, R, nkv, d = c["b"], c["R"], c["nkv"], c["d"]
    i = torch.arange(R, device="cuda")
    live = i[None] <= st["n"][:, None]
    node = st["path"].long().clamp(min=0)
    row = (st["len"].long()[:, None] + i)[:, None, :, None].expand(b, nkv, R, d)
    pick = node[:, :, None, None].expand(b, R, nkv, d)
    for cache, tree in ((st["k"], st["kt"]), (st["v"], st["vt"])):
        for l in range(c["L"]):
            new = tree[l].gather(1, pick).transpose(1, 2)
            cache[l].scatter_(2, row, torch.where(live[:, None, :, None], new, cache[l].gather(2, row)))
    hid = st["hid"].gather(1, node[:, :, None].expand(b, R, c["hid"]))
    st["hid_out"].copy_(torch.where(live[:, :, None], hid, st["hid_out"]))
    return st["k"], st["v"], st["len"] + st["n"] + 1, st["hid_out"]


def _own(st):
    from block_diffusion_speculative_draft_gb300 import api
    op = st["case"]["op"]
    if op == "attend":
        api.dflash_tree_attention(st["q"], st["kv"], 1, st["kt"], st["vt"], st["mask"], st["out"], n_nodes=st["nodes"],
                                  lse_out=st["lse"], ws=st["ws"])
        return st["out"], st["lse"]
    if op == "adjust":
        api.dflash_adjust_logits(st["z"], st["out"], hist=st["hist"], n_hist=st["n_hist"], n_prompt=st["n_prompt"],
                                 draft=st["draft"], path=st["path"], repetition=st["rep"], frequency=st["freq"],
                                 presence=st["pres"], bias_idx=st["bi"], bias_val=st["bv"], allow=st["allow"],
                                 allow_row=st["allow_row"])
        return st["out"]
    if op == "walk":
        api.dflash_tree_mask(st["parent"], st["mask"], n_nodes=st["nodes"], depth_out=st["depth"])
        api.dflash_tree_accept(st["want"], st["tree"], st["parent"], st["n"], st["corr"], st["path"],
                               n_nodes=st["nodes"], emitted=st["emitted"], next_tok=st["next"])
        return tuple(st[x] for x in ("mask", "depth", "n", "corr", "path", "emitted", "next"))
    api.dflash_tree_commit(st["kv"], st["kt"], st["vt"], st["path"], st["n"], hid=st["hid"], hid_out=st["hid_out"],
                           len_out=st["len_out"], ws=st["ws"])
    return st["k"], st["v"], st["len_out"], st["hid_out"]


PLAIN = dict(attend=_plain_attend, adjust=_plain_adjust, walk=_plain_walk, commit=_plain_commit)


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------- exact ---
def _exact_attend(case, st):
    """One query head at a time over its own list of keys, in 64 bits."""
    b, N, nq, nkv, d = case["b"], case["N"], case["nq"], case["nkv"], case["d"]
    bit = _host_bits(st["mask"], N)
    out, lse = torch.zeros((b, N, nq, d), dtype=torch.float64), torch.zeros((b, N, nq), dtype=torch.float64)
    for j in range(b):
        C, n = int(st["len"][j]), int(st["nodes"][j])
        block = torch.as_tensor(np.where(bit[j, :n, :n], 0.0, -np.inf), device="cuda")
        for h in range(nq):
            q = st["q"][j, :n, h].double() / math.sqrt(d)
            old = q @ st["k"][1, j, h * nkv // nq, :C].double().T
            new = q @ st["kt"][j, :n, h * nkv // nq].double().T + block
            both = torch.logsumexp(torch.cat([old, new], 1), 1, keepdim=True)
            o = torch.exp(old - both) @ st["v"][1, j, h * nkv // nq, :C].double()
            o += torch.exp(new - both) @ st["vt"][j, :n, h * nkv // nq].double()
            out[j, :n, h], lse[j, :n, h] = o.cpu(), both[:, 0].cpu()
    return out, lse


def _host_bits(words, n):
    w = words.cpu().numpy().view(np.uint32).view(np.uint8)
    return np.unpackbits(w, axis=-1, bitorder="little")[..., :n].astype(bool)


def _exact_adjust(case, st):
    """Row by row: only the tokens that something changes are worked on."""
    b, R, V = case["b"], case["R"], case["V"]
    if b * R * V > 200_000_000:
        return None
    host = {x: None if st[x] is None else st[x].cpu().numpy() for x in
            ("hist", "n_hist", "n_prompt", "rep", "freq", "pres", "draft", "bi", "bv", "allow_row")}
    path = None if st["path"] is None else _host_bits(st["path"], R)
    allow = None if st["allow"] is None else _host_bits(st["allow"], V)
    out = torch.empty((b, R, V), dtype=torch.float64)
    for j in range(b):
        rows = st["z"][j].double().cpu().numpy()
        for r in range(R):
            x = rows[r]
            if host["hist"] is not None:
                a, e = int(host["n_prompt"][j]), int(host["n_hist"][j])
                made = list(host["hist"][j, a:e])
                if host["draft"] is not None:
                    d = host["draft"][j]
                    made += list(d[path[j, r]]) if path is not None else list(d[:r])
                ids, c = np.unique(np.array(made, np.int64), return_counts=True)
                both = np.union1d(ids, host["hist"][j, :a]).astype(np.int64)
                rho = float(host["rep"][j])
                x[both] = np.where(x[both] > 0, x[both] / rho, x[both] * rho)
                x[ids] -= float(host["freq"][j]) * c + float(host["pres"][j])
            if host["bi"] is not None:
                for t, w in zip(host["bi"][j], host["bv"][j]):
                    if t >= 0:
                        x[t] += float(w)
            if allow is not None and host["allow_row"][j, r] >= 0:
                x[~allow[host["allow_row"][j, r]]] = -np.inf
        out[j] = torch.from_numpy(rows)
    return out


def exact(case, seed):
    if case["op"] not in ("attend", "adjust"):
        return None  # whole numbers and copies
    st = prepare(case, seed)
    return (_exact_attend if case["op"] == "attend" else _exact_adjust)(case, st)


# ---------------------------------------------------------------------- work ---
def work(case):
    op, b = case["op"], case["b"]
    if op == "attend":
        N, nq, nkv, d = case["N"], case["nq"], case["nkv"], case["d"]
        # a ragged batch's contexts are about half of the longest one, its trees three quarters
        keys = case["ctx"] * (0.5 if case["ragged"] and b > 1 else 1.0) + N
        rows = N * (0.75 if case["ragged"] else 1.0)
        return dict(bytes=int(b * (4 * keys * nkv * d + 4 * rows * nq * d + 4 * rows * nq)),
                    flops=int(4 * b * rows * nq * d * keys))
    if op == "adjust":
        n, V = b * case["R"], case["V"]
        masks = 0 if case["kind"] == "penalties" else min(64, n) * V // 8
        return dict(bytes=2 * n * V * ESIZE[case["dtype"]] + masks + 4 * b * case["hist"] * (case["kind"] != "grammar"),
                    flops=6 * n * V)
    if op == "walk":
        N, R = case["N"], case["R"]
        return dict(bytes=b * (12 * N + 4 * N * ((N + 31) // 32) + 4 * N + 8 * R + 16), flops=b * N)
    # half of the batch's paths on average
    rows = b * (case["R"] + 1) / 2
    return dict(bytes=int(rows * 2 * (case["L"] * case["nkv"] * case["d"] * 4 + case["hid"] * 2)), flops=0)
