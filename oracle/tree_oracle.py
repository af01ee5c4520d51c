"""Plain float64 numpy forms of the operators on a tree of drafts and of the
adjustments of logits: one sequence (or row) at a time, written from the
formulas.  Test infrastructure only."""
import numpy as np


def tree_mask(parent, n=None):
    """(sees [N][N] truth values, depth [N]): node i sees itself and its
    ancestors; nodes that are not there, whose parent is out of range or that
    hang from such a node see nothing and have depth -1."""
    N = len(parent)
    n = N if n is None else n
    sees, depth = np.zeros((N, N), bool), np.full(N, -1)
    for i in range(n):
        p = int(parent[i])
        if p == -1:
            depth[i] = 0
        elif 0 <= p < i and depth[p] >= 0:
            sees[i] = sees[p]
            depth[i] = depth[p] + 1
        if depth[i] >= 0:
            sees[i, i] = True
    return sees, depth


def pack_bits(sees):
    """Truth values along the last axis as int32 words, lowest bit first."""
    W = (sees.shape[-1] + 31) // 32
    full = np.zeros(sees.shape[:-1] + (W * 32,), np.uint8)
    full[..., :sees.shape[-1]] = sees
    return np.packbits(full, axis=-1, bitorder="little").view(np.uint32).view(np.int32)


def tree_attention(q, k, v, kt, vt, sees, scale):
    """q [n][nq][d] over cached keys k, v [C][nkv][d] and the nodes' kt, vt
    [n][nkv][d] that sees [n][n] allows: (o [n][nq][d], lse [n][nq], spread):
    spread [n][nq][d] is sum p |v| / sum p."""
    n, nq, d = q.shape
    nkv = kt.shape[1]
    o, lse, spread = np.zeros((n, nq, d)), np.full((n, nq), -np.inf), np.zeros((n, nq, d))
    for h in range(nq):
        g = h * nkv // nq
        keys = np.concatenate([k[:, g], kt[:, g]]).astype(np.float64)
        vals = np.concatenate([v[:, g], vt[:, g]]).astype(np.float64)
        s = scale * (q[:, h].astype(np.float64) @ keys.T)
        s[:, len(k):][~sees] = -np.inf
        m = s.max(1, initial=-np.inf)
        p = np.exp(s - np.where(np.isneginf(m), 0.0, m)[:, None])
        total = p.sum(1)
        some = total > 0
        o[some, h] = (p @ vals)[some] / total[some, None]
        spread[some, h] = (p @ np.abs(vals))[some] / total[some, None]
        lse[some, h] = m[some] + np.log(total[some])
    return o, lse, spread


def tree_accept(tok, tree, parent, R, n=None):
    """(steps, corr, path [R], emitted [R], next token) of the walk."""
    n = len(tok) if n is None else n
    path, emitted = [-1] * R, [-1] * R
    if n == 0:
        return -1, -1, path, emitted, -1
    cur, steps = 0, 0
    path[0] = 0
    while steps + 1 < R and tok[cur] >= 0:
        kids = [c for c in range(cur + 1, n) if parent[c] == cur and tree[c] == tok[cur]]
        if not kids:
            break
        cur = kids[0]
        steps += 1
        path[steps] = cur
        emitted[steps - 1] = int(tree[cur])
    corr = int(tok[cur]) if tok[cur] >= 0 else -1
    emitted[steps] = corr
    return steps, corr, path, emitted, corr if corr >= 0 else int(tree[cur])


def adjust_row(z, prompt=(), made=(), repetition=1.0, frequency=0.0, presence=0.0, bias=(), allowed=None):
    """One row: prompt and made are lists of tokens, bias of (token, value),
    allowed truth values [V] (None: no grammar).  Returns (row, size): size
    bounds every intermediate value's magnitude."""
    x = np.array(z, np.float64)
    V = x.size
    c = np.zeros(V)
    there = np.zeros(V, bool)
    for t in made:
        if 0 <= t < V:
            c[t] += 1
    for t in prompt:
        if 0 <= t < V:
            there[t] = True
    seen = there | (c > 0)
    size = np.abs(x)
    with np.errstate(invalid="ignore"):
        x = np.where(seen, np.where(x > 0, x / repetition, x * repetition), x)
        size = np.maximum(size, np.abs(x))
        x = x - frequency * c - presence * (c > 0)
        size = size + abs(frequency) * c + abs(presence) * (c > 0)
        for t, w in bias:
            if 0 <= t < V:
                x[t] += w
                size[t] += abs(w)
    if allowed is not None:
        x = np.where(allowed, x, -np.inf)
    return x, size
