"""Measured cases of the vocabulary-row operators: filtered sampling, the
filtered speculative accept, top logits with log-sum-exp, and distillation
from a teacher's top logits.

`run` computes an operator either in its plain form (elementary torch
operations, 64 bits where decisions sit next to a border) or, with `own` set,
through the library's entry points.  All inputs are seeded and made on the
GPU.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2}
# what a row's request asks for, in turn over the rows of a "mixed" batch
MIX = ["kp", "p", "k", "m", "none", "greedy", "kpm"]


def listed():
    return [
        # one decoded token of one sequence: latency
        dict(name="sample-1", op="sample", rows=1, V=151936, pad=0, dtype="bf16", mode="kp"),
        # a decode batch of unlike requests on fp32 logits (filters, greedy and unfiltered rows)
        dict(name="sample-64-mixed", op="sample", rows=64, V=151936, pad=0, dtype="f32", mode="mixed"),
        # odd vocabulary, rows padded by an odd stride
        dict(name="sample-37-odd", op="sample", rows=37, V=50021, pad=11, dtype="f16", mode="kpm"),
        # a large decode batch under top-p alone (no bound on the kept tokens)
        dict(name="sample-512-p", op="sample", rows=512, V=151936, pad=0, dtype="bf16", mode="p"),
        # one block of 16 verified rows
        dict(name="accept-1x16", op="accept", b=1, R=16, D=15, V=151936, pad=0, dtype="f32", mode="kp"),
        # eight sequences of blocks, unlike requests
        dict(name="accept-8x16-mixed", op="accept", b=8, R=16, D=15, V=151936, pad=0, dtype="bf16", mode="mixed"),
        # sixteen sequences of 32-row blocks
        dict(name="accept-16x32", op="accept", b=16, R=32, D=31, V=151936, pad=0, dtype="bf16", mode="kp"),
        # the teacher's rows of one verified block
        dict(name="top-16", op="top", rows=16, V=151936, pad=0, dtype="f32", K=64, T=1.0),
        # the teacher's rows of a training batch
        dict(name="top-1024", op="top", rows=1024, V=151936, pad=0, dtype="bf16", K=256, T=2.0),
        # one block's loss and gradient
        dict(name="distill-15", op="distill", rows=15, V=151936, pad=0, dtype="f32", K=64, T=1.0, rest=True,
             mode="grad"),
        # odd sizes, loss first and the gradient by a second call from a given upstream gradient
        dict(name="distill-1023-two", op="distill", rows=1023, V=50021, pad=3, dtype="f16", K=37, T=1.5, rest=False,
             mode="two"),
        # a training batch's loss and gradient
        dict(name="distill-2048", op="distill", rows=2048, V=151936, pad=0, dtype="bf16", K=128, T=1.0, rest=True,
             mode="grad"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "accept", "top", "distill"])
    V = rng.choice([151936, _log_int(rng, 1000, 260000), _log_int(rng, 1000, 260000)])
    c = dict(op=op, V=V, dtype=rng.choice(["f32", "f16", "bf16"]), pad=rng.choice([0, 0, 0, rng.randrange(1, 40)]))
    room = 75_000_000 // (V + c["pad"])  # rows that keep a case below the largest listed one
    if op == "sample":
        c.update(rows=_log_int(rng, 1, min(512, room)),
                 mode=rng.choice(["kp", "p", "k", "m", "none", "kpm", "mixed", "mixed"]))
    elif op == "accept":
        R = rng.randrange(2, 33)
        c.update(b=_log_int(rng, 1, max(1, min(32, room // R))), R=R, D=rng.choice([R - 1, R - 1, R]),
                 mode=rng.choice(["kp", "p", "k", "kpm", "mixed", "mixed"]))
    elif op == "top":
        c.update(rows=_log_int(rng, 1, min(1024, room)), K=_log_int(rng, 1, 1000), T=rng.choice([1.0, 0.7, 2.0]))
    else:
        c.update(rows=_log_int(rng, 1, min(2048, room)), K=_log_int(rng, 1, 512), T=rng.choice([1.0, 0.7, 2.0]),
                 rest=rng.random() < 0.5, mode=rng.choice(["loss", "grad", "grad", "two"]))
    return c


# ------------------------------------------------------------------ inputs ---
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _places(n, K, V, g):
    """K distinct token ids for each of n rows."""
    step = 1 + (torch.rand((n, 1), device="cuda", generator=g) * (V // K - 1)).long()
    return (torch.randint(0, V, (n, 1), device="cuda", generator=g) + step * torch.arange(K, device="cuda")) % V


def _rows(case, rows, g):
    """Logits of `rows` rows: a normal bulk under a head of likely tokens
    whose probabilities fall as a power of their rank; every ninth row has no
    head (a high-entropy position)."""
    V, ld = case["V"], case["V"] + case["pad"]
    buf = torch.empty((rows, ld), dtype=DTYPES[case["dtype"]], device="cuda")
    H = min(192, V // 4)
    fall = 1.3 * torch.log1p(torch.arange(H, device="cuda", dtype=torch.float32))
    for r0 in range(0, rows, 256):
        n = min(256, rows - r0)
        z = torch.randn((n, ld), device="cuda", generator=g).mul_(2.0)
        top = 18.0 + 1.5 * torch.randn((n, 1), device="cuda", generator=g)
        head = top - fall + 0.5 * torch.randn((n, H), device="cuda", generator=g)
        at = _places(n, H, V, g)
        lift = ((r0 + torch.arange(n, device="cuda")) % 9 != 8).unsqueeze(1)
        z.scatter_(1, at, torch.where(lift, head, z.gather(1, at)))
        buf[r0:r0 + n] = z
    return buf[:, :V]


def _params(mode, n, g):
    """Per-request temperature, top-k, top-p and min-p (an unset filter at its
    neutral value)."""
    T = 0.6 + 0.6 * torch.rand(n, device="cuda", generator=g)
    k = torch.randint(20, 101, (n,), device="cuda", generator=g)
    p = 0.8 + 0.18 * torch.rand(n, device="cuda", generator=g)
    mp = 0.02 + 0.08 * torch.rand(n, device="cuda", generator=g)
    kinds = [MIX[i % len(MIX)] if mode == "mixed" else mode for i in range(n)]
    has = lambda ch: torch.tensor([q not in ("none", "greedy") and ch in q for q in kinds], device="cuda")
    greedy = torch.tensor([q == "greedy" for q in kinds], device="cuda")
    return dict(T=torch.where(greedy, torch.zeros_like(T), T),
                k=torch.where(has("k"), k, torch.zeros_like(k)).to(torch.int32),
                p=torch.where(has("p"), p, torch.ones_like(p)),
                m=torch.where(has("m"), mp, torch.zeros_like(mp)))


def _uniforms(shape, g):
    """Uniforms strictly inside (0, 1)."""
    return torch.rand(shape, device="cuda", generator=g).clamp_(min=2.0 ** -25)


def prepare(case, seed):
    g = _gen(seed, 17)
    op, V = case["op"], case["V"]
    st = dict(case=case)
    if op == "sample":
        n = case["rows"]
        st["z"] = _rows(case, n, g)
        st.update(_params(case["mode"], n, g))
        st["u"] = _uniforms((n, V), g)
        st["tok"] = torch.empty(n, dtype=torch.int32, device="cuda")
        st["lp"] = torch.empty(n, dtype=torch.float32, device="cuda")
    elif op == "accept":
        b, R, D = case["b"], case["R"], case["D"]
        z = _rows(case, b * R, g)
        best = torch.topk(z.float(), 4, dim=1).indices.view(b, R, 4)
        which = (torch.rand((b, D, 1), device="cuda", generator=g) < 0.2).long()
        which = which * torch.randint(1, 4, (b, D, 1), device="cuda", generator=g)
        pick = best[:, :D].gather(2, which)
        st["draft"] = pick.squeeze(2).to(torch.int32).contiguous()
        # where the drafter agrees with the target both are sure: blocks keep
        # several drafts before the first rejection
        agree = torch.rand((b, D, 1), device="cuda", generator=g) < 0.95
        at = (torch.arange(b, device="cuda")[:, None] * R + torch.arange(D, device="cuda"))[agree[:, :, 0]]
        z[at, pick[agree]] = z[at].amax(1) + 4
        st["z"] = z.unflatten(0, (b, R))
        st.update(_params(case["mode"], b, g))
        st["ua"] = _uniforms((b, D), g)
        st["u"] = _uniforms((b, V), g)
        for name in ("n", "corr", "next"):
            st[name] = torch.empty(b, dtype=torch.int32, device="cuda")
        st["emitted"] = torch.empty((b, R), dtype=torch.int32, device="cuda")
        if own:
            from block_diffusion_speculative_draft_gb300 import api
            st["ws"] = torch.zeros(api.dflash_verify_filtered_workspace_size(b, R, V), dtype=torch.uint8,
                                   device="cuda")
    elif op == "top":
        n, K = case["rows"], case["K"]
        st["z"] = _rows(case, n, g)
        st["val"] = torch.empty((n, K), dtype=torch.float32, device="cuda")
        st["idx"] = torch.empty((n, K), dtype=torch.int32, device="cuda")
        st["lse"] = torch.empty(n, dtype=torch.float32, device="cuda")
    else:
        n, K = case["rows"], case["K"]
        z = _rows(case, n, g)
        # the teacher's K top tokens: distinct places, falling logits, and a
        # student that has learnt part of them
        at = _places(n, K, V, g)
        t = 20.0 - 1.2 * torch.log1p(torch.arange(K, device="cuda", dtype=torch.float32)) \
            + 0.4 * torch.randn((n, K), device="cuda", generator=g)
        z.scatter_(1, at, (t - 1.0 + 0.8 * torch.randn((n, K), device="cuda", generator=g)).to(z.dtype))
        st["z"], st["tv"], st["ti"] = z, t, at.to(torch.int32)
        st["tl"] = None
        if case["rest"]:  # the listed entries hold all but a few per cent of the teacher's mass
            rest = 0.01 + 0.05 * torch.rand(n, device="cuda", generator=g)
            st["tl"] = torch.logsumexp(t / case["T"], 1) - torch.log1p(-rest)
        st["w"] = 0.5 + torch.rand(n, device="cuda", generator=g)
        st["w"][torch.rand(n, device="cuda", generator=g) < 0.03] = 0.0  # positions left out of the loss
        st["loss"] = torch.empty(n, dtype=torch.float32, device="cuda")
        st["stats"] = torch.empty((n, 4), dtype=torch.float32, device="cuda")
        st["dz"] = None if case["mode"] == "loss" else torch.empty((n, V), dtype=z.dtype, device="cuda")
    return st


# --------------------------------------------------------------- plain forms ---
def _weights(z, T):
    """z with NaN masked, (z - max)/T and its exponential, in 64 bits."""
    z = z.double()
    z = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
    m = z.amax(1, keepdim=True)
    x = torch.where(z == m, torch.zeros_like(z), (z - m) / torch.where(T > 0, T, torch.ones_like(T)).double()[:, None])
    return z, m, x


def _kept(z, m, x, T, k, p, mp):
    """Truth value of each logit: kept by top-k, then top-p over what is left,
    then min-p."""
    V = z.shape[1]
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    w = torch.exp(x.gather(1, order))
    rank = torch.arange(V, device=z.device)[None]
    kk = torch.where(k > 0, k, torch.full_like(k, V))[:, None]
    keep = rank < kk
    w = torch.where(keep, w, torch.zeros_like(w))
    before = torch.cumsum(w, 1) - w
    pp = p.double()[:, None]
    keep &= (before < pp * w.sum(1, keepdim=True)) | (pp >= 1) | (rank == 0)
    keep &= (mp[:, None] <= 0) | (zs >= m + T.double()[:, None] * torch.log(mp.double())[:, None])
    keep &= (zs > -math.inf) & ((T[:, None] > 0) | (rank == 0))
    return torch.zeros_like(keep).scatter_(1, order, keep)


def _plain_sample(st):
    z, m, x = _weights(st["z"], st["T"])
    keep = _kept(z, m, x, st["T"], st["k"], st["p"], st["m"])
    none = torch.full_like(x, -math.inf)
    score = torch.where(keep, x - torch.log(-torch.log(st["u"].double())), none)
    best = score.amax(1, keepdim=True)
    at = torch.arange(z.shape[1], device=z.device)[None].expand_as(z)
    tok = torch.where(keep & (score == best), at, torch.full_like(at, z.shape[1])).amin(1)
    total = torch.where(keep, torch.exp(x), torch.zeros_like(x)).sum(1)
    lp = x.gather(1, tok[:, None])[:, 0] - torch.log(total)
    return tok.to(torch.int32), lp.float()


def _plain_accept(st):
    z3, draft = st["z"], st["draft"].long()
    b, R, V = z3.shape
    D = draft.shape[1]
    per_row = lambda a: a.repeat_interleave(R)
    T = per_row(st["T"])
    z, m, x = _weights(z3.reshape(b * R, V), T)
    keep = _kept(z, m, x, T, per_row(st["k"]), per_row(st["p"]), per_row(st["m"]))
    w = torch.where(keep, torch.exp(x), torch.zeros_like(x))
    prob = (w / w.sum(1, keepdim=True)).view(b, R, V)[:, :D].gather(2, draft[:, :, None])[:, :, 0]
    n = torch.cumprod((st["ua"].double() < prob).long(), 1).sum(1)
    row = n.clamp(max=R - 1)
    pick = torch.arange(b, device=z.device) * R + row
    score = torch.where(keep[pick], x[pick] - torch.log(-torch.log(st["u"].double())),
                        torch.full_like(x[pick], -math.inf))
    out = draft.gather(1, n.clamp(max=D - 1)[:, None])
    at = torch.arange(V, device=z.device)[None]
    score = torch.where((at == out) & (n < D)[:, None], torch.full_like(score, -math.inf), score)
    best = score.amax(1, keepdim=True)
    corr = torch.where((score == best) & (score > -math.inf), at.expand_as(score), torch.full_like(score, V).long()).amin(1)
    corr = torch.where(n < R, corr, torch.full_like(corr, -1))
    nxt = torch.where(corr >= 0, corr, draft.gather(1, (n - 1).clamp(min=0)[:, None])[:, 0])
    q = torch.arange(R, device=z.device)[None]
    ext = torch.nn.functional.pad(draft, (0, R - D))
    emitted = torch.where(q < n[:, None], ext, torch.where(q == n[:, None], corr[:, None], torch.full_like(ext, -1)))
    i32 = lambda a: a.to(torch.int32)
    return i32(n), i32(corr), i32(emitted), i32(nxt)


def _plain_top(st):
    K, T = st["case"]["K"], st["case"]["T"]
    z = st["z"].float()
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    m = zs[:, :1]
    lse = m[:, 0] / T + torch.log(torch.exp((z - m) / T).sum(1))
    return zs[:, :K].contiguous(), order[:, :K].to(torch.int32).contiguous(), lse


def _plain_distill(st):
    """Sums and statistics in 32 bits; the rest's probability, a difference
    from one, in 64."""
    c, w = st["case"], st["w"]
    T = c["T"]
    z = st["z"].float() / T
    t = st["tv"] / T
    at = st["ti"].long()
    lt = torch.logsumexp(t, 1) if st["tl"] is None else st["tl"]
    lp = t - lt[:, None]
    p = torch.exp(lp)
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lq = z.gather(1, at) - m - torch.log(total)
    loss = (p * (lp - lq)).sum(1)
    mass = p.sum(1)
    scale = mass[:, None]
    if st["tl"] is not None:
        pr = (1.0 - torch.exp(st["tv"].double() / T - lt.double()[:, None]).sum(1)).clamp(min=0).float()
        qr = e.scatter(1, at, 0.0).sum(1) / total[:, 0]
        loss = loss + pr * (torch.log(pr) - torch.log(qr))
        mass = mass + pr
        scale = (mass - pr / qr)[:, None]
    loss = loss * w
    if c["mode"] == "loss":
        return loss
    q = e / total
    grad = q * scale
    grad = grad.scatter(1, at, q.gather(1, at) * mass[:, None] - p)
    return loss, (grad * (w / T)[:, None]).to(st["z"].dtype)


def _own(st):
    from block_diffusion_speculative_draft_gb300 import api
    c = st["case"]
    if c["op"] == "sample":
        api.dflash_sample(st["z"], st["T"], st["u"], st["tok"], top_k=st["k"], top_p=st["p"], min_p=st["m"],
                          logprob_out=st["lp"])
        return st["tok"], st["lp"]
    if c["op"] == "accept":
        api.dflash_verify_accept_filtered(st["z"], st["draft"], st["T"], st["ua"], st["u"], st["n"], st["corr"],
                                          top_k=st["k"], top_p=st["p"], min_p=st["m"], emitted=st["emitted"],
                                          next_tok=st["next"], ws=st["ws"])
        return st["n"], st["corr"], st["emitted"], st["next"]
    if c["op"] == "top":
        api.dflash_top_logits(st["z"], c["K"], st["val"], st["idx"], lse_out=st["lse"], temperature=c["T"])
        return st["val"], st["idx"], st["lse"]
    if c["mode"] == "two":
        api.dflash_distill_loss(st["z"], st["tv"], st["ti"], st["loss"], t_lse=st["tl"], temperature=c["T"],
                                stats_out=st["stats"])
        api.dflash_distill_backward(st["z"], st["tv"], st["ti"], st["stats"], st["w"], st["dz"], t_lse=st["tl"],
                                    temperature=c["T"])
        return st["loss"] * st["w"], st["dz"]
    api.dflash_distill_loss(st["z"], st["tv"], st["ti"], st["loss"], t_lse=st["tl"], temperature=c["T"],
                            weight=st["w"], dlogits=st["dz"])
    return st["loss"] if st["dz"] is None else (st["loss"], st["dz"])


PLAIN = dict(sample=_plain_sample, accept=_plain_accept, top=_plain_top, distill=_plain_distill)


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------- exact ---
def _prefix(z, T, k, p, mp):
    """Kept token ids of one row in descending order of logit, with their
    weights, by walking the sorted row (64-bit numpy)."""
    z = np.where(np.isnan(z), -np.inf, z)
    m = z.max()
    if T == 0:
        i = int(np.argmax(z))
        return np.array([i]), np.ones(1)
    ids = np.lexsort((np.arange(z.size), -z))
    if k > 0:
        ids = ids[:k]
    ids = ids[z[ids] > -np.inf]
    w = np.exp((z[ids] - m) / T)
    if p < 1:
        c = np.concatenate([[0.0], np.cumsum(w)])
        ids = ids[:max(1, int(np.searchsorted(c[:-1], p * c[-1], side="left")))]
    if mp > 0:
        ids = ids[z[ids] >= m + T * np.log(mp)]
    return ids, np.exp((z[ids] - m) / T)


def _host(t, dtype=np.float64):
    return t.double().cpu().numpy().astype(dtype)


def _gumbel_pick(ids, w, u, drop=None):
    s = np.log(w) - np.log(-np.log(u[ids]))
    if drop is not None:
        s = np.where(ids == drop, -np.inf, s)
    best = s.max()
    return int(ids[s == best].min())


def exact(case, seed):
    elements = case["V"] * (case["b"] * case["R"] if case["op"] == "accept" else case["rows"])
    limit = 40_000_000 if case["op"] in ("sample", "accept") else 200_000_000
    if elements > limit:
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op in ("sample", "accept"):
        T, p, mp = (_host(st[a]) for a in ("T", "p", "m"))
        k = st["k"].cpu().numpy()
    if op == "sample":
        tok, lp = [], []
        for r in range(case["rows"]):
            z, u = _host(st["z"][r]), _host(st["u"][r])
            ids, w = _prefix(z, T[r], int(k[r]), p[r], mp[r])
            i = _gumbel_pick(ids, w, u)
            tok.append(i)
            lp.append(math.log(float(w[ids == i][0]) / math.fsum(w)))
        return torch.tensor(tok, dtype=torch.int32), torch.tensor(lp, dtype=torch.float64)
    if op == "accept":
        draft, ua = st["draft"].cpu().numpy(), _host(st["ua"])
        R, D = case["R"], case["D"]
        out = [[], [], [], []]
        for j in range(case["b"]):
            n, drop = 0, None
            while n < R:
                ids, w = _prefix(_host(st["z"][j, n]), T[j], int(k[j]), p[j], mp[j])
                if n >= D:
                    break
                x = int(draft[j, n])
                pr = float(w[ids == x].sum()) / math.fsum(w)
                if not ua[j, n] < pr:
                    drop = x
                    break
                n += 1
            corr = _gumbel_pick(ids, w, _host(st["u"][j]), drop) if n < R else -1
            em = [int(v) for v in draft[j, :n]] + ([corr] if n < R else [])
            out[0].append(n)
            out[1].append(corr)
            out[3].append(em[-1])
            out[2].append(em + [-1] * (R - len(em)))
        return tuple(torch.tensor(o, dtype=torch.int32) for o in out)
    z = st["z"].double()
    if op == "top":
        # the composite order by two passes of a selection, apart from sort
        v, i = torch.topk(z, case["K"], dim=1)
        last = v[:, -1:]
        idx = []
        for r in range(case["rows"]):
            zr = z[r]
            sure = torch.nonzero(zr > last[r])[:, 0]
            tied = torch.nonzero(zr == last[r])[:, 0][:case["K"] - sure.numel()]
            ids = torch.cat([sure, tied]).cpu().numpy()
            vals = zr[torch.as_tensor(ids, device=zr.device)].cpu().numpy()
            idx.append(ids[np.lexsort((ids, -vals))])
        idx = torch.as_tensor(np.stack(idx))
        val = z.cpu().gather(1, idx) if elements < 5_000_000 else v.cpu()
        lse = torch.logsumexp(z / case["T"], 1).cpu()
        return val, idx.to(torch.int32), lse
    T, w, at = case["T"], st["w"].double(), st["ti"].long()
    zt, t = z / T, st["tv"].double() / T
    mine = torch.logsumexp(zt, 1)
    log_p = t - (torch.logsumexp(t, 1) if st["tl"] is None else st["tl"].double())[:, None]
    p = log_p.exp()
    loss = (p * log_p).sum(1) - (p * zt.gather(1, at)).sum(1) + p.sum(1) * mine
    pr = torch.zeros_like(mine)
    outside = torch.logsumexp(zt.scatter(1, at, -math.inf), 1)
    if st["tl"] is not None:
        pr = (1 - p.sum(1)).clamp(min=0)
        loss = loss + torch.xlogy(pr, pr) - pr * (outside - mine)
    loss = loss * w
    if case["mode"] == "loss":
        return loss
    # d/dz of -sum p z - pr * lse(outside) + (sum p + pr) lse
    grad = torch.exp(zt - mine[:, None]) * (p.sum(1) + pr)[:, None]
    grad -= (pr[:, None] * torch.exp(zt - outside[:, None])).scatter(1, at, 0.0)
    grad.scatter_add_(1, at, -p)
    return loss, grad * (w / T)[:, None]


# ---------------------------------------------------------------------- work ---
def _unfiltered(mode, n):
    if mode == "none":
        return n
    return sum(MIX[i % len(MIX)] == "none" for i in range(n)) if mode == "mixed" else 0


def work(case):
    V, es, op = case["V"], ESIZE[case["dtype"]], case["op"]
    if op == "sample":
        # logits once; every uniform only where no filter leaves tokens out
        n = case["rows"]
        return dict(bytes=n * V * es + 4 * V * _unfiltered(case["mode"], n) + n * 24, flops=4 * n * V)
    if op == "accept":
        b, R = case["b"], case["R"]
        return dict(bytes=b * R * V * es + 4 * V * _unfiltered(case["mode"], b) + b * (16 + 12 * R), flops=4 * b * R * V)
    n, K = case["rows"], case["K"]
    if op == "top":
        return dict(bytes=n * V * es + n * (8 * K + 4), flops=4 * n * V)
    sides = 1 if case["mode"] == "loss" else 2
    return dict(bytes=n * V * es * sides + n * (8 * K + 12), flops=(4 if sides == 1 else 6) * n * V)
