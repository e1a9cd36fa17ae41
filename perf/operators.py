"""The operators of a speculative-decoding step and of training its draft model, as measured cases.

- ``tree_attention``: attention of a tree of drafted tokens over a layer's K/V cache;
- ``sample``: sampling with temperature, top-k, top-p and min-p from given random numbers;
- ``tree_accept``: the accepted path of a sampled tree, and its K/V moved into the cache;
- ``distill_topk``: distillation from a teacher's top logits, loss and logit gradient.

``run`` computes a case either in its plain form (elementary torch operations) or, with ``own`` set, by the
framework's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def _attn(B, N, H, Hkv, D, T_max, len_lo, len_hi, window, dtype, ragged=False):
    return dict(kind="attn", B=B, N=N, H=H, Hkv=Hkv, D=D, T_max=T_max, len_lo=len_lo, len_hi=len_hi, window=window,
                dtype=dtype, ragged=ragged)


def _sample(M, V, params):
    return dict(kind="sample", M=M, V=V, params=params)


def _accept(B, N, L, Hkv, D, T_max, acc, dtype):
    return dict(kind="accept", B=B, N=N, L=L, Hkv=Hkv, D=D, T_max=T_max, acc=acc, dtype=dtype)


def _distill(M, V, K, cap, tau, dz, weighted):
    return dict(kind="distill", M=M, V=V, K=K, cap=cap, tau=tau, dz=dz, weighted=weighted)


def listed():
    return [
        # one user's short chat: a chain-like draft of four tokens over 300 kept positions (d20's heads)
        dict(_attn(1, 4, 10, 10, 128, 2048, 300, 300, 0, "fp16"), name="attn chat B1 N4"),
        # a small serving batch at the 2048-token context, grouped heads (the d26 GQA model's)
        dict(_attn(8, 32, 16, 4, 128, 2048, 900, 1990, 0, "bf16"), name="attn gqa B8 N32"),
        # a layer with the 512-key window, 64-wide heads, trees of different sizes padded to 27 nodes
        dict(_attn(16, 27, 12, 12, 64, 4096, 700, 3900, 512, "fp16", True), name="attn window D64 B16 N27"),
        # a large batch of long contexts, wide trees: the heaviest step
        dict(_attn(32, 64, 16, 4, 128, 8192, 3000, 8100, 0, "fp16"), name="attn long B32 N64"),
        # the next token of one user, the usual filters
        dict(_sample(1, 32768, "usual"), name="sample M1"),
        # one decode step of 32 requests, each with settings of its own
        dict(_sample(32, 32768, "mixed"), name="sample M32 mixed"),
        # every node of 16 trees of 64, temperature alone; a vocabulary that is no multiple of 4
        dict(_sample(1024, 32749, "pure"), name="sample M1024 pure"),
        # one user's tree of eight nodes, 20 layers (d20's cache)
        dict(_accept(1, 8, 20, 10, 128, 256, 3, "fp16"), name="accept B1 N8"),
        # 32 users' trees of 64 nodes, 26 layers of the d26 GQA model
        dict(_accept(32, 64, 26, 4, 128, 256, 5, "bf16"), name="accept B32 N64"),
        # a short distillation batch on a small vocabulary
        dict(_distill(64, 512, 8, 15.0, 1.0, "fp32", False), name="distill V512"),
        # a training micro-batch of two 2048-token rows: loss and the 16-bit logit gradient
        dict(_distill(4096, 32768, 64, 15.0, 2.0, "bf16", True), name="distill train M4096"),
        # the same loss as an evaluation, without the gradient
        dict(_distill(2048, 32768, 32, 15.0, 1.0, "none", False), name="distill eval M2048"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b = most.setdefault(c["kind"], {"bytes": 0, "flops": 0})
        for k in b:
            b[k] = max(b[k], w[k])
    kind = rng.choice(["attn", "attn", "sample", "sample", "accept", "distill", "distill"])
    while True:
        if kind == "attn":
            Hkv = rng.choice([1, 2, 4, 5, 8, 10, 12])
            G = rng.choice([1, 1, 2, 3, 4, 8])
            hi = _log(rng, 1, 8000)
            T = hi + rng.randint(0, 300)
            c = _attn(_log(rng, 1, 32), _log(rng, 1, 64), Hkv * G, Hkv, rng.choice([64, 128]), T, rng.randint(0, hi), hi,
                      rng.choice([0, 0, _log(rng, 16, 2000)]), rng.choice(["fp16", "bf16"]), rng.random() < 0.3)
        elif kind == "sample":
            c = _sample(_log(rng, 1, 1024), _log(rng, 500, 60000), rng.choice(["usual", "mixed", "pure", "topp"]))
        elif kind == "accept":
            N = _log(rng, 2, 128)
            c = _accept(_log(rng, 1, 32), N, rng.randint(2, 26), rng.choice([1, 2, 4, 5, 10]), rng.choice([64, 128]),
                        rng.randint(160, 300), rng.randint(1, min(N, 9)), rng.choice(["fp16", "bf16"]))
        else:
            V = _log(rng, 512, 50000)
            c = _distill(_log(rng, 1, 4096), V, _log(rng, 1, 128), rng.choice([0.0, 15.0]), rng.choice([1.0, 1.5, 2.0]),
                         rng.choice(["none", "fp32", "bf16", "fp16"]), rng.random() < 0.5)
        w = work(c)
        if all(w[k] <= most[kind][k] for k in w):
            return c


def _lens(c):
    """Committed lengths of the rows: spread evenly over [len_lo, len_hi] (one row: len_hi)."""
    B = c["B"]
    return [c["len_hi"] if B == 1 else c["len_lo"] + (c["len_hi"] - c["len_lo"]) * b // (B - 1) for b in range(B)]


def _nodes(c):
    """Nodes in use of each row's tree."""
    B, N = c["B"], c["N"]
    lo = (N + 3) // 4
    return [N if not c["ragged"] or B == 1 else lo + (N - lo) * b // (B - 1) for b in range(B)]


def work(c):
    k = c["kind"]
    if k == "attn":
        B, N, H, Hkv, D, W = c["B"], c["N"], c["H"], c["Hkv"], c["D"], c["window"]
        keys = [n if W <= 0 else min(n, W - 1) for n in _lens(c)]
        nodes = _nodes(c)
        kv = 2 * Hkv * D * 2
        return {"bytes": sum(keys) * kv + sum(nodes) * kv + 2 * B * N * H * D * 2 + B * N * 4 * ((N + 31) // 32) + 4 * B,
                "flops": 4 * D * H * sum(n * (x + 1 + math.log2(n)) for n, x in zip(nodes, keys))}
    if k == "sample":
        return {"bytes": c["M"] * (c["V"] * 4 + 4 + 16 + 8), "flops": 3 * c["M"] * c["V"]}
    if k == "accept":
        B, N, L = c["B"], c["N"], c["L"]
        return {"bytes": 2 * L * B * c["acc"] * 2 * c["Hkv"] * c["D"] * 2 + B * N * 4 * (3 + (N + 31) // 32 + 1) + 16 * B,
                "flops": B * N * N}
    M, V, K = c["M"], c["V"], c["K"]
    out = {"none": 0, "fp32": 4, "bf16": 2, "fp16": 2}[c["dz"]]
    return {"bytes": M * V * (4 + out) + M * K * 8 + M * 4 * (2 if c["weighted"] else 1),
            "flops": M * V * (8 if out else 4)}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _tree(rs, N, n, chain=None):
    """Parents of a random tree of n nodes padded to N (-1: the root, -2: unused); `chain`: a path that it holds."""
    p = np.full(N, -2, np.int32)
    p[0] = -1
    for i in range(1, n):
        p[i] = rs.randint(0, i)
    if chain is not None:
        for a, b in zip(chain[:-1], chain[1:]):
            p[b] = a
    return p


def _mask_words(parents):
    """[B, N, W] int32: bit j of node i's words is set where j is i or an ancestor of i."""
    B, N = parents.shape
    W = (N + 31) // 32
    bits = np.zeros((B, N, W * 32), np.uint8)
    for i in range(N):
        p = parents[:, i]
        for b in range(B):
            if p[b] == -2:
                continue
            if p[b] >= 0:
                bits[b, i] = bits[b, p[b]]
            bits[b, i, i] = 1
    return np.packbits(bits, axis=-1, bitorder="little").view(np.int32).reshape(B, N, W)


def _prepare_attn(c, seed):
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    B, N, H, Hkv, D = c["B"], c["N"], c["H"], c["Hkv"], c["D"]
    dt = DTYPES[c["dtype"]]
    order = rs.permutation(B)
    lens, nodes = np.array(_lens(c))[order], np.array(_nodes(c))[order]
    parents = np.stack([_tree(rs, N, n) for n in nodes])
    q = _randn((B, N, H, D), g, dt)
    return {"case": c, "q": q, "kv": _randn((B, N, 2, Hkv, D), g, dt),
            "cache": _randn((B, c["T_max"], 2, Hkv, D), g, dt), "lens": _int(lens), "mask": _int(_mask_words(parents)),
            "out": torch.empty_like(q)}


def _prepare_sample(c, seed):
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    M, V, how = c["M"], c["V"], c["params"]
    # logits as a language model's: a bell of unlikely tokens with an exponential tail of likely ones, soft-capped at 15
    z = 1.5 * _randn((M, V), g)
    z -= 1.2 * torch.rand((M, V), generator=g, device=DEV).clamp_min_(1e-7).log_()
    s = {"case": c, "logits": 15.0 * torch.tanh(z / 15.0), "u": torch.rand(M, generator=g, device=DEV)}
    f32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV)  # noqa: E731
    none = {"temperature": None, "top_k": None, "top_p": None, "min_p": None}
    if how == "usual":
        none.update(temperature=f32(np.full(M, 0.8)), top_k=_int(np.full(M, 50)), top_p=f32(np.full(M, 0.95)))
    elif how == "mixed":
        none.update(temperature=f32(rs.choice([0.0, 0.6, 0.8, 1.0, 1.2], M)), top_k=_int(rs.choice([0, 20, 50, 200], M)),
                    top_p=f32(rs.choice([0.8, 0.9, 0.95, 1.0], M)), min_p=f32(rs.choice([0.0, 0.02, 0.05], M)))
    elif how == "topp":
        none.update(temperature=f32(rs.uniform(0.5, 1.5, M)), top_p=f32(rs.uniform(0.3, 0.99, M)))
    else:
        none.update(temperature=f32(np.full(M, 1.0)))
    s.update(none)
    s["tokens"] = torch.empty(M, dtype=torch.int32, device=DEV)
    s["logprob"] = torch.empty(M, dtype=torch.float32, device=DEV)
    return s


def _prepare_accept(c, seed):
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    B, N, L, Hkv, D, V = c["B"], c["N"], c["L"], c["Hkv"], c["D"], 32768
    dt = DTYPES[c["dtype"]]
    parents, tokens, sampled = (np.zeros((B, N), np.int32) for _ in range(3))
    for b in range(B):
        chain = np.concatenate([[0], np.sort(rs.choice(np.arange(1, N), c["acc"] - 1, replace=False))])
        parents[b] = _tree(rs, N, N, chain)
        t = rs.permutation(V)[:2 * N + 1]
        tokens[b], sampled[b] = t[:N], t[N:2 * N]  # no drafted token is sampled ...
        sampled[b, chain[:-1]] = tokens[b, chain[1:]]  # ... but along the chain
    lens = rs.randint(0, c["T_max"] - N + 1, B)
    out = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"case": c, "tokens": _int(tokens), "parents": _int(parents), "mask": _int(_mask_words(parents)),
            "sampled": _int(sampled), "lens": _int(lens), "kv": _randn((L, B, N, 2, Hkv, D), g, dt),
            "cache": _randn((L, B, c["T_max"], 2, Hkv, D), g, dt), "path": out(B, N), "count": out(B), "next": out(B),
            "lens_out": out(B)}


def _prepare_distill(c, seed):
    g = _gen(seed)
    M, V, K = c["M"], c["V"], c["K"]
    z = 3.0 * _randn((M, V), g)
    # the teacher agrees with the student in part: its top logits are those of a noisy copy
    cap = c["cap"]
    t = z + 1.5 * _randn((M, V), g)
    t = cap * torch.tanh(t / cap) if cap > 0 else t
    tl, ti = torch.topk(t, K, dim=1)
    del t
    return {"case": c, "z": z, "teacher_idx": ti.to(torch.int32).contiguous(), "teacher_logits": tl.contiguous(),
            "row_weight": torch.rand(M, generator=g, device=DEV) if c["weighted"] else None,
            "token_loss": torch.empty(M, device=DEV),
            "dz": None if c["dz"] == "none" else torch.empty((M, V), dtype=DTYPES[c["dz"]], device=DEV)}


def prepare(case, seed):
    return {"attn": _prepare_attn, "sample": _prepare_sample, "accept": _prepare_accept,
            "distill": _prepare_distill}[case["kind"]](case, seed)


# ------------------------------------------------------------------ plain forms

def _bits(mask, N):
    """[B, N, N] truth values of the packed words."""
    j = torch.arange(N, device=mask.device)
    return (mask[:, :, j // 32] >> (j % 32)) & 1 == 1


def _plain_attn(s):
    c, q, kv, cache, lens = s["case"], s["q"], s["kv"], s["cache"], s["lens"]
    B, N, H, D = q.shape
    T, Hkv, W = cache.shape[1], cache.shape[3], c["window"]
    anc = _bits(s["mask"], N)
    used = anc.diagonal(dim1=1, dim2=2)
    depth = anc.sum(-1) - 1
    t = torch.arange(T, device=q.device)
    see = (t < lens[:, None])[:, None, :] & used[:, :, None]
    tree = anc & used[:, :, None]
    if W > 0:
        see = see & ((lens[:, None] + depth)[:, :, None] - t < W)
        tree = tree & (depth[:, :, None] - depth[:, None, :] < W)
    see = torch.cat([see, tree], 2)  # [B, N, T + N]
    k = torch.cat([cache[:, :, 0], kv[:, :, 0]], 1).float().permute(0, 2, 3, 1)
    v = torch.cat([cache[:, :, 1], kv[:, :, 1]], 1).float().permute(0, 2, 1, 3)
    G = H // Hkv
    qg = q.float().view(B, N, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * N, D)
    sc = (torch.matmul(qg, k) / math.sqrt(D)).view(B, Hkv, G, N, T + N)
    sc = sc.masked_fill(~see[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * N, T + N), v).view(B, Hkv, G, N, D)
    o = torch.where(l > 0, o / l, 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, N, H, D).to(q.dtype)


def _plain_sample(s):
    l = s["logits"].double()
    M, V = l.shape
    one = torch.ones((M, 1), dtype=torch.float64, device=l.device)
    T = one if s["temperature"] is None else s["temperature"].double()[:, None]
    mx, best = l.max(1, keepdim=True)
    best = (l == mx).to(torch.uint8).argmax(1, keepdim=True)  # the lowest index of the largest
    w = torch.exp((l - mx) / torch.where(T > 0, T, 1.0))
    wi = w
    if s["top_k"] is not None or s["top_p"] is not None:
        order = torch.sort(l, dim=1, descending=True, stable=True)[1]
        ws = w.gather(1, order)
        rank = torch.arange(V, device=l.device)[None]
        keep = torch.ones((M, V), dtype=torch.bool, device=l.device)
        if s["top_k"] is not None:
            k = s["top_k"].long()[:, None]
            keep &= (rank < k) | (k <= 0)
        wk = ws * keep
        if s["top_p"] is not None:
            p = s["top_p"].double()[:, None]
            before = wk.cumsum(1) - wk
            keep &= (before < p * wk.sum(1, keepdim=True)) | (p >= 1) | (rank == 0)
        wi = w * torch.zeros_like(keep).scatter_(1, order, keep)
    if s["min_p"] is not None:
        wi = wi * (w >= s["min_p"].double()[:, None])
    cdf = wi.cumsum(1)
    total = cdf[:, -1:]
    tok = (cdf <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    last = V - 1 - (wi.flip(1) > 0).to(torch.uint8).argmax(1, keepdim=True)
    tok = torch.minimum(tok, last)
    lp = torch.log(wi.gather(1, tok) / total)
    tok = torch.where(T > 0, tok, best)
    lp = torch.where(T > 0, lp, 0.0)
    return tok[:, 0].to(torch.int32), lp[:, 0].float()


def _plain_accept(s):
    tok, par, smp, lens, kv, cache = (s[k] for k in ("tokens", "parents", "sampled", "lens", "kv", "cache"))
    B, N = tok.shape
    T_max = cache.shape[2]
    anc = _bits(s["mask"], N)
    up = par.clamp_min(0).long()
    hit = (smp.gather(1, up) == tok) & (par >= 0)
    twin = (par[:, :, None] == par[:, None, :]) & (tok[:, :, None] == tok[:, None, :])  # [b, j, i]
    first = ~(twin & torch.ones(N, N, dtype=torch.bool, device=tok.device).tril(-1)).any(2)
    ok = hit & first
    ok[:, 0] = True
    took = ~(anc & ~ok[:, None, :]).any(2) & anc[:, :, 0] & anc.diagonal(dim1=1, dim2=2)
    rank = took.cumsum(1) - 1
    took = took & (lens[:, None] + rank < T_max)
    count = took.sum(1)
    node = torch.arange(N, device=tok.device)
    path = torch.full((B, N + 1), -1, dtype=torch.int32, device=tok.device)
    path.scatter_(1, torch.where(took, rank, N), node.to(torch.int32).expand(B, N).contiguous())
    path = path[:, :N].contiguous()
    last = path.gather(1, (count - 1).clamp_min(0)[:, None]).clamp_min(0).long()
    nxt = torch.where(count[:, None] > 0, smp.gather(1, last), tok[:, :1])[:, 0]
    b, j = took.nonzero(as_tuple=True)
    cache[:, b, (lens[:, None] + rank)[b, j]] = kv[:, b, j]
    return path, count.to(torch.int32), nxt, lens + count.to(torch.int32), cache


def _plain_distill(s):
    c, z, ti, tl = s["case"], s["z"], s["teacher_idx"].long(), s["teacher_logits"]
    cap, tau = c["cap"], c["tau"]
    th = torch.tanh(z / cap) if cap > 0 else None
    x = (cap * th if cap > 0 else z) / tau
    x = x - x.amax(1, keepdim=True)
    e = torch.exp(x)
    tot = e.sum(1, keepdim=True)
    t = tl / tau
    t = t - t.amax(1, keepdim=True)
    te = torch.exp(t)
    tt = te.sum(1, keepdim=True)
    q = te / tt
    loss = tau * tau * (q * ((t - torch.log(tt)) - (x.gather(1, ti) - torch.log(tot)))).sum(1)
    w = s["row_weight"]
    if s["dz"] is None:
        return loss,
    d = e / tot
    d = d.scatter_add(1, ti, -q)
    d = d * (tau if w is None else tau * w[:, None])
    if cap > 0:
        d = d * (1 - th * th)
    return loss, d.to(s["dz"].dtype)


# ------------------------------------------------------------------ the framework's calls

def _own_run(s):
    import decoder_only_transformer_nc_b200 as nc
    kind = s["case"]["kind"]
    if kind == "attn":
        nc.tree_attention(s["q"], s["kv"], s["cache"], s["lens"], s["mask"], s["out"], s["case"]["window"])
        return s["out"]
    if kind == "sample":
        nc.sample(s["logits"], s["u"], s["tokens"], s["logprob"], temperature=s["temperature"], top_k=s["top_k"],
                  top_p=s["top_p"], min_p=s["min_p"])
        return s["tokens"], s["logprob"]
    if kind == "accept":
        nc.tree_accept(s["tokens"], s["parents"], s["mask"], s["sampled"], s["lens"], s["kv"], s["cache"], s["path"],
                       s["count"], s["next"], s["lens_out"])
        return s["path"], s["count"], s["next"], s["lens_out"], s["cache"]
    nc.distill_topk(s["z"], s["teacher_idx"], s["teacher_logits"], s["token_loss"], s["dz"], tau=s["case"]["tau"],
                    cap=s["case"]["cap"], row_weight=s["row_weight"])
    return (s["token_loss"],) if s["dz"] is None else (s["token_loss"], s["dz"])


def run(state):
    if own:
        return _own_run(state)
    return {"attn": _plain_attn, "sample": _plain_sample, "accept": _plain_accept,
            "distill": _plain_distill}[state["case"]["kind"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_attn(c, s):
    B, N, H, Hkv, D, W = c["B"], c["N"], c["H"], c["Hkv"], c["D"], c["window"]
    lens, words = s["lens"].tolist(), s["mask"].cpu().numpy().view(np.uint32)
    out = torch.zeros((B, N, H, D), dtype=torch.float64, device=DEV)
    for b in range(B):
        n = lens[b]
        sees = [[j for j in range(N) if words[b, i, j // 32] >> (j % 32) & 1] for i in range(N)]
        vis = np.zeros((N, n + N), bool)
        for i in range(N):
            if i not in sees[i]:
                continue
            p = n + len(sees[i]) - 1
            vis[i, (max(0, p - W + 1) if W > 0 else 0):n] = True
            for j in sees[i]:
                vis[i, n + j] = W <= 0 or len(sees[i]) - len(sees[j]) < W
        see = torch.from_numpy(vis).to(DEV)
        for g in range(Hkv):
            k = torch.cat([s["cache"][b, :n, 0, g], s["kv"][b, :, 0, g]]).double()
            v = torch.cat([s["cache"][b, :n, 1, g], s["kv"][b, :, 1, g]]).double()
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                a = s["q"][b, :, h].double() @ k.T * D ** -0.5
                a = torch.where(see, a, torch.full_like(a, -math.inf))
                top = torch.logsumexp(a, 1, keepdim=True)
                out[b, :, h] = torch.where(torch.isinf(top), torch.zeros_like(a), torch.exp(a - top)) @ v
    return out


def _exact_sample(c, s):
    M = c["M"]
    if M * c["V"] > 1 << 26:
        return None
    get = lambda k, d: [d] * M if s[k] is None else s[k].tolist()  # noqa: E731
    Ts, ks, ps, ms, us = get("temperature", 1.0), get("top_k", 0), get("top_p", 1.0), get("min_p", 0.0), s["u"].tolist()
    lp = np.zeros(M)
    rows = s["logits"].cpu().numpy().astype(np.float64)
    for m in range(M):
        if Ts[m] <= 0:
            continue
        x = rows[m] / Ts[m]
        by = np.lexsort((np.arange(len(x)), -rows[m]))
        if ks[m] > 0:
            by = by[:ks[m]]
        pr = np.exp(x[by] - x[by[0]])
        if ps[m] < 1:
            n = int(np.searchsorted(np.cumsum(pr), ps[m] * pr.sum(), side="left")) + 1
            by, pr = by[:n], pr[:n]
        at = np.sort(by[pr >= ms[m]])
        pr = np.exp(x[at] - x[at].max())
        cdf = np.cumsum(pr)
        i = min(int(np.searchsorted(cdf, us[m] * cdf[-1], side="right")), len(at) - 1)
        lp[m] = math.log(pr[i] / cdf[-1])
    return None, lp


def _exact_accept(c, s):
    par, tok, smp, lens = (s[k].cpu().numpy() for k in ("parents", "tokens", "sampled", "lens"))
    cache = s["cache"]
    for b in range(c["B"]):
        at, walk = 0, []
        while at is not None and lens[b] + len(walk) < c["T_max"]:
            cache[:, b, lens[b] + len(walk)] = s["kv"][:, b, at]
            walk.append(at)
            at = next((j for j in range(at + 1, c["N"]) if par[b, j] == at and tok[b, j] == smp[b, at]), None)
    return None, None, None, None, cache


def _exact_distill(c, s):
    M, cap, tau = c["M"], c["cap"], c["tau"]
    loss = torch.empty(M, dtype=torch.float64, device=DEV)
    dz = None if s["dz"] is None else torch.empty(s["dz"].shape, dtype=torch.float64, device=DEV)
    for a in range(0, M, 256):
        z, i = s["z"][a:a + 256].double(), s["teacher_idx"][a:a + 256].long()
        l = cap * torch.tanh(z / cap) if cap > 0 else z
        logp = torch.log_softmax(l / tau, 1)
        logq = torch.log_softmax(s["teacher_logits"][a:a + 256].double() / tau, 1)
        loss[a:a + 256] = tau ** 2 * (logq.exp() * (logq - logp.gather(1, i))).sum(1)
        if dz is not None:
            d = logp.exp()
            d.scatter_add_(1, i, -logq.exp())
            d *= tau if s["row_weight"] is None else tau * s["row_weight"][a:a + 256, None].double()
            dz[a:a + 256] = d * (1 - (l / cap) ** 2) if cap > 0 else d
    return (loss,) if dz is None else (loss, dz)


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "sample": _exact_sample, "accept": _exact_accept,
            "distill": _exact_distill}[case["kind"]](case, s)
