"""The drafted-tree operators, sampling and distillation against their 64-bit definitions."""
import math

import numpy as np
import pytest
import torch

from oracle import tree as o64

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _mask_i32(m):
    return _dev(m.view(np.int32))


def _trees(rng, B, N, how):
    p = np.full((B, N), -2, np.int32)
    for b in range(B):
        n = N if how != "ragged" else int(rng.integers(0, N + 1))
        for i in range(n):
            if how == "chain":
                p[b, i] = i - 1
            elif how == "forest":
                p[b, i] = -1 if i % 3 == 0 else int(rng.integers(0, i))
            else:
                p[b, i] = -1 if i == 0 else int(rng.integers(0, i))
    return p


# ------------------------------------------------------------------ masks

@pytest.mark.parametrize("N", [1, 5, 32, 33, 64, 100, 128])
def test_tree_mask(gpu, N):
    rng = np.random.default_rng(N)
    p = np.concatenate([_trees(rng, 2, N, h) for h in ("chain", "random", "ragged", "forest")])
    wild = rng.integers(-5, N + 5, (4, N)).astype(np.int32)  # parents that lead nowhere, or to themselves
    wild[0] = np.array([0x7fffffff, -0x80000000] * N)[:N]
    p = np.concatenate([p, wild])
    out = torch.full((len(p), N, (N + 31) // 32), -1, dtype=torch.int32, device=DEV)
    gpu.tree_mask(_dev(p), out)
    assert np.array_equal(out.cpu().numpy().view(np.uint32), o64.tree_mask(p))


# ------------------------------------------------------------------ attention

def _attn_case(seed, B, N, H, Hkv, D, T, lens, dt, how):
    rng = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DT[dt])  # noqa: E731
    q, kv, cache = t(B, N, H, D), t(B, N, 2, Hkv, D), t(B, T, 2, Hkv, D)
    mask = o64.tree_mask(_trees(rng, B, N, how))
    return q, kv, cache, np.array(lens, np.int32), mask


def _check_attn(got, q, kv, cache, lens, mask, window, dt, what=""):
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    q, kv, cache = f(q), f(kv), f(cache)
    lens = np.clip(lens, 0, cache.shape[1])
    want = o64.tree_attention(q, kv, cache, lens, mask, window)
    av = lambda x: np.concatenate([x[:, :, :1], np.abs(x[:, :, 1:])], 2)  # noqa: E731
    A = o64.tree_attention(q, av(kv), av(cache), lens, mask, window)  # sum of p |v|
    half = torch.finfo(DT[dt]).eps / 2
    # a weight (<= 1, their sum >= 1) is rounded to 16 bits once: half a step of it, or for
    # fp16's subnormal weights 2^-25; the output once; the scores are fp32 sums of D products
    # (2 D 2^-24 of about 8 = sum |q k| / sqrt(D) of unit normals), the rest is far below
    n = cache.shape[1] + kv.shape[1]
    sub = n * 2.0 ** -25 * 6 if dt == "fp16" else 0.0
    tol = half * (A + np.abs(want)) + 2 * q.shape[-1] * 2.0 ** -24 * 8 * A + sub
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"{what}: worst error / tolerance {np.nanmax(err / np.maximum(tol, 1e-30)):.2f}"


ATTN = [
    # B, N, H, Hkv, D, T, lens, window, dtype, tree
    (1, 1, 1, 1, 64, 1, [0], 0, "fp16", "chain"),          # one node, empty cache
    (1, 1, 2, 1, 128, 40, [40], 0, "bf16", "chain"),       # a plain decode step, full cache
    (2, 4, 10, 10, 128, 300, [300, 1], 0, "fp16", "chain"),
    (3, 7, 6, 2, 64, 200, [199, 0, 64], 0, "bf16", "random"),
    (2, 27, 12, 12, 64, 260, [259, 130], 100, "bf16", "ragged"),
    (2, 32, 4, 1, 128, 130, [63, 65], 0, "fp16", "random"),
    (2, 33, 8, 1, 64, 90, [90, 17], 7, "fp16", "forest"),  # a window shorter than the tree
    (1, 64, 4, 2, 128, 700, [650], 512, "bf16", "chain"),
    (1, 128, 3, 1, 128, 50, [50], 0, "fp16", "random"),    # three heads a group
    (4, 100, 8, 1, 64, 33, [0, 1, 32, 33], 1, "bf16", "ragged"),  # a window of one: a node sees itself
    (2, 17, 5, 5, 128, 1500, [1411, 1500], 0, "bf16", "ragged"),
    # more rows a kv head than the small kernel takes
    (7, 40, 2, 2, 128, 400, [0, 1, 127, 128, 129, 399, 400], 0, "fp16", "random"),
    (7, 33, 2, 1, 64, 400, [0, 1, 127, 128, 129, 399, 400], 0, "bf16", "ragged"),
    (3, 64, 8, 2, 128, 600, [600, 5, 257], 0, "bf16", "ragged"),    # two row tiles a unit
    (2, 100, 3, 1, 64, 500, [500, 333], 129, "fp16", "forest"),     # three row tiles of 42 nodes
    (1, 64, 4, 1, 128, 3000, [2999], 0, "fp16", "random"),          # one unit over every SM
    (5, 128, 4, 4, 64, 300, [300, 299, 0, 150, 1], 200, "fp16", "chain"),
    (1, 3, 128, 1, 64, 260, [260], 0, "bf16", "random"),            # 128 heads a group
    (1, 2, 200, 1, 64, 130, [130], 0, "bf16", "random"),            # more heads a group than a tile has rows
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"B{c[0]}N{c[1]}H{c[2]}kv{c[3]}D{c[4]}W{c[7]}{c[8]}{c[9]}")
def test_tree_attention(gpu, case):
    B, N, H, Hkv, D, T, lens, window, dt, how = case
    q, kv, cache, lens, mask = _attn_case(sum(case[:6]), B, N, H, Hkv, D, T, lens, dt, how)
    out = torch.full_like(q, 7.0).to(DEV)
    gpu.tree_attention(q.to(DEV), kv.to(DEV), cache.to(DEV), _dev(lens), _mask_i32(mask), out, window)
    _check_attn(out, q, kv, cache, lens, mask, window, dt)
    again = torch.full_like(out, 3.0)
    gpu.tree_attention(q.to(DEV), kv.to(DEV), cache.to(DEV), _dev(lens), _mask_i32(mask), again, window)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("H,W", [(4, 40), (16, 0), (16, 140), (8, 0)])
def test_tree_attention_reads_nothing_unseen(gpu, dt, H, W):
    """NaN behind a row's length, before the window, in unused nodes' q, K and V; lengths out
    of range are clamped; a strided q."""
    B, N, Hkv, D, T = 3, 21, 2, 64, 350
    q, kv, cache, lens, mask = _attn_case(5, B, N, H, Hkv, D, T, [350, 77, 0], dt, "ragged")
    mask[0] = o64.tree_mask(_trees(np.random.default_rng(1), 1, N, "random"))[0]
    mask[1, 9:] = 0
    clean = (kv.clone(), cache.clone(), q.clone())
    for b in range(B):
        cache[b, lens[b]:] = math.nan
        if W:
            cache[b, :max(0, lens[b] - W + 1)] = math.nan
        for i in range(N):
            if not (mask[b, i, 0] >> i) & 1:
                kv[b, i] = math.nan
                q[b, i] = math.nan
    packed = torch.full((B, N, (H + 2 * Hkv) * D), math.nan, dtype=DT[dt])
    packed[:, :, :H * D] = q.reshape(B, N, H * D)
    qs = packed.to(DEV)[:, :, :H * D].view(B, N, H, D)
    out = torch.empty((B, N, H, D), dtype=DT[dt], device=DEV)
    wild = lens.copy()
    wild[0], wild[2] = 1 << 30, -5
    gpu.tree_attention(qs, kv.to(DEV), cache.to(DEV), _dev(wild), _mask_i32(mask), out, W)
    _check_attn(out, clean[2], clean[0], clean[1], lens, mask, W, dt)


def test_tree_attention_many_rows_strided_q_and_own_workspace(gpu):
    """More rows of the cache than the tensor-core kernel plans for (trees of a size that it takes else);
    the q columns of a packed projection, and a workspace of the caller's, one too small refused."""
    B, N, H, Hkv, D, T = 1030, 40, 1, 1, 64, 24
    lens = [(7 * b) % 25 for b in range(B)]
    q, kv, cache, lens, mask = _attn_case(8, B, N, H, Hkv, D, T, lens, "fp16", "ragged")
    out = torch.full_like(q, 7.0).to(DEV)
    assert gpu.lib().nc_tree_attention_workspace_bytes(B, N, H, Hkv, D, T, 0) == 0
    gpu.tree_attention(q.to(DEV), kv.to(DEV), cache.to(DEV), _dev(lens), _mask_i32(mask), out)
    _check_attn(out, q, kv, cache, lens, mask, 0, "fp16")
    B, N, H, Hkv, D, T = 3, 50, 6, 2, 128, 700
    q, kv, cache, lens, mask = _attn_case(9, B, N, H, Hkv, D, T, [700, 1, 300], "bf16", "random")
    need = gpu.lib().nc_tree_attention_workspace_bytes(B, N, H, Hkv, D, T, 0)
    assert need > 0
    packed = torch.full((B, N, (H + 2 * Hkv) * D), math.nan, dtype=DT["bf16"])
    packed[:, :, :H * D] = q.reshape(B, N, H * D)
    qs = packed.to(DEV)[:, :, :H * D].view(B, N, H, D)
    args = (qs, kv.to(DEV), cache.to(DEV), _dev(lens), _mask_i32(mask))
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.empty((B, N, H, D), dtype=DT["bf16"], device=DEV)
    for w in (ws[:need - 1], ws[:0]):
        with pytest.raises(gpu.NcError) as e:
            gpu.tree_attention(*args, out, workspace=w)
        assert e.value.code == 5
    gpu.tree_attention(*args, out, workspace=ws[:need], status=st)
    _check_attn(out, q, kv, cache, lens, mask, 0, "bf16")
    assert (ws[need:] == 255).all() and int(st) == 0


@pytest.mark.parametrize("N", [5, 64])  # each of the kernels
def test_offsets_past_32_bits(gpu, N):
    """A cache of 2^31 elements a row: the last positions of three rows under a window, the accepted K/V
    there, and logits rows 2^31 elements apart."""
    B, H, Hkv, D, T, W = 3, 8, 8, 128, 1 << 20, 200
    lens = [T - 130, T - 200, 1000]
    q, kv, near, _, mask = _attn_case(2, B, N, H, Hkv, D, 300, [0] * B, "bf16", "random")
    cache = torch.empty((1, B, T, 2, Hkv, D), dtype=DT["bf16"], device=DEV)
    for b in range(B):
        cache[0, b, lens[b] - 300:lens[b]] = near[b].to(DEV)
    out = torch.empty((B, N, H, D), dtype=DT["bf16"], device=DEV)
    words = _mask_i32(mask)
    gpu.tree_attention(q.to(DEV), kv.to(DEV), cache[0], _dev(np.array(lens, np.int32)), words, out, W)
    _check_attn(out, q, kv, near, np.array([300] * B), mask, W, "bf16")
    par = np.full((B, N), -1, np.int32)
    par[:, 1:] = np.arange(N - 1)
    words = _mask_i32(o64.tree_mask(par))
    tok = torch.arange(B * N, dtype=torch.int32, device=DEV).view(B, N)
    path, (count, nxt, lo) = torch.empty_like(tok), torch.empty((3, B), dtype=torch.int32, device=DEV)
    gpu.tree_accept(tok, _dev(par), words, tok + 1, _dev(np.array(lens, np.int32)), kv.to(DEV)[None], cache, path, count,
                    nxt, lo)
    assert count.tolist() == [N] * B
    for b in range(B):
        assert torch.equal(cache[0, b, lens[b]:lens[b] + N], kv[b].to(DEV))
        assert torch.equal(cache[0, b, lens[b] - 300:lens[b]], near[b].to(DEV))
    del cache
    V, ld = 5000, 1 << 31
    x = torch.empty(ld + V, device=DEV).as_strided((2, V), (ld, 1))
    x.copy_(3 * torch.randn((2, V), device=DEV))
    u, a, b = torch.rand(2, device=DEV), *torch.empty((2, 2), dtype=torch.int32, device=DEV)
    gpu.sample(x, u, a)
    gpu.sample(x.contiguous(), u, b)
    assert torch.equal(a, b)


def test_tree_attention_calls_side_by_side(gpu):
    """The same and another problem on four streams at once, each call with its own workspace."""
    cases = [(4, 64, 4, 2, 128, 500, [500, 7, 256, 0]), (2, 33, 8, 2, 128, 900, [900, 640])]
    ins, want = [], []
    for i, (B, N, H, Hkv, D, T, lens) in enumerate(cases):
        q, kv, cache, lens, mask = _attn_case(30 + i, B, N, H, Hkv, D, T, lens, "bf16", "random")
        a = [q.to(DEV), kv.to(DEV), cache.to(DEV), _dev(lens), _mask_i32(mask)]
        out = torch.empty_like(a[0])
        gpu.tree_attention(*a, out)
        ins.append(a)
        want.append(out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [[torch.empty_like(ins[k % 2][0]) for k in range(4)] for _ in range(6)]
    for turn in outs:
        for k, s in enumerate(streams):
            gpu.tree_attention(*ins[k % 2], turn[k], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[k % 2]) for turn in outs for k, o in enumerate(turn))


# ------------------------------------------------------------------ acceptance

@pytest.mark.parametrize("B,N,L,Hkv,D,T", [(1, 1, 1, 1, 64, 3), (3, 8, 4, 2, 64, 20), (5, 33, 2, 1, 128, 40),
                                           (2, 128, 3, 3, 64, 131), (4, 64, 1, 1, 4, 70)])
@pytest.mark.parametrize("vocab", [2, 1000])
def test_tree_accept(gpu, B, N, L, Hkv, D, T, vocab):
    rng = np.random.default_rng(N + vocab)
    par = np.concatenate([_trees(rng, 1, N, h) for h in ("chain", "random", "ragged", "forest", "chain")])[:B]
    tok, smp = (rng.integers(0, vocab, (B, N)).astype(np.int32) for _ in range(2))
    if vocab == 1000:  # drafts that are mostly right
        for b in range(B):
            for i in range(1, N):
                if par[b, i] >= 0 and rng.random() < 0.9:
                    smp[b, par[b, i]] = tok[b, i]
    mask = o64.tree_mask(par)
    lens = rng.integers(0, T + 1, B).astype(np.int32)
    lens[0] = T - 1
    kv = torch.randn((L, B, N, 2, Hkv, D), dtype=torch.bfloat16, device=DEV)
    cache = torch.randn((L, B, T, 2, Hkv, D), dtype=torch.bfloat16, device=DEV)
    want = cache.clone()
    path, (count, nxt, lo) = torch.full((B, N), 9, dtype=torch.int32, device=DEV), torch.zeros((3, B), dtype=torch.int32, device=DEV)
    gpu.tree_accept(_dev(tok), _dev(par), _mask_i32(mask), _dev(smp), _dev(lens), kv, cache, path, count, nxt, lo)
    for b, (p, n) in enumerate(o64.tree_accept(tok, par, mask, smp, lens, T)):
        assert path[b].tolist() == p + [-1] * (N - len(p))
        assert (int(count[b]), int(nxt[b]), int(lo[b])) == (len(p), n, lens[b] + len(p))
        for k, j in enumerate(p):
            want[:, b, lens[b] + k] = kv[:, b, j]
    assert torch.equal(cache, want)  # what is behind the accepted rows is left as it was


# ------------------------------------------------------------------ sampling

def _sample(gpu, l, u, **kw):
    M = l.shape[0]
    tok = torch.full((M,), -7, dtype=torch.int32, device=DEV)
    lp = torch.full((M,), math.nan, device=DEV)
    dev = {k: None if v is None else _dev(np.asarray(v, np.int32 if k == "top_k" else np.float32)) for k, v in kw.items()}
    gpu.sample(l if isinstance(l, torch.Tensor) else _dev(l.astype(np.float32)), _dev(np.asarray(u, np.float32)), tok, lp, **dev)
    return tok.cpu().numpy(), lp.cpu().numpy()


def _check_sample(l, u, tok, lp, T=None, top_k=None, top_p=None, min_p=None):
    l = l.cpu().numpy() if isinstance(l, torch.Tensor) else l.astype(np.float32)
    g = lambda a, d, m: d if a is None else float(np.float32(a[m]))  # noqa: E731
    for m in range(len(l)):
        w = o64.sample_row(l[m], float(np.float32(u[m])), g(T, 1.0, m), int(g(top_k, 0, m)), g(top_p, 1.0, m), g(min_p, 0.0, m))
        # a running mass is off by less than V units of 2^-sh, sh >= 46 here
        assert tok[m] == w[0] or w[2] < 1e-9, (m, tok[m], w)
        if tok[m] == w[0]:
            assert lp[m] == w[1] or abs(lp[m] - w[1]) <= 2.0 ** -23 * abs(w[1]) + 1e-9, (m, lp[m], w)


@pytest.mark.parametrize("V", [1, 2, 31, 1000, 1025, 4099, 32768, 50257])
@pytest.mark.parametrize("how", ["plain", "k", "p", "m", "all", "kp"])
def test_sample(gpu, V, how):
    M = 6
    rng = np.random.default_rng(V * 7 + len(how))
    l = (1.5 * rng.standard_normal((M, V)) + rng.exponential(1.2, (M, V))).astype(np.float32)
    u = rng.random(M).astype(np.float32)
    u[0], u[1] = 0.0, np.nextafter(np.float32(1), np.float32(0))
    T = np.array([1.0, 0.7, 1.5, 0.0, 0.3, 40.0])
    kw = {}
    if how in ("k", "all", "kp"):
        kw["top_k"] = np.array([50, 1, 7, 5, 2000, V + 5])
    if how in ("p", "all", "kp"):
        kw["top_p"] = np.array([0.95, 0.5, 0.99, 0.9, 0.05, 0.999])
    if how in ("m", "all"):
        kw["min_p"] = np.array([0.02, 0.5, 0.001, 0.1, 0.0, 0.9])
    tok, lp = _sample(gpu, l, u, temperature=T, **kw)
    _check_sample(l, u, tok, lp, T, **kw)


def test_sample_ties_and_extremes(gpu):
    V = 3001
    rng = np.random.default_rng(3)
    l = np.zeros((12, V), np.float32)
    l[1] = np.where(np.arange(V) % 2, 0.0, -0.0)      # +0 and -0 tie
    l[2] = rng.integers(0, 4, V)                       # heavy ties
    l[3] = rng.integers(-3, 2, V)
    l[4, ::2] = -np.inf
    l[5] = -np.inf
    l[6] = np.nan
    l[7] = rng.standard_normal(V)
    l[7, 5], l[7, 6] = np.nan, -np.inf
    l[8] = rng.standard_normal(V)
    l[8, 17] = l[8, 40] = np.inf
    l[9] = rng.standard_normal(V) * 1e30
    l[10] = -3.4e38
    l[10, 2000:2010] = np.arange(10) * 0.1
    l[11] = rng.standard_normal(V) * 1e-30
    u = rng.random(12).astype(np.float32)
    for kw in [{}, dict(top_k=np.full(12, 100)), dict(top_p=np.full(12, 0.5)), dict(top_p=np.full(12, 0.0)),
               dict(top_k=np.full(12, 7), top_p=np.full(12, 0.7)), dict(min_p=np.full(12, 1.0)),
               dict(min_p=np.full(12, 7.0)), dict(top_k=np.full(12, -1), top_p=np.full(12, 2.0), min_p=np.full(12, -1.0)),
               dict(top_k=np.full(12, 2900), top_p=np.full(12, 0.9), min_p=np.full(12, 0.2))]:
        tok, lp = _sample(gpu, l, u, **kw)
        _check_sample(l, u, tok, lp, **kw)
        assert tok[5] == tok[6] == -1 and lp[5] == lp[6] == -np.inf
    for bad_u in (1.0, 2.0):
        tok, lp = _sample(gpu, l, np.full(12, bad_u, np.float32))
        _check_sample(l, np.full(12, 1.0), tok, lp)
    tok, _ = _sample(gpu, l, np.full(12, np.nan, np.float32))
    tok0, _ = _sample(gpu, l, np.zeros(12, np.float32))
    assert np.array_equal(tok, tok0)
    T = np.array([np.inf, 1e-38, 1e38, 1e-3, 1.0, 1, 1, 2, 1, 1, np.nan, -1.0])
    tok, lp = _sample(gpu, l, u, temperature=T)
    _check_sample(l, u, tok, lp, T)


@pytest.mark.parametrize("V,M", [(300000, 2), (1 << 20, 1), (140001, 3), (32749, 300)])
def test_sample_large_vocabularies_and_many_rows(gpu, V, M):
    rng = np.random.default_rng(V)
    l = (1.5 * rng.standard_normal((M, V)) + rng.exponential(1.2, (M, V))).astype(np.float32)
    u = rng.random(M).astype(np.float32)
    for kw in [{}, dict(top_k=np.full(M, 40)), dict(top_p=np.full(M, 0.9)), dict(top_k=np.full(M, 20000), top_p=np.full(M, 0.8)),
               dict(top_k=np.full(M, 3000), min_p=np.full(M, 0.05))]:
        tok, lp = _sample(gpu, l, u, **kw)
        _check_sample(l, u, tok, lp, **kw)


@pytest.mark.parametrize("scale", [1e-6, 0.01, 1.0, 30.0, 1e4])
def test_sample_logits_of_any_spread(gpu, scale):
    """Logits packed into few histogram bins, or spread far past them."""
    rng = np.random.default_rng(4)
    M, V = 4, 20011
    l = (scale * rng.standard_normal((M, V))).astype(np.float32)
    l[2] = np.round(l[2] / scale) * np.float32(scale)   # about ten values: thousands of ties
    l[3, ::3] = -3e38
    u = rng.random(M).astype(np.float32)
    for T in (1.0, scale):
        for kw in [{}, dict(top_k=np.array([1, 1500, 4000, 12000])), dict(top_p=np.array([0.1, 0.5, 0.9, 0.999])),
                   dict(top_k=np.full(M, 9000), top_p=np.full(M, 0.6)), dict(top_k=np.full(M, 50), top_p=np.full(M, 0.95), min_p=np.full(M, 0.1))]:
            tok, lp = _sample(gpu, l, u, temperature=np.full(M, T), **kw)
            _check_sample(l, u, tok, lp, np.full(M, T), **kw)


@pytest.mark.parametrize("M", [30, 180])  # one row an SM, and several
def test_sample_maxima_far_above_the_rest(gpu, M):
    """One or a few tokens anywhere in the row, from e^2 to e^5000 (and infinitely) above the others."""
    V = 32768
    rng = np.random.default_rng(M)
    l = rng.standard_normal((M, V)).astype(np.float32)
    for m in range(M):
        h = [2, 5, 8, 9, 12, 60, 80, 88, 90, 120, 176, 178, 200, 300, 1000, 5000, np.inf][m % 17]
        at = rng.integers(0, V, 1 + m % 3)
        l[m, at] += np.float32(h)
        if m % 5 == 0:  # and all the first of every part far below
            for s in range(0, V, 2048):
                l[m, s:s + 512] -= 500
    u = rng.random(M).astype(np.float32)
    tok, lp = _sample(gpu, l, u)
    _check_sample(l, u, tok, lp)


@pytest.mark.parametrize("M", [24, 200])  # one row an SM, and several
@pytest.mark.parametrize("how", ["plain", "p", "kp", "m"])
def test_sample_at_the_borders(gpu, M, how):
    """u (and top_p) as near to a border between two tokens as fp32 numbers come, some 1e-8 of the mass."""
    V = 32768
    rng = np.random.default_rng(M + len(how))
    l = (1.5 * rng.standard_normal((M, V)) + rng.exponential(1.2, (M, V))).astype(np.float32)
    kw = {"p": dict(top_p=np.zeros(M)), "kp": dict(top_p=np.zeros(M), top_k=np.full(M, 9000)), "m": dict(min_p=np.full(M, 1e-3)),
          "plain": {}}[how]
    u = np.empty(M, np.float32)
    for m in range(M):
        w = np.exp(l[m].astype(np.float64) - l[m].max())
        order = np.argsort(-l[m], kind="stable")
        if how == "kp":
            order = order[:9000]
        if "top_p" in kw:  # between n and n + 1 tokens
            cum = np.cumsum(w[order])
            n = int(rng.integers(20, 0.9 * len(order)))
            kw["top_p"][m] = np.float32(cum[n - 1] / cum[-1])
            order = order[:n + int(kw["top_p"][m] > cum[n - 1] / cum[-1])]
        if how == "m":
            order = order[w[order] >= np.float32(1e-3)]
        cum = np.cumsum(w[np.sort(order)])
        u[m] = cum[rng.integers(0, max(1, len(cum) - 1))] / cum[-1]
    tok, lp = _sample(gpu, l, u, **kw)
    _check_sample(l, u, tok, lp, **kw)


def test_sample_strided_rows_and_no_logprob(gpu):
    x = torch.randn((5, 4, 777), device=DEV)
    l = x[:, 2]
    u = torch.rand(5, device=DEV)
    a, b = (torch.empty(5, dtype=torch.int32, device=DEV) for _ in range(2))
    gpu.sample(l, u, a)
    gpu.sample(l.contiguous(), u, b)
    assert torch.equal(a, b)
    _check_sample(l, u.cpu().numpy(), a.cpu().numpy(), np.array([o64.sample_row(r, v)[1] for r, v in zip(l.cpu().numpy(), u.cpu().numpy())]))


# ------------------------------------------------------------------ distillation

def _check_distill(gpu, z, idx, t, tau, cap, weight, dzt):
    M, V = z.shape
    loss = torch.full((M,), math.nan, device=DEV)
    dz = None if dzt is None else torch.full((M, V), math.nan, dtype=dzt, device=DEV)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    gpu.distill_topk(_dev(z), _dev(idx), _dev(t), loss, dz, tau=tau, cap=cap, status=st,
                     row_weight=None if weight is None else _dev(weight))
    for m in range(M):
        w = 1.0 if weight is None else float(weight[m])
        wl, wd = o64.distill_row(z[m], idx[m], t[m], tau, cap, w)
        R = cap if cap > 0 else np.abs(z[m][np.isfinite(z[m])]).max()
        # a logit l / tau and a log-sum-exp are each within a few steps of their size, at
        # most R / tau + log V; so a probability is off by this share of it
        rel = 2.0 ** -24 * (16 * max(R, np.abs(t[m][idx[m] >= 0]).max(initial=0.0)) / tau + 32)
        assert abs(float(loss[m]) - wl) <= tau * tau * 2 * rel + 2.0 ** -23 * abs(wl), (m, float(loss[m]), wl)
        if dz is not None:
            got = dz[m].double().cpu().numpy()
            l = cap * np.tanh(z[m].astype(np.float64) / cap) if cap > 0 else z[m].astype(np.float64)
            p = np.exp(l / tau - (l / tau).max())
            p /= p.sum()
            slope = 1 - (l / cap) ** 2 if cap > 0 else np.ones(V)
            pq = np.abs(wd) + 2 * abs(w) * tau * p * slope  # at least w tau (p + q) slope
            half = torch.finfo(dzt).eps / 2
            tiny = torch.finfo(dzt).smallest_normal * torch.finfo(dzt).eps
            # 1 - t^2 loses t's half step where t is near 1
            tol = half * np.abs(wd) + rel * pq + abs(w) * tau * (p + np.abs(wd)) * 2.0 ** -22 + tiny
            if cap > 0:
                tol += 2.0 ** -21 * (np.abs(wd) / np.maximum(slope, 1e-12))
            assert (np.abs(got - wd) <= tol).all(), (m, np.abs(got - wd).max(), (np.abs(got - wd) / tol).max())
    return loss, dz, st


@pytest.mark.parametrize("M,V,K", [(1, 1, 1), (3, 7, 3), (5, 512, 8), (4, 1001, 1), (3, 4096, 64), (2, 32768, 128),
                                   (2, 50257, 33), (2, 1000, 1000)])
@pytest.mark.parametrize("dz", ["fp32", "bf16", "fp16", "none"])
@pytest.mark.parametrize("cap,tau", [(15.0, 1.0), (0.0, 2.0), (15.0, 0.5)])
def test_distill(gpu, M, V, K, dz, cap, tau):
    rng = np.random.default_rng(V + K)
    z = (3 * rng.standard_normal((M, V))).astype(np.float32)
    idx = np.stack([rng.permutation(V)[:K] for _ in range(M)]).astype(np.int32)
    t = (4 * rng.standard_normal((M, K))).astype(np.float32)
    w = rng.random(M).astype(np.float32) if K % 2 else None
    dzt = {"fp32": torch.float32, "none": None, **DT}[dz]
    _, _, st = _check_distill(gpu, z, idx, t, tau, cap, w, dzt)
    assert int(st[0]) == 0


@pytest.mark.parametrize("V", [65536, 65537, 70001, 140000])  # the last that fits registers, and beyond
@pytest.mark.parametrize("dz,cap", [("fp32", 15.0), ("bf16", 0.0), ("fp16", 15.0), ("none", 15.0)])
def test_distill_long_rows(gpu, V, dz, cap):
    rng = np.random.default_rng(V)
    M, K = 3, 40
    z = (3 * rng.standard_normal((M, V))).astype(np.float32)
    idx = rng.integers(0, V, (M, K)).astype(np.int32)
    idx[0, 1], idx[0, 2], idx[1, 5:] = idx[0, 0], -1, -1
    idx[2] = -1
    idx[0, 3], idx[0, 4] = 0, V - 1
    t = (2 * rng.standard_normal((M, K))).astype(np.float32)
    _check_distill(gpu, z, idx, t, 1.0, cap, rng.random(M).astype(np.float32), {"fp32": torch.float32, "none": None, **DT}[dz])


@pytest.mark.parametrize("cap,tau", [(2.0 ** -16, 2.0 ** -12), (0.3, 1.0), (300.0, 30.0), (65536.0, 65536.0)])
def test_distill_caps_of_any_size(gpu, cap, tau):
    rng = np.random.default_rng(4)
    M, V, K = 3, 5000, 20
    z = (cap * rng.standard_normal((M, V)) * np.array([[0.1], [1.0], [4.0]])).astype(np.float32)
    idx = np.stack([rng.permutation(V)[:K] for _ in range(M)]).astype(np.int32)
    t = (tau * rng.standard_normal((M, K))).astype(np.float32)
    _check_distill(gpu, z, idx, t, tau, cap, None, torch.float32)


@pytest.mark.parametrize("dz", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,zo,do", [(33, 1, 0), (4099, 3, 1), (8192, 1, 1), (8192, 2, 3), (32768, 0, 1), (70001, 1, 2)])
def test_distill_at_any_alignment(gpu, V, zo, do, dz):
    """z and dz that start anywhere: equal to the aligned call to the order of the sums, and nothing
    beside dz is written."""
    dzt = {"fp32": torch.float32, **DT}[dz]
    M, K = 5, 16
    z = 3 * torch.randn((M, V), device=DEV)
    idx = torch.randint(0, V, (M, K), dtype=torch.int32, device=DEV)
    t = torch.randn((M, K), device=DEV)
    zb = torch.full((M * V + 8,), math.nan, device=DEV)
    zb[zo:zo + M * V] = z.flatten()
    db = torch.full((M * V + 8,), 7.0, dtype=dzt, device=DEV)
    la, lb, da = torch.empty(M, device=DEV), torch.empty(M, device=DEV), torch.empty((M, V), dtype=dzt, device=DEV)
    gpu.distill_topk(z, idx, t, la, da, tau=0.7)
    gpu.distill_topk(zb[zo:zo + M * V].view(M, V), idx, t, lb, db[do:do + M * V].view(M, V), tau=0.7)
    # sums of p in another order: V / 4096 + 20 additions of at most half a step each a side
    rel = 2.0 ** -24 * 2 * (V / 4096 + 20) + 2.0 ** -24 * 16 * 15 / 0.7
    assert (la - lb).abs().max().item() <= 0.49 * 2 * rel + 2.0 ** -22 * la.abs().max().item()
    got, want = db[do:do + M * V].view(M, V).double(), da.double()
    tiny = torch.finfo(dzt).smallest_normal * torch.finfo(dzt).eps
    # 0.7 p (1 - t^2) of an entry is at most 0.7, and p - q of a teacher's entry cancels
    assert ((got - want).abs() <= torch.finfo(dzt).eps * want.abs() + rel * (want.abs() + 0.7) * 2 + tiny).all()
    assert (db[:do] == 7).all() and (db[do + M * V:] == 7).all()


def test_distill_many_rows(gpu):
    """More rows than one launch takes; the rows around the border against the definition."""
    M, V, K = 65535 + 9, 70, 4
    rng = np.random.default_rng(6)
    z = (3 * rng.standard_normal((M, V))).astype(np.float32)
    idx = rng.integers(-1, V, (M, K)).astype(np.int32)
    t = rng.standard_normal((M, K)).astype(np.float32)
    w = rng.random(M).astype(np.float32)
    loss, dz = torch.full((M,), math.nan, device=DEV), torch.full((M, V), math.nan, device=DEV)
    gpu.distill_topk(_dev(z), _dev(idx), _dev(t), loss, dz, tau=1.0, cap=15.0, row_weight=_dev(w))
    assert not loss.isnan().any() and not dz.isnan().any()
    s = slice(65535 - 6, None)
    a, b, _ = _check_distill(gpu, z[s], idx[s], t[s], 1.0, 15.0, w[s], torch.float32)
    assert (a - loss[s]).abs().max().item() <= 1e-5 and (b - dz[s]).abs().max().item() <= 1e-5


def test_distill_repeated_missing_and_bad_entries(gpu):
    rng = np.random.default_rng(9)
    M, V, K = 7, 300, 6
    z = (3 * rng.standard_normal((M, V))).astype(np.float32)
    z[5] = 40.0 * np.sign(z[5])
    idx = rng.integers(0, V, (M, K)).astype(np.int32)
    t = rng.standard_normal((M, K)).astype(np.float32)
    idx[0] = 4                     # one index six times
    idx[1, 2:] = -1                # a short row
    idx[2] = -1                    # an empty row
    t[3, 1:4] = -np.inf
    t[4] = -np.inf
    idx[6, 0] = V - 1
    for dz in (torch.float32, torch.bfloat16):
        loss, d, st = _check_distill(gpu, z, idx, t, 1.0, 15.0, None, dz)
        assert int(st[0]) == 0
        assert float(loss[2]) == float(loss[4]) == 0.0 and not d[2].any() and not d[4].any()
    idx[3, 0], idx[6, 1] = V, -2
    _, _, st = _check_distill(gpu, z, idx, t, 1.0, 15.0, None, torch.float32)
    assert int(st[0]) == 2  # NC_DEV_TARGET_RANGE
    z[0, :] = -np.inf              # tokens that are masked out of the student, no cap
    z[0, 4], z[0, 9] = 1.0, 2.0
    _check_distill(gpu, z, idx, t, 2.0, 0.0, None, torch.float32)


def test_distill_gradient_against_differences(gpu):
    """dz against central differences of the kernel's own loss.  With h = 2^-3 the difference's
    third-order term is h^2 / 6 |d3 loss| <= 2.6e-3 |w| (the loss's third derivative in one logit is at
    most p (1 + cap terms) < 1), and each loss is within 1e-5."""
    rng = np.random.default_rng(2)
    V, K, h = 64, 5, 0.125
    z0 = rng.standard_normal(V).astype(np.float32)
    z = np.stack([z0] + [z0 + s * h * np.eye(V, dtype=np.float32)[i] for i in range(V) for s in (1, -1)]).astype(np.float32)
    M = len(z)
    idx = np.tile(rng.permutation(V)[:K].astype(np.int32), (M, 1))
    t = np.tile(rng.standard_normal(K).astype(np.float32), (M, 1))
    loss, dz = torch.empty(M, device=DEV), torch.empty((M, V), device=DEV)
    gpu.distill_topk(_dev(z), _dev(idx), _dev(t), loss, dz, tau=1.0, cap=15.0)
    num = (loss[1::2] - loss[2::2]) / (2 * h)
    assert (num - dz[0]).abs().max().item() < 2.6e-3 + 1e-5 / h


# ------------------------------------------------------------------ streams, graphs, devices

def test_operators_on_another_stream_and_in_one_graph(gpu):
    """Attention, sampling and acceptance captured together, replayed on changed inputs,
    equal to the calls made one by one."""
    rng = np.random.default_rng(11)
    B, N, H, D, T, V, L = 2, 9, 2, 64, 96, 500, 2
    par = _trees(rng, B, N, "random")
    q, kv, cache, lens, mask = _attn_case(3, B, N, H, H, D, T, [60, 0], "bf16", "random")
    q, kv1, cache1 = q.to(DEV), kv.to(DEV), cache.to(DEV)
    lens, parents = _dev(lens), _dev(par)
    words = torch.zeros((B, N, 1), dtype=torch.int32, device=DEV)
    logits, u = torch.randn((B * N, V), device=DEV), torch.rand(B * N, device=DEV)
    tok = torch.randint(0, V, (B, N), dtype=torch.int32, device=DEV)
    kvL, cacheL = torch.randn((L, B, N, 2, H, D), device=DEV).bfloat16(), torch.zeros((L, B, T, 2, H, D), device=DEV).bfloat16()
    out, smp = torch.empty_like(q), torch.empty(B * N, dtype=torch.int32, device=DEV)
    path, (count, nxt, lo) = torch.empty((B, N), dtype=torch.int32, device=DEV), torch.empty((3, B), dtype=torch.int32, device=DEV)

    def step():
        gpu.tree_mask(parents, words)
        gpu.tree_attention(q, kv1, cache1, lens, words, out, 0)
        gpu.sample(logits, u, smp)
        gpu.tree_accept(tok, parents, words, smp.view(B, N), lens, kvL, cacheL, path, count, nxt, lo)

    res = lambda: [t.clone() for t in (words, out, smp, path, count, nxt, lo, cacheL)]  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    first = res()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    cacheL.zero_()
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, res()))
    u.copy_(torch.rand(B * N, device=DEV))
    q.mul_(0.5)
    cacheL.zero_()
    g.replay()
    got = res()
    cacheL.zero_()
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, res()))
    a = torch.empty_like(smp)
    gpu.sample(logits, u, a, stream=s)  # an explicit stream
    s.synchronize()
    assert torch.equal(a, got[2])
