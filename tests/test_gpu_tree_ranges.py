"""Tree attention and sampling where the ranges of their number formats end: far weights in fp16, weights
under the unit of sampling's integers."""
import math

import numpy as np
import pytest
import torch

from oracle import tree as o64

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ attention: weights far below the largest

@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("first", [True, False])  # the large key before the others, or behind them
@pytest.mark.parametrize("N,H,T", [(4, 2, 300), (20, 2, 300), (40, 2, 300), (40, 4, 700), (4, 1, 9000)])
def test_far_weights_count(gpu, N, H, T, first, D, dt):
    """One key 18 (in the exponent) above all the others, with a V of zeros: the output is the others' sum, each
    of a weight of e^-18 = 2^-25.97, below fp16's smallest number if it were held as it is.  They are held times 2^7
    at least (2^-18.97, to a step of 2^-24): half a step is 2^-6.03 of it; the output's own rounding and the
    fp32 scores (of 18, 2^-23 of it each) are below 2^-10.  bf16: 2^-8 a rounding, twice."""
    B = 2
    rng = np.random.default_rng(N + T)
    t = lambda a: torch.from_numpy(a.astype(np.float32)).to(DT[dt])  # noqa: E731
    q = np.zeros((B, N, H, D))
    q[..., 0] = 2 * math.sqrt(D) if D == 64 else 16
    a = 9.0 if D == 64 else 18 * math.sqrt(D) / 16  # q k / sqrt(D) = 18
    kv, cache = np.zeros((B, N, 2, 1, D)), np.zeros((B, T, 2, 1, D))
    kv[:, :, 1] = rng.uniform(1000, 2000, (B, N, 1, D))
    cache[:, :, 1] = rng.uniform(1000, 2000, (B, T, 1, D))
    at = 0 if first else T - 1
    cache[:, at, 0, 0, 0] = a
    cache[:, at, 1] = 0
    q, kv, cache = t(q), t(kv), t(cache)
    par = np.tile(np.arange(N, dtype=np.int32) - 1, (B, 1))
    mask = o64.tree_mask(par)
    out = torch.full_like(q, 7.0).to(DEV)
    lens = np.full(B, T, np.int32)
    gpu.tree_attention(q.to(DEV), kv.to(DEV), cache.to(DEV), torch.from_numpy(lens).to(DEV),
                       torch.from_numpy(mask.view(np.int32)).to(DEV), out, 0)
    f = lambda x: x.double().numpy()  # noqa: E731
    want = o64.tree_attention(f(q), f(kv), f(cache), lens, mask, 0)
    assert want.min() > 1e-3  # normal numbers in fp16 too
    rel = 2.0 ** -6.03 + 2.0 ** -10 if dt == "fp16" else 2.0 ** -7 + 2.0 ** -10
    err = np.abs(out.double().cpu().numpy() - want) / want
    assert err.max() <= rel, f"relative error {err.max():.3g}"


@pytest.mark.parametrize("N,H,T", [(4, 2, 300), (40, 2, 300), (40, 4, 700)])
def test_values_near_the_end_of_bf16(gpu, N, H, T):
    """V of 1e38 at a key whose weight is nearly all of its row's: what fp32 has room for, without a factor.  The other
    keys, 30 in the exponent below, have V of 1.  Errors: the weight (1) is exact, the output is rounded once (2^-9),
    the division and the sum add 2^-22."""
    B, D = 2, 64
    q = torch.zeros((B, N, H, D))
    q[..., 0] = 16
    kv, cache = torch.zeros((B, N, 2, 1, D)), torch.zeros((B, T, 2, 1, D))
    kv[:, :, 1] = cache[:, :, 1] = 1.0
    cache[:, T // 2, 0, 0, 0] = 15.0
    cache[:, T // 2, 1] = 1e38
    q, kv, cache = (x.bfloat16().to(DEV) for x in (q, kv, cache))
    mask = o64.tree_mask(np.tile(np.arange(N, dtype=np.int32) - 1, (B, 1)))
    out = torch.empty_like(q)
    gpu.tree_attention(q, kv, cache, torch.full((B,), T, dtype=torch.int32, device=DEV),
                       torch.from_numpy(mask.view(np.int32)).to(DEV), out, 0)
    want = cache[0, T // 2, 1, 0, 0].double().item()
    assert ((out.double() - want).abs() <= want * 2.0 ** -8).all()


# ------------------------------------------------------------------ sampling: weights under the unit

def _sample(gpu, l, u, **kw):
    M = len(l)
    tok, lp = torch.full((M,), -7, dtype=torch.int32, device=DEV), torch.full((M,), math.nan, device=DEV)
    dev = lambda a, t: torch.from_numpy(np.full(M, a, t)).to(DEV)  # noqa: E731
    gpu.sample(l, torch.from_numpy(u).to(DEV), tok, lp,
               **{k: dev(v, np.int32 if k == "top_k" else np.float32) for k, v in kw.items()})
    return tok.cpu().numpy(), lp.cpu().numpy()


def _check_units(gpu, l, u, **kw):
    """l [M, V] and u [M] of rows that differ, or one row [V] and its u, M times over (kw: M)."""
    M = kw.pop("M", len(l))
    rows = l if l.ndim == 2 else l[None]
    tok, lp = _sample(gpu, torch.from_numpy(rows).to(DEV).expand(M, -1).contiguous(),
                      np.broadcast_to(np.asarray(u, np.float32), (M,)).copy(), **kw)
    names = {"temperature": "T"}
    V = rows.shape[1]
    for m in range(len(rows)):
        want = o64.sample_units(rows[m], float(np.float32(np.atleast_1d(u)[m])),
                                **{names.get(k, k): v if k == "top_k" else float(np.float32(v)) for k, v in kw.items()})
        # logprob: fp32 of a logarithm; the mass in it may come from fp32 weights (4.5e-7) and hold
        # what the units drop (V half units)
        tol = 2.0 ** -23 * abs(want[1]) + 4.5e-7 + V * 2.0 ** -(63 - (V - 1).bit_length())
        same = slice(m, m + 1) if l.ndim == 2 else slice(None)
        assert (tok[same] == want[0]).all(), (m, tok[same], want, kw)
        assert (np.abs(lp[same] - want[1]) <= tol).all(), (m, lp[same], want, kw)


@pytest.mark.parametrize("M", [3, 200])  # one row an SM, and several
@pytest.mark.parametrize("V", [700, 32768])
@pytest.mark.parametrize("T,tail", [(1.0, -40.0), (5.0, -200.0), (1.0, -60.0)])
def test_top_p_ties_over_a_tail_of_nothing(gpu, M, V, T, tail):
    """2 n equal tokens, the others' weights under half a unit: they count as 0, so exactly n tokens hold half of
    the mass, whichever way the row takes."""
    rng = np.random.default_rng(V + M)
    for n in (1, 2, 40):
        l = np.full((M, V), tail, np.float32)
        for m in range(M):
            l[m, rng.permutation(V)[:2 * n]] = 0.0
        u = rng.random(M).astype(np.float32)
        _check_units(gpu, l, u, temperature=T, top_p=0.5)
        _check_units(gpu, l, u, temperature=T, top_p=0.5, top_k=V - 1)
        _check_units(gpu, l, u, temperature=T, top_p=0.5, min_p=0.25)


@pytest.mark.parametrize("M,V", [(1, 1 << 17), (1, 1 << 20), (1, 1 << 22), (150, 1 << 17), (150, 1 << 20)])
def test_large_vocabularies_count_in_units(gpu, V, M):
    """A tail of tokens just under half a unit (2^-sh, sh = 62 less the bits of V).  They count as 0 and are not
    sampled, though together they are V / 2 units: 2^-24 of the mass at V = 2^20, 2^-20 at 2^22."""
    sh = 62 - (V - 1).bit_length()
    l = np.full(V, math.log(0.49) - sh * math.log(2.0), np.float32)
    l[0] = 0.0
    u = np.nextafter(np.float32(1), np.float32(0))
    _check_units(gpu, l, u, M=M)
    l[V // 3] = 0.0
    for top_p in (0.5, 0.9):
        _check_units(gpu, l, u, M=M, top_p=top_p)
        _check_units(gpu, l, u, M=M, top_p=top_p, temperature=1.0, top_k=V // 2)


@pytest.mark.parametrize("M", [2, 160])
@pytest.mark.parametrize("units,kept", [(127.6, True), (127.4, False)])
@pytest.mark.parametrize("kw", [{}, dict(top_p=0.9999999), dict(top_k=30000)], ids=["m", "mp", "mk"])
def test_min_p_of_a_few_units(gpu, M, units, kept, kw):
    """min_p = 2^-40 is 128 units at V = 32768; weights of 127.6 are 128 of them and kept, of 127.4 are not.  With u = 2^-26
    the kept ones, 2^-25 of the mass before the largest token, hold the target."""
    V, sh = 32768, 47
    l = np.full(V, math.log(units) - sh * math.log(2.0), np.float32)
    l[-1] = 0.0
    _check_units(gpu, l, 2.0 ** -26, M=M, min_p=2.0 ** -40, **kw)
    want = o64.sample_units(l, 2.0 ** -26, min_p=2.0 ** -40)[0]
    assert (want < V - 1) == kept  # the case is what it says
