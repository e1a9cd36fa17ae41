"""Tree attention and sampling where the ranges of their number formats end."""
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
