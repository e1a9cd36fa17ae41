"""Outputs that may share an input's memory: attention over its queries, sampling over a per-row array."""
import numpy as np
import pytest
import torch

from oracle import tree as o64

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("B,N,H,Hkv,D,T", [(2, 5, 4, 2, 64, 300), (3, 40, 8, 2, 128, 700), (1, 128, 4, 1, 64, 2000)])
def test_attention_over_its_queries(gpu, B, N, H, Hkv, D, T):
    g = torch.Generator(device=DEV).manual_seed(N)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).half()  # noqa: E731
    q, kv, cache = r(B, N, H, D), r(B, N, 2, Hkv, D), r(B, T, 2, Hkv, D)
    rng = np.random.default_rng(N)
    par = np.array([[-1] + [int(rng.integers(0, i)) for i in range(1, N)]] * B, np.int32)
    mask = torch.from_numpy(o64.tree_mask(par).view(np.int32)).to(DEV)
    lens = torch.tensor([T - 7 * b for b in range(B)], dtype=torch.int32, device=DEV)
    want = torch.empty_like(q)
    gpu.tree_attention(q, kv, cache, lens, mask, want)
    for _ in range(20):
        x = q.clone()
        gpu.tree_attention(x, kv, cache, lens, mask, x)
        assert torch.equal(x, want)


@pytest.mark.parametrize("M", [5, 300])
def test_sampling_over_its_own_numbers(gpu, M):
    g = torch.Generator(device=DEV).manual_seed(M)
    l, u = 3 * torch.randn((M, 5000), generator=g, device=DEV), torch.rand(M, generator=g, device=DEV)
    k = torch.randint(1, 2000, (M,), generator=g, device=DEV, dtype=torch.int32)
    p = torch.rand(M, generator=g, device=DEV)
    tok, lp = torch.empty_like(k), torch.empty_like(u)
    gpu.sample(l, u, tok, lp, top_k=k, top_p=p)
    for over in ("u", "p"):
        a = {"u": u.clone(), "p": p.clone()}
        t = k.clone()
        gpu.sample(l, a["u"], t, a[over], top_k=t, top_p=a["p"])
        assert torch.equal(t, tok) and torch.equal(a[over], lp)
