"""Refusals of the drafted-tree, sampling and distillation entry points, and pins of
their 64-bit definitions (CPU only)."""
import math

import numpy as np
import pytest
import torch

from oracle import tree as o64


def _i(*s):
    return torch.zeros(s, dtype=torch.int32)


def _f(*s):
    return torch.zeros(s)


def _h(*s):
    return torch.zeros(s, dtype=torch.float16)


def _code(nclib, fn, *a, **k):
    with pytest.raises(nclib.NcError) as e:
        fn(*a, **k)
    return e.value.code


A = 1 << 40  # an aligned address that no check dereferences


def _c_attn(nc, q=A, qs=512, kv=A, cache=A, lens=A, mask=A, out=A, B=1, N=4, H=4, Hkv=2, D=128, T=64, win=0, dt=1, ws=None,
            wn=0):
    return nc.lib().nc_tree_attention(q, qs, kv, cache, lens, mask, out, B, N, H, Hkv, D, T, win, dt, ws, wn, None, None)


def test_tree_attention_refusals(nclib):
    for bad, want in [(dict(q=None), 1), (dict(mask=None), 1), (dict(Hkv=3), 1), (dict(dt=2), 1), (dict(B=-1), 1),
                      (dict(D=96, qs=384), 3), (dict(N=0), 3), (dict(N=129), 3), (dict(T=0), 3), (dict(B=65536), 3),
                      (dict(qs=504), 1), (dict(qs=513), 1), (dict(q=A + 2), 4), (dict(kv=A + 8), 4),
                      (dict(cache=A + 4), 4), (dict(out=A + 2), 4), (dict(ws=A + 8), 4),
                      (dict(N=64, ws=None), 5), (dict(N=64, ws=A, wn=1000), 5)]:
        assert _c_attn(nclib, **bad) == want, bad
    good = dict(q=_h(2, 3, 4, 64), kv=_h(2, 3, 2, 2, 64), cache=_h(2, 9, 2, 2, 64), lens=_i(2), mask=_i(2, 3, 1),
                out=_h(2, 3, 4, 64))
    assert _code(nclib, nclib.tree_attention, **good) == 8  # nothing but the device is wrong
    for name, t, want in [("kv", _h(2, 4, 2, 2, 64), 3), ("cache", _h(1, 9, 2, 2, 64), 3), ("lens", _i(3), 3),
                          ("mask", _i(2, 3, 2), 3), ("out", _h(2, 3, 4, 128)[..., ::2], 1),
                          ("q", _h(2, 4, 3, 64).transpose(1, 2), 1)]:
        assert _code(nclib, nclib.tree_attention, **{**good, name: t}) == want, name
    for name, t in [("kv", good["kv"].bfloat16()), ("lens", _f(2)), ("q", _f(2, 3, 4, 64))]:
        with pytest.raises(TypeError):
            nclib.tree_attention(**{**good, name: t})


def test_tree_accept_and_mask_refusals(nclib):
    L = nclib.lib()

    def acc(tokens=A, lens=A + 64, kv=A, cache=A, lens_out=A, B=2, N=4, L_=3, Hkv=2, D=64, T=32):
        return L.nc_tree_accept(tokens, A, A, A, lens, kv, cache, A, A, A, lens_out, B, N, L_, Hkv, D, T, None)

    for bad, want in [(dict(tokens=None), 1), (dict(lens_out=A + 64), 1), (dict(B=-1), 1), (dict(N=0), 3),
                      (dict(N=129), 3), (dict(L_=0), 3), (dict(T=0), 3), (dict(kv=A + 2), 4), (dict(cache=A + 8), 4),
                      (dict(Hkv=1, D=2), 3)]:
        assert acc(**bad) == want, bad
    assert L.nc_tree_mask(None, A, 1, 4, None) == 1
    assert L.nc_tree_mask(A, A, 1, 129, None) == 3
    assert _code(nclib, nclib.tree_mask, _i(2, 33), _i(2, 33, 1)) == 3
    b = dict(tokens=_i(2, 3), parents=_i(2, 3), mask=_i(2, 3, 1), sampled=_i(2, 3), lens=_i(2),
             kv=_h(2, 2, 3, 2, 1, 64), cache=_h(2, 2, 9, 2, 1, 64), path=_i(2, 3), count=_i(2), next=_i(2),
             lens_out=_i(2))
    assert _code(nclib, nclib.tree_accept, **b) == 8
    for name, t, want in [("cache", _h(1, 2, 9, 2, 1, 64), 3), ("path", _i(2, 4), 3), ("sampled", _i(3, 2).T, 1)]:
        assert _code(nclib, nclib.tree_accept, **{**b, name: t}) == want, name


def test_sample_refusals(nclib):
    L = nclib.lib()

    def smp(logits=A, ld=100, u=A, tokens=A, M=2, V=100):
        return L.nc_sample(logits, ld, u, None, None, None, None, tokens, None, M, V, None)

    for bad, want in [(dict(logits=None), 1), (dict(u=None), 1), (dict(tokens=None), 1), (dict(M=-1), 1),
                      (dict(V=0), 3), (dict(V=(1 << 24) + 1, ld=1 << 25), 3), (dict(ld=99), 1)]:
        assert smp(**bad) == want, bad
    b = dict(logits=_f(2, 10), u=_f(2), tokens=_i(2))
    assert _code(nclib, nclib.sample, **b) == 8
    for name, t, want in [("u", _f(3), 3), ("temperature", _f(1), 3), ("logits", _f(2, 20)[:, ::2], 1),
                          ("logits", _f(2, 2, 5), 3), ("logits", _f(1, 10).expand(2, 10), 1), ("u", None, 1)]:
        assert _code(nclib, nclib.sample, **{**b, name: t}) == want, name
    for name, t in [("top_k", _f(2)), ("logits", _h(2, 10)), ("tokens", _i(2).long())]:
        with pytest.raises(TypeError):
            nclib.sample(**{**b, name: t})


def test_distill_refusals(nclib):
    L = nclib.lib()

    def dis(z=A, idx=A, loss=A, dz=A + 64, dt=0, M=2, V=10, K=2, tau=1.0, cap=15.0):
        return L.nc_distill_topk(z, idx, A, None, loss, dz, dt, M, V, K, tau, cap, None, None)

    for bad, want in [(dict(z=None), 1), (dict(loss=None), 1), (dict(dz=None), 1), (dict(dt=3), 1), (dict(dt=4), 1),
                      (dict(dz=A), 1), (dict(tau=0.0), 1), (dict(tau=math.inf), 1), (dict(tau=math.nan), 1),
                      (dict(cap=-1.0), 1), (dict(cap=math.nan), 1), (dict(K=0), 3), (dict(K=1025), 3), (dict(V=0), 3),
                      (dict(V=(1 << 24) + 1), 3), (dict(tau=1e-5), 1), (dict(tau=1e5), 1), (dict(cap=1e-5), 1),
                      (dict(cap=1e5), 1)]:
        assert dis(**bad) == want, bad
    b = dict(z=_f(2, 10), teacher_idx=_i(2, 3), teacher_logits=_f(2, 3), token_loss=_f(2), dz=_f(2, 10))
    assert _code(nclib, nclib.distill_topk, **b) == 8
    for name, t, want in [("teacher_logits", _f(2, 4), 3), ("dz", _f(2, 9), 3), ("row_weight", _f(3), 3),
                          ("z", _f(10, 2).T, 1), ("token_loss", None, 1)]:
        assert _code(nclib, nclib.distill_topk, **{**b, name: t}) == want, name
    with pytest.raises(TypeError):
        nclib.distill_topk(**{**b, "dz": _i(2, 10)})


def test_status_words_and_empty_batches(nclib):
    a = dict(q=_h(2, 3, 4, 64), kv=_h(2, 3, 2, 2, 64), cache=_h(2, 9, 2, 2, 64), lens=_i(2), mask=_i(2, 3, 1),
             out=_h(2, 3, 4, 64))
    d = dict(z=_f(2, 10), teacher_idx=_i(2, 3), teacher_logits=_f(2, 3), token_loss=_f(2), dz=_f(2, 10))
    byte = torch.zeros(16, dtype=torch.uint8)
    byte = byte[-byte.data_ptr() % 4:]
    for fn, args in [(nclib.tree_attention, a), (nclib.distill_topk, d)]:
        # a wrong word is found before the call, a right one gets as far as the missing device
        for t, want in [(byte[:3], 5), (byte[1:9], 4), (_i(4)[::2], 1), (byte[:4], 8), (_i(1), 8)]:
            assert _code(nclib, fn, **args, status=t) == want, (fn.__name__, t.shape)
    # no rows: nothing is done
    nclib.tree_mask(_i(0, 5), _i(0, 5, 1))
    nclib.tree_attention(_h(0, 3, 4, 64), _h(0, 3, 2, 2, 64), _h(0, 9, 2, 2, 64), _i(0), _i(0, 3, 1), _h(0, 3, 4, 64))
    nclib.sample(_f(0, 10), _f(0), _i(0))
    nclib.distill_topk(_f(0, 10), _i(0, 3), _f(0, 3), _f(0))
    nclib.tree_accept(_i(0, 3), _i(0, 3), _i(0, 3, 1), _i(0, 3), _i(0), _h(2, 0, 3, 2, 1, 64), _h(2, 0, 9, 2, 1, 64),
                      _i(0, 3), _i(0), _i(0), _i(0))


def test_tree_workspace_and_step_refusals(nclib):
    import ctypes
    L = nclib.lib()
    c = nclib.init_config(2, 64, 64, 0, 256, 512)
    assert nclib.tree_workspace_bytes(c, 2, 8) > 0
    assert [nclib.tree_workspace_bytes(c, *bn) for bn in [(0, 8), (2, 0), (2, 129), (65536, 1)]] == [0] * 4
    sb, wb = L.nc_session_bytes(ctypes.byref(c), 2, 64), nclib.tree_workspace_bytes(c, 2, 8)

    def acc(cfg=c, B=2, N=8, lens_out=A + 64, sess=A, s_bytes=sb, T=64, ws=A, w_bytes=wb):
        return L.nc_accept_tree(ctypes.byref(cfg), A, A, A, A, B, N, A, A, A, lens_out, sess, s_bytes, T, ws, w_bytes,
                                None)

    for bad, want in [(dict(N=129), 3), (dict(B=0), 3), (dict(T=257), 3), (dict(s_bytes=sb - 1), 5),
                      (dict(w_bytes=wb - 1), 5), (dict(sess=A + 16), 4), (dict(ws=A + 16), 4), (dict(lens_out=A), 1),
                      (dict(ws=None), 1)]:
        assert acc(**bad) == want, bad
    f8 = nclib.NcConfig.from_buffer_copy(c)
    f8.fp8 = 1
    assert acc(cfg=f8) == 2


def test_definitions_on_hand_made_cases():
    par = np.array([[-1, 0, 0, 1, -2, 5, 4]], np.int32)
    m = o64.tree_mask(par)[0, :, 0]
    assert list(m) == [1, 3, 5, 11, 0, 0, 0]  # 4: unused; 5: its own parent; 6: under an unused node
    l = np.log(np.array([0.1, 0.4, 0.2, 0.3], np.float32))
    assert [o64.sample_row(l, u)[0] for u in (0.0, 0.05, 0.15, 0.65, 0.99, 1.0)] == [0, 0, 1, 2, 3, 3]
    assert [o64.sample_row(l, u, top_k=2)[0] for u in (0.0, 0.56, 0.58)] == [1, 1, 3]
    assert [o64.sample_row(l, u, top_p=0.8)[0] for u in (0.0, 0.5, 0.99)] == [1, 2, 3]  # 0.4 + 0.3 < 0.8
    assert [o64.sample_row(l, u, min_p=0.6)[0] for u in (0.0, 0.99)] == [1, 3]
    assert o64.sample_row(l, 0.5, T=0.0)[:2] == (1, 0.0)
    # the gradient against differences of the loss
    rng = np.random.default_rng(0)
    z, idx, t = rng.normal(size=9) * 4, np.array([3, 1, 3, -1], np.int64), rng.normal(size=4)
    for tau, cap in [(1.0, 15.0), (2.0, 0.0), (0.7, 3.0)]:
        _, d = o64.distill_row(z, idx, t, tau, cap)
        for i in range(9):
            h = np.zeros(9)
            h[i] = 1e-5
            num = (o64.distill_row(z + h, idx, t, tau, cap)[0] - o64.distill_row(z - h, idx, t, tau, cap)[0]) / 2e-5
            assert abs(num - d[i]) < 1e-8
