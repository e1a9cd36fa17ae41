"""The drafted-tree calls on streams of their own: temporaries, work queued ahead, several threads."""
import threading

import numpy as np
import pytest
import torch

from workloads import SHAPES, make_tokens, make_weights

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def _model(nc, s):
    cfg = nc.make_config(s.n_layer, s.d_model, s.n_head, s.n_kv_head, s.head_dim, s.seq_len, s.vocab, s.short_window)
    return nc.Model.from_numpy(cfg, make_weights(s))


def _hold(stream):
    """Some tens of ms of products queued on the stream."""
    with torch.cuda.stream(stream):
        a = torch.ones((8192, 8192), device=DEV)
        for _ in range(8):
            a @ a
    return a


@pytest.mark.parametrize("drop", [False, True])
def test_temporaries_on_a_stream_that_is_held_back(gpu, drop):
    """Tokens, parents and samples given as temporaries to a stream that is behind; their memory is asked for
    again at once on the default stream.  drop: the tree is given up by the next one instead of accepted."""
    s, B, N = SHAPES["tiny"], 2, 6
    model = _model(gpu, s)
    x, _ = make_tokens(s, batch=B, seed=3)
    par = np.tile(np.array([-1, 0, 1, 1, 0, 2], np.int32), (B, 1))
    tok = x[:, 20:20 + N].astype(np.int32)
    smp = np.full((B, N), -1, np.int32)
    smp[:, 0], smp[:, 1], smp[:, 2] = tok[:, 1], tok[:, 2], tok[:, 5]
    ref = gpu.Session(model, B, 64)
    ref.prefill(_dev(x[:, :20]))
    want_logits = ref.decode_tree(_dev(tok), _dev(par))
    want = ref.accept_tree(_dev(smp))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    sess = gpu.Session(model, B, 64)
    sess.prefill(_dev(x[:, :20]))
    torch.cuda.synchronize()
    keep = _hold(st)
    logits = sess.decode_tree(_dev(tok), _dev(par), stream=st)
    junk = []
    if drop:
        other = (_dev(tok[:, ::-1].copy()), _dev(par))
        sess.decode_tree(*other, stream=st)
    else:
        got = sess.accept_tree(_dev(smp), stream=st)
    for _ in range(64):
        junk.append(torch.full((B, N), 7, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    # the same products in the order of their atomic sums, as for a decode step (1e-3 over two layers)
    assert (logits - want_logits).abs().max().item() <= 1e-3
    if not drop:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert got[1].tolist() == [4] * B and torch.equal(sess.lens, ref.lens)
    del keep, junk


def test_threads_side_by_side(gpu):
    """Two threads, each with a stream, a session, a workspace and another tree: what each gets is what it gets
    alone."""
    s = SHAPES["tiny"]
    model = _model(gpu, s)
    x, _ = make_tokens(s, batch=4, seed=9)

    def work(k, stream, out):
        B, N = 2 + k, 5 + 35 * k
        with torch.cuda.stream(stream):
            sess = gpu.Session(model, B, 128)
            sess.prefill(_dev(x[:B, :30]))
            rng = np.random.default_rng(k)
            par = np.array([[-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, N)]] * B, np.int32)
            g = torch.Generator(device=DEV).manual_seed(k)
            q, kv, cache = (torch.randn(z, generator=g, device=DEV).half() for z in
                            ((B, N, 8, 64), (B, N, 2, 2, 64), (B, 600, 2, 2, 64)))
            mask = torch.empty((B, N, (N + 31) // 32), dtype=torch.int32, device=DEV)
            lens = torch.full((B,), 500, dtype=torch.int32, device=DEV)
            z, u = torch.randn((B * N, 3001), generator=g, device=DEV), torch.rand(B * N, generator=g, device=DEV)
            ti = torch.randint(0, 3001, (B * N, 9), generator=g, device=DEV, dtype=torch.int32)
            tl = torch.randn((B * N, 9), generator=g, device=DEV)
            for turn in range(12):
                tok = _dev(rng.integers(0, s.vocab, (B, N)))
                parents = _dev(par)
                sess.decode_tree(tok, parents)
                smp = tok[:, [1] + list(range(1, N))].contiguous()
                path, count, nxt = sess.accept_tree(smp)
                o, t, loss, dz = torch.empty_like(q), torch.empty(B * N, dtype=torch.int32, device=DEV), torch.empty(
                    B * N, device=DEV), torch.empty_like(z)
                gpu.tree_mask(parents, mask)
                gpu.tree_attention(q, kv, cache, lens, mask, o)
                gpu.sample(z, u, t, top_p=torch.full_like(u, 0.9))
                gpu.distill_topk(z, ti, tl, loss, dz)
                out.append([a.clone() for a in (path, count, nxt, o, t, loss, dz)])
            stream.synchronize()

    alone, both = [[], []], [[], []]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for k in range(2):
        work(k, streams[k], alone[k])
    errors = []

    def run(k):
        try:
            work(k, streams[k], both[k])
        except Exception as e:  # noqa: BLE001  (shown below)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for a, b in zip(alone, both):
        assert len(a) == len(b) == 12
        assert all(torch.equal(p, q) for x, y in zip(a, b) for p, q in zip(x, y))


@pytest.mark.parametrize("extras", [False, True])
def test_trees_of_hundreds_of_rows(gpu, extras):
    """Trees of 100 nodes, 300 rows of the projections, padded and of parted lengths: every node against the oracle."""
    from test_gpu_tree_session import _check_nodes, _model as both_models
    s, B, N = SHAPES["tiny"], 3, 100
    w, ex, model = both_models(gpu, s, extras)
    x, _ = make_tokens(s, batch=B, seed=6)
    rng = np.random.default_rng(1)
    sess = gpu.Session(model, B, 128)
    sess.prefill(_dev(x[:, :40]))
    text = [list(r) for r in x[:, :40]]
    for turn in range(2):
        par = np.full((B, N), -2, np.int32)
        for b in range(B):
            for i in range(N - 30 * b):
                par[b, i] = -1 if i == 0 else int(rng.integers(max(0, i - 40), i))
        tok = rng.integers(0, s.vocab, (B, N)).astype(np.int32)
        logits = sess.decode_tree(_dev(tok), _dev(par))
        assert sess.status() == 0
        _check_nodes(s, w, ex, text, tok, par, logits)
        smp = np.full((B, N), -1, np.int32)
        for b in range(1, B):  # rows 1 and 2 accept a child of the root, row 2 a grandchild too, where there is one
            at = 0
            for _ in range(b):
                kids = np.flatnonzero(par[b] == at)
                if len(kids):
                    smp[b, at], at = tok[b, kids[0]], kids[0]
        path, count, _ = sess.accept_tree(_dev(smp))
        for b in range(B):
            text[b] += [int(tok[b, j]) for j in path[b].tolist() if j >= 0]
        assert count.tolist() == [len(t) - 40 for t in text] if turn == 0 else True
        assert sess.lens.tolist() == [len(t) for t in text]
