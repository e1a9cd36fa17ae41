"""Trees of drafted tokens over a KV-cache session (Session.decode_tree / sample /
accept_tree) against the oracle: a node's logits are those of the whole forward over the
row's prefix followed by the node's path.  Bars as for the forward: logits max-abs <= 3e-2.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import tree as o64
from workloads import SHAPES, ModelShape, make_extras, make_tokens, make_weights

pytestmark = pytest.mark.gpu

DEV = "cuda"
BAR = 3e-2
GQA = ModelShape("gqa", 3, 256, 6, 2, 128, 256, 512, 2, 64)  # three query heads a kv head: no decode step has that


def _oracle_cfg(s):
    return oracle.OracleConfig(s.n_layer, s.d_model, s.n_head, s.n_kv_head, s.head_dim, s.seq_len, s.vocab,
                               short_window=s.short_window)


def _model(nc, s, extras):
    w = make_weights(s)
    ex = make_extras(s, layers=[l for l in range(s.n_layer) if oracle.value_embed_layers(s.n_layer)[l]]) if extras else None
    cfg = nc.make_config(s.n_layer, s.d_model, s.n_head, s.n_kv_head, s.head_dim, s.seq_len, s.vocab, s.short_window,
                         extras=nc.EXTRA_ALL if extras else 0)
    return w, ex, nc.Model.from_numpy(cfg, w, extras=ex)


def _path(parents, i):
    p = []
    while i >= 0:
        p.append(i)
        i = parents[i]
    return p[::-1]


def _want(s, w, ex, seq):
    """Logits of the last position of each sequence, one forward per length."""
    out = {}
    for n in sorted({len(q) for q in seq}):
        rows = [i for i, q in enumerate(seq) if len(q) == n]
        kw = {} if ex is None else {"extras": ex}
        lo = oracle.forward(_oracle_cfg(s), w, np.array([seq[i] for i in rows], np.int32), **kw)["logits"][:, -1]
        out.update(zip(rows, lo))
    return np.stack([out[i] for i in range(len(seq))])


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def _check_nodes(s, w, ex, prefix, tokens, parents, logits):
    seq, where = [], []
    for b in range(len(tokens)):
        for i in range(tokens.shape[1]):
            if parents[b, i] >= -1:
                seq.append(list(prefix[b]) + [int(tokens[b, j]) for j in _path(parents[b], i)])
                where.append((b, i))
    got = np.stack([logits[b, i].cpu().numpy() for b, i in where])
    err = np.abs(got - _want(s, w, ex, seq)).max()
    assert err <= BAR, f"logits max-abs {err:.3e}"


@pytest.mark.parametrize("shape,extras,N,T0", [(SHAPES["tiny"], False, 7, 90), (SHAPES["tiny"], True, 7, 90),
                                               (SHAPES["tiny"], True, 5, 0), (GQA, False, 24, 70), (GQA, True, 9, 1)],
                         ids=["tiny", "tiny-extras", "tiny-extras-empty", "gqa", "gqa-extras"])
def test_speculative_steps_match_the_forward(gpu, shape, extras, N, T0):
    """Three rounds of draft, check, accept: rows accept paths of different lengths, so their
    lengths part; every node's logits against the oracle on the row's own text."""
    s, B = shape, 3
    w, ex, model = _model(gpu, s, extras)
    rng = np.random.default_rng(N + T0)
    x, _ = make_tokens(s, batch=B, seed=3)
    prefix = [list(r) for r in x[:, :T0]]
    sess = gpu.Session(model, B, s.seq_len)
    sess.prefill(_dev(x[:, :T0]) if T0 else torch.empty((B, 0), dtype=torch.int32, device=DEV))
    root, parted = x[:, T0].copy(), False
    for turn in range(3):
        parents = np.full((B, N), -2, np.int32)
        for b in range(B):
            for i in range(N - b):  # smaller trees are padded
                parents[b, i] = -1 if i == 0 else (i - 1 if i < 4 else rng.integers(0, i))
        tokens = rng.integers(0, s.vocab, (B, N)).astype(np.int32)
        tokens[:, 0] = root
        tokens[parents == -2] = -1  # an unused node's token is not looked at
        logits = sess.decode_tree(_dev(tokens), _dev(parents))
        assert sess.status() == 0
        _check_nodes(s, w, ex, prefix, tokens, parents, logits)
        # the samples confirm b + turn nodes behind the root, then nothing
        sampled = np.full((B, N), s.vocab + 7, np.int32)
        for b in range(B):
            at = 0
            for _ in range((b + turn) % 3):
                kids = [j for j in range(N) if parents[b, j] == at and (tokens[b, :j] != tokens[b, j])[parents[b, :j] == at].all()]
                if not kids:
                    break
                sampled[b, at] = tokens[b, kids[-1]]
                at = kids[-1]
            sampled[b, at] = root[b] = rng.integers(0, s.vocab)
        path, count, nxt = sess.accept_tree(_dev(sampled))
        for b in range(B):
            p = [j for j in path[b].tolist() if j >= 0]
            assert len(p) == int(count[b]) and p[0] == 0 and all(parents[b, j] == i for i, j in zip(p, p[1:]))
            prefix[b] += [int(tokens[b, j]) for j in p]
        assert np.array_equal(nxt.cpu().numpy(), root)
        assert sess.lens.tolist() == [len(q) for q in prefix]
        parted = parted or len({len(q) for q in prefix}) > 1
    assert parted
    with pytest.raises(gpu.NcError):
        sess.decode(_dev(root))
    with pytest.raises(gpu.NcError):
        sess.accept_tree(_dev(sampled))


def test_tree_of_one_is_a_decode_step(gpu):
    """N = 1 over equal lengths against nc_decode_step: the same projections and cache, so the
    logits agree to the order of the atomic sums (1e-3 over two layers)."""
    s, B = SHAPES["tiny"], 4
    _, _, model = _model(gpu, s, False)
    x, _ = make_tokens(s, batch=B, seed=8)
    a, b = gpu.Session(model, B, 64), gpu.Session(model, B, 64)
    a.prefill(_dev(x[:, :20]))
    b.prefill(_dev(x[:, :20]))
    par = torch.full((B, 1), -1, dtype=torch.int32, device=DEV)
    for t in range(20, 26):
        la = a.decode(_dev(x[:, t]))
        lb = b.decode_tree(_dev(x[:, t:t + 1]), par)[:, 0]
        assert (la - lb).abs().max().item() <= 1e-3
        _, count, _ = b.accept_tree(_dev(x[:, t + 1:t + 2]))
        assert count.tolist() == [1] * B


def test_trees_from_an_empty_text_and_refusals(gpu):
    """The first tokens of a text by trees; what decode_tree and accept_tree need before them; calls
    on other streams than the one that made the session's tensors."""
    s, B = SHAPES["tiny"], 2
    w, ex, model = _model(gpu, s, False)
    x, _ = make_tokens(s, batch=B, seed=21)
    parents = np.array([[-1, 0, 1]] * B, np.int32)
    sess = gpu.Session(model, B, 40)
    tok, par = _dev(x[:, :3]), _dev(parents)
    with pytest.raises(gpu.NcError):
        sess.decode_tree(tok, par)
    sess.prefill(torch.empty((B, 0), dtype=torch.int32, device=DEV))
    with pytest.raises(gpu.NcError):
        sess.accept_tree(tok)
    text = [[] for _ in range(B)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(6):
        tok = _dev(x[:, 3 * k:3 * k + 3])
        sampled = _dev(np.stack([x[:, 3 * k + 1], x[:, 3 * k + 2], x[:, 3 * k + 3]], 1))
        torch.cuda.synchronize()
        logits = sess.decode_tree(tok, par, stream=streams[k % 2])
        torch.cuda.synchronize()
        _check_nodes(s, w, ex, text, x[:, 3 * k:3 * k + 3], parents, logits)
        _, count, nxt = sess.accept_tree(sampled, stream=streams[(k + 1) % 2])
        torch.cuda.synchronize()
        assert count.tolist() == [3] * B and nxt.tolist() == x[:, 3 * k + 3].tolist()
        text = [t + [int(v) for v in x[b, 3 * k:3 * k + 3]] for b, t in enumerate(text)]
    assert sess.lens.tolist() == [18] * B
    with pytest.raises(gpu.NcError):
        sess.decode(_dev(x[:, 18]))


def test_sampled_generation_in_one_graph(gpu):
    """decode_tree, sample and acceptance captured together (the entry points on preallocated
    buffers) and replayed until the cache is full: at every step the logits are the oracle's for
    the row's text, and the samples, paths and lengths are those of the definitions on the
    step's own logits."""
    import ctypes
    s, B, N, T_max = SHAPES["tiny"], 2, 4, 64
    w, ex, model = _model(gpu, s, False)
    x, _ = make_tokens(s, batch=B, seed=5)
    L = gpu.lib()
    parents = np.array([[-1, 0, 1, 1]] * B, np.int32)
    par, mask = _dev(parents), o64.tree_mask(parents)
    gen = torch.Generator(device=DEV).manual_seed(1)
    temp = torch.full((B * N,), 0.7, device=DEV)
    topk = torch.full((B * N,), 3, dtype=torch.int32, device=DEV)
    sess = gpu.Session(model, B, T_max)
    sess.prefill(_dev(x[:, :50]))
    ws = torch.empty(gpu.tree_workspace_bytes(model.cfg, B, N), dtype=torch.uint8, device=DEV)
    i32 = lambda *z: torch.zeros(z, dtype=torch.int32, device=DEV)  # noqa: E731
    tok, smp, path, count, nxt, lens, lens2 = i32(B, N), i32(B * N), i32(B, N), i32(B), i32(B), i32(B), i32(B)
    logits, u = torch.zeros((B, N, s.vocab), device=DEV), torch.zeros(B * N, device=DEV)
    cfg, wts = ctypes.byref(model.cfg), ctypes.byref(model.weights)

    def step():
        st = torch.cuda.current_stream().cuda_stream
        assert L.nc_decode_tree(cfg, wts, tok.data_ptr(), par.data_ptr(), lens.data_ptr(), B, N, logits.data_ptr(),
                                sess.buffer.data_ptr(), sess.buffer.numel(), T_max, ws.data_ptr(), ws.numel(), st) == 0
        gpu.sample(logits.view(B * N, -1), u, smp, temperature=temp, top_k=topk)
        assert L.nc_accept_tree(cfg, tok.data_ptr(), par.data_ptr(), smp.data_ptr(), lens.data_ptr(), B, N,
                                path.data_ptr(), count.data_ptr(), nxt.data_ptr(), lens2.data_ptr(),
                                sess.buffer.data_ptr(), sess.buffer.numel(), T_max, ws.data_ptr(), ws.numel(), st) == 0

    def start():
        lens.fill_(50)
        tok.copy_(_dev(x[:, 50:50 + N]))
        u.copy_(torch.rand(B * N, generator=gen, device=DEV))

    start()
    step()  # eagerly once; what it put behind position 50 is written again below
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    start()
    text = [list(r) for r in x[:, :50]]
    for k in range(20):
        g.replay()
        t, sm, ln = tok.cpu().numpy(), smp.cpu().numpy().reshape(B, N), lens.cpu().numpy()
        lg, uu = logits.cpu().numpy(), u.cpu().numpy().reshape(B, N)
        if all(v + 2 < T_max for v in ln):  # every node's position is inside the cache
            _check_nodes(s, w, ex, text, t, parents, logits)
        for b in range(B):
            for i in range(N):
                want = o64.sample_row(lg[b, i], float(uu[b, i]), float(np.float32(0.7)), 3)
                assert sm[b, i] == want[0] or want[2] < 1e-9
        for b, (p, n) in enumerate(o64.tree_accept(t, parents, mask, sm, ln, T_max)):
            assert path[b].tolist() == p + [-1] * (N - len(p)) and int(nxt[b]) == n
            assert int(lens2[b]) == ln[b] + len(p)
            text[b] += [int(t[b, j]) for j in p]
        lens.copy_(lens2)
        tok[:, 0] = nxt
        tok[:, 1:] = torch.randint(0, s.vocab, (B, N - 1), generator=gen, device=DEV, dtype=torch.int32)
        tok[:, 1] = torch.where(torch.arange(B, device=DEV) == k % B, smp.view(B, N)[:, 1], tok[:, 1])
        u.copy_(torch.rand(B * N, generator=gen, device=DEV))
    assert lens.tolist() == [T_max] * B and count.tolist() == [0] * B
