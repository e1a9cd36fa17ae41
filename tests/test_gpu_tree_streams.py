"""The drafted-tree calls on streams of their own: temporaries, work queued ahead, several threads."""
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
