"""Session.decode_tree / accept_tree: the tensors they hold on to, without a GPU (the launches are recorded)."""
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture
def session(nclib, monkeypatch):
    sess = nclib.Session.__new__(nclib.Session)
    sess.model = SimpleNamespace(cfg=nclib.init_config(2, 64, 64, 0, 256, 512), weights=nclib.NcWeights())
    sess.B, sess.T_max, sess.pos = 2, 64, 4
    sess.buffer = torch.zeros(16, dtype=torch.uint8)
    sess._graph, sess._filled = None, True
    sess._lens = sess._tree = sess._tree_ws = None
    used = []
    monkeypatch.setattr(nclib, "_launch", lambda *a: None)
    monkeypatch.setattr(nclib.Session, "_used_on", lambda self, stream, *t: used.append([x.data_ptr() for x in t]))
    return sess, used


def test_a_tree_held_by_the_session_outlives_calls_on_another_stream(session):
    """From decode_tree on the session may hold the last references to tokens and parents; both calls
    that read them mark them as used on the stream they run on."""
    sess, used = session
    tok, par = torch.zeros((2, 3), dtype=torch.int32), torch.tensor([[-1, 0, 1]] * 2, dtype=torch.int32)
    want = {tok.data_ptr(), par.data_ptr()}
    sess.decode_tree(tok, par)
    assert want <= set(sum(used, []))
    used.clear()
    ws = sess._tree_ws.data_ptr()
    smp = torch.zeros((2, 3), dtype=torch.int32)
    sess.accept_tree(smp)
    assert want | {ws, smp.data_ptr()} <= set(sum(used, []))


def test_prefill_marks_its_workspace(session, nclib):
    """Its workspace is freed when the call returns, maybe before the stream has come to it."""
    sess, used = session
    made = []
    empty = torch.empty
    torch_empty = lambda *a, **k: made.append(empty(*a, **k)) or made[-1]  # noqa: E731
    with pytest.MonkeyPatch.context() as m:
        m.setattr(torch, "empty", torch_empty)
        with pytest.raises(nclib.NcError):  # the launch: the session's buffer is a stand-in
            sess.prefill(torch.zeros((2, 3), dtype=torch.int32), stream=SimpleNamespace(cuda_stream=0))
    assert len(made) == 1 and made[0].data_ptr() in sum(used, [])
