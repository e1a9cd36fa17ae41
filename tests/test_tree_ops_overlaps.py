"""Calls whose outputs overlap their inputs or one another are refused before anything runs (CPU only: addresses
that nothing dereferences)."""
import ctypes
import itertools

P = 1 << 40  # each array has its own 2^30 bytes from here on


def _places(names):
    return {n: P + (i << 30) for i, n in enumerate(names)}


def test_tree_accept_overlaps(nclib):
    L = nclib.lib()
    B, N, layers, Hkv, D, T = 2, 40, 3, 2, 64, 128
    names = ["tokens", "parents", "mask", "sampled", "lens", "kv", "cache", "path", "count", "next", "lens_out"]
    size = dict(tokens=B * N * 4, parents=B * N * 4, mask=B * N * 8, sampled=B * N * 4, lens=B * 4, count=B * 4, next=B * 4,
                lens_out=B * 4, path=B * N * 4, kv=layers * B * N * 2 * Hkv * D * 2, cache=layers * B * T * 2 * Hkv * D * 2)

    def code(**at):
        return L.nc_tree_accept(*{**_places(names), **at}.values(), B, N, layers, Hkv, D, T, None)

    assert code() == 8  # nothing but the device is wrong
    outs = ["cache", "path", "count", "next", "lens_out"]
    for o, i in itertools.permutations(names, 2):
        if o not in outs and i not in outs:
            continue
        base = _places(names)[i]
        # the same start, the last 16 bytes (4 of the small ones), and just beside
        assert code(**{o: base}) == 1, (o, i)
        step = 16 if size[i] >= 16 and size[i] % 16 == 0 else 4
        if o not in ("kv", "cache") or step == 16:
            assert code(**{o: base + size[i] - step}) == 1, (o, i)
            assert code(**{o: base + size[i] + 16 - size[i] % 16}) == 8, (o, i)
    # inputs may share memory
    assert code(tokens=_places(names)["sampled"], parents=_places(names)["sampled"]) == 8


def test_accept_tree_overlaps(nclib):
    L = nclib.lib()
    c = nclib.init_config(2, 64, 64, 0, 256, 512)
    B, N, T = 2, 8, 64
    sb, wb = L.nc_session_bytes(ctypes.byref(c), B, T), nclib.tree_workspace_bytes(c, B, N)
    names = ["tokens", "parents", "sampled", "lens", "path", "count", "next", "lens_out", "session", "ws"]

    def code(**at):
        a = {**_places(names), **at}
        return L.nc_accept_tree(ctypes.byref(c), *[a[k] for k in names[:4]], B, N, *[a[k] for k in names[4:8]], a["session"],
                                sb, T, a["ws"], wb, None)

    assert code() == 8
    for o in names[4:8]:
        for i in names:
            if i != o:
                assert code(**{o: _places(names)[i]}) == 1, (o, i)
                assert code(**{o: _places(names)[i] + 4}) == 1, (o, i)
    assert code(path=P + (9 << 30) + wb - 4) == 1 and code(path=P + (9 << 30) + wb) == 8


def test_distill_overlaps(nclib):
    L = nclib.lib()
    M, V, K = 6, 70, 8
    names = ["z", "idx", "teacher", "weight", "loss", "dz"]
    size = dict(z=M * V * 4, idx=M * K * 4, teacher=M * K * 4, weight=M * 4, loss=M * 4)
    for dt, es in ((0, 2), (1, 2), (2, 4), (3, 0)):
        size["dz"] = M * V * es

        def code(**at):
            a = {**_places(names), **at}
            if not es:
                a["dz"] = None
            return L.nc_distill_topk(*[a[k] for k in names], dt, M, V, K, 1.0, 15.0, None, None)

        assert code() == 8 and code(weight=None) == 8
        for o in ["loss", "dz"] if es else ["loss"]:
            for i in names:
                if i == o or not size[i]:
                    continue
                base = _places(names)[i]
                assert code(**{o: base}) == 1, (o, i)
                assert code(**{o: base + size[i] - 4}) == 1, (o, i)
                assert code(**{o: base - size[o] + 4}) == 1, (o, i)
                assert code(**{o: base + size[i]}) == 8 and code(**{o: base - size[o]}) == 8, (o, i)
        assert code(weight=_places(names)["teacher"]) == 8  # inputs may share memory


def test_tree_mask_overlaps(nclib):
    L = nclib.lib()
    for N, W in ((20, 1), (40, 2)):
        assert L.nc_tree_mask(P, P + 3 * N * 4, 3, N, None) == 8 and L.nc_tree_mask(P + 3 * N * W * 4, P, 3, N, None) == 8
        for d in (0, 4, 3 * N * 4 - 4):
            assert L.nc_tree_mask(P, P + d, 3, N, None) == 1
        assert L.nc_tree_mask(P + 3 * N * W * 4 - 4, P, 3, N, None) == 1


def test_tree_attention_overlaps(nclib):
    L = nclib.lib()
    names = ["q", "kv", "cache", "lens", "mask", "out", "ws"]
    for B, N, H, Hkv, D, T, stride in ((2, 4, 4, 2, 64, 96, 256), (2, 64, 4, 2, 128, 900, 512), (1, 3, 4, 4, 64, 96, 768)):
        W = (N + 31) // 32
        need = L.nc_tree_attention_workspace_bytes(B, N, H, Hkv, D, T, 0)
        size = dict(q=((B * N - 1) * stride + H * D) * 2, kv=B * N * 2 * Hkv * D * 2, cache=B * T * 2 * Hkv * D * 2, lens=B * 4,
                    mask=B * N * W * 4, out=B * N * H * D * 2, ws=need)

        def code(**at):
            a = {**_places(names), **at}
            return L.nc_tree_attention(a["q"], stride, a["kv"], a["cache"], a["lens"], a["mask"], a["out"], B, N, H, Hkv, D, T, 0,
                                       1, a["ws"] if need else None, need, None, None)

        assert code() == 8
        for o in ("out", "ws") if need else ("out",):
            for i in names:
                if i == o or not size[i]:
                    continue
                base = _places(names)[i]
                whole = o == "out" and i == "q" and stride == H * D
                assert code(**{o: base}) == (8 if whole else 1), (o, i)
                assert code(**{o: base + (size[i] - 1) // 16 * 16}) == 1, (o, i)
                assert code(**{o: base + (size[i] + 15) // 16 * 16}) == 8, (o, i)


def test_sample_overlaps(nclib):
    L = nclib.lib()
    M, V, ld = 6, 70, 100
    names = ["logits", "u", "t", "k", "p", "m", "tokens", "logprob"]

    def code(**at):
        a = {**_places(names), **at}
        return L.nc_sample(a["logits"], ld, a["u"], a["t"], a["k"], a["p"], a["m"], a["tokens"], a["logprob"], M, V, None)

    assert code() == 8 and code(logprob=None) == 8
    end = ((M - 1) * ld + V) * 4
    for o in ("tokens", "logprob"):
        assert code(**{o: _places(names)["logits"]}) == 1 and code(**{o: _places(names)["logits"] + end - 4}) == 1
        assert code(**{o: _places(names)["logits"] + end}) == 8
        for i in names[1:]:
            if i == o:
                continue
            base = _places(names)[i]
            assert code(**{o: base}) == (1 if i in ("tokens", "logprob") else 8), (o, i)
            assert code(**{o: base + 4}) == 1 and code(**{o: base - 4}) == 1 and code(**{o: base + M * 4}) == 8, (o, i)
    # between two rows of the logits there is room
    at = _places(names)["logits"]
    assert code(tokens=at + V * 4) == 8 and code(tokens=at + (ld + V) * 4, logprob=at + (ld - M) * 4) == 8
    assert code(tokens=at + V * 4 - 4) == 1 and code(tokens=at + (ld - M + 1) * 4) == 1
    assert code(tokens=at - M * 4) == 8 and code(tokens=at - M * 4 + 4) == 1


def test_tree_attention_output_between_the_queries(nclib):
    L = nclib.lib()
    B, N, H, Hkv, D, T, stride = 1, 2, 2, 2, 64, 32, 512  # q: 256 bytes of every 1024; out: 512 bytes
    names = ["q", "kv", "cache", "lens", "mask", "out"]

    def code(out):
        a = _places(names)
        return L.nc_tree_attention(a["q"], stride, a["kv"], a["cache"], a["lens"], a["mask"], out, B, N, H, Hkv, D, T, 0, 1, None, 0,
                                   None, None)

    assert [code(P + d) for d in (0, 240, 256, 512, 528, 1024, 1264, 1280, -512, -496)] == [1, 1, 8, 8, 1, 1, 1, 8, 8, 1]
