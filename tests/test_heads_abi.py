"""The operators around a draft head on the host: size queries, and argument
errors that are found before anything is enqueued.  No kernel is launched."""
import ctypes

import pytest
import torch

import draft_verification_row_amd as sv

OK, EINVAL, EDTYPE, EWORKSPACE = 0, 1, 2, 3
P = 4096
WS = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return sv.load_library()


def test_size_queries(lib):
    q = lib.spec_logprobs_workspace_bytes
    assert q(1, 6, 128256, 5) > 0 and q(0, 6, 128256, 32) % 256 == 0
    assert q(2, 6, 128256, 5) == 0 and q(1, 0, 128256, 5) == 0 and q(1, 6, 0, 5) == 0
    assert q(1, 6, 262145, 5) == 0 and q(1, 6, 100, 33) == 0 and q(1, 6, 100, -1) == 0
    assert q(1, 1 << 24, 100, 0) == 0  # one tile a row, 2^24 rows
    k = lib.spec_draft_kl_workspace_bytes
    assert k(1, 32, 5, 128256) > 0 and k(1, 0, 5, 100) == 0 and k(1, 1, 0, 100) == 0 and k(3, 1, 1, 100) == 0
    for f in (lib.spec_linear_workspace_bytes, lib.spec_linear_grad_workspace_bytes):
        assert f(1, 8, 16, 32) > 0 and f(0, 8, 16, 32) > 0
        assert f(2, 8, 16, 32) == 0 and f(1, 0, 16, 32) == 0 and f(1, 8, 0, 32) == 0 and f(1, 8, 16, 0) == 0
        assert f(1, (1 << 20) + 1, 16, 32) == 0 and f(1, 1 << 20, 1 << 20, 1) == 0


def test_logprobs_argument_errors(lib):
    need = lib.spec_logprobs_workspace_bytes(1, 4, 100, 5)

    def f(**over):
        a = dict(X=P, dt=1, tok=P, rows=4, V=100, top=5, lp=P, ent=P, tt=P, tl=P, st=P, stats=None, ws=WS,
                 wsb=need, stream=None)
        a.update(over)
        return lib.spec_token_logprobs(*a.values())

    assert f(dt=2) == EDTYPE and f(dt=-1) == EDTYPE
    for bad in (dict(rows=0), dict(rows=-1), dict(V=0), dict(V=262145), dict(top=-1), dict(top=33), dict(X=None),
                dict(tok=None), dict(lp=None), dict(ent=None), dict(tt=None), dict(tl=None), dict(st=None),
                dict(rows=1 << 24), dict(stats=P + 4)):
        assert f(**bad) == EINVAL, bad
    assert f(ws=None) == EWORKSPACE and f(ws=WS + 8) == EWORKSPACE and f(wsb=0) == EWORKSPACE
    g = lib.spec_token_logprobs_grad
    assert g(P, 5, P, P, P, P, 4, 100, P, None) == EDTYPE
    assert g(None, 1, P, P, P, P, 4, 100, P, None) == EINVAL
    assert g(P, 1, None, P, P, P, 4, 100, P, None) == EINVAL
    assert g(P, 1, P, None, P, P, 4, 100, P, None) == EINVAL
    assert g(P, 1, P, P, P, P, 0, 100, P, None) == EINVAL
    assert g(P, 1, P, P + 8, P, P, 4, 100, P, None) == EINVAL
    assert g(P, 1, P, P, P, P, 4, 100, None, None) == EINVAL


def test_kl_argument_errors(lib):
    need = lib.spec_draft_kl_workspace_bytes(1, 2, 3, 100)

    def f(**over):
        a = dict(T=P, D=P, dt=1, mask=None, B=2, K=3, Kt=4, V=100, kl=P, stats=None, ws=WS, wsb=need, stream=None)
        a.update(over)
        return lib.spec_draft_kl(*a.values())

    assert f(dt=7) == EDTYPE
    for bad in (dict(T=None), dict(D=None), dict(kl=None), dict(B=0), dict(K=0), dict(Kt=2), dict(V=0),
                dict(V=262145), dict(stats=P + 4)):
        assert f(**bad) == EINVAL, bad
    assert f(ws=None) == EWORKSPACE and f(wsb=0) == EWORKSPACE and f(ws=WS + 16) == EWORKSPACE
    g = lib.spec_draft_kl_grad
    assert g(P, P, 2, None, P, P, 2, 3, 4, 100, P, None) == EDTYPE
    for i in (0, 1, 4, 5, 10):
        a = [P, P, 1, None, P, P, 2, 3, 4, 100, P, None]
        a[i] = None
        assert g(*a) == EINVAL, i


def test_linear_argument_errors(lib):
    need = lib.spec_linear_workspace_bytes(1, 4, 8, 16)

    def f(**over):
        a = dict(x=P, w=P, b=None, r=None, dt=1, ot=1, act=0, M=4, N=8, K=16, y=P, z=None, ws=WS, wsb=need,
                 stream=None)
        a.update(over)
        return lib.spec_linear(*a.values())

    assert f(dt=3) == EDTYPE and f(ot=2) == EDTYPE and f(dt=0, ot=1) == EDTYPE
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(M=0), dict(N=0), dict(K=0), dict(act=4),
                dict(act=-1), dict(M=1 << 21), dict(M=1 << 20, N=1 << 16)):
        assert f(**bad) == EINVAL, bad
    assert f(ws=None) == EWORKSPACE and f(ws=WS + 64) == EWORKSPACE and f(wsb=need - 1) == EWORKSPACE
    gneed = lib.spec_linear_grad_workspace_bytes(1, 4, 8, 16)

    def g(**over):
        a = dict(x=P, w=P, z=P, gy=P, dt=1, ot=1, act=3, M=4, N=8, K=16, gx=P, gw=P, gb=P, ws=WS, wsb=gneed,
                 stream=None)
        a.update(over)
        return lib.spec_linear_grad(*a.values())

    assert g(dt=0, ot=1) == EDTYPE
    for bad in (dict(gy=None), dict(z=None), dict(x=None), dict(w=None), dict(act=9), dict(M=0)):
        assert g(**bad) == EINVAL, bad
    assert g(wsb=gneed - 1) == EWORKSPACE and g(ws=None) == EWORKSPACE


def test_binding_refuses_host_tensors():
    X = torch.zeros(2, 50)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_token_logprobs(X, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_draft_kl(X[None], X[None])
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_linear(X, X)


def test_a_capture_refuses_leaves_of_another_streams_graph():
    """The rule behind captured backward passes, on the host: streams are
    numbers here."""
    from draft_verification_row_amd.heads import _note_stream
    x, y = torch.ones(3, requires_grad=True), torch.ones(3)
    graph = x * y
    _note_stream(graph.grad_fn.next_functions, 1, False)
    again = x * 2
    _note_stream(again.grad_fn.next_functions, 2, False)   # eager calls may use any stream
    _note_stream(again.grad_fn.next_functions, 1, True)    # a capture on the same one too
    with pytest.raises(sv.SpecVerifyError):
        _note_stream(again.grad_fn.next_functions, 2, True)
    _note_stream((again * 3).grad_fn.next_functions, 2, True)  # no leaf
    del graph, again
    _note_stream((x * 2).grad_fn.next_functions, 2, True)  # the graphs are gone


@pytest.mark.gpu
def test_binding_refusals():
    X = torch.zeros(2, 4, 50, device="cuda")
    tok = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    E = sv.SpecVerifyError
    bad = [
        lambda: sv.spec_token_logprobs(X.half(), tok), lambda: sv.spec_token_logprobs(X, tok.long()),
        lambda: sv.spec_token_logprobs(X, tok[:1]), lambda: sv.spec_token_logprobs(X, tok, top_n=33),
        lambda: sv.spec_token_logprobs(X, tok, top_n=-1), lambda: sv.spec_token_logprobs(X, tok.cpu()),
        lambda: sv.spec_token_logprobs(X.transpose(0, 1), tok), lambda: sv.spec_token_logprobs(X[..., :0], tok),
        lambda: sv.spec_token_logprobs(torch.zeros(1, 262145, device="cuda"), tok[0, :1]),
        lambda: sv.spec_draft_kl(X, X.bfloat16()), lambda: sv.spec_draft_kl(X[:, :3], X),
        lambda: sv.spec_draft_kl(X, X[..., :40].contiguous()), lambda: sv.spec_draft_kl(X[0], X[0]),
        lambda: sv.spec_draft_kl(X, X, mask=tok), lambda: sv.spec_draft_kl(X.clone().requires_grad_(), X),
        lambda: sv.spec_draft_kl(X, X, mask=torch.ones(2, 3, dtype=torch.bool, device="cuda")),
        lambda: sv.spec_linear(X, X[0, :, :49].contiguous()), lambda: sv.spec_linear(X, X[0].bfloat16()),
        lambda: sv.spec_linear(X, X[0], activation="tanh"), lambda: sv.spec_linear(X, X[0], X[0, 0]),
        lambda: sv.spec_linear(X, X[0], out_dtype=torch.bfloat16), lambda: sv.spec_linear(X, X[0].t()),
        lambda: sv.spec_linear(X, X[0], residual=X), lambda: sv.spec_linear(X.half(), X[0].half()),
        lambda: sv.spec_linear(X, X[0, :0]), lambda: sv.spec_linear(X, X[0], torch.zeros(4)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(E):
            f()
            print("not refused:", i)
