"""spec_embedding against its definition in float64, forward and gradient.

Tolerances.  u = 2^-24, h half a step of a type.  Forward: one product, rounded
to float32 and then to the type: off by at most (h + u) |y| (u alone where the
type is float32).  A token's n positions are summed in float32 in any order and
scaled: off by at most (n + 1) u times the sum of magnitudes, then h.
"""
import math

import pytest
import torch

import draft_verification_row_amd as sv

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def half(dt):
    return torch.finfo(dt).eps / 2


def at_offset(t, off):
    buf = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
    buf[off:] = t.reshape(-1)
    return buf[off:].view(t.shape)


def close(got, want, tol, what):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), want[bad][:3].tolist())


def check(n, V, H, dtype, scale=1.0, seed=0, off=0, tokens=None):
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed + n + V + H)
    w = at_offset(torch.randn(V, H, generator=g, device="cuda").to(dt), off).requires_grad_()
    if tokens is None:
        tokens = torch.randint(-1, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    gy = at_offset(torch.randn(n, H, generator=g, device="cuda").to(dt), off)
    y = sv.spec_embedding(w, tokens, scale=scale)
    assert y.dtype == dt and y.shape == (n, H)
    live = (tokens >= 0) & (tokens < V)
    at = tokens.long().clamp(0, V - 1)
    want = torch.where(live[:, None], w.detach().double()[at] * scale, 0.0)
    close(y, want, (half(dt) + 2 * U) * want.abs(), "y")
    gw, = torch.autograd.grad([y], [w], [gy])
    index = at[live]
    add = lambda rows: torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, index, rows)  # noqa: E731
    want = add(gy[live].double()) * scale
    size = add(gy[live].double().abs()) * abs(scale)
    count = torch.bincount(index, minlength=V)[:, None]
    err = (count + 2) * U * size
    close(gw, want, err + half(dt) * (want.abs() + err), "grad")
    assert (gw[torch.bincount(index, minlength=V) == 0] == 0).all()
    return y, gw


SIZES = [(1, 1, 1), (1, 10, 7), (6, 1000, 64), (63, 50, 8), (64, 3, 40), (65, 300, 136), (129, 7, 512), (1000, 999, 264),
         (3001, 5000, 77), (5000, 17, 1032), (20000, 30000, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,H", SIZES)
def test_embedding_sizes(n, V, H, dtype):
    check(n, V, H, dtype, scale=math.sqrt(H) if n % 2 else 1.0)


@pytest.mark.parametrize("dtype,off", [("bf16", 1), ("bf16", 4), ("f32", 1)])
@pytest.mark.parametrize("n,V,H", [(7, 30, 24), (200, 9, 65), (300, 40, 2048)])
def test_embedding_alignment(n, V, H, dtype, off):
    check(n, V, H, dtype, scale=-0.37, off=off)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [64, 127, 128, 700, 5000])
def test_embedding_one_token_everywhere(n, dtype):
    """Long runs, which are summed in parts; then two tokens, of long runs each,
    at the table's ends."""
    tok = torch.full((n,), 3, dtype=torch.int32, device="cuda")
    check(n, 8, 72, dtype, tokens=tok)
    tok = torch.where(torch.arange(n, device="cuda") % 3 == 0, 0, 7).int()
    check(n, 8, 72, dtype, tokens=tok)


def test_embedding_padding_and_tokens_outside():
    V, H = 50, 40
    w = torch.randn(V, H, device="cuda").requires_grad_()
    tok = torch.tensor([[3, -1, 50], [-2, 49, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    y = sv.spec_embedding(w, tok, scale=2.0)
    assert y.shape == (2, 3, H)
    assert torch.equal(y[0, 0], w[3] * 2) and (y[0, 1] == 0).all() and torch.equal(y[1, 1], w[49] * 2)
    assert y[0, 2].isnan().all() and y[1, 0].isnan().all() and y[1, 2].isnan().all()
    gy = torch.full((2, 3, H), math.nan, device="cuda")
    gy[0, 0], gy[1, 1] = 1.0, 5.0
    g, = torch.autograd.grad([y], [w], [gy])  # the others' gradients are not read
    want = torch.zeros(V, H, device="cuda")
    want[3], want[49] = 2.0, 10.0
    assert torch.equal(g, want)
    allpad = sv.spec_embedding(w, torch.full((5,), -1, dtype=torch.int32, device="cuda"))
    g, = torch.autograd.grad([allpad.sum()], [w])
    assert (allpad == 0).all() and (g == 0).all()


def test_embedding_shapes():
    w = torch.randn(20, 16, device="cuda", requires_grad=True)
    one = sv.spec_embedding(w, torch.tensor(4, dtype=torch.int32, device="cuda"))
    assert one.shape == (16,) and torch.equal(one, w[4])
    none = sv.spec_embedding(w, torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    assert none.shape == (0, 3, 16)
    none.sum().backward()
    assert (w.grad == 0).all()
    y = sv.spec_embedding(w, torch.tensor([1, 1], dtype=torch.int32, device="cuda"))
    w.grad = None
    y.sum().backward()  # an expanded gradient
    assert (w.grad[1] == 2).all() and w.grad.sum() == 32


def test_embedding_order_is_fixed():
    n, V, H = 30000, 40, 96
    tok = torch.randint(0, V, (n,), dtype=torch.int32, device="cuda")
    w = torch.randn(V, H, device="cuda", requires_grad=True)
    gy = torch.randn(n, H, device="cuda")
    grads = [torch.autograd.grad([sv.spec_embedding(w, tok)], [w], [gy])[0] for _ in range(3)]
    assert torch.equal(grads[0], grads[1]) and torch.equal(grads[0], grads[2])


def test_embedding_past_32_bits_of_offset():
    V, H = 262144, 8448
    w = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    w[-1] = 3.0
    w.requires_grad_()
    tok = torch.tensor([V - 1, 0, V - 1], dtype=torch.int32, device="cuda")
    y = sv.spec_embedding(w, tok, scale=2.0)
    assert (y[0] == 6).all() and (y[1] == 0).all() and (y[2] == 6).all()
    g, = torch.autograd.grad([y.sum()], [w])
    assert (g[-1] == 4).all() and (g[0] == 2).all() and g.count_nonzero() == 2 * H


def test_embedding_writes_nothing_behind_its_outputs():
    lib = sv.load_library()
    st = torch.cuda.current_stream().cuda_stream
    for n, V, H, dt, code in ((5, 9, 24, torch.bfloat16, 1), (70, 33, 7, torch.float32, 0)):
        w, gy = torch.randn(V, H, device="cuda").to(dt), torch.randn(n, H, device="cuda").to(dt)
        tok = torch.randint(0, V, (n,), dtype=torch.int32, device="cuda")
        out = torch.full((n * H + 512,), 7.0, dtype=dt, device="cuda")
        assert lib.spec_embedding(w.data_ptr(), code, tok.data_ptr(), 1.0, n, V, H, out.data_ptr(), st) == 0
        size = lib.spec_embedding_grad_workspace_bytes(code, n, V, H)
        ws = torch.full((size + 256,), 3, dtype=torch.uint8, device="cuda")
        gw = torch.full((V * H + 512,), 7.0, dtype=dt, device="cuda")
        assert lib.spec_embedding_grad(tok.data_ptr(), gy.data_ptr(), code, 1.0, n, V, H, gw.data_ptr(), ws.data_ptr(), size, st) == 0
        torch.cuda.synchronize()
        assert (out[n * H:] == 7).all() and (gw[V * H:] == 7).all() and (ws[size:] == 3).all()
