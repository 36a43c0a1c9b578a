"""spec_linear against its definition in float64, forward and gradients.

Tolerances.  u = 2^-24, h half a step of a type.  A product summed in float32
in any order is off by at most (K + 8) 2u sum |x| |w| (2u a step: the matrix
instructions need not round to nearest).  The activations have slopes of at
most 1.13 and are evaluated to a few u of |z| + 1.  For the gradients, z is
kept in the operands' type and dz rounded to it: with |act''| <= 0.8, dz is
off by |dy| (0.8 (h |z| + its own error) + 8 u) + h |dz|, and the products'
errors follow from their definition.
"""
import math

import pytest
import torch

import draft_verification_row_amd as sv

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "gelu", "silu"]


def half(dt):
    return torch.finfo(dt).eps / 2


def act(z, name):
    return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * 0.5 * torch.erfc(-z / math.sqrt(2))}[name]()


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def at_offset(t, off):
    buf = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
    buf[off:] = t.reshape(-1)
    return buf[off:].view(t.shape)


def make(M, N, K, dt, ot, bias, residual, seed, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = dict(x=r(M, K).to(dt), w=(r(N, K) / math.sqrt(K)).to(dt), b=(r(N) * 0.5).to(dt) if bias else None,
             r=r(M, N).to(ot) if residual else None)
    t = {k: v if v is None else at_offset(v, off) for k, v in t.items()}
    return t, r(M, N).to(ot)


def close(got, want, tol, what):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), want[bad][:3].tolist())


def check(M, N, K, dtype="bf16", out=None, activation="none", bias=False, residual=False, backward=True, seed=0,
          off=0):
    dt = DT[dtype]
    ot = DT[out] if out else dt
    t, gy = make(M, N, K, dt, ot, bias, residual, seed + M + N + K, off)
    live = {k: v.requires_grad_(backward) for k, v in t.items() if v is not None}
    y = sv.spec_linear(t["x"], t["w"], t["b"], residual=t["r"], activation=activation, out_dtype=ot)
    assert y.dtype == ot and y.shape == (M, N)
    x, w = t["x"].detach().double(), t["w"].detach().double()
    b = t["b"].detach().double() if bias else torch.zeros(N, device="cuda", dtype=torch.float64)
    r = t["r"].detach().double() if residual else 0.0
    z = x @ w.t() + b
    ez = 2 * U * ((K + 8) * (x.abs() @ w.abs().t()) + b.abs() + z.abs())
    f = act(z, activation)
    want = f + r
    ey = 1.13 * ez + 8 * U * (z.abs() + 1) + 2 * U * want.abs()
    close(y, want, ey + half(ot) * (want.abs() + ey), "y")
    if not backward:
        return y
    names = list(live)
    got = dict(zip(names, torch.autograd.grad([y], [live[n] for n in names], [gy])))
    dy = gy.double()
    s = slope(z, activation)
    dz = dy * s
    h = half(dt)
    if activation == "none":
        edz = h * dz.abs()
    elif activation == "relu":
        near = z.abs() <= ez + h * z.abs() * 2  # may fall on either side of 0
        edz = h * dz.abs() + torch.where(near & (z.abs() < 1e-3), dy.abs(), 0.0)
    else:
        edz = dy.abs() * (0.8 * (h * z.abs() + ez * 1.01) + 8 * U * (1 + z.abs())) * 1.01 + 1.01 * h * dz.abs()
    full = dz.abs() + edz

    def one(name, val, err):
        close(got[name], val, err + h * (val.abs() + err) + 1e-37, "grad " + name)

    one("x", dz @ w, edz @ w.abs() + 2 * U * (N + 8) * (full @ w.abs()))
    one("w", dz.t() @ x, edz.t() @ x.abs() + 2 * U * (M + 8) * (full.t() @ x.abs()))
    if bias:
        one("b", dz.sum(0), edz.sum(0) + U * (M + 8) * full.sum(0))
    if residual:
        assert torch.equal(got["r"], gy)
    return y


SIZES = [(1, 1, 1), (1, 7, 3), (2, 64, 64), (3, 100, 31), (1, 4096, 4096), (5, 1000, 513), (16, 256, 128),
         (17, 129, 257), (33, 640, 72), (64, 512, 1024), (65, 130, 130), (100, 1001, 777), (127, 255, 127),
         (128, 128, 128), (129, 257, 264), (256, 256, 64), (300, 700, 520), (513, 384, 192), (1025, 300, 8)]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_sizes(M, N, K, dtype, out):
    check(M, N, K, dtype, out, ACTS[(M + N) % 4], bias=(M + K) % 2 == 0, residual=N % 2 == 0)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("M,N,K", [(4, 96, 160), (140, 264, 136), (300, 520, 96)])
def test_linear_epilogues(M, N, K, activation, dtype, out):
    for bias in (False, True):
        for residual in (False, True):
            check(M, N, K, dtype, out, activation, bias, residual, seed=bias + 2 * residual)


@pytest.mark.parametrize("dtype,off", [("bf16", 1), ("bf16", 4), ("f32", 1)])
@pytest.mark.parametrize("M,N,K", [(2, 72, 64), (40, 130, 96), (270, 264, 128)])
def test_linear_alignment(M, N, K, dtype, off):
    """Operands whose memory starts at any element."""
    check(M, N, K, dtype, None, "silu", True, True, off=off)


@pytest.mark.parametrize("M,N,K", [(1, 128256, 256), (32, 32000, 512), (700, 4096, 2048), (2048, 2304, 1024), (4096, 512, 512),
                                   (1500, 2000, 777), (4000, 4100, 131)])
def test_linear_larger(M, N, K):
    check(M, N, K, "bf16", "bf16", "silu", True, True)


def test_linear_long_sums():
    check(3, 40, 100000, "bf16", "f32", "none", backward=True)
    check(100000, 24, 16, "bf16", "bf16", "gelu", bias=True)
    check(70, 90, 50001, "f32", "f32", "none", backward=False)


def test_linear_few_tiles_split():
    """Few outputs of a long sum: K over several workgroups."""
    for M, N, K in ((100, 300, 4000), (70, 129, 5001), (65, 64, 16384)):
        check(M, N, K, "bf16", "bf16", "gelu", True, True)
        check(M, N, K, "f32", "f32", "silu", True, True)
    check(300, 6, 9000, "bf16", "f32", "relu", True, False)


def test_linear_special_values():
    """NaN and infinities stay in their rows; activations at the ends."""
    x = torch.randn(5, 64, device="cuda").bfloat16()
    w = torch.randn(70, 64, device="cuda").bfloat16()
    clean = sv.spec_linear(x, w, activation="relu")
    x[2, 5] = math.nan
    y = sv.spec_linear(x, w, activation="relu")
    keep = [0, 1, 3, 4]
    assert y[2].isnan().all() and torch.equal(y[keep], clean[keep])
    big = torch.tensor([[-300.0], [-20.0], [0.0], [20.0], [300.0]], device="cuda")
    one = torch.ones(1, 1, device="cuda")
    for name in ("silu", "gelu"):
        b = big.clone().requires_grad_()
        v = sv.spec_linear(b, one, activation=name)
        g, = torch.autograd.grad([v.sum()], [b])
        assert (v.double() - act(big.double(), name)).abs().max() < 1e-5
        assert (g.double() - slope(big.double(), name)).abs().max() < 1e-5


def test_linear_shapes_and_single_gradients():
    x = torch.randn(2, 3, 40, device="cuda", requires_grad=True)
    w = torch.randn(20, 40, device="cuda")
    y = sv.spec_linear(x, w)
    assert y.shape == (2, 3, 20)
    y.sum().backward()  # an expanded gradient; only x's is wanted
    assert (x.grad - w.sum(0)).abs().max() < 1e-4
    wg = w.clone().requires_grad_()
    sv.spec_linear(x.detach(), wg, activation="silu").square().sum().backward()
    xd, wd = x.detach().double().view(6, 40), w.double()
    z = xd @ wd.t()
    want = (2 * act(z, "silu") * slope(z, "silu")).t() @ xd
    assert (wg.grad.double() - want).abs().max() < 1e-3
    vec = sv.spec_linear(x[0, 0].detach(), w)
    assert vec.shape == (20,)


def test_linear_no_rows():
    x = torch.empty(0, 40, device="cuda", requires_grad=True)
    w = torch.randn(20, 40, device="cuda", requires_grad=True)
    b = torch.randn(20, device="cuda", requires_grad=True)
    y = sv.spec_linear(x, w, b, activation="gelu")
    assert y.shape == (0, 20)
    y.sum().backward()
    assert x.grad.shape == (0, 40) and (w.grad == 0).all() and (b.grad == 0).all()


def test_linear_gradient_against_differences():
    """Directional derivatives by central differences of the float64
    definition; the third derivatives are of order K^1.5 v^3 / M."""
    M, N, K, h = 6, 50, 70, 1e-4
    t, gy = make(M, N, K, torch.float32, torch.float32, True, True, 5)
    live = [t[k].requires_grad_() for k in "xwbr"]
    y = sv.spec_linear(live[0], live[1], live[2], residual=live[3], activation="silu")
    grads = torch.autograd.grad([y], live, [gy])
    dirs = [torch.randn(v.shape, device="cuda").double() for v in live]

    def f(s):
        x, w, b, r = (v.detach().double() + s * d for v, d in zip(live, dirs))
        return ((act(x @ w.t() + b, "silu") + r) * gy.double()).sum()

    slope_fd = float((f(h) - f(-h)) / (2 * h))
    got = float(sum((g.double() * d).sum() for g, d in zip(grads, dirs)))
    assert abs(got - slope_fd) < 1e-2 + 1e-5 * abs(slope_fd)


def test_linear_captured_and_replayed():
    """Forward and backward in a graph, with eager calls between its replays."""
    t, gy = make(150, 200, 136, torch.bfloat16, torch.bfloat16, True, True, 3)
    live = [t[k].requires_grad_() for k in "xwbr"]

    def work():
        y = sv.spec_linear(live[0], live[1], live[2], residual=live[3], activation="gelu")
        one = sv.spec_linear(live[0][:2].detach(), live[1].detach())
        return [v.detach() for v in (y, one, *torch.autograd.grad([y], live, [gy]))]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        eager = [v.clone() for v in work()]
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = work()
    for rep in range(3):
        for v in outs[:-1]:  # the last is the gradient of y itself
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, outs):
            assert torch.equal(a, b), rep
        check(40, 64, 64)


def test_linear_capture_is_refused_while_an_eager_graph_lives():
    t, _ = make(8, 16, 32, torch.bfloat16, torch.bfloat16, True, False, 3)
    live = [t[k].requires_grad_() for k in "xwb"]
    kept = sv.spec_linear(*live, activation="silu")
    g = torch.cuda.CUDAGraph()
    with pytest.raises(sv.SpecVerifyError):
        with torch.cuda.graph(g):
            sv.spec_linear(*live)
    torch.cuda.synchronize()
    kept.sum().backward()
    assert all(v.grad.isfinite().all() for v in live)


def test_linear_repeatable_on_two_streams():
    a, _ = make(64, 4096, 4096, torch.bfloat16, torch.bfloat16, True, False, 3)
    first = sv.spec_linear(a["x"], a["w"], a["b"], activation="silu")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        outs = []
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(sv.spec_linear(a["x"], a["w"], a["b"], activation="silu"))
        torch.cuda.synchronize()
        assert torch.equal(outs[0], first) and torch.equal(outs[1], first)


def test_linear_writes_nothing_behind_its_output():
    lib = sv.load_library()
    for M, N, K in ((3, 70, 64), (130, 129, 72), (300, 264, 128)):
        x, w = torch.randn(M, K, device="cuda").bfloat16(), torch.randn(N, K, device="cuda").bfloat16()
        out = torch.full((M * N + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
        n = lib.spec_linear_workspace_bytes(1, M, N, K)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        assert lib.spec_linear(x.data_ptr(), w.data_ptr(), None, None, 1, 1, 0, M, N, K, out.data_ptr(), None,
                               ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert (out[M * N:] == 7).all()


def test_linear_past_32_bits_of_offset():
    """A weight of more than 2^31 elements, and an output of as many."""
    N, K = 262144, 8448
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    w[-1], w[5] = 1.0, 2.0
    x = torch.ones(2, K, dtype=torch.bfloat16, device="cuda")
    y = sv.spec_linear(x, w, out_dtype=torch.float32)
    assert (y[:, -1] == K).all() and (y[:, 5] == 2 * K).all() and y.count_nonzero() == 4
    del w
    M, N, K = 8400, 262144, 64
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-1] = 1.0
    w = torch.ones(N, K, dtype=torch.bfloat16, device="cuda")
    y = sv.spec_linear(x, w)
    assert (y[-1] == K).all() and (y[:-1].sum(0) == 0).all()
