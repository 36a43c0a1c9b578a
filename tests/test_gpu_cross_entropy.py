"""spec_cross_entropy against its definition in float64, forward and gradients.

Tolerances.  u = 2^-24, h half a step of a type.  A logit's product summed in
float32 in any order is off by at most e = (K + 9) 2u (sum |x| |w| + |b|) (2u a
step: the matrix instructions need not round to nearest); E is a row's largest.
The sum of exponentials joins at most 400 values one after the other along any
path, each of whose exponents rounds by a few u of its size, and |d| e^-|d| < 1:
it is off by at most 600 u of itself.  So the log-sum-exp is off by E + 600 u and
its own rounding, the loss by 2 E + 600 u and its roundings, and p, relative, by
e + E + u (600 + 6 |ln p|).  dz is rounded to the type (not for the bias), and
the gradients' products are sums as above.
"""
import math

import pytest
import torch

import draft_verification_row_amd as sv
from test_gpu_embedding import DT, U, at_offset, close, half

pytestmark = pytest.mark.gpu


def make(M, V, K, dt, bias, masked, pad, seed, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = r(V, K) * 2 / math.sqrt(K)
    tok = torch.randint(0, V, (M,), generator=g, device="cuda")
    x = r(M, K) + 3 * torch.rand(M, 1, generator=g, device="cuda") * w[tok]
    b = r(V) * 0.5 if bias else None
    if masked:
        b[torch.rand(V, generator=g, device="cuda") < masked] = -math.inf
    tok = tok.masked_fill(torch.rand(M, generator=g, device="cuda") < pad, -1).int()
    t = [at_offset(v.to(dt), off) if v is not None else None for v in (x, w, b)]
    return t, tok, r(M).abs() + 0.1, r(M)


def check(M, V, K, dtype="bf16", bias=False, masked=0.0, pad=0.2, lse=True, backward=True, seed=0, off=0, edit=None):
    dt = DT[dtype]
    h = half(dt)
    (x, w, b), tok, gl, ge = make(M, V, K, dt, bias, masked, pad, seed + M + V + K, off)
    if edit:
        edit(x, w, b, tok)
    live = [t.requires_grad_() for t in (x, w, b) if t is not None] if backward else []
    out = sv.spec_cross_entropy(x, w, tok, b)
    assert out.loss.shape == out.lse.shape == (M,) and (out.status == 0).all()
    xd, wd = x.detach().double(), w.detach().double()
    bd = b.detach().double() if bias else torch.zeros(V, device="cuda", dtype=torch.float64)
    on = tok >= 0
    at = tok.long().clamp_min(0)[:, None]
    xd = torch.where(on[:, None], xd, 0.0)
    z = xd @ wd.t() + bd
    some = bd > -math.inf
    e = 2 * U * (K + 9) * (xd.abs() @ wd.abs().t() + bd.masked_fill(~some, 0.0).abs())
    E = torch.where(some, e, 0.0).amax(1)
    n = torch.logsumexp(z, 1)
    zt = z.gather(1, at)[:, 0]
    loss = torch.where(zt == -math.inf, math.inf, n - zt)  # also where nothing is left
    loss = torch.where(on, loss, 0.0)
    n = torch.where(on, n, 0.0)
    fine = loss.isfinite()
    size = n.masked_fill(~n.isfinite(), 0.0).abs()
    assert torch.equal(out.loss[~fine].double(), loss[~fine]) and torch.equal(out.lse[~n.isfinite()].double(), n[~n.isfinite()])
    close(out.lse[n.isfinite()], n[n.isfinite()], (E + U * (600 + 4 * size))[n.isfinite()], "lse")
    close(out.loss[fine], loss[fine], (2 * E + U * (600 + 4 * size + 4 * loss.abs()))[fine], "loss")
    if not backward:
        return out
    ends, weights = ([out.loss, out.lse], [gl, ge]) if lse else ([out.loss], [gl])
    got = torch.autograd.grad(ends, live, weights)
    real = on & n.isfinite()
    one = torch.where(real, gl.double(), 0.0)[:, None]
    both = one + (torch.where(real, ge.double(), 0.0)[:, None] if lse else 0.0)
    lp = torch.where(real[:, None] & some, z - n[:, None], -math.inf)
    p = torch.exp(lp)
    dz = both * p
    edz = both.abs() * p * (e + E[:, None] + U * (600 + 6 * torch.where(p > 0, lp.abs(), 0.0))) + 4 * U * dz.abs()
    dz = dz.scatter_add(1, at, -one)
    edz = edz.scatter_add(1, at, 4 * U * one)
    if bias:
        err = edz.sum(0) + U * (M + 8) * (dz.abs() + edz).sum(0)
        want = dz.sum(0)
        close(got[2], want, err + h * (want.abs() + err) + 1e-37, "grad bias")
    edz = edz + h * (dz.abs() + edz) + 1e-40
    full = dz.abs() + edz
    want, err = dz @ wd, edz @ wd.abs() + 2 * U * (V + 8) * (full @ wd.abs())
    close(got[0], want, err + h * (want.abs() + err) + 1e-37, "grad x")
    assert (got[0][~real] == 0).all()
    want, err = dz.t() @ xd, edz.t() @ xd.abs() + 2 * U * (M + 8) * (full.t() @ xd.abs())
    close(got[1], want, err + h * (want.abs() + err) + 1e-37, "grad weight")
    return out


SIZES = [(1, 1, 1), (1, 7, 3), (2, 64, 64), (3, 1000, 31), (6, 5000, 256), (31, 129, 72), (33, 640, 40), (64, 512, 128),
         (65, 130, 130), (100, 1001, 777), (127, 255, 127), (128, 128, 128), (129, 257, 264), (300, 700, 520), (513, 384, 192),
         (1025, 300, 8), (2000, 50, 24)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,V,K", SIZES)
def test_entropy_sizes(M, V, K, dtype):
    check(M, V, K, dtype, bias=(M + K) % 2 == 0, lse=V % 2 == 0, pad=0.3 if M > 3 else 0.0)


@pytest.mark.parametrize("dtype,off", [("bf16", 1), ("bf16", 4), ("f32", 1)])
@pytest.mark.parametrize("M,V,K", [(2, 72, 64), (40, 130, 96), (270, 264, 128)])
def test_entropy_alignment(M, V, K, dtype, off):
    check(M, V, K, dtype, bias=True, off=off)


# every tile of each product, whole and ragged, and rows that are padded first
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,V,K", [(1, 32000, 256), (48, 20000, 512), (700, 4096, 2048), (2048, 8192, 128), (2050, 8001, 1032),
                                   (4096, 4097, 4096), (1500, 2000, 777), (66, 33000, 64)])
def test_entropy_larger(M, V, K, dtype):
    check(M, V, K, dtype, bias=M % 4 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,V,K", [(6, 100, 8000), (40, 1000, 5001), (100, 300, 4096), (300, 1501, 8192)])
def test_entropy_few_tiles_split(M, V, K, dtype):
    """Few logits of long sums: K over several workgroups."""
    check(M, V, K, dtype, bias=True, masked=0.2)
    check(M, V, K, dtype)


@pytest.mark.parametrize("dtype,V", [("bf16", 50001), ("f32", 30000)])
def test_entropy_in_pieces_of_the_vocabulary(dtype, V):
    """More than 512 MiB of dz: the second piece adds to x's gradient."""
    check(8192, V, 64, dtype, bias=True, pad=0.0)


@pytest.mark.parametrize("M", [5, 50, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_entropy_masks(M, dtype):
    """-inf in the bias: tokens out of the vocabulary, the rows' own among them
    (loss +inf), and everything (rows of -inf alone)."""
    check(M, 700, 64, dtype, bias=True, masked=0.4)

    def nothing(x, w, b, tok):
        b.fill_(-math.inf)

    out = check(M, 300, 64, dtype, bias=True, edit=nothing)
    on = out.lse != 0
    assert on.any() and (out.loss[on] == math.inf).all() and (out.lse[on] == -math.inf).all()

    def one_left(x, w, b, tok):
        b.fill_(-math.inf)
        b[77] = 1.0
        tok.fill_(77)

    out = check(M, 300, 64, dtype, bias=True, edit=one_left)
    assert (out.loss == 0).all()
    lowest = torch.finfo(DT[dtype]).min  # an ordinary logit
    x, w, b = make(M, 300, 64, DT[dtype], True, 0, 0, 3)[0]
    b.fill_(lowest)
    x.zero_()
    tok = torch.arange(M, device="cuda").int() % 300
    out = sv.spec_cross_entropy(x, w, tok, b)
    assert (out.loss - math.log(300)).abs().max() < 1e-5 and (out.lse == lowest).all()


@pytest.mark.parametrize("M", [5, 50, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_entropy_padded_rows_are_not_used(M, dtype):
    """NaN in the rows of padded tokens changes nothing; all rows padded."""
    def poison(x, w, b, tok):
        x[tok < 0] = math.nan

    check(M, 400, 72, dtype, pad=0.5, edit=poison)

    def all_padded(x, w, b, tok):
        x.fill_(math.inf)
        tok.fill_(-1)

    check(M, 400, 72, dtype, bias=True, edit=all_padded)


def test_entropy_special_values():
    for M in (5, 300):
        x = torch.randn(M, 64, device="cuda")
        w = torch.randn(700, 64, device="cuda")
        tok = torch.randint(0, 700, (M,), device="cuda", dtype=torch.int32)
        clean = sv.spec_cross_entropy(x, w, tok)
        x[2, 5] = math.nan
        out = sv.spec_cross_entropy(x, w, tok)
        keep = [i for i in range(M) if i != 2]
        assert out.loss[2].isnan() and out.lse[2].isnan()
        assert torch.equal(out.loss[keep], clean.loss[keep]) and torch.equal(out.lse[keep], clean.lse[keep])


def test_entropy_tokens_outside():
    for M in (6, 200):
        x = torch.randn(M, 40, device="cuda", requires_grad=True)
        w = torch.randn(30, 40, device="cuda", requires_grad=True)
        tok = torch.randint(0, 30, (M,), device="cuda", dtype=torch.int32)
        tok[0], tok[1], tok[2], tok[3] = 30, -2, 2 ** 31 - 1, -1
        out = sv.spec_cross_entropy(x, w, tok)
        assert out.status.tolist() == [1, 1, 1] + [0] * (M - 3)
        assert (out.loss[:4] == 0).all() and (out.lse[:4] == 0).all() and (out.loss[4:] > 0).all()
        gx, gw = torch.autograd.grad([out.loss.sum()], [x, w])
        assert (gx[:4] == 0).all() and (gx[4:] != 0).any(1).all() and gw.isfinite().all()


def test_entropy_shapes_and_single_gradients():
    x, w, b = torch.randn(2, 3, 40, device="cuda"), torch.randn(50, 40, device="cuda"), torch.randn(50, device="cuda")
    tok = torch.randint(0, 50, (2, 3), device="cuda", dtype=torch.int32)
    full = [t.clone().requires_grad_() for t in (x, w, b)]
    out = sv.spec_cross_entropy(full[0], full[1], tok, full[2])
    assert out.loss.shape == out.lse.shape == out.status.shape == (2, 3)
    want = torch.autograd.grad([out.loss.sum()], full)  # an expanded gradient
    for i in range(3):
        one = [t.clone().requires_grad_(j == i) for j, t in enumerate((x, w, b))]
        got, = torch.autograd.grad([sv.spec_cross_entropy(one[0], one[1], tok, one[2]).loss.sum()], [one[i]])
        assert torch.equal(got, want[i]), i
    assert torch.equal(sv.spec_cross_entropy(x, w, tok, b).loss, out.loss)
    alone = sv.spec_cross_entropy(x[0, 0], w, tok[0, 0], b)
    assert alone.loss.shape == ()
    # the log-sum-exp's gradient alone: softmax
    xs = x.clone().requires_grad_()
    g, = torch.autograd.grad([sv.spec_cross_entropy(xs, w, tok, b).lse.sum()], [xs])
    p = torch.softmax((x.double() @ w.double().t() + b), -1)
    assert (g - p @ w.double()).abs().max() < 1e-4


def test_entropy_no_rows():
    x = torch.empty(0, 40, device="cuda", requires_grad=True)
    w = torch.randn(20, 40, device="cuda", requires_grad=True)
    out = sv.spec_cross_entropy(x, w, torch.empty(0, dtype=torch.int32, device="cuda"))
    out.loss.sum().backward()
    assert out.loss.shape == (0,) and x.grad.shape == (0, 40) and (w.grad == 0).all()


def test_entropy_agrees_with_the_logits_operators():
    """The same rows by spec_linear and spec_token_logprobs: both sums are float32's."""
    (x, w, b), tok, _, _ = make(90, 3000, 128, torch.float32, True, 0, 0.2, 1)
    out = sv.spec_cross_entropy(x, w, tok, b)
    lp = sv.spec_token_logprobs(sv.spec_linear(x, w, b), tok)
    assert (out.loss + lp.logprob).abs().max() < 1e-4


def test_entropy_gradient_against_differences():
    M, V, K, h = 6, 50, 70, 1e-4
    (x, w, b), tok, gl, ge = make(M, V, K, torch.float32, True, 0, 0.0, 5)
    live = [t.requires_grad_() for t in (x, w, b)]
    out = sv.spec_cross_entropy(x, w, tok, b)
    grads = torch.autograd.grad([out.loss, out.lse], live, [gl, ge])
    dirs = [torch.randn(v.shape, device="cuda").double() for v in live]

    def f(s):
        xs, ws, bs = (v.detach().double() + s * d for v, d in zip(live, dirs))
        z = xs @ ws.t() + bs
        n = torch.logsumexp(z, 1)
        return ((n - z.gather(1, tok.long()[:, None])[:, 0]) * gl.double() + n * ge.double()).sum()

    want = float((f(h) - f(-h)) / (2 * h))
    got = float(sum((g.double() * d).sum() for g, d in zip(grads, dirs)))
    assert abs(got - want) < 1e-2 + 1e-5 * abs(want)


def test_entropy_writes_nothing_behind_its_outputs():
    lib = sv.load_library()
    st = torch.cuda.current_stream().cuda_stream
    for M, V, K in ((3, 70, 64), (130, 129, 72), (300, 264, 129), (70, 5001, 200)):
        (x, w, b), tok, gl, ge = make(M, V, K, torch.bfloat16, True, 0, 0.3, 1)
        f = lambda n, dt=torch.float32: torch.full((n + 512,), 7, dtype=dt, device="cuda")  # noqa: E731
        loss, lse, status, stats = f(M), f(M), f(M, torch.int32), f(2 * M)
        grads = [f(n, torch.bfloat16) for n in (M * K, V * K, V)]
        n1, n2 = lib.spec_cross_entropy_workspace_bytes(1, M, V, K), lib.spec_cross_entropy_grad_workspace_bytes(1, M, V, K)
        w1, w2 = (torch.full((n + 256,), 3, dtype=torch.uint8, device="cuda") for n in (n1, n2))
        assert lib.spec_cross_entropy(x.data_ptr(), w.data_ptr(), b.data_ptr(), 1, tok.data_ptr(), M, V, K, loss.data_ptr(),
                                      lse.data_ptr(), status.data_ptr(), stats.data_ptr(), w1.data_ptr(), n1, st) == 0
        assert lib.spec_cross_entropy_grad(x.data_ptr(), w.data_ptr(), b.data_ptr(), 1, tok.data_ptr(), stats.data_ptr(), gl.data_ptr(),
                                           ge.data_ptr(), M, V, K, *(g.data_ptr() for g in grads), w2.data_ptr(), n2, st) == 0
        torch.cuda.synchronize()
        for t, n in ((loss, M), (lse, M), (status, M), (stats, 2 * M), (grads[0], M * K), (grads[1], V * K), (grads[2], V)):
            assert (t[n:] == 7).all()
        assert (w1[n1:] == 3).all() and (w2[n2:] == 3).all()


def test_entropy_past_32_bits_of_offset():
    """A weight of more than 2^31 elements."""
    V, K = 262144, 8448
    w = torch.zeros(V, K, dtype=torch.bfloat16, device="cuda")
    w[-1] = 0.01
    for M in (2, 80):
        x = torch.ones(M, K, dtype=torch.bfloat16, device="cuda").requires_grad_()
        ws = w.detach().requires_grad_()
        out = sv.spec_cross_entropy(x, ws, torch.full((M,), V - 1, dtype=torch.int32, device="cuda"))
        z = float(w[-1, 0]) * K
        lse = math.log(math.exp(z) + V - 1)
        assert (out.lse - lse).abs().max() < 1e-3 and (out.loss - (lse - z)).abs().max() < 1e-3
        gx, gw = torch.autograd.grad([out.loss.sum()], [x, ws])
        p = math.exp(z - lse)
        assert (gx.float() - (p - 1) * float(w[-1, 0])).abs().max() < 1e-4
        assert (gw[-1].float() - M * (p - 1)).abs().max() < M * 0.01 and (gw[5] != 0).all()
