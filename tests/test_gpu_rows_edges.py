"""Edges of spec_token_logprobs and spec_draft_kl: gradients of any weight on
masked rows, terms at the ends of the exponent range.  Against float64, with
the bounds of test_gpu_rows.py.
"""
import math

import pytest
import torch

import draft_verification_row_amd as sv
from test_gpu_rows import DT, Ref, check_kl, close, half, pair, rows_of, tokens_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weight", [1.2, 1.5, 100.0, 65536.0, 1e30])
@pytest.mark.parametrize("V", [33, 16500])
def test_entropy_gradient_of_any_weight(V, weight, dtype):
    """Entropy gradients of either sign on rows with -inf and the type's lowest
    value in places: 0 where p = 0, the formula elsewhere."""
    dt = DT[dtype]
    X = rows_of(8, V, dt, seed=9).clone()
    tok = tokens_of(8, V, 9)
    X[0:2, ::3] = -math.inf
    X[2:4, ::2] = torch.finfo(dt).min
    X[4:6, : V - 2] = -math.inf
    X[6:8] = torch.finfo(dt).min
    X[6:8, 5] = 3.0
    X.requires_grad_()
    ref = Ref(X, tok)
    ge = weight * torch.tensor([1.0, -1.0], device="cuda").repeat(4)
    gl = torch.linspace(-1, 1, 8, device="cuda")
    r = sv.spec_token_logprobs(X, tok)
    for a in (gl, None):
        outs, ws = ([r.logprob, r.entropy], [gl, ge]) if a is not None else ([r.entropy], [ge])
        got, = torch.autograd.grad(outs, [X], ws, retain_graph=True)
        want, err = ref.grad(torch.zeros_like(gl) if a is None else a, ge)
        close(got, want, err + half(dt) * want.abs() + 1e-38, "grad")
        # a masked place's gradient is exactly 0, but for the row's own token
        masked = (ref.p == 0).scatter(1, ref.at, False)
        assert (got[masked] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_entropy_gradient_of_a_scaled_loss(dtype):
    """(2 * entropy).sum().backward() under a sampling mask."""
    X = rows_of(4, 5000, DT[dtype], seed=2).clone()
    X[:, 100:] = -math.inf
    X.requires_grad_()
    (2 * sv.spec_token_logprobs(X, tokens_of(4, 100, 3)).entropy).sum().backward()
    assert X.grad.isfinite().all() and (X.grad[:, 100:] == 0).all() and (X.grad[:, :100] != 0).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_rows_have_nan_gradients(dtype):
    """A NaN logit stays visible in its own row's gradient, and in no other."""
    X = rows_of(3, 4000, DT[dtype], seed=4).clone()
    X[1, 7] = math.nan
    X[:, 9] = -math.inf
    X.requires_grad_()
    r = sv.spec_token_logprobs(X, tokens_of(3, 4000, 5))
    g, = torch.autograd.grad((r.logprob + 3 * r.entropy).sum(), [X])
    assert g[1].isnan().all() and g[0].isfinite().all() and g[2].isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gap", [60, 100, 500, 704, 800, 1024])
@pytest.mark.parametrize("V", [40, 20000, 128256])
def test_kl_of_an_excluded_unlikely_token(V, gap, dtype):
    """A draft's -inf on a token that lies `gap` nats under the target's
    largest, first, in the middle and last of the row, alone there and among
    others as unlikely: infinite while the target's p is positive as a
    double."""
    T, D = (t.clone() for t in pair(1, 6, 6, V, DT[dtype], 3))
    top = T.float().amax(-1)
    for k, at in enumerate((0, V // 2, V - 1)):
        T[0, k, at] = top[0, k] - gap
        D[0, k, at] = -math.inf
    for k, part in ((3, slice(0, V // 2)), (4, slice(V // 4, V - 2))):
        T[0, k, part] = T[0, k].float().amax() - gap  # the part's own largest
        T[0, k, V - 1] = T[0, k].float().amax() + gap
        D[0, k, V // 4 + 1] = -math.inf
    T[0, 5, 3] = torch.finfo(DT[dtype]).min  # the usual masks of either side
    D[0, 5, 3] = -math.inf
    kl, _ = check_kl(T, D)
    assert kl[0, 5].isfinite()
    assert (kl[0, :3] == math.inf).all() if gap < 740 else kl[0, :3].isfinite().all()


def test_kl_infinities_of_split_and_unsplit_rows():
    """The same rows one at a time, split over workgroups, and 600 at once."""
    V = 32000
    T, D = (t.clone() for t in pair(1, 600, 600, V, torch.bfloat16, 5))
    T[0, :, 17] = -120.0
    D[0, ::2, 17] = -math.inf
    kl = sv.spec_draft_kl(T, D)
    assert (kl[0, ::2] == math.inf).all() and kl[0, 1::2].isfinite().all()
    for k in (0, 1, 598, 599):
        one = sv.spec_draft_kl(T[:, k:k + 1].contiguous(), D[:, k:k + 1].contiguous())
        assert torch.isposinf(one[0, 0]) == torch.isposinf(kl[0, k])


# Rows of n equal maxima, whose sum is exactly n, with tokens d = -16 .. -20
# under them (multiples of 2^-6, so that d is exact), which add less than
# 2^-26 of it.  p = 2^(d log2 e) / n then has these errors: the product's
# rounding, half a step of [16, 32) times ln 2, 11.1 u; log2 e's own, 1.34e-8
# |d|, 4.5 u at -20; the exponential's step, 2 u; 1 / n and the last product,
# u each; the sum's, below u.
P_TOL = 21 * 2.0 ** -24


def flat_rows(rows, V, n, seed):
    at = torch.randperm(V, generator=torch.Generator().manual_seed(seed)).cuda()
    d = -16.0 - torch.arange(256, device="cuda") / 64
    X = torch.full((rows, V), -math.inf, device="cuda")
    X[:, at[:n]] = 3.0
    X[:, at[n:n + 256]] = 3.0 + d
    return X, at[n:n + 256], torch.exp(d.double()) / (n + torch.exp(d.double()).sum())


@pytest.mark.parametrize("n", [1000, 3001, 4095])
@pytest.mark.parametrize("rows", [1, 600])
def test_gradients_of_unlikely_tokens_are_good_to_their_exponent(rows, n):
    V = 8192
    X, at, p = flat_rows(rows, V, n, n)
    tok = torch.full((rows,), int((X[0] == 3.0).nonzero()[0]), dtype=torch.int32, device="cuda")
    X.requires_grad_()
    g, = torch.autograd.grad(sv.spec_token_logprobs(X, tok).logprob.sum(), [X])
    assert ((-g[:, at].double() - p).abs() <= P_TOL * p).all()
    T = torch.full((1, rows, V), -math.inf, device="cuda")
    T[:, :, tok[0]] = 1.0
    gd, = torch.autograd.grad(sv.spec_draft_kl(T, X[None]).sum(), [X])
    assert ((gd[:, at].double() - p).abs() <= P_TOL * p).all()


@pytest.mark.parametrize("rows", [1, 600])
@pytest.mark.parametrize("n,more", [(1000, 24), (3000, 1), (4000, 96), (1, 1), (7, 4000)])
def test_kl_of_flat_rows_is_good_to_its_quotient(rows, n, more):
    """Uniform over n tokens against uniform over n + more: ln(1 + more / n),
    off by the quotient's half step and the logarithm's own steps."""
    V = 8192
    T, D = torch.full((2, 1, rows, V), -math.inf, device="cuda")
    D[..., 50:50 + n + more] = -2.0
    T[..., 51:51 + n] = 5.0
    want = math.log1p(more / n)
    kl = sv.spec_draft_kl(T, D).double()
    assert ((kl - want).abs() <= 2.0 ** -24 * (1 + 4 * want)).all()
