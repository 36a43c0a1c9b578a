"""spec_token_logprobs and spec_draft_kl against their definitions in float64,
forward and gradient.

Tolerances.  u = 2^-24 is half a step of float32.  A row's sum of V terms
e^d, d = l - max <= 0, is added in chains of at most ceil(V / 256) + 16 terms
and each term carries its argument's rounding, |d| u, and a few u of the
exponential; so ln S is off by at most (chain + 8) u plus E|d| u, with E the
mean under p, and a log-prob by that and 2 |lp| u.  Sums weighted by |d| or
|u| scale alike.  A gradient's element is off by p times its bracket's error,
plus half a step of its type.
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


def rows_of(rows, V, dt, seed, offset=0, scale=2.5):
    """Contiguous logits that start `offset` elements into their memory."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, V, generator=g, device="cuda") * scale
    x[:, seed % V] += 6
    buf = torch.empty(rows * V + offset, dtype=dt, device="cuda")
    buf[offset:] = x.to(dt).reshape(-1)
    return buf[offset:].view(rows, V)


def tokens_of(rows, V, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    return torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)


class Ref:
    """The definitions in float64, and the bounds above."""

    def __init__(self, X, tokens):
        x = X.detach().double()
        V = x.shape[-1]
        m = x.amax(-1, keepdim=True)
        d = torch.where(m > -math.inf, x - m, torch.full_like(x, -math.inf))
        S = torch.exp(d).sum(-1, keepdim=True)
        self.lp = d - torch.log(S)  # of every token; an empty row has NaN
        self.p = torch.nan_to_num(torch.exp(self.lp), nan=0.0)
        plp = torch.where(self.p > 0, self.p * self.lp, 0.0)
        self.H = -plp.sum(-1)
        self.live = (tokens >= 0) & (tokens < V) & (m[:, 0] > -math.inf)
        self.skip = (tokens < 0) | (tokens >= V)
        at = tokens.clamp(0, V - 1).long()[:, None]
        self.logprob = torch.where(self.live, self.lp.gather(1, at)[:, 0], -math.inf)
        self.logprob[self.skip] = 0
        self.H = torch.where(self.live, self.H, 0.0)
        chain = math.ceil(V / 256) + 16
        ed = torch.where(self.p > 0, self.p * d.abs(), 0.0).sum(-1)
        self.tol = U * (chain + 8 + ed + 2 * self.lp.gather(1, at)[:, 0].abs().nan_to_num(posinf=0))
        self.tolH = U * 2 * (chain + 12) * (1 + ed)
        self.at = at

    def grad(self, gl, ge):
        gl = torch.where(self.live, gl.double(), 0.0)[:, None]
        ge = torch.where(self.live, ge.double(), 0.0)[:, None]
        plp = torch.where(self.p > 0, self.p * self.lp, 0.0)
        g = -gl * self.p - ge * (plp + self.p * self.H[:, None])
        g.scatter_add_(1, self.at, gl)
        lp = torch.where(self.p > 0, self.lp, 0.0).abs()
        bracket = gl.abs() + ge.abs() * (lp + self.H[:, None])
        tol = (self.tol[:, None] + (lp + 8) * U)
        err = self.p * (bracket * 2 * tol + ge.abs() * (tol + self.tolH[:, None])) + 4 * U * gl.abs() * self.p
        err.scatter_add_(1, self.at, 2 * U * gl.abs())
        return g, err


def close(got, want, tol, what):
    got, want = got.double(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~same & ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist())


def check_top(r, X, ref, top_n):
    """Alternatives: by value, then lowest index; -1 past the possible ones."""
    x = X.detach().double()
    V = x.shape[1]
    n = min(top_n, V)
    order = torch.sort(x + 0.0, dim=-1, descending=True, stable=True).indices[:, :n]
    lp = ref.lp.gather(1, order)
    some = ref.live[:, None] & (lp > -math.inf)
    want = torch.where(some, order, -1).to(torch.int32)
    assert torch.equal(r.top_tokens[:, :n], want), (r.top_tokens[:, :n] != want).nonzero()[:4]
    wlp = torch.where(some, lp, -math.inf)
    wlp[ref.skip] = 0
    tol = ref.tol[:, None] + 2 * U * torch.where(some, lp, 0.0).abs()
    close(r.top_logprob[:, :n], wlp, tol, "top_logprob")
    assert (r.top_tokens[:, n:] == -1).all()
    rest = torch.where(ref.skip, 0.0, -math.inf)[:, None].expand(-1, top_n - n)
    assert torch.equal(r.top_logprob[:, n:].double(), rest.double())


def check(X, tokens, top_n=0, backward=True, seed=0):
    X = X.detach().requires_grad_(backward)
    ref = Ref(X, tokens)
    r = sv.spec_token_logprobs(X, tokens, top_n=top_n)
    close(r.logprob, ref.logprob, ref.tol, "logprob")
    close(r.entropy, ref.H, ref.tolH, "entropy")
    check_top(r, X, ref, top_n)
    V = X.shape[1]
    assert torch.equal(r.status, ((tokens < -1) | (tokens >= V)).int())
    if backward:
        g = torch.Generator(device="cuda").manual_seed(seed)
        gl = torch.randn(X.shape[0], generator=g, device="cuda")
        ge = torch.randn(X.shape[0], generator=g, device="cuda")
        for a, b in ((gl, ge), (gl, None), (None, ge)):
            outs = [o for o, w in ((r.logprob, a), (r.entropy, b)) if w is not None]
            got, = torch.autograd.grad(outs, [X], [w for w in (a, b) if w is not None],
                                       retain_graph=True)
            zero = torch.zeros_like(gl)
            want, err = ref.grad(zero if a is None else a, zero if b is None else b)
            close(got, want, err + half(X.dtype) * want.abs() + 1e-38, "grad")
    return r


SIZES = [(1, 1), (3, 2), (2, 7), (5, 64), (1, 255), (4, 1001), (2, 8191), (3, 8192), (3, 8193),
         (2, 16384), (1, 50257), (6, 128256), (1, 262143), (1, 262144), (300, 513), (70, 32000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", SIZES)
def test_logprobs_sizes(rows, V, dtype):
    X = rows_of(rows, V, DT[dtype], seed=rows + V)
    check(X, tokens_of(rows, V, V), top_n=20)


@pytest.mark.parametrize("dtype,offset", [("bf16", 1), ("bf16", 3), ("bf16", 7), ("bf16", 8), ("f32", 1), ("f32", 3)])
@pytest.mark.parametrize("rows,V", [(3, 5), (4, 4099), (2, 40000), (3, 128256)])
def test_logprobs_alignment(rows, V, dtype, offset):
    """Logits whose first element and rows start at any element."""
    X = rows_of(rows, V, DT[dtype], seed=V, offset=offset)
    check(X, tokens_of(rows, V, V), top_n=5)


@pytest.mark.parametrize("top_n", [0, 1, 2, 5, 31, 32])
@pytest.mark.parametrize("rows,V", [(2, 3), (3, 33), (5, 20000), (1100, 1500)])
def test_logprobs_top_n(rows, V, top_n):
    check(rows_of(rows, V, torch.bfloat16, seed=top_n + V), tokens_of(rows, V, 3), top_n=top_n, backward=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 9000, 70001])
def test_logprobs_ties(V, dtype):
    """Equal logits everywhere, two values, +0 beside -0: lowest index first."""
    dt = DT[dtype]
    X = torch.zeros(5, V, dtype=dt, device="cuda")
    X[1, ::2] = -0.0
    X[2, V // 2:] = 1.0
    X[3, V - 3:] = 1.0
    X[4] = (torch.arange(V, device="cuda") % 7).to(dt)
    check(X, tokens_of(5, V, 5), top_n=32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [33, 16500, 128256])
def test_logprobs_masks(V, dtype):
    """-inf entries, one finite entry, a row of -inf, the type's lowest value
    in places and everywhere, a token under the mask."""
    dt = DT[dtype]
    low = torch.finfo(dt).min
    X = rows_of(7, V, dt, seed=9).clone()
    tok = tokens_of(7, V, 9)
    X[0, ::3] = -math.inf
    X[1] = -math.inf
    X[1, V - 1] = -4.0
    tok[1] = V - 1
    X[2] = -math.inf
    X[3, ::2] = low
    X[4] = low
    X[5, 5] = -math.inf
    tok[5] = 5
    X[6, : V - 2] = -math.inf
    r = check(X, tok, top_n=8)
    assert r.logprob[1] == 0 and r.entropy[1] == 0
    assert r.logprob[2] == -math.inf and r.entropy[2] == 0
    assert r.logprob[5] == -math.inf


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lanes", [(31, 7, 7, 7), (31, 31, 31, 31), (64, 0, 0, 0), (3, 0, 1, 9), (0, 0, 0, 1)])
def test_logprobs_uneven_masks(lanes, dtype):
    """Finite logits under a few of each wave's lanes only, so that the waves'
    bounds are loose and a tile may have more candidates than its list holds."""
    dt = DT[dtype]
    vec = 8 if dtype == "bf16" else 4
    V = 40000
    t = torch.arange(V, device="cuda") // vec % 256
    keep = torch.tensor(lanes, device="cuda")[t // 64] > t % 64
    X = rows_of(3, V, dt, seed=7).masked_fill(~keep, -math.inf)
    X[1] = torch.where(keep, 1.0, -math.inf).to(dt)   # all of them tied
    check(X.contiguous(), tokens_of(3, V, 7), top_n=32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 700])
def test_logprobs_rising_rows(rows, dtype):
    """Logits that rise along the row, in steps and strictly: every tile has
    better tokens than the last."""
    V = 30000
    x = torch.arange(V, device="cuda") / 500
    X = torch.stack([x, x.floor(), -x, x % 17] * ((rows + 3) // 4))[:rows].to(DT[dtype]).contiguous()
    check(X, tokens_of(rows, V, 3), top_n=32, backward=False)


@pytest.mark.parametrize("V", [100, 20001])
def test_logprobs_padded_rows_are_not_read(V):
    """Token -1: NaN and +inf logits behind it do not matter; a token outside
    the vocabulary is reported and treated alike."""
    X = rows_of(6, V, torch.bfloat16, seed=4).clone()
    tok = tokens_of(6, V, 4)
    X[1], tok[1] = math.nan, -1
    X[3], tok[3] = math.inf, -1
    X[4], tok[4] = math.nan, V
    tok[5] = -2
    r = sv.spec_token_logprobs(X.requires_grad_(), tok, top_n=3)
    g, = torch.autograd.grad(r.logprob.sum() + r.entropy.sum(), [X])
    for i in (1, 3, 4, 5):
        assert r.logprob[i] == 0 and r.entropy[i] == 0 and (g[i] == 0).all()
        assert (r.top_tokens[i] == -1).all() and (r.top_logprob[i] == 0).all()
    assert r.status.tolist() == [0, 0, 0, 0, 1, 1]
    assert g[0].isfinite().all() and (g[2] != 0).any()


@pytest.mark.parametrize("V", [50, 30000])
def test_logprobs_nan_rows(V):
    """A NaN or +inf makes its own row NaN, and no other."""
    X = rows_of(4, V, torch.float32, seed=6).clone()
    clean = sv.spec_token_logprobs(X, tokens_of(4, V, 6), top_n=4)
    X[1, V // 2] = math.nan
    X[2, 3] = math.inf
    r = sv.spec_token_logprobs(X, tokens_of(4, V, 6), top_n=4)
    assert r.logprob[1:3].isnan().all() and r.entropy[1:3].isnan().all()
    assert ((r.top_tokens >= -1) & (r.top_tokens < V)).all()
    for a, b in zip(r, clean):
        assert torch.equal(a[0], b[0]) and torch.equal(a[3], b[3])


def test_logprobs_leading_shapes_and_verify_output():
    """[B][K+1][V] logits with the verifier's own padded tokens."""
    B, K, V = 4, 3, 5000
    T, D = rows_of(B * (K + 1), V, torch.bfloat16, 1).view(B, K + 1, V), rows_of(B * K, V, torch.bfloat16, 2).view(B, K, V)
    x = tokens_of(B * K, V, 3).view(B, K)
    u = torch.rand(B, K + 1, device="cuda")
    v = sv.spec_verify_exact(T, D, x, u)
    r = sv.spec_token_logprobs(T, v.tokens, top_n=4)
    assert r.logprob.shape == (B, K + 1) and r.top_tokens.shape == (B, K + 1, 4)
    pad = v.tokens < 0
    assert pad.any() and (r.logprob[pad] == 0).all() and (r.status == 0).all()
    assert (r.logprob - v.target_logprob).abs().max() < 1e-4
    one = sv.spec_token_logprobs(T[0, 0], v.tokens[0, 0].reshape(()))  # no leading dimension
    assert one.logprob.shape == () and torch.allclose(one.logprob, r.logprob[0, 0])
    none = sv.spec_token_logprobs(T[:0], v.tokens[:0], top_n=2)        # no rows
    assert none.logprob.shape == (0, K + 1) and none.top_tokens.shape == (0, K + 1, 2)


@pytest.mark.parametrize("V", [257, 9001])
def test_logprobs_gradient_against_differences(V):
    """Directional derivatives of the float64 definition by central
    differences; h^2 times a third derivative of order 1 stays under 1e-6."""
    X = rows_of(3, V, torch.float32, seed=V)
    tok = tokens_of(3, V, V)
    Xg = X.clone().requires_grad_()
    r = sv.spec_token_logprobs(Xg, tok)
    g, = torch.autograd.grad(r.logprob.sum() + 0.7 * r.entropy.sum(), [Xg])
    v = torch.randn(3, V, device="cuda").double()
    h = 1e-4

    def f(x):
        q = Ref(x, tok)
        return q.logprob + 0.7 * q.H

    slope = (f(X.double() + h * v) - f(X.double() - h * v)) / (2 * h)
    want, err = Ref(X, tok).grad(torch.ones(3, device="cuda"), torch.full((3,), 0.7, device="cuda"))
    assert ((g.double() * v).sum(-1) - slope).abs().max() < 1e-5 + (err * v.abs()).sum(-1).max()


# ------------------------------------------------------------------ divergence
def kl_ref(T, D, mask):
    K = D.shape[1]
    t, d = T[:, :K].double(), D.detach().double()
    V = t.shape[-1]
    m, n = t.amax(-1, keepdim=True), d.amax(-1, keepdim=True)
    lp, lq = torch.log_softmax(t, -1), torch.log_softmax(d, -1)
    p, q = lp.exp().nan_to_num(nan=0.0), lq.exp().nan_to_num(nan=0.0)
    kl = torch.where(p > 0, p * (lp - lq), 0.0).sum(-1)
    empty_t, empty_d = m[..., 0] == -math.inf, n[..., 0] == -math.inf
    kl = torch.where(empty_d, math.inf, kl)
    kl = torch.where(empty_t, 0.0, kl)
    skip = ~mask if mask is not None else torch.zeros_like(empty_t)
    kl = torch.where(skip, 0.0, kl)
    chain = math.ceil(V / 256) + 16
    gap = torch.where((p > 0) & (q > 0), p * ((t - m) - (d - n)).abs(), 0.0).nan_to_num().sum(-1)
    ed = torch.where(p > 0, p * (t - m).abs(), 0.0).nan_to_num().sum(-1)
    eq = torch.where(q > 0, q * (d - n).abs(), 0.0).nan_to_num().sum(-1)
    tol = U * (2 * (chain + 12) * (1 + gap) + ed * (1 + gap) + eq + 40)
    dead = skip | empty_t | empty_d
    diff = torch.where(dead[..., None], 0.0, q - p)
    lpa, lqa = torch.where(p > 0, lp, 0.0).abs(), torch.where(q > 0, lq, 0.0).abs()
    err = U * torch.where(dead[..., None], 0.0,
                          p * (chain + 24 + ed[..., None] + 4 * lpa) + q * (chain + 24 + eq[..., None] + 4 * lqa))
    return kl, tol, diff, err


def check_kl(T, D, mask=None):
    D = D.detach().requires_grad_()
    kl = sv.spec_draft_kl(T, D, mask=mask)
    want, tol, diff, err = kl_ref(T, D, mask)
    close(kl, want, tol, "kl")
    w = torch.rand(kl.shape, device="cuda") + 0.5
    g, = torch.autograd.grad([kl], [D], [w])
    wd = w.double()[..., None]
    close(g, diff * wd, wd * err + (half(D.dtype) + 2 * U) * (diff * wd).abs() + 1e-38, "kl grad")
    return kl, g


def pair(B, K, Kt, V, dt, seed, off_t=0, off_d=0):
    T = rows_of(B * Kt, V, dt, seed, off_t).view(B, Kt, V)
    noise = torch.randn(B, K, V, generator=torch.Generator(device="cuda").manual_seed(seed + 5), device="cuda")
    buf = torch.empty(B * K * V + off_d, dtype=dt, device="cuda")
    buf[off_d:] = (T[:, :K].float() + 0.7 * noise).to(dt).reshape(-1)
    return T, buf[off_d:].view(B, K, V)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,K,Kt,V", [(1, 1, 1, 1), (1, 1, 2, 3), (2, 3, 4, 33), (2, 1, 1, 4096), (3, 2, 3, 8193),
                                      (1, 5, 6, 32000), (4, 3, 3, 50257), (2, 5, 6, 128256), (1, 1, 2, 262144),
                                      (300, 2, 5, 700)])
def test_kl_sizes(B, K, Kt, V, dtype):
    T, D = pair(B, K, Kt, V, DT[dtype], seed=V + K)
    mask = torch.rand(B, K, device="cuda") < 0.8
    check_kl(T, D)
    check_kl(T, D, mask)


@pytest.mark.parametrize("dtype,off_t,off_d", [("bf16", 1, 0), ("bf16", 3, 6), ("bf16", 0, 5), ("f32", 1, 2)])
@pytest.mark.parametrize("V", [9, 4100, 40001])
def test_kl_alignment(V, dtype, off_t, off_d):
    T, D = pair(2, 3, 4, V, DT[dtype], V, off_t, off_d)
    check_kl(T, D)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 20000])
def test_kl_masks(V, dtype):
    dt = DT[dtype]
    low = torch.finfo(dt).min
    T, D = (t.clone() for t in pair(1, 9, 9, V, dt, 3))
    hide = torch.rand(V, device="cuda") < 0.4
    hide[3 % V] = False
    T[0, 0, hide], D[0, 0, hide] = -math.inf, -math.inf  # one mask on both
    T[0, 1, hide] = -math.inf                            # the target's alone
    D[0, 2, hide] = -math.inf                            # the draft's alone: infinite
    T[0, 3] = -math.inf                                  # nothing left of the target
    D[0, 4] = -math.inf                                  # nothing left of the draft
    T[0, 5], D[0, 5] = -math.inf, -math.inf
    T[0, 6, hide], D[0, 6, hide] = low, low
    T[0, 7], D[0, 7] = low, low                          # both uniform
    D[0, 8] = T[0, 8]                                    # equal: 0
    kl, g = check_kl(T, D)
    assert kl[0, 2] == math.inf and kl[0, 3] == 0 and kl[0, 4] == math.inf and kl[0, 7] == 0
    assert (g[0, 3:6] == 0).all() and kl[0, 8].abs() < 1e-5


def test_kl_masked_rows_are_not_read():
    T, D = (t.clone() for t in pair(2, 2, 3, 9000, torch.bfloat16, 3))
    mask = torch.tensor([[True, False], [False, True]], device="cuda")
    T[0, 1], D[1, 0] = math.nan, math.nan
    T[:, 2] = math.nan  # the bonus row
    D.requires_grad_()
    kl = sv.spec_draft_kl(T, D, mask=mask)
    g, = torch.autograd.grad([kl.sum()], [D])
    assert kl.isfinite().all() and g.isfinite().all()
    assert kl[0, 1] == 0 and kl[1, 0] == 0 and (g[0, 1] == 0).all() and (g[1, 0] == 0).all()
    assert (g[0, 0] != 0).any() and kl[1, 1] > 0


def test_kl_offsets_cancel():
    """A constant on a row changes nothing: the logits are multiples of 2^-6,
    so the sums are exact."""
    T, D = pair(2, 2, 2, 5000, torch.float32, 8)
    T, D = (T * 64).round() / 64, (D * 64).round() / 64
    a = sv.spec_draft_kl(T, D)
    b = sv.spec_draft_kl(T + 512, D - 256)
    r = kl_ref(T + 512, D - 256, None)
    close(b, r[0], r[1], "kl with offsets")
    assert (a - b).abs().max() < 1e-4


def test_kl_gradient_against_differences():
    T, D = pair(1, 2, 3, 700, torch.float32, 12)
    Dg = D.clone().requires_grad_()
    g, = torch.autograd.grad([sv.spec_draft_kl(T, Dg).sum()], [Dg])
    v = torch.randn(D.shape, device="cuda").double()
    h = 1e-4
    f = lambda d: kl_ref(T, d, None)[0].sum()  # noqa: E731
    slope = (f(D.double() + h * v) - f(D.double() - h * v)) / (2 * h)
    err = (kl_ref(T, D, None)[3] * v.abs()).sum()
    assert abs(float((g.double() * v).sum() - slope)) < 1e-5 + float(err)


# ------------------------------------------------- streams, graphs, workspaces
def test_rows_expanded_gradients_and_chained_graph():
    """A gradient that arrives expanded (from a sum) and logits that are an
    intermediate result."""
    base = torch.randn(3, 900, device="cuda", requires_grad=True)
    tok = tokens_of(3, 900, 1)
    sv.spec_token_logprobs(base * 2, tok).logprob.sum().backward()
    ref = torch.log_softmax(base.detach().double() * 2, -1).exp() * -2
    ref.scatter_add_(1, tok.long()[:, None], torch.full((3, 1), 2.0, device="cuda", dtype=torch.float64))
    assert (base.grad.double() - ref).abs().max() < 1e-5


def test_rows_captured_and_replayed():
    """Both operators with their gradients, captured twice; replays with eager
    calls of the same and other shapes between them equal the eager results."""
    V = 30001
    X = rows_of(9, V, torch.bfloat16, 1).requires_grad_()
    tok = tokens_of(9, V, 2)
    T, D = pair(2, 3, 4, V, torch.bfloat16, 3)
    D.requires_grad_()

    def work():
        r = sv.spec_token_logprobs(X, tok, top_n=6)
        kl = sv.spec_draft_kl(T, D)
        gx, = torch.autograd.grad([r.logprob, r.entropy], [X], [torch.ones_like(r.logprob)] * 2)
        gd, = torch.autograd.grad([kl], [D], [torch.ones_like(kl)])
        return [t.detach() for t in (*r, kl, gx, gd)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        eager = [t.clone() for t in work()]
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, work()))
    for rep in range(3):
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for (g, outs), st in zip(graphs, streams):  # both at once
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for _, outs in graphs:
            for a, b in zip(eager, outs):
                assert torch.equal(a, b), rep
        sv.spec_token_logprobs(rows_of(3, 777, torch.float32, rep), tokens_of(3, 777, 1), top_n=32)
        torch.cuda.synchronize()


def test_rows_two_streams_at_once_and_repeatable():
    V = 128256
    sets = [(rows_of(12, V, torch.bfloat16, s), tokens_of(12, V, s)) for s in (1, 2)]
    alone = [[t.clone() for t in sv.spec_token_logprobs(x, t, top_n=20)] for x, t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        outs = []
        for (x, t), st in zip(sets, streams):
            with torch.cuda.stream(st):
                outs.append(sv.spec_token_logprobs(x, t, top_n=20))
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            for i, j in zip(a, b):
                assert torch.equal(i, j)


def test_rows_workspace_is_left_zero():
    """The library's zero-filled workspace serves a rule, these calls and the
    rule again."""
    lib = sv.load_library()
    V, rows = 128256, 12
    X, tok = rows_of(rows, V, torch.bfloat16, 5), tokens_of(rows, V, 5)
    n = max(lib.spec_logprobs_workspace_bytes(1, rows, V, 32), lib.spec_draft_kl_workspace_bytes(1, 2, 5, V),
            sv.spec_verify_workspace_bytes(2, 6, V))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    T = X.view(2, 6, V)
    before = sv.spec_verify_greedy(T, tok.view(2, 6)[:, :5].contiguous(), workspace=ws)
    o = [torch.empty(rows * 32, dtype=d, device="cuda") for d in (torch.float32, torch.float32, torch.int32, torch.float32, torch.int32)]
    st = torch.cuda.current_stream().cuda_stream
    assert lib.spec_token_logprobs(X.data_ptr(), 1, tok.data_ptr(), rows, V, 32, *(t.data_ptr() for t in o),
                                   None, ws.data_ptr(), n, st) == 0
    torch.cuda.synchronize()
    assert (ws == 0).all()
    D = X.view(2, 6, V)[:, :5].contiguous()
    assert lib.spec_draft_kl(X.data_ptr(), D.data_ptr(), 1, None, 2, 5, 6, V, o[0].data_ptr(), None,
                             ws.data_ptr(), n, st) == 0
    torch.cuda.synchronize()
    assert (ws == 0).all()
    after = sv.spec_verify_greedy(T, tok.view(2, 6)[:, :5].contiguous(), workspace=ws)
    for a, b in zip(before, after):
        assert torch.equal(a, b)


def test_rows_past_32_bits_of_offset():
    """Rows beyond 2^31 elements of one tensor."""
    V, rows = 262144, 8200
    X = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    X[-1] = rows_of(1, V, torch.bfloat16, 3)[0]
    tok = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    tok[-1] = 77
    r = sv.spec_token_logprobs(X, tok, top_n=3)
    one = sv.spec_token_logprobs(X[-1:].clone(), tok[-1:], top_n=3)
    assert torch.equal(r.logprob[-1:], one.logprob) or (r.logprob[-1] - one.logprob[0]).abs() < 1e-5
    assert torch.equal(r.top_tokens[-1:], one.top_tokens) and (r.logprob[:-1] == 0).all()


@pytest.mark.parametrize("dtype,rows", [("bf16", 1100), ("f32", 1030)])
@pytest.mark.parametrize("V", [128256, 128255])
def test_rows_beyond_the_caches(V, rows, dtype):
    """Logits of more than 256 MiB, which are read and whose gradients are
    written past the caches, equal their halves' results bit for bit."""
    X = rows_of(rows, V, DT[dtype], 21).requires_grad_()
    tok = tokens_of(rows, V, 21)
    tok[::7] = -1
    assert X.numel() * X.element_size() > 256 << 20
    w = torch.rand(rows, device="cuda")

    def run(x, t, w, draft):
        r = sv.spec_token_logprobs(x, t, top_n=3)
        g, = torch.autograd.grad([r.logprob, r.entropy], [x], [w, 1 - w])
        kl = sv.spec_draft_kl(draft, x[None], mask=(t >= 0)[None])
        gk, = torch.autograd.grad([kl], [x], [w[None]])
        return [v.detach() for v in (*r, g, kl[0], gk)]

    T = rows_of(rows, V, DT[dtype], 22)
    def piece(x, s):
        """A copy of some rows that starts at the same place of 16 bytes: the
        order of a row's sums follows its alignment."""
        x = x.detach()
        off = s.start * V % (16 // x.element_size())
        buf = torch.empty(x[s].numel() + off, dtype=x.dtype, device="cuda")
        buf[off:] = x[s].reshape(-1)
        return buf[off:].view(-1, V)

    whole = run(X, tok, w, T[None])
    for half in (slice(0, rows // 2), slice(rows // 2, rows)):
        part = run(piece(X, half).requires_grad_(), tok[half], w[half], piece(T, half)[None])
        for a, b in zip(whole, part):
            assert torch.equal(a[half], b)
