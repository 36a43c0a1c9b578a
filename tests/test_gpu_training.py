"""The operators together, as a draft head's training uses them: head_loss of a
HeadModel with gated and residual blocks, its gradients against float64 and
against differences, captured and replayed, on two streams; and the driver on
the same model."""
import threading

import pytest
import torch

import draft_verification_row_amd as sv
import draft_verification_row_amd.markov as mk

pytestmark = pytest.mark.gpu


def head(V, H, F, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    blocks = [mk.GatedBlock(*((r(*s) / s[1] ** 0.5).to(dtype) for s in ((F, H), (F, H), (H, F)))),
              ((r(H, H) / H ** 0.5).to(dtype), (0.3 * r(H)).to(dtype))]
    return mk.HeadModel(r(V, H).to(dtype), blocks, (2 * r(V, H) / H ** 0.5).to(dtype))


def params(m):
    return [m.embedding, *(t for b in m.blocks for t in b), m.output]


def model_of(ps):
    return mk.HeadModel(ps[0], [mk.GatedBlock(*ps[1:4]), (ps[4], ps[5])], ps[6])


def batch(V, B, L, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(0, V, (B, L + 1), generator=g, device="cuda", dtype=torch.int32)
    for b in range(B):  # ragged: padded behind each sequence
        tokens[b, max(1, L - 2 * b):] = -1
    weight = torch.rand(B, L, generator=g, device="cuda")
    return tokens[:, :-1].contiguous(), tokens[:, 1:].contiguous(), weight


def reference(ps, tokens, targets):
    """Losses in float64 by torch's own autograd on the CPU."""
    emb, gate, up, down, w, b, out = ps
    on = tokens >= 0
    h = torch.where(on[..., None], emb[tokens.long().clamp_min(0)], 0.0)
    g = h @ gate.t()
    h = h + (g * torch.sigmoid(g) * (h @ up.t())) @ down.t()
    z = h @ w.t() + b
    h = h + z * torch.sigmoid(z)
    lp = torch.log_softmax(h @ out.t(), -1)
    loss = -lp.gather(-1, targets.long().clamp_min(0)[..., None])[..., 0]
    return torch.where(targets >= 0, loss, 0.0)


@pytest.mark.parametrize("V,H,F,B,L", [(97, 40, 56, 3, 6), (1000, 128, 200, 9, 33), (3001, 65, 100, 7, 20)])
def test_training_step_gradients(V, H, F, B, L):
    """float32 throughout.  Every stage is a few hundred roundings of 2^-24 from
    exact and the layers' gains are of order 1, so the gradients agree to 1e-4
    of their largest element."""
    ps = [p.requires_grad_() for p in params(head(V, H, F, torch.float32, 3))]
    tokens, targets, weight = batch(V, B, L, 5)
    loss = mk.head_loss(model_of(ps), tokens, targets)
    assert loss.shape == tokens.shape and (loss[targets < 0] == 0).all()
    grads = torch.autograd.grad((loss * weight).sum(), ps)
    rs = [p.detach().double().cpu().requires_grad_() for p in ps]
    want = reference(rs, tokens.cpu(), targets.cpu())
    assert (loss.detach().double().cpu() - want.detach()).abs().max() < 1e-4
    ref = torch.autograd.grad((want * weight.double().cpu()).sum(), rs)
    for a, b in zip(grads, ref):
        assert (a.double().cpu() - b).abs().max() < 1e-4 * b.abs().max()


def test_tied_embedding_and_output():
    V, H = 200, 48
    ps = params(head(V, H, 64, torch.float32, 4))
    tokens, targets, _ = batch(V, 4, 12, 6)
    one = ps[0].clone().requires_grad_()
    two = [ps[0].clone().requires_grad_() for _ in range(2)]
    tied, = torch.autograd.grad(mk.head_loss(model_of([one, *ps[1:6], one]), tokens, targets).sum(), [one])
    a, b = torch.autograd.grad(mk.head_loss(model_of([two[0], *ps[1:6], two[1]]), tokens, targets).sum(), two)
    assert torch.equal(tied, a + b) or (tied - (a + b)).abs().max() <= 2 ** -23 * (a.abs() + b.abs()).max()


def test_losses_agree_with_the_logits():
    m = head(500, 64, 96, torch.float32, 8)
    tokens, targets, _ = batch(500, 5, 17, 7)
    loss = mk.head_loss(m, tokens, targets)
    on = targets >= 0
    lp = sv.spec_token_logprobs(mk.head_logits(m, tokens.clamp_min(0)), targets).logprob
    assert ((loss + lp)[on].abs() < 1e-4).all()


def test_driver_on_gated_blocks():
    """The eager driver and the captured one give the same tokens, and the rule's
    log probs are those of the model's losses."""
    V, B, K, rounds = 300, 12, 3, 4
    draft, target = head(V, 64, 96, torch.bfloat16, 1), head(V, 64, 160, torch.bfloat16, 2)
    start = torch.randint(0, V, (B,), dtype=torch.int32, device="cuda")
    ud, uv = torch.rand(rounds, B, K, device="cuda"), torch.rand(rounds, B, K + 1, device="cuda")
    tr = mk.generate_speculative(target, draft, start, ud, uv)
    g = mk.SpeculativeGraph(target, draft, B, K, rounds)
    for rep in range(3):
        out = g.run(start, ud, uv)
        torch.cuda.synchronize()
        assert torch.equal(out.emitted, tr.emitted) and torch.equal(out.accept_len, tr.accept_len), rep
        mk.generate_speculative(target, draft, start.flip(0), ud, uv)
        torch.cuda.synchronize()
    emitted = tr.emitted[0]
    tokens = torch.cat([start[:, None], emitted[:, :-1]], 1).contiguous()
    losses = mk.head_loss(target, tokens, emitted)
    logits = mk.head_logits(target, tokens.clamp_min(0), out_dtype=torch.float32)
    want = sv.spec_token_logprobs(logits, emitted).logprob
    on = emitted >= 0
    # a bfloat16 head's hidden states may come out a rounding apart from other
    # numbers of rows
    assert ((losses + want)[on].abs() < 0.1).all() and (losses[~on] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_captured_and_replayed(dtype):
    """A whole training step in a graph, with eager steps between its replays;
    two graphs of the same leaves."""
    ps = [p.requires_grad_() for p in params(head(700, 72, 104, dtype, 3))]
    tokens, targets, weight = batch(700, 12, 13, 5)

    def step():
        loss = mk.head_loss(model_of(ps), tokens, targets)
        return [loss.detach(), *torch.autograd.grad([loss], ps, [weight])]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        eager = [v.clone() for v in step()]
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        graphs.append((g, outs))
    for rep in range(3):
        for g, outs in graphs:
            for v in outs:
                v.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, outs in graphs:
            for a, b in zip(eager, outs):
                assert torch.equal(a, b), rep
        step()
        torch.cuda.synchronize()
    # new tokens in the same buffers: the graph reads them anew
    tokens.copy_(tokens.flip(0))
    targets.copy_(targets.flip(0))
    want = [v.clone() for v in step()]
    for g, outs in graphs:
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_capture_is_refused_while_an_eager_graph_lives():
    ps = [p.requires_grad_() for p in params(head(60, 24, 32, torch.bfloat16, 3))]
    tokens, targets, _ = batch(60, 3, 5, 5)
    W, x = ps[6], torch.randn(4, 24, device="cuda").bfloat16()
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    for f in (lambda: sv.spec_embedding(ps[0], tok), lambda: sv.spec_gated_linear(x, ps[1], ps[2]),
              lambda: sv.spec_cross_entropy(x, W, tok).loss, lambda: mk.head_loss(model_of(ps), tokens, targets)):
        kept = f()
        with pytest.raises(sv.SpecVerifyError):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                f()
        torch.cuda.synchronize()
        kept.sum().backward()
        del kept


def test_calls_on_side_streams_and_threads():
    """Two threads on two streams, each with its own inputs, equal the calls alone."""
    sets = []
    for s in range(2):
        ps = [p.requires_grad_() for p in params(head(900, 96, 128, torch.bfloat16, 10 + s))]
        sets.append((ps, *batch(900, 15, 20, s)))

    def work(ps, tokens, targets, weight):
        loss = mk.head_loss(model_of(ps), tokens, targets)
        return [loss.detach(), *torch.autograd.grad([loss], ps, [weight])]

    alone = [[t.clone() for t in work(*s)] for s in sets]
    torch.cuda.synchronize()
    out = [None, None]

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(8):
                out[i] = work(*sets[i])
            torch.cuda.current_stream().synchronize()

    th = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    [t.start() for t in th]
    [t.join() for t in th]
    for a, b in zip(alone, out):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
