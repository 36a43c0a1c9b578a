"""The operators together, as a draft head uses them: a HeadModel's logits, its
distillation step against float64, the driver on a head, log probs of what it
emitted."""
import pytest
import torch

import draft_verification_row_amd as sv
import draft_verification_row_amd.markov as mk

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def head(V, H, blocks, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return mk.HeadModel(r(V, H).to(dtype), [((r(H, H) / H ** 0.5).to(dtype), (0.3 * r(H)).to(dtype)) for _ in range(blocks)],
                        (2 * r(V, H) / H ** 0.5).to(dtype))


def params(m):
    return [m.embedding, *(t for b in m.blocks for t in b), m.output]


def reference_loss(ps, tokens, target, weight):
    """The distillation loss in float64, by torch's own autograd on the CPU."""
    emb, *blocks, out = ps
    h = emb[tokens]
    for i in range(0, len(blocks), 2):
        z = h @ blocks[i].t() + blocks[i + 1]
        h = h + z * torch.sigmoid(z)
    lq = torch.log_softmax(h @ out.t(), -1)
    lp = torch.log_softmax(target, -1)
    return ((lp.exp() * (lp - lq)).sum(-1) * weight).sum()


@pytest.mark.parametrize("V,H,B,K,blocks", [(97, 40, 5, 3, 1), (1000, 128, 30, 4, 2)])
def test_distillation_step_gradients(V, H, B, K, blocks):
    """float32 throughout.  Every stage is a few hundred roundings of u from
    exact and the layers' gains are of order 1, so the gradients agree to
    1e-4 of their largest element."""
    m = head(V, H, blocks, torch.float32, 3)
    ps = [p.requires_grad_() for p in params(m)]
    g = torch.Generator(device="cuda").manual_seed(5)
    tokens = torch.randint(0, V, (B, K), generator=g, device="cuda")
    target = torch.randn(B, K + 1, V, generator=g, device="cuda") * 2
    mask = torch.rand(B, K, generator=g, device="cuda") < 0.8
    kl = sv.spec_draft_kl(target, mk.head_logits(m, tokens), mask=mask)
    grads = torch.autograd.grad(kl.sum(), ps)
    rs = [p.detach().double().cpu().requires_grad_() for p in ps]
    loss = reference_loss(rs, tokens.cpu(), target[:, :K].double().cpu(), mask.double().cpu())
    want = torch.autograd.grad(loss, rs)
    assert abs(float(kl.detach().sum()) - float(loss.detach())) < 1e-5 * abs(float(loss.detach()))
    for a, b in zip(grads, want):
        assert (a.double().cpu() - b).abs().max() < 1e-4 * b.abs().max()


@pytest.mark.parametrize("target_is_head,dtype", [(False, torch.bfloat16), (False, torch.float32), (True, torch.bfloat16)])
def test_driver_on_heads(target_is_head, dtype):
    """One round by hand on the same logits, the eager driver and the captured
    one give the same tokens; the emitted tokens' log probs follow."""
    V, H, B, K, rounds = 300, 64, 12, 3, 5
    draft = head(V, H, 1, torch.bfloat16, 1)
    target = head(V, H, 2, torch.bfloat16, 2) if target_is_head else (torch.randn(V, V, device="cuda") * 2).to(dtype)
    start = torch.randint(0, V, (B,), dtype=torch.int32, device="cuda")
    ud = torch.rand(rounds, B, K, device="cuda")
    uv = torch.rand(rounds, B, K + 1, device="cuda")
    tr = mk.generate_speculative(target, draft, start, ud, uv)
    prev = [start]
    for i in range(K):
        q = mk.head_logits(draft, prev[-1], out_dtype=dtype)
        prev.append(sv.spec_sample_drafts(q, ud[0, :, i].contiguous()).tokens)
    idx = torch.stack(prev, 1)
    T = mk.head_logits(target, idx, out_dtype=dtype) if target_is_head else target[idx]
    D = mk.head_logits(draft, idx[:, :K], out_dtype=dtype)
    r = sv.spec_verify_exact(T, D, idx[:, 1:].contiguous(), uv[0])
    assert torch.equal(r.tokens, tr.emitted[0]) and torch.equal(r.accept_len, tr.accept_len[0])
    lp = sv.spec_token_logprobs(T, tr.emitted[0], top_n=3)
    assert (lp.logprob - r.target_logprob).abs().max() < 1e-4
    assert (lp.top_logprob[..., 0] >= lp.logprob).all() and (lp.status == 0).all()
    kl = sv.spec_draft_kl(T, D)
    assert (kl >= 0).all() and kl.isfinite().all()
    eager = (tr.emitted.clone(), tr.accept_len.clone())
    g = mk.SpeculativeGraph(target, draft, B, K, rounds)
    for rep in range(3):
        out = g.run(start, ud, uv)
        torch.cuda.synchronize()
        assert torch.equal(out.emitted, eager[0]) and torch.equal(out.accept_len, eager[1]), rep
        mk.generate_speculative(target, draft, start.flip(0), ud, uv)
        torch.cuda.synchronize()


def test_head_models_are_checked():
    m = head(50, 16, 1, torch.bfloat16, 1)
    table = torch.randn(50, 50, device="cuda")
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    u = torch.rand(1, 2, 2, device="cuda")
    v = torch.rand(1, 2, 3, device="cuda")
    bad = [m._replace(output=m.output[:40]), m._replace(embedding=m.embedding.float()),
           m._replace(blocks=[(m.blocks[0][0], m.blocks[0][1][:8])]), head(60, 16, 0, torch.bfloat16, 1),
           head(50, 16, 0, torch.float32, 1)]
    for i, b in enumerate(bad):
        with pytest.raises(sv.SpecVerifyError):
            mk.generate_speculative(table.bfloat16(), b, start, u, v)
            print("not refused:", i)
    mk.generate_speculative(table, m, start, u, v)  # float32 logits from a bfloat16 head


def test_calls_on_a_side_stream_and_threads():
    """Two threads on two streams, each with its own inputs, equal the calls alone."""
    import threading
    sets = []
    for s in range(2):
        m = head(400, 96, 1, torch.bfloat16, 10 + s)
        tok = torch.randint(0, 400, (7, 4), device="cuda")
        T = torch.randn(7, 5, 400, device="cuda").bfloat16()
        sets.append((m, tok, T))

    def work(m, tok, T):
        with torch.no_grad():
            D = mk.head_logits(m, tok)
            r = sv.spec_token_logprobs(T, tok.new_zeros(7, 5).int(), top_n=7)
            return [D, sv.spec_draft_kl(T, D), *r]

    alone = [[t.clone() for t in work(*s)] for s in sets]
    torch.cuda.synchronize()
    out = [None, None]

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                out[i] = work(*sets[i])
            torch.cuda.current_stream().synchronize()

    th = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    [t.start() for t in th]
    [t.join() for t in th]
    for a, b in zip(alone, out):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
