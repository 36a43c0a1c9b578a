"""The driver on draft heads: what it hands to the rule, and what it keeps."""
import pytest
import torch

import draft_verification_row_amd as sv
import draft_verification_row_amd.markov as mk
from test_gpu_heads import head

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,K,H,blocks", [(12, 3, 64, 1), (4, 5, 512, 2), (16, 8, 96, 0), (1, 1, 64, 1), (33, 2, 64, 1)])
def test_the_rule_gets_the_logits_the_drafts_were_drawn_from(monkeypatch, B, K, H, blocks):
    """Bit for bit, also where B rows and B * K rows take different kernels of
    the product (B = 12, K = 3: 12 rows and 36)."""
    V, rounds = 300, 3
    draft = head(V, H, blocks, torch.bfloat16, 1)
    target = (torch.randn(V, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) * 2).bfloat16()
    g = torch.Generator(device="cuda").manual_seed(3)
    start = torch.randint(0, V, (B,), dtype=torch.int32, device="cuda", generator=g)
    ud = torch.rand(rounds, B, K, device="cuda", generator=g)
    uv = torch.rand(rounds, B, K + 1, device="cuda", generator=g)
    drawn, given = [], []
    sample, verify = mk.spec_sample_drafts, mk.spec_verify_exact

    def sampled(q, *a, **k):
        drawn.append(q.clone())
        return sample(q, *a, **k)

    def verified(T, D, x, *a, **k):
        given.append((D.clone(), x.clone()))
        return verify(T, D, x, *a, **k)

    monkeypatch.setattr(mk, "spec_sample_drafts", sampled)
    monkeypatch.setattr(mk, "spec_verify_exact", verified)
    tr = mk.generate_speculative(target, draft, start, ud, uv)
    monkeypatch.undo()
    assert len(drawn) == rounds * K and len(given) == rounds
    for r in range(rounds):
        assert torch.equal(given[r][0], torch.stack(drawn[r * K:(r + 1) * K], 1)), r
    # and the captured driver makes the same calls
    out = mk.SpeculativeGraph(target, draft, B, K, rounds).run(start, ud, uv)
    torch.cuda.synchronize()
    assert torch.equal(out.emitted, tr.emitted) and torch.equal(out.accept_len, tr.accept_len)


def test_head_logits_of_views_of_tokens():
    """Any integer tensor of tokens, whatever its strides."""
    m = head(200, 64, 2, torch.bfloat16, 4)
    tok = torch.randint(0, 200, (6, 10, 4), device="cuda")
    for view in (tok.transpose(0, 1), tok[:, ::2, 1:3], tok[0, 0].expand(5, 4), tok.int().permute(2, 0, 1), tok[1, 2, 3]):
        got = mk.head_logits(m, view)
        assert got.shape == (*view.shape, 200) and torch.equal(got, mk.head_logits(m, view.contiguous()))
    # and with a gradient to the embedding: the rows' sums, of at most 240 terms
    # in float32, may be added in another order
    m = head(200, 64, 1, torch.float32, 4)
    m = m._replace(embedding=m.embedding.requires_grad_())
    a, b = (torch.autograd.grad(mk.head_logits(m, t).sum(), [m.embedding])[0]
            for t in (tok.transpose(0, 1), tok.transpose(0, 1).contiguous()))
    assert (a - b).abs().max() < 1e-4 * b.abs().max()


def test_a_captured_driver_keeps_its_heads_tensors():
    """A head's list of blocks that is changed after the capture: the graph
    still reads the weights it was captured with."""
    V, H, B, K, rounds = 300, 512, 4, 3, 2
    model = head(V, H, 2, torch.bfloat16, 1)
    blocks = list(model.blocks)
    draft = model._replace(blocks=blocks)
    target = (torch.randn(V, V, device="cuda") * 2).bfloat16()
    start = torch.randint(0, V, (B,), dtype=torch.int32, device="cuda")
    ud, uv = torch.rand(rounds, B, K, device="cuda"), torch.rand(rounds, B, K + 1, device="cuda")
    g = mk.SpeculativeGraph(target, draft, B, K, rounds)
    want = [t.clone() for t in g.run(start, ud, uv)]
    torch.cuda.synchronize()
    del model
    held = [weight.data_ptr() for weight, _ in blocks]
    blocks.clear()
    fill = [torch.full((H, H), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    assert not {t.data_ptr() for t in fill} & set(held)
    out = g.run(start, ud, uv)
    torch.cuda.synchronize()
    assert torch.equal(out.emitted, want[0]) and torch.equal(out.accept_len, want[1])


def test_a_captured_step_of_cast_weights_is_refused_while_an_eager_one_lives():
    """float32 weights, cast for each call: the eager graph has to go first;
    then the step is captured and its replays equal the eager gradients."""
    V, H = 150, 64
    m = head(V, H, 1, torch.float32, 6)
    (w, b), out = m.blocks[0], m.output
    ps = [w.requires_grad_(), b.requires_grad_(), out.requires_grad_()]
    emb = m.embedding.bfloat16()
    tok = torch.randint(0, V, (5, 3), device="cuda")
    gy = torch.randn(5, 3, V, device="cuda")

    def forward():
        return mk.head_logits(mk.HeadModel(emb, [(w.bfloat16(), b.bfloat16())], out.bfloat16()), tok, out_dtype=torch.float32)

    def step():
        return torch.autograd.grad([forward()], ps, [gy])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = [g.clone() for g in step()]
    torch.cuda.current_stream().wait_stream(s)
    kept = forward()
    with pytest.raises(sv.SpecVerifyError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            forward()
    torch.cuda.synchronize()
    del kept
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for rep in range(3):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), rep
        step()
        torch.cuda.synchronize()
