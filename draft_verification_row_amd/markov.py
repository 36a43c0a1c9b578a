"""Multi-round speculative sampling with toy Markov models on the GPU.

The loop of the spec-decode README ("How it works", and generate_speculative
under "Use it"): each round the draft proposes K tokens one after another
from its own next-token distribution, the target scores all K+1 positions at
once, the exact rule accepts a prefix and emits one more token, and the next
round continues from the last emitted token.  A toy model's next_dist(prefix)
is the row of its logit table picked by the last token, so its "forward pass"
is a row lookup (torch indexing), or, for a HeadModel, a small network on the
last token's embedding, whose products run in spec_linear; every draw and
every decision runs in the library's kernels: spec_sample_drafts for the K
draft tokens, spec_verify_exact for the verification.

SpeculativeGraph captures every round of one shape in a single HIP graph,
so a run is one graph launch instead of some 35 launches per round from the
host; its replays give the same tokens as the eager loop, bit for bit.

Run statistics follow the README's report: target passes (one per round per
sequence), acceptance rate = accepted drafts / proposed drafts, tokens per
target pass, and the speedup over target-only sampling when one draft step
costs `draft_cost` target passes: tokens / (passes * (1 + K * draft_cost)).
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import (SpecVerifyError, _check, spec_linear, spec_sample_drafts,
               spec_sample_workspace_bytes, spec_verify_exact, spec_verify_workspace_bytes)

__all__ = ["HeadModel", "SpeculativeTrace", "SpeculativeGraph", "generate_speculative",
           "head_logits", "trace_stats"]


class HeadModel(NamedTuple):
    """A next-token model made of a draft head's parts, one dtype throughout:
    the last token's embedding h, residual blocks h + silu(h W^T + b), and the
    output layer.  It may stand wherever a logit table may."""
    embedding: torch.Tensor                                # [V][H]
    blocks: Sequence[Tuple[torch.Tensor, torch.Tensor]]    # (W [H][H], b [H]) each
    output: torch.Tensor                                   # [V][H]


def head_logits(model: HeadModel, tokens: torch.Tensor, *,
                out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """The model's next-token logits after each of `tokens` (an integer tensor
    on the GPU): [*tokens.shape][V] in out_dtype (the model's by default).  The
    parameters have gradients."""
    h = model.embedding[tokens].contiguous()  # a view of tokens gives a view
    for weight, bias in model.blocks:
        h = spec_linear(h, weight, bias, residual=h, activation="silu")
    return spec_linear(h, model.output, out_dtype=out_dtype)


class SpeculativeTrace(NamedTuple):
    emitted: torch.Tensor     # int32 [rounds][B][K+1]: emitted tokens, -1 padded
    accept_len: torch.Tensor  # int32 [rounds][B]: accepted drafts per round


def _model(model, name):
    """(vocabulary, dtype or None where the logits' dtype is free) of a table
    or a HeadModel, checked."""
    if not isinstance(model, HeadModel):
        P = _check(model, name)
        if P.dim() != 2 or P.shape[0] != P.shape[1]:
            raise SpecVerifyError(f"{name} must be [V][V]")
        return P.shape[0], P.dtype
    E = _check(model.embedding, f"{name}.embedding")
    if E.dim() != 2:
        raise SpecVerifyError(f"{name}.embedding must be [V][H]")
    V, H = E.shape
    _check(model.output, f"{name}.output", E.dtype, (V, H))
    for i, (weight, bias) in enumerate(model.blocks):
        _check(weight, f"{name}.blocks[{i}] weight", E.dtype, (H, H))
        _check(bias, f"{name}.blocks[{i}] bias", E.dtype, (H,))
    return V, None if E.dtype == torch.bfloat16 else E.dtype


class _Models(NamedTuple):
    target: object
    draft: object
    V: int
    dtype: torch.dtype      # of both models' logits
    device: torch.device


def _models(target, draft) -> _Models:
    """Both models' logits have one dtype: a table's own, float32 from float32
    heads, either from bfloat16 heads (bfloat16 where both are heads)."""
    V, dt = _model(target, "target_table")
    Vd, dd = _model(draft, "draft_table")
    dtype = dt or dd or torch.bfloat16
    if Vd != V or dd not in (None, dtype):
        raise SpecVerifyError(f"draft_table must have target_table's vocabulary {V} and dtype "
                              f"{dtype}, got {Vd} and {dd}")
    dev = (target.embedding if isinstance(target, HeadModel) else target).device
    return _Models(_held(target), _held(draft), V, dtype, dev)


def _held(model):
    """The model with its blocks in tuples, which no one else can change."""
    if isinstance(model, HeadModel):
        return model._replace(blocks=tuple((weight, bias) for weight, bias in model.blocks))
    return model


def _logits(model, tokens, dtype):
    if isinstance(model, HeadModel):
        return head_logits(model, tokens, out_dtype=dtype)
    return model[tokens]


def _workspaces(m, B, K):
    """Workspaces of the round's two library calls."""
    V = m.V
    u8 = dict(dtype=torch.uint8, device=m.device)
    # zero-filled: the library reads published words as "not written" while
    # they are zero and leaves every byte zero after each call
    return (torch.zeros(spec_sample_workspace_bytes(B, V), **u8),
            torch.zeros(spec_verify_workspace_bytes(B, 2 * K + 1, V), **u8))


def _round(m, cur, udt_r, uv_r, ws, rows, emitted_r, accept_r):
    """One round from the last emitted tokens `cur` int32 [B]: K draft draws
    (udt_r [K][B]: draft step i's uniforms are row i), one exact verification;
    writes the round's outputs and returns the next cur.  rows = arange(B)."""
    K = udt_r.shape[0]
    if K < 1:
        raise SpecVerifyError("K must be positive")
    ws_s, ws_v = ws
    # The rule has to take the very logits the drafts were drawn from.  A head's
    # would come out a rounding apart if all K steps were computed at once, so
    # they are kept; a table's rows are looked up again in one call, which costs
    # less (V = 4096, B = 32, K = 4, us a round: 92.6 captured and 147 eager;
    # 93.7 and 159 with the rows kept).
    keep = isinstance(m.draft, HeadModel)
    prev, steps = [cur], []
    for i in range(K):
        q = _logits(m.draft, prev[-1], m.dtype)
        prev.append(spec_sample_drafts(q, udt_r[i], logprobs=False, workspace=ws_s).tokens)
        if keep:
            steps.append(q)
    idx = torch.stack(prev, 1)
    D = torch.stack(steps, 1) if keep else m.draft[idx[:, :K]]
    res = spec_verify_exact(_logits(m.target, idx, m.dtype), D, idx[:, 1:].contiguous(), uv_r,
                            logprobs=False, workspace=ws_v)
    emitted_r.copy_(res.tokens)
    accept_r.copy_(res.accept_len)
    return res.tokens[rows, res.accept_len]


@torch.no_grad()
def generate_speculative(target_table, draft_table,
                         start: torch.Tensor, u_draft: torch.Tensor,
                         u_verify: torch.Tensor) -> SpeculativeTrace:
    """target_table, draft_table: [V][V] logits (row s: the next token after s,
    bfloat16 or float32, one dtype), or a HeadModel each; start int32 [B]; u_draft float32
    [rounds][B][K] and u_verify float32 [rounds][B][K+1] uniforms in [0,1)."""
    m = _models(target_table, draft_table)
    ud = _check(u_draft, "u_draft", torch.float32)
    rounds, B, K = ud.shape
    uv = _check(u_verify, "u_verify", torch.float32, (rounds, B, K + 1))
    cur = _check(start, "start", torch.int32, (B,)).clone()
    emitted = torch.empty((rounds, B, K + 1), dtype=torch.int32, device=m.device)
    accept = torch.empty((rounds, B), dtype=torch.int32, device=m.device)
    ws = _workspaces(m, B, K)
    udt = ud.transpose(1, 2).contiguous()
    rows = torch.arange(B, dtype=torch.int32, device=m.device)
    for r in range(rounds):
        cur = _round(m, cur, udt[r], uv[r], ws, rows, emitted[r], accept[r])
    return SpeculativeTrace(emitted, accept)


class SpeculativeGraph:
    """generate_speculative for a fixed (B, K, rounds) on fixed models,
    captured once in one HIP graph.  run() copies the start tokens and
    uniforms into the graph's input buffers and replays it; the returned
    trace's tensors are the graph's output buffers, overwritten by the next
    run.  Replays are ordered on the stream current at run()."""

    @torch.no_grad()
    def __init__(self, target_table, draft_table, B: int, K: int, rounds: int):
        m = _models(target_table, draft_table)
        self.P, self.Q = target_table, draft_table
        if B < 1 or K < 1 or rounds < 1:
            raise SpecVerifyError("B, K and rounds must be positive")
        dev = m.device
        self.B, self.K, self.rounds = B, K, rounds
        self.start = torch.zeros((B,), dtype=torch.int32, device=dev)
        self.u_draft_t = torch.zeros((rounds, K, B), dtype=torch.float32, device=dev)
        self.u_verify = torch.zeros((rounds, B, K + 1), dtype=torch.float32, device=dev)
        self.emitted = torch.empty((rounds, B, K + 1), dtype=torch.int32, device=dev)
        self.accept = torch.empty((rounds, B), dtype=torch.int32, device=dev)
        # Buffers made before the capture and read by the graph belong to the
        # ordinary allocator, so they are held here for the graph's lifetime:
        # freed, their blocks could go to other tensors between replays.  The
        # heads' tensors too, whatever becomes of the caller's list of blocks.
        self._models = m
        self._ws = _workspaces(m, B, K)
        self._rows = torch.arange(B, dtype=torch.int32, device=dev)
        self.graph = torch.cuda.CUDAGraph()
        cap = torch.cuda.Stream(device=dev)
        torch.cuda.synchronize(dev)
        with torch.cuda.graph(self.graph, stream=cap):
            cur = self.start.clone()
            for r in range(rounds):
                cur = _round(m, cur, self.u_draft_t[r], self.u_verify[r], self._ws,
                             self._rows, self.emitted[r], self.accept[r])
        torch.cuda.synchronize(dev)

    def run(self, start: torch.Tensor, u_draft: torch.Tensor,
            u_verify: torch.Tensor) -> SpeculativeTrace:
        B, K, R = self.B, self.K, self.rounds
        self.start.copy_(_check(start, "start", torch.int32, (B,)))
        self.u_draft_t.copy_(_check(u_draft, "u_draft", torch.float32, (R, B, K)).transpose(1, 2))
        self.u_verify.copy_(_check(u_verify, "u_verify", torch.float32, (R, B, K + 1)))
        self.graph.replay()
        return SpeculativeTrace(self.emitted, self.accept)


def trace_stats(accept_len, K: int, draft_cost: float = 0.1) -> dict:
    """accept_len [rounds][B] (tensor or array) -> the README's run report."""
    a = torch.as_tensor(accept_len).to("cpu", torch.float64)
    passes = a.numel()
    accepted = float(a.sum())
    tokens = accepted + passes
    return {"target_passes": passes, "tokens": int(tokens),
            "acceptance_rate": accepted / (K * passes),
            "tokens_per_target_pass": tokens / passes,
            "draft_cost": draft_cost,
            "speedup": tokens / (passes * (1.0 + K * draft_cost))}
