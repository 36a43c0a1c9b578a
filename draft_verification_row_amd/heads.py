"""Operators around a draft head, with their gradients: the log probabilities
of given tokens (entropy, top alternatives), the divergence of a draft from
its target, and the matrix product with bias, activation and residual that a
head is made of.

They take contiguous GPU tensors like the rules, on one device, and run on
that device's current stream.  Where an input requires a gradient the results
carry one (first order).  Calls may be captured into a graph: a captured call
gets a workspace of its own, which lives as long as the graph.  Before a
backward pass is captured, graphs of the same leaves that were built on other
streams have to be gone (the capture is refused while one of these operators'
lives, of leaves that they take as they are or cast, viewed or looked up).
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import SpecVerifyError, _check, _dtype_code, _raise, load_library

__all__ = ["LogprobResult", "spec_token_logprobs", "spec_draft_kl", "spec_linear", "SPEC_MAX_TOP"]

SPEC_MAX_TOP = 32
_ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "silu": 3}


class LogprobResult(NamedTuple):
    logprob: torch.Tensor       # float32 [...]
    entropy: torch.Tensor       # float32 [...]
    top_tokens: torch.Tensor    # int32 [..., top_n], -1 past the possible tokens
    top_logprob: torch.Tensor   # float32 [..., top_n]
    status: torch.Tensor        # int32 [...]: 1 for a token outside [-1, V)


# ---------------------------------------------------------------- helpers
_workspaces = {}


def _stream(index: int) -> int:
    """The device's current stream, as its handle."""
    return torch.cuda.current_stream(index).cuda_stream


# the same without making a stream object, some 5 us of host time a call
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)


def _capturing(index: int) -> bool:
    """Whether the device's current stream, which the calls run on, is being
    captured: torch answers for the current device alone."""
    if index == torch.cuda.current_device():
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(index):
        return torch.cuda.is_current_stream_capturing()


def _workspace_bytes(query: str, *sizes: int) -> int:
    """The library's answer to a size query; what it does not take, and what
    its 32-bit sizes cannot hold, is refused."""
    n = getattr(load_library(), query)(*sizes) if max(sizes) < 1 << 31 else 0
    if n == 0:
        raise SpecVerifyError("sizes outside the supported range")
    return n


def _zeroed(device: torch.device, nbytes: int) -> torch.Tensor:
    """A zero-filled workspace: one per (device, stream) for eager calls, a
    fresh one for a captured call, so that graphs share none."""
    if _capturing(device.index):
        return torch.zeros(nbytes, dtype=torch.uint8, device=device)
    key = (device.index, _stream(device.index))
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _workspaces[key] = torch.zeros(nbytes, dtype=torch.uint8, device=device)
    return ws


def _same_device(device: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise SpecVerifyError(f"{name} is on {t.device}, expected {device}")


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _call(name: str, device: torch.device, *args) -> None:
    """The library's entry point `name` on the device's current stream."""
    fn = getattr(load_library(), name)
    stream = _stream(device.index)
    if device.index == torch.cuda.current_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != 0:
        _raise(rc, name)


def _wants_grad(*tensors) -> bool:
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _mark_leaves(out: torch.Tensor) -> None:
    """Notes the stream on the gradient nodes of the leaves that `out` was
    computed from.  A leaf's node works on the stream it was made on; a backward
    pass that is captured on another stream would draw that stream into the
    capture, which ends the process.  So a leaf whose node an earlier, still
    living graph of these operators made on another stream is refused in a
    capture.  A leaf counts where an operator takes it, and behind casts, views,
    lookups and whatever else has one input that requires a gradient."""
    _note_stream([(_behind(node), 0) for node, _ in out.grad_fn.next_functions],
                 _stream(out.device.index), _capturing(out.device.index))


_CHAIN = 8  # nodes that are looked past; each costs about a microsecond


def _behind(node):
    """The gradient node behind up to _CHAIN nodes of one edge each."""
    for _ in range(_CHAIN):
        if node is None or type(node).__name__ == "AccumulateGrad":
            break
        edges = [n for n, _ in node.next_functions if n is not None]
        if len(edges) != 1:
            break
        node = edges[0]
    return node


def _note_stream(edges, stream: int, capturing: bool) -> None:
    for node, _ in edges:
        if type(node).__name__ == "AccumulateGrad":
            if node.metadata.setdefault("spec_stream", stream) != stream and capturing:
                raise SpecVerifyError(
                    "a tensor that requires a gradient still belongs to a graph built on another "
                    "stream: let go of that graph before capturing")


def _grad_in(g: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return None if g is None else g.contiguous()


# ----------------------------------------------------- token log probabilities
def _logprobs(X, tokens, top_n, stats):
    lead, V = X.shape[:-1], X.shape[-1]
    dev = X.device
    f32 = dict(dtype=torch.float32, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    out = LogprobResult(torch.empty(lead, **f32), torch.empty(lead, **f32),
                        torch.empty((*lead, top_n), **i32), torch.empty((*lead, top_n), **f32),
                        torch.empty(lead, **i32))
    rows = tokens.numel()
    st = torch.empty((*lead, 4), **f32) if stats else None
    if rows:
        code = _dtype_code(X)
        ws = _zeroed(dev, _workspace_bytes("spec_logprobs_workspace_bytes", code, rows, V, top_n))
        _call("spec_token_logprobs", dev, _p(X), code, _p(tokens), rows, V, top_n, _p(out.logprob),
              _p(out.entropy), _p(out.top_tokens), _p(out.top_logprob), _p(out.status), _p(st),
              _p(ws), ws.numel())
    return out, st


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top_n):
        out, st = _logprobs(logits, tokens, top_n, True)
        ctx.save_for_backward(logits, tokens, st)
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(out.top_tokens, out.top_logprob, out.status)
        return tuple(out)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_logprob, g_entropy, *_):
        logits, tokens, st = ctx.saved_tensors
        if g_logprob is None and g_entropy is None:
            return None, None, None
        grad = torch.empty_like(logits)
        if tokens.numel():
            gl, ge = _grad_in(g_logprob), _grad_in(g_entropy)
            _call("spec_token_logprobs_grad", logits.device, _p(logits), _dtype_code(logits),
                  _p(tokens), _p(st), _p(gl), _p(ge), tokens.numel(), logits.shape[-1], _p(grad))
        return grad, None, None


def spec_token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, *, top_n: int = 0
                        ) -> LogprobResult:
    """log p(token) under softmax(row) for one token per logit row, the row's
    entropy, and its top_n most probable tokens with their log-probs (lowest
    index first among equals).

    logits [..., V] bfloat16 or float32; tokens int32 with logits' leading
    shape.  A token of -1 pads its row, as in the rules' outputs: the row's
    logits are not read and it gets 0, 0 and alternatives -1.  logprob and
    entropy have a gradient to the logits; the alternatives have none.
    """
    X = _check(logits, "logits")
    if X.dim() < 1 or X.shape[-1] < 1:
        raise SpecVerifyError("logits must have a vocabulary dimension")
    _dtype_code(X)
    tok = _check(tokens, "tokens", torch.int32, X.shape[:-1])
    _same_device(X.device, tokens=tok)
    top_n = int(top_n)
    if not 0 <= top_n <= SPEC_MAX_TOP:
        raise SpecVerifyError(f"top_n must be in 0..{SPEC_MAX_TOP}")
    if _wants_grad(X):
        out = LogprobResult(*_TokenLogprobs.apply(X, tok, top_n))
        _mark_leaves(out.logprob)
        return out
    return _logprobs(X, tok, top_n, False)[0]


# ---------------------------------------------------------- draft divergence
def _kl(T, D, mask, stats):
    B, K, V = D.shape
    kl = torch.empty((B, K), dtype=torch.float32, device=D.device)
    st = torch.empty((B, K, 4), dtype=torch.float32, device=D.device) if stats else None
    if B * K:
        code = _dtype_code(D)
        ws = _zeroed(D.device, _workspace_bytes("spec_draft_kl_workspace_bytes", code, B, K, V))
        _call("spec_draft_kl", D.device, _p(T), _p(D), code, _p(mask), B, K, T.shape[1], V,
              _p(kl), _p(st), _p(ws), ws.numel())
    return kl, st


class _DraftKl(torch.autograd.Function):
    @staticmethod
    def forward(ctx, target, draft, mask):
        kl, st = _kl(target, draft, mask, True)
        ctx.save_for_backward(target, draft, mask, st)
        return kl

    @staticmethod
    @once_differentiable
    def backward(ctx, g_kl):
        T, D, mask, st = ctx.saved_tensors
        B, K, V = D.shape
        grad = torch.empty_like(D)
        if B * K:
            g = g_kl.contiguous()
            _call("spec_draft_kl_grad", D.device, _p(T), _p(D), _dtype_code(D), _p(mask), _p(st),
                  _p(g), B, K, T.shape[1], V, _p(grad))
        return None, grad, None


def spec_draft_kl(target_logits: torch.Tensor, draft_logits: torch.Tensor, *,
                  mask: Optional[torch.Tensor] = None) -> torch.Tensor:
    """KL(p || q) of each draft row q from its target row p, float32 [B][K], on
    the tensors the exact rule takes: target_logits [B][K+1][V] (or [B][K][V];
    rows past K are not read), draft_logits [B][K][V], one dtype.  mask bool
    [B][K]: rows that are False are not read and give 0.  The gradient is to
    draft_logits; the target is a constant."""
    T, D = _check(target_logits, "target_logits"), _check(draft_logits, "draft_logits")
    if T.dim() != 3 or D.dim() != 3 or D.shape[2] < 1:
        raise SpecVerifyError("target_logits must be [B][K+1][V] and draft_logits [B][K][V]")
    B, K, V = D.shape
    if T.shape[0] != B or T.shape[2] != V or not K <= T.shape[1] < 1 << 31:
        raise SpecVerifyError(f"target_logits has shape {tuple(T.shape)}, expected "
                              f"{(B, K + 1, V)} or {(B, K, V)}")
    _dtype_code(D)
    if T.dtype != D.dtype:
        raise SpecVerifyError(f"target_logits must be {D.dtype}, got {T.dtype}")
    if mask is not None:
        _check(mask, "mask", torch.bool, (B, K))
    _same_device(D.device, target_logits=T, mask=mask)
    if _wants_grad(T):
        raise SpecVerifyError("target_logits requires a gradient, which is not computed: detach it")
    if _wants_grad(D):
        kl = _DraftKl.apply(T, D, mask)
        _mark_leaves(kl)
        return kl
    return _kl(T, D, mask, False)[0]


# ------------------------------------------------------------- matrix product
def _linear(x, weight, bias, residual, act, out_dtype, preact):
    N, K = weight.shape
    M = x.numel() // K
    out = torch.empty((*x.shape[:-1], N), dtype=out_dtype, device=x.device)
    z = torch.empty((M, N), dtype=x.dtype, device=x.device) if preact else None
    if M:
        code = _dtype_code(x)
        ws = torch.empty(_workspace_bytes("spec_linear_workspace_bytes", code, M, N, K),
                         dtype=torch.uint8, device=x.device)
        _call("spec_linear", x.device, _p(x), _p(weight), _p(bias), _p(residual), code,
              _dtype_code(out), act, M, N, K, _p(out), _p(z), _p(ws), ws.numel())
    return out, z


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, act, out_dtype):
        need = ctx.needs_input_grad
        keep = act != 0 and any(need[:3])
        y, z = _linear(x, weight, bias, residual, act, out_dtype, keep)
        # x is read for the weight's gradient, the weight for x's
        ctx.save_for_backward(x if need[1] else None, weight if need[0] else None, z)
        ctx.act, ctx.sizes = act, (x.shape, weight.shape, x.dtype)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g_y):
        x, weight, z = ctx.saved_tensors
        x_shape, (N, K), dtype = ctx.sizes
        need = ctx.needs_input_grad
        dev = g_y.device
        M = g_y.numel() // N
        gx = torch.empty(x_shape, dtype=dtype, device=dev) if need[0] else None
        # with no rows the sums over them are 0
        make = torch.empty if M else torch.zeros
        gw = make((N, K), dtype=dtype, device=dev) if need[1] else None
        gb = make((N,), dtype=dtype, device=dev) if need[2] else None
        if M and any(need[:3]):
            g = g_y.contiguous()
            code = 1 if dtype == torch.bfloat16 else 0
            ws = torch.empty(_workspace_bytes("spec_linear_grad_workspace_bytes", code, M, N, K),
                             dtype=torch.uint8, device=dev)
            _call("spec_linear_grad", dev, _p(x), _p(weight), _p(z), _p(g), code, _dtype_code(g),
                  ctx.act, M, N, K, _p(gx), _p(gw), _p(gb), _p(ws), ws.numel())
        return gx, gw, gb, g_y if need[3] else None, None, None


def spec_linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                residual: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """residual + activation(x W^T + bias), summed in float32 and rounded once.

    x [..., K], weight [N][K] and bias [N] in one dtype, bfloat16 or float32;
    the result [..., N] and the residual, of the result's shape, in out_dtype
    (x's by default; float32 logits from bfloat16 operands with
    torch.float32).  activation: None, "relu", "gelu" (by the normal
    distribution function) or "silu".  Every tensor input has a gradient.
    """
    _check(x, "x")
    _dtype_code(x)
    _check(weight, "weight", x.dtype)
    if x.dim() < 1 or weight.dim() != 2 or weight.shape[1] != x.shape[-1] or weight.numel() == 0:
        raise SpecVerifyError(f"x must be [..., K] and weight [N][K], got {tuple(x.shape)} and "
                              f"{tuple(weight.shape)}")
    N = weight.shape[0]
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype not in (x.dtype, torch.float32):
        raise SpecVerifyError(f"out_dtype must be {x.dtype} or torch.float32, got {out_dtype}")
    if activation not in _ACTIVATIONS:
        raise SpecVerifyError(f"activation must be one of relu, gelu, silu, got {activation!r}")
    if bias is not None:
        _check(bias, "bias", x.dtype, (N,))
    if residual is not None:
        _check(residual, "residual", out_dtype, (*x.shape[:-1], N))
    _same_device(x.device, weight=weight, bias=bias, residual=residual)
    act = _ACTIVATIONS[activation]
    if _wants_grad(x, weight, bias, residual):
        y = _Linear.apply(x, weight, bias, residual, act, out_dtype)
        _mark_leaves(y)
        return y
    return _linear(x, weight, bias, residual, act, out_dtype, False)[0]
