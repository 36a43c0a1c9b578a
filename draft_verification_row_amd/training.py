"""Operators that train a draft head beside its plain matrix products, with
their gradients: the embedding lookup, a gated block's projections, and the
cross entropy of the output layer, whose logits are never kept.

They follow the operators of `heads`: contiguous GPU tensors on one device, run
on that device's current stream; results carry a gradient (first order) where
an input requires one; calls may be captured into a graph, with the same
condition on other graphs of the same leaves.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import SpecVerifyError, _check, _dtype_code
from .heads import (_ACTIVATIONS, _call, _grad_in, _mark_leaves, _p, _same_device, _wants_grad,
                    _workspace_bytes)

__all__ = ["spec_embedding", "spec_gated_linear", "spec_cross_entropy", "CrossEntropyResult"]


class CrossEntropyResult(NamedTuple):
    loss: torch.Tensor    # float32 [...]
    lse: torch.Tensor     # float32 [...]
    status: torch.Tensor  # int32 [...]: 1 for a token outside [-1, V)


def _room(query: str, device: torch.device, *sizes: int) -> torch.Tensor:
    """An uninitialized workspace of the size that the library asks for."""
    return torch.empty(_workspace_bytes(query, *sizes), dtype=torch.uint8, device=device)


# ------------------------------------------------------------ embedding lookup
def _embedding(weight, tokens, scale):
    V, H = weight.shape
    n = tokens.numel()
    out = torch.empty((*tokens.shape, H), dtype=weight.dtype, device=weight.device)
    if n:
        code = _dtype_code(weight)
        _workspace_bytes("spec_embedding_grad_workspace_bytes", code, n, V, H)  # checks the sizes
        _call("spec_embedding", weight.device, _p(weight), code, _p(tokens), scale, n, V, H, _p(out))
    return out


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, tokens, scale):
        ctx.save_for_backward(tokens)
        ctx.scale, ctx.sizes, ctx.dtype = scale, weight.shape, weight.dtype
        return _embedding(weight, tokens, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_y):
        tokens, = ctx.saved_tensors
        V, H = ctx.sizes
        n, dev = tokens.numel(), g_y.device
        make = torch.empty if n else torch.zeros
        grad = make((V, H), dtype=ctx.dtype, device=dev)
        if n:
            g = g_y.contiguous()
            code = _dtype_code(g)
            ws = _room("spec_embedding_grad_workspace_bytes", dev, code, n, V, H)
            _call("spec_embedding_grad", dev, _p(tokens), _p(g), code, ctx.scale, n, V, H, _p(grad),
                  _p(ws), ws.numel())
        return grad, None, None


def spec_embedding(weight: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0
                   ) -> torch.Tensor:
    """scale * weight[tokens], rounded once: [*tokens.shape][H].

    weight [V][H] bfloat16 or float32; tokens int32.  A token of -1 pads its
    position, as in the rules' outputs, and gives zeros; any other outside
    [0, V) gives NaN.  The weight has a gradient, a whole table: each token's
    positions are summed in float32, in a fixed order.
    """
    W = _check(weight, "weight")
    if W.dim() != 2 or W.numel() == 0:
        raise SpecVerifyError(f"weight must be [V][H], got {tuple(W.shape)}")
    _dtype_code(W)
    _check(tokens, "tokens", torch.int32)
    _same_device(W.device, tokens=tokens)
    scale = float(scale)
    if not abs(scale) <= torch.finfo(torch.float32).max:
        raise SpecVerifyError(f"scale must be finite in float32, got {scale}")
    if _wants_grad(W):
        y = _Embedding.apply(W, tokens, scale)
        _mark_leaves(y)
        return y
    return _embedding(W, tokens, scale)


# ------------------------------------------------------------ gated projections
def _gated(x, gate, up, act, keep):
    N, K = gate.shape
    M = x.numel() // K
    out = torch.empty((*x.shape[:-1], N), dtype=x.dtype, device=x.device)
    g, u = ((torch.empty((M, N), dtype=torch.float32, device=x.device) for _ in range(2)) if keep
            else (None, None))
    if M:
        code = _dtype_code(x)
        ws = _room("spec_gated_linear_workspace_bytes", x.device, code, M, N, K)
        _call("spec_gated_linear", x.device, _p(x), _p(gate), _p(up), code, act, M, N, K, _p(out),
              _p(g), _p(u), _p(ws), ws.numel())
    return out, g, u


class _GatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, up, act):
        need = ctx.needs_input_grad
        y, g, u = _gated(x, gate, up, act, True)
        # x is read for the weights' gradients, the weights for x's
        ctx.save_for_backward(x if need[1] or need[2] else None, gate if need[0] else None,
                              up if need[0] else None, g, u)
        ctx.act, ctx.sizes = act, (x.shape, gate.shape, x.dtype)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g_y):
        x, gate, up, g, u = ctx.saved_tensors
        x_shape, (N, K), dtype = ctx.sizes
        need = ctx.needs_input_grad
        dev = g_y.device
        M = g_y.numel() // N
        gx = torch.empty(x_shape, dtype=dtype, device=dev) if need[0] else None
        make = torch.empty if M else torch.zeros  # with no rows the sums over them are 0
        gg, gu = (make((N, K), dtype=dtype, device=dev) if n else None for n in need[1:3])
        if M:
            g_y = g_y.contiguous()
            code = _dtype_code(g_y)
            ws = _room("spec_gated_linear_grad_workspace_bytes", dev, code, M, N, K)
            _call("spec_gated_linear_grad", dev, _p(x), _p(gate), _p(up), _p(g), _p(u), _p(g_y),
                  code, ctx.act, M, N, K, _p(gx), _p(gg), _p(gu), _p(ws), ws.numel())
        return gx, gg, gu, None


def spec_gated_linear(x: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, *,
                      activation: Optional[str] = "silu") -> torch.Tensor:
    """activation(x gate^T) * (x up^T), element by element, from float32 sums
    and rounded once: the gated block's half before its down projection (for
    which spec_linear takes the block's input as residual).

    x [..., K], gate and up [N][K] in one dtype, bfloat16 or float32; the
    result [..., N] too.  activation as spec_linear's.  Every tensor input has
    a gradient; for it both products are kept in float32.
    """
    _check(x, "x")
    _dtype_code(x)
    _check(gate, "gate", x.dtype)
    if x.dim() < 1 or gate.dim() != 2 or gate.shape[1] != x.shape[-1] or gate.numel() == 0:
        raise SpecVerifyError(f"x must be [..., K] and gate [N][K], got {tuple(x.shape)} and "
                              f"{tuple(gate.shape)}")
    _check(up, "up", x.dtype, gate.shape)
    if activation not in _ACTIVATIONS:
        raise SpecVerifyError(f"activation must be one of relu, gelu, silu, got {activation!r}")
    _same_device(x.device, gate=gate, up=up)
    act = _ACTIVATIONS[activation]
    if _wants_grad(x, gate, up):
        y = _GatedLinear.apply(x, gate, up, act)
        _mark_leaves(y)
        return y
    return _gated(x, gate, up, act, False)[0]


# --------------------------------------------------------------- cross entropy
def _cross_entropy(x, weight, bias, tokens, keep):
    V, K = weight.shape
    M, dev = tokens.numel(), x.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = CrossEntropyResult(torch.empty(tokens.shape, **f32), torch.empty(tokens.shape, **f32),
                             torch.empty(tokens.shape, dtype=torch.int32, device=dev))
    stats = torch.empty((M, 2), **f32) if keep else None
    if M:
        code = _dtype_code(x)
        ws = _room("spec_cross_entropy_workspace_bytes", dev, code, M, V, K)
        _call("spec_cross_entropy", dev, _p(x), _p(weight), _p(bias), code, _p(tokens), M, V, K,
              _p(out.loss), _p(out.lse), _p(out.status), _p(stats), _p(ws), ws.numel())
    return out, stats


class _CrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, tokens):
        out, stats = _cross_entropy(x, weight, bias, tokens, True)
        ctx.save_for_backward(x, weight, bias, tokens, stats)
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(out.status)
        return tuple(out)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_loss, g_lse, _):
        x, weight, bias, tokens, stats = ctx.saved_tensors
        if g_loss is None and g_lse is None:
            return None, None, None, None
        need = ctx.needs_input_grad
        V, K = weight.shape
        M = tokens.numel()
        make = torch.empty_like if M else torch.zeros_like
        gx, gw, gb = (make(t) if n else None for t, n in zip((x, weight, bias), need))
        if M:
            code = _dtype_code(x)
            gl, ge = _grad_in(g_loss), _grad_in(g_lse)
            ws = _room("spec_cross_entropy_grad_workspace_bytes", x.device, code, M, V, K)
            _call("spec_cross_entropy_grad", x.device, _p(x), _p(weight), _p(bias), code,
                  _p(tokens), _p(stats), _p(gl), _p(ge), M, V, K, _p(gx), _p(gw), _p(gb), _p(ws),
                  ws.numel())
        return gx, gw, gb, None


def spec_cross_entropy(x: torch.Tensor, weight: torch.Tensor, tokens: torch.Tensor,
                       bias: Optional[torch.Tensor] = None) -> CrossEntropyResult:
    """-log softmax(x weight^T + bias)[token] for one token per row of x, and the
    row's log-sum-exp, without the logits in memory: forward a tile leaves only
    its rows' maxima and sums, backward the logits are made again a piece of the
    vocabulary at a time.

    x [..., K], weight [V][K] and bias [V] in one dtype, bfloat16 or float32;
    tokens int32 with x's leading shape.  A token of -1 pads its row, as in the
    rules' outputs: the row enters no result and gets 0 and 0.  A bias of -inf
    takes a token out of the vocabulary.  x, weight and bias have gradients.
    """
    _check(x, "x")
    _dtype_code(x)
    _check(weight, "weight", x.dtype)
    if x.dim() < 1 or weight.dim() != 2 or weight.shape[1] != x.shape[-1] or weight.numel() == 0:
        raise SpecVerifyError(f"x must be [..., K] and weight [V][K], got {tuple(x.shape)} and "
                              f"{tuple(weight.shape)}")
    _check(tokens, "tokens", torch.int32, x.shape[:-1])
    if bias is not None:
        _check(bias, "bias", x.dtype, weight.shape[:1])
    _same_device(x.device, weight=weight, tokens=tokens, bias=bias)
    if _wants_grad(x, weight, bias):
        out = CrossEntropyResult(*_CrossEntropy.apply(x, weight, bias, tokens))
        _mark_leaves(out.loss)
        return out
    return _cross_entropy(x, weight, bias, tokens, False)[0]
