"""Autograd form of the layer for training.

The Sparse-BitNet Guide's module ("End-to-End Implementation: Building a
Sparse-BitLinear Layer") keeps fp32 latent weights, rebuilds the N:M mask and
the ternary weights from them on every forward, and trains them through the
straight-through estimator ("Training Stability & The Straight-Through
Estimator").  Here every step of that runs in the library's kernels:

    forward   sbl_prepare_weights (mask, scale, ternarise, pack; every call,
              so the mask follows the latent weights), sbl_quant_act (the
              int8 activations kept for the backward) and sbl_linear_q on
              those (sbl_linear, which quantises x itself, when K % 64 != 0);
    backward  sbl_linear_backward (dX = dY . (scale * W_t) to the activations,
              dW = dY^T . (x_q / s_t) to every latent weight).

The guide's module normalises x with an RMSNorm first; here that is a module of
its own (SparseBitNorm: sbl_norm, sbl_norm_backward), so SparseBitLinear's x is
the layer's input as quantised.  What else a training step around the layer
needs: SparseBitFeedForward, a gated block whose gate and up products, activation
and gradients run in sbl_ffn_gated and sbl_ffn_gated_backward, and
LinearCrossEntropy, the vocabulary projection with its loss
(sbl_linear_cross_entropy and its backward), which never holds the logits.
Argument marshalling only: no arithmetic of these layers runs in PyTorch.
"""
from __future__ import annotations

import contextlib
import math

import torch
from torch.autograd.function import once_differentiable

from . import _lib, api


def _on_device_of(x: torch.Tensor):
    # The weight preparation, the linear layers and the status word belong to
    # the current device, which need not be x's.
    return torch.cuda.device(x.device) if x.is_cuda else contextlib.nullcontext()


def _stop_on_nonfinite(where: str) -> None:
    # The kernels do not pass NaN or Inf through: a non-finite latent
    # weight or activation only sets the device status word while the
    # outputs stay finite, so a diverging run would keep training on
    # garbage.  Read the word (this waits for the stream) and stop.
    status = api.sbl_device_status()
    if status == _lib.SBL_ERR_NONFINITE:
        raise FloatingPointError(f"{where}: non-finite latent weights or activations")
    if status == _lib.SBL_ERR_INVALID_ARG:
        # never the caller's own: it prepares its weights in its own pattern
        raise _lib.SblError(status, f"found by {where} and set by an earlier call (sbl_linear_cross_entropy for a target "
                                    "outside the vocabulary, or sbl_linear for weights not in their pattern)")
    if status != _lib.SBL_OK:
        raise _lib.SblError(status, f"{where} forward")


class SparseBitLinearFunction(torch.autograd.Function):
    """y = dequant(int8(x) . ternary_NM(W)^T) with straight-through gradients.

    x: bf16 [T, K] (contiguous), weight: fp32 [O, K] latent weights; returns fp32 [T, O]."""

    @staticmethod
    def forward(ctx, x, weight, n, m, dw_ternary, check_finite=True):
        w = api.sbl_prepare_weights(weight.detach(), n, m)
        xq, s = api.sbl_quant_act(x)
        # contract the x_q kept for the backward (x is quantised once); the
        # contraction on quantised activations needs K % 64 == 0
        y = api.sbl_linear_q(xq, s, w) if weight.shape[1] % 64 == 0 else api.sbl_linear(x, w)
        if check_finite:
            _stop_on_nonfinite("SparseBitLinear")
        ctx.save_for_backward(xq, s, w.packed, w.row_scale)
        ctx.layer = (n, m, weight.shape[1], x.dtype, bool(dw_ternary))
        return y

    @staticmethod
    def backward(ctx, dy):
        xq, s, packed, row_scale = ctx.saved_tensors
        n, m, K, x_dtype, dw_ternary = ctx.layer
        need_dx, need_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        if not (need_dx or need_dw):
            return None, None, None, None, None, None
        w = api.PreparedWeights(packed, row_scale, n, m, K)
        dX, dW = api.sbl_linear_backward(dy.float().contiguous(), xq, s, w, need_dx=need_dx, need_dw=need_dw,
                                         dw_ternary=dw_ternary)
        return (dX.to(x_dtype) if need_dx else None), dW, None, None, None, None


class SparseBitLinear(torch.nn.Module):
    """The guide's Sparse-BitLinear layer without its RMSNorm: fp32 latent
    weights [out_features, in_features], N:M-sparse ternary in the forward.

    ``dw_ternary`` selects the guide module's weight gradient (taken at the
    ternary matrix, i.e. scaled by the row scale) instead of the
    straight-through gradient of the dequantised weight.  Inputs of any
    leading shape with last dimension in_features are cast to bf16 (the
    library's activation type); the output is fp32.

    With ``check_finite`` (the default) every forward reads the library's
    device status word and raises FloatingPointError when a latent weight or
    an activation was NaN or Inf (the kernels flag such values rather than
    propagate them).  Reading it waits for the stream; ``check_finite=False``
    skips the wait and the check."""

    def __init__(self, in_features: int, out_features: int, n: int = 2, m: int = 4, dw_ternary: bool = False,
                 device=None, check_finite: bool = True):
        super().__init__()
        self.in_features, self.out_features = in_features, out_features
        self.n, self.m, self.dw_ternary, self.check_finite = n, m, dw_ternary, check_finite
        self.weight = torch.nn.Parameter(torch.empty((out_features, in_features), dtype=torch.float32,
                                                     device=device))
        self.reset_parameters()

    def reset_parameters(self) -> None:
        # the same initialisation as the guide's module (torch's Linear default)
        torch.nn.init.kaiming_uniform_(self.weight, a=math.sqrt(5))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        lead = x.shape[:-1]
        x2 = x.reshape(-1, self.in_features).to(torch.bfloat16).contiguous()
        y = SparseBitLinearFunction.apply(x2, self.weight, self.n, self.m, self.dw_ternary, self.check_finite)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, {self.n}:{self.m}"


class SparseBitNormFunction(torch.autograd.Function):
    """sbl_norm with its gradients.  x: fp32 or bf16 [T, K] (contiguous), weight and
    bias (or None): fp32 [K]; returns [T, K] in x's type."""

    @staticmethod
    def forward(ctx, x, weight, bias, kind, eps):
        y, mean, rstd = api.sbl_norm(x, weight.detach(), None if bias is None else bias.detach(), kind=kind, eps=eps,
                                     with_stats=True)
        ctx.save_for_backward(x, weight, rstd, *(() if mean is None else (mean,)))
        ctx.kind = kind
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, rstd, *mean = ctx.saved_tensors
        need = ctx.needs_input_grad[:3]
        if not any(need):
            return None, None, None, None, None
        dx, dw, db = api.sbl_norm_backward(dy.to(x.dtype).contiguous(), x, weight.detach(), mean[0] if mean else None, rstd,
                                           kind=ctx.kind, need_dx=need[0], need_dw=need[1], need_db=need[2])
        return dx, dw, db, None, None


class SparseBitNorm(torch.nn.Module):
    """RMS norm (``kind="rms"``, the guide module's, with torch's epsilon) or layer
    norm (``"layer"``) over the last dimension: fp32 weight and optional bias,
    output in the input's type (types other than fp32 and bf16 go through fp32)."""

    def __init__(self, features: int, kind: str = "rms", bias: bool = False, eps: float = api.RMSNORM_EPS_F32,
                 device=None):
        super().__init__()
        self.features, self.kind, self.eps = features, kind, eps
        self.weight = torch.nn.Parameter(torch.ones((features,), dtype=torch.float32, device=device))
        self.bias = torch.nn.Parameter(torch.zeros((features,), dtype=torch.float32, device=device)) if bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        x2 = x.reshape(-1, self.features)
        x2 = (x2 if x2.dtype in (torch.float32, torch.bfloat16) else x2.float()).contiguous()
        y = SparseBitNormFunction.apply(x2, self.weight, self.bias, self.kind, self.eps)
        return y.to(x.dtype).reshape(x.shape)

    def extra_repr(self) -> str:
        return f"{self.features}, kind={self.kind}, bias={self.bias is not None}, eps={self.eps}"


class SparseBitGatedFunction(torch.autograd.Function):
    """h = act(gate(x)) * up(x) with straight-through gradients.  x: bf16 [T, K]
    (contiguous), gate and up: fp32 [F, K] latent weights; returns fp32 [T, F].
    Only x and the prepared weights are kept: the backward computes both
    products again."""

    @staticmethod
    def forward(ctx, x, gate, up, n, m, act, dw_ternary, check_finite=True):
        g, u = api.sbl_prepare_weights_grouped([gate.detach(), up.detach()], n, m)
        h = api.sbl_ffn_gated(x, g, u, act=act)
        if check_finite:
            _stop_on_nonfinite("SparseBitFeedForward")
        ctx.save_for_backward(x, g.packed, g.row_scale, u.packed, u.row_scale)
        ctx.layer = (n, m, gate.shape[1], act, bool(dw_ternary))
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, gp, gs, up, us = ctx.saved_tensors
        n, m, K, act, dw_ternary = ctx.layer
        need = ctx.needs_input_grad[:3]
        if not any(need):
            return (None,) * 8
        dx, dg, du = api.sbl_ffn_gated_backward(dh.float().contiguous(), x, api.PreparedWeights(gp, gs, n, m, K),
                                                api.PreparedWeights(up, us, n, m, K), act=act, need_dx=need[0],
                                                need_dgate=need[1], need_dup=need[2], dw_ternary=dw_ternary)
        return (None if dx is None else dx.to(x.dtype)), dg, du, None, None, None, None, None


class SparseBitFeedForward(torch.nn.Module):
    """A gated feed-forward block of Sparse-BitLinear layers: down(act(gate(x)) * up(x)).

    ``gate`` and ``up`` are fp32 latent weights [hidden_features, in_features],
    ``down`` a SparseBitLinear back to in_features (both sizes multiples of 16);
    ``act`` is "silu" or "relu2" (the squared ReLU).  x of any leading shape is cast to bf16; the output is
    fp32.  h enters ``down`` in bf16, and the gradients of h and of x are rounded to bf16 on
    their way.  ``dw_ternary`` and ``check_finite`` as in SparseBitLinear."""

    def __init__(self, in_features: int, hidden_features: int, n: int = 2, m: int = 4, act: str = "silu",
                 dw_ternary: bool = False, device=None, check_finite: bool = True):
        super().__init__()
        if in_features % 16 or hidden_features % 16:
            raise ValueError(f"in_features and hidden_features must be multiples of 16, got {in_features}, "
                             f"{hidden_features}")
        self.in_features, self.hidden_features = in_features, hidden_features
        self.n, self.m, self.act = n, m, act
        self.dw_ternary, self.check_finite = dw_ternary, check_finite
        new = lambda: torch.nn.Parameter(torch.empty((hidden_features, in_features), dtype=torch.float32, device=device))
        self.gate, self.up = new(), new()
        for w in (self.gate, self.up):
            torch.nn.init.kaiming_uniform_(w, a=math.sqrt(5))
        self.down = SparseBitLinear(hidden_features, in_features, n, m, dw_ternary=dw_ternary, device=device,
                                    check_finite=check_finite)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        x2 = x.reshape(-1, self.in_features).to(torch.bfloat16).contiguous()
        with _on_device_of(x):
            h = SparseBitGatedFunction.apply(x2, self.gate, self.up, self.n, self.m, self.act, self.dw_ternary,
                                             self.check_finite)
            return self.down(h).reshape(x.shape)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, hidden_features={self.hidden_features}, {self.n}:{self.m}, "
                f"act={self.act}")


class LinearCrossEntropyFunction(torch.autograd.Function):
    """Per-token softmax cross entropy of x . W^T (fp32 [T]) without the logits.
    x: bf16 [T, D], W: bf16 [V, D] (both contiguous), target: int64 [T]."""

    @staticmethod
    def forward(ctx, x, W, target, ignore_index):
        loss, lse = api.sbl_linear_cross_entropy(x, W.detach(), target, ignore_index=ignore_index)
        ctx.save_for_backward(x, W, target, lse)
        ctx.ignore_index = ignore_index
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        x, W, target, lse = ctx.saved_tensors
        need = ctx.needs_input_grad[:2]
        if not any(need):
            return None, None, None, None
        dx, dw = api.sbl_linear_cross_entropy_backward(dloss.float().contiguous(), x, W.detach(), target, lse,
                                                       ignore_index=ctx.ignore_index, need_dx=need[0], need_dw=need[1])
        return dx, dw, None, None


class LinearCrossEntropy(torch.nn.Module):
    """A vocabulary projection and its softmax cross entropy: the loss of hidden
    states [..., in_features] against targets [...] of int64 words.

    ``weight`` is fp32 [vocab, in_features], cast to bf16 (as x is) for the
    products; its gradient is rounded to bf16 once.  ``reduction``: "mean" over the tokens whose target is not
    ``ignore_index``, "sum", or "none" (per token, 0 for ignored ones).

    With ``check_targets`` (the default) a forward whose targets are neither words nor
    ``ignore_index`` raises IndexError before it runs.  Reading them waits for the stream;
    ``check_targets=False``, and a forward captured in a graph, skip the wait and the
    check: the loss of such a token is then NaN, and sbl_device_status reports it."""

    def __init__(self, in_features: int, vocab: int, ignore_index: int = -100, reduction: str = "mean", device=None,
                 check_targets: bool = True):
        super().__init__()
        if reduction not in ("mean", "sum", "none"):
            raise ValueError(f"reduction must be mean, sum or none, got {reduction!r}")
        self.in_features, self.vocab = in_features, vocab
        self.ignore_index, self.reduction, self.check_targets = ignore_index, reduction, check_targets
        self.weight = torch.nn.Parameter(torch.empty((vocab, in_features), dtype=torch.float32, device=device))
        torch.nn.init.normal_(self.weight, std=0.02)

    def _stop_on_bad_targets(self, t: torch.Tensor) -> None:
        if t.is_cuda and torch.cuda.is_current_stream_capturing():
            return
        bad = ((t < 0) | (t >= self.vocab)) & (t != self.ignore_index)
        if bad.any():
            raise IndexError(f"LinearCrossEntropy: target {t[bad][0].item()} is neither one of {self.vocab} words nor "
                             f"ignore_index={self.ignore_index}")

    def forward(self, x: torch.Tensor, target: torch.Tensor) -> torch.Tensor:
        if x.shape[:-1] != target.shape or x.shape[-1] != self.in_features:
            raise ValueError(f"x {tuple(x.shape)} and target {tuple(target.shape)} do not match in_features="
                             f"{self.in_features}")
        x2 = x.reshape(-1, self.in_features).to(torch.bfloat16).contiguous()
        t = target.reshape(-1).contiguous()
        if self.check_targets:
            self._stop_on_bad_targets(t)
        loss = LinearCrossEntropyFunction.apply(x2, self.weight.to(torch.bfloat16), t, self.ignore_index)
        if self.reduction == "none":
            return loss.reshape(target.shape)
        if self.reduction == "sum":
            return loss.sum()
        return loss.sum() / (t != self.ignore_index).sum()

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, vocab={self.vocab}, reduction={self.reduction}"
