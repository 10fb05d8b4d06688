"""PyTorch autograd glue over the C ABI: the layer as a torch.autograd.Function and
an nn.Module holding its weights.

Marshalling only.  The forward runs moe_forward_ws with MOE_PATH_TRAIN when a
gradient is needed (moe_forward otherwise), the backward runs moe_backward_ws
on the workspace the forward kept; every step is the library's kernels.

The layer is the one of include/moe.h: router scores Wg x, top-k with softmax
gates over the k, SwiGLU experts W2 (SiLU(W1 x) * W3 x), gate-weighted sum
("Mistral/Mixtral architecture" page, section "MoEの数学 — ルーターとゲーティング機構").
With alpha != 0 the gradient also holds the load-balance loss alpha E sum f p of
the batch's routing (subsection "ロードバランス損失"); its value comes from
moe_route_stats.

GroupedLinear is the grouped product alone (moe_grouped_mm with both gradients), for
experts of another form around moe_dispatch's segments; clip_grad_norm_ clips the
.grad of a list of parameters by their global norm (moe_clip_grads).
"""
from __future__ import annotations

import math

import torch

from . import (MOE_DTYPE_BF16, MOE_DTYPE_F32, MOE_PATH_TRAIN, moe_backward_ws, moe_clip_grads, moe_forward,
               moe_forward_ws, moe_grouped_dgrad, moe_grouped_mm, moe_grouped_wgrad, moe_train_workspace_size)


def _operand(t):
    """t as the kernels take it: contiguous and 16-byte aligned.  A gradient may be a view at any offset of a
    larger one, as that of a tensor that was flattened into a concatenation."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class MoEFunction(torch.autograd.Function):
    """out = MoE(x) with weights (Wg, W1, W3, W2); gradients for x and every weight.

    Weight gradients are summed in fp32 and rounded once to each weight's dtype
    (for bf16 weights, inside the GEMM epilogue).
    """

    @staticmethod
    def forward(ctx, x, Wg, W1, W3, W2, k: int, alpha: float = 0.0):
        T, d = x.shape
        E, F, _ = W1.shape
        code = MOE_DTYPE_BF16 if x.dtype == torch.bfloat16 else MOE_DTYPE_F32
        ws = torch.empty(max(moe_train_workspace_size(T, d, F, E, k, code), 1), dtype=torch.uint8, device=x.device)
        out = moe_forward_ws(x, Wg, W1, W3, W2, k, path=MOE_PATH_TRAIN, workspace=ws)
        ctx.save_for_backward(x, Wg, W1, W3, W2)
        ctx.ws, ctx.k, ctx.alpha = ws, k, float(alpha)
        return out

    @staticmethod
    def backward(ctx, dout):
        x, Wg, W1, W3, W2 = ctx.saved_tensors
        wd = torch.bfloat16 if W1.dtype == torch.bfloat16 else torch.float32
        g, _ = moe_backward_ws(x, Wg, W1, W3, W2, _operand(dout), ctx.k, ctx.ws, alpha=ctx.alpha, wgrad_dtype=wd)
        ctx.ws = None
        grads = (g["dx"], g["dWg"].to(Wg.dtype), g["dW1"].to(W1.dtype), g["dW3"].to(W3.dtype), g["dW2"].to(W2.dtype))
        if torch.is_grad_enabled():   # create_graph: the gradients are functions of all of these
            grads = FirstDerivatives.apply(len(grads), *grads, x, Wg, W1, W3, W2, dout)
        return (*grads, None, None)


class FirstDerivatives(torch.autograd.Function):
    """The layer's gradients beside what they are functions of: a derivative of them is not built, and raises
    instead of being left out of a sum."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tensors[:n]

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("second derivatives of the MoE layer are not supported")


class SparseMoE(torch.nn.Module):
    """The MoE feed-forward layer with its weights as parameters (nn.Linear layouts):
    Wg [E][d], W1 [E][F][d], W3 [E][F][d], W2 [E][d][F].  Input [..., d]."""

    def __init__(self, d: int, ffn: int, E: int = 8, k: int = 2, alpha: float = 0.0, dtype=torch.bfloat16,
                 device="cuda"):
        super().__init__()
        self.k, self.alpha = k, alpha
        kw = dict(dtype=dtype, device=device)
        self.Wg = torch.nn.Parameter(torch.randn(E, d, **kw) / math.sqrt(d))
        self.W1 = torch.nn.Parameter(torch.randn(E, ffn, d, **kw) / math.sqrt(d))
        self.W3 = torch.nn.Parameter(torch.randn(E, ffn, d, **kw) / math.sqrt(d))
        self.W2 = torch.nn.Parameter(torch.randn(E, d, ffn, **kw) / math.sqrt(ffn))

    def forward(self, x):
        shape = x.shape
        x2 = _operand(x.reshape(-1, shape[-1]))
        weights = (self.Wg, self.W1, self.W3, self.W2)
        if torch.is_grad_enabled() and (x2.requires_grad or any(w.requires_grad for w in weights)):
            out = MoEFunction.apply(x2, *weights, self.k, self.alpha)
        else:
            out = moe_forward(x2, *(w.detach() for w in weights), self.k)
        return out.reshape(shape)


class GroupedMmFunction(torch.autograd.Function):
    """y_r = W_e x_r for the rows of every expert's segment, with gradients for x and W.

    Rows in no segment are zero in y and in the gradient of x.  The gradients are functions with gradients of
    their own, the same three products over again, so derivatives of any order are right.
    """

    @staticmethod
    def forward(ctx, x, W, offsets, counts=None):
        y = torch.zeros((x.shape[0], W.shape[1]), dtype=x.dtype, device=x.device)
        moe_grouped_mm(x, W, offsets, counts, out=y)
        ctx.save_for_backward(x, W, offsets, counts)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, W, offsets, counts = ctx.saved_tensors
        dy = _operand(dy)
        dx = dW = None
        if ctx.needs_input_grad[0]:
            dx = GroupedDgradFunction.apply(dy, W, offsets, counts)
        if ctx.needs_input_grad[1]:
            dW = GroupedWgradFunction.apply(dy, x, offsets, counts)
        return dx, dW, None, None


class GroupedDgradFunction(torch.autograd.Function):
    """dx_r = W_e^T dy_r for the rows of every expert's segment, zero elsewhere."""

    @staticmethod
    def forward(ctx, dy, W, offsets, counts=None):
        dx = torch.zeros((dy.shape[0], W.shape[2]), dtype=dy.dtype, device=dy.device)
        moe_grouped_dgrad(dy, W, offsets, counts, out=dx)
        ctx.save_for_backward(dy, W, offsets, counts)
        return dx

    @staticmethod
    def backward(ctx, g):
        dy, W, offsets, counts = ctx.saved_tensors
        g = _operand(g)
        ddy = GroupedMmFunction.apply(g, W, offsets, counts) if ctx.needs_input_grad[0] else None
        dW = GroupedWgradFunction.apply(dy, g, offsets, counts) if ctx.needs_input_grad[1] else None
        return ddy, dW, None, None


class GroupedWgradFunction(torch.autograd.Function):
    """dW_e = sum over segment e's rows of dy_r x_r^T."""

    @staticmethod
    def forward(ctx, dy, x, offsets, counts=None):
        ctx.save_for_backward(dy, x, offsets, counts)
        return moe_grouped_wgrad(dy, x, offsets, counts)

    @staticmethod
    def backward(ctx, g):
        dy, x, offsets, counts = ctx.saved_tensors
        g = _operand(g)
        ddy = GroupedMmFunction.apply(x, g, offsets, counts) if ctx.needs_input_grad[0] else None
        dx = GroupedDgradFunction.apply(dy, g, offsets, counts) if ctx.needs_input_grad[1] else None
        return ddy, dx, None, None


class GroupedLinear(torch.nn.Module):
    """One bias-free linear map per expert over ragged segments of rows: W [E][out][in]."""

    def __init__(self, E: int, in_features: int, out_features: int, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.W = torch.nn.Parameter(torch.randn(E, out_features, in_features, dtype=dtype, device=device) /
                                    math.sqrt(in_features))

    def forward(self, x, offsets, counts=None):
        return GroupedMmFunction.apply(_operand(x), self.W, offsets, counts)


def _contiguous_alike(g):
    """The elements of g in the order of its memory where they fill it (a transposed gradient does), else a copy."""
    if g.is_contiguous():
        return g
    v = g.permute(sorted(range(g.dim()), key=g.stride, reverse=True))
    return v if v.is_contiguous() else g.contiguous()


@torch.no_grad()
def clip_grad_norm_(parameters, max_norm: float, eps: float = 1e-6):
    """Clip the gradients of the parameters (one, or an iterable) in place by their global 2-norm; returns
    the norm before clipping (float32 [1], on the parameters' device).  No host synchronisation."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    parameters = list(parameters)
    grads = [p.grad for p in parameters if p.grad is not None]
    if not grads:
        return torch.zeros(1, device=parameters[0].device if parameters else None)
    flat = [_contiguous_alike(g) for g in grads]
    norm = moe_clip_grads(flat, max_norm, eps=eps)[0]
    for g, f in zip(grads, flat):
        if f.data_ptr() != g.data_ptr():
            g.copy_(f)
    return norm
