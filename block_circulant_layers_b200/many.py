"""PyTorch autograd of the many-adapter operators: a bank of n adapters beside a projection that
all tokens share, each token of a batch using one of them or none (adapter_plan).

    plan = rd.adapter_plan(ids, n)            # once per step, for every layer
    y = bank(x, plan, base=shared(x))         # y_t = base_t + adapter_k(x_t)

Parameters are fp32, activations bf16 or fp32. The gradients of the parameters are summed in a
fixed order (the same bits on every run). As with any autograd function, a backward pass that is
captured into a CUDA graph must be the only live graph of its leaves: drop the outputs of eager
steps first.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import _binding as _b


def _base2(base, shape, dtype):
    if base is None:
        return None
    if base.shape != shape:
        raise ValueError(f"base must have shape {tuple(shape)}")
    return base.reshape(-1, shape[-1]).contiguous().to(dtype)


class _LowRankFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, a, b, plan, scale, base):
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        a2, b2 = a.detach().to(x.dtype).contiguous(), b.detach().to(x.dtype).contiguous()
        shape = x.shape[:-1] + (b.shape[1],)
        u = torch.empty(plan.T, a.shape[1], dtype=torch.float32, device=x.device) if ctx.needs_input_grad[2] else None
        y = _b.lora_fwd(x2, a2, b2, plan, scale=scale, base=_base2(base, shape, x.dtype), u=u)
        ctx.save_for_backward(x2, a2, b2, u, scale, plan.buf)
        ctx.plan, ctx.base_dtype, ctx.x_shape = plan, None if base is None else base.dtype, x.shape
        return y.reshape(shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        x2, a2, b2, u, scale, _ = ctx.saved_tensors         # fails if the plan was made again
        need = ctx.needs_input_grad
        g2 = gy.reshape(-1, gy.shape[-1]).contiguous().to(x2.dtype)
        gx = ga = gb = None
        if need[0] or need[1] or need[2]:
            gx, ga, gb = _b.lora_bwd(g2, x2, a2, b2, ctx.plan, u, scale=scale, need_grad_x=need[0],
                                     need_grad_a=need[1], need_grad_b=need[2])
        if gx is not None:
            gx = gx.reshape(ctx.x_shape)
        return gx, ga, gb, None, None, gy.to(ctx.base_dtype) if need[5] else None


class _CirculantManyFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, c, p, plan, base):
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        c_hat = _b.rdfft_fwd(c.detach().clone(memory_format=torch.contiguous_format), p)
        y = _b.circ_fwd_many(x2, c_hat, p, plan, base=_base2(base, x.shape, x.dtype))
        ctx.save_for_backward(x2, c_hat, plan.buf)
        ctx.p, ctx.plan, ctx.base_dtype = p, plan, None if base is None else base.dtype
        return y.reshape(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        x2, c_hat, _ = ctx.saved_tensors                      # fails if the plan was made again
        need = ctx.needs_input_grad
        gx = gc = None
        if need[0] or need[1]:
            g2 = gy.reshape(-1, gy.shape[-1]).contiguous().to(x2.dtype)
            gx, gc = _b.circ_bwd_many(g2, x2, c_hat, ctx.p, ctx.plan, need_grad_x=need[0], need_grad_c=need[1])
        if gx is not None:
            gx = gx.reshape(gy.shape)
        return gx, gc, None, None, gy.to(ctx.base_dtype) if need[4] else None


def low_rank_many(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, plan: _b.AdapterPlan,
                  scale: torch.Tensor | None = None, base: torch.Tensor | None = None) -> torch.Tensor:
    """y_t = base_t + scale_k b_k (a_k x_t); a (n, r, K), b (n, N, r) and base are used in x's dtype,
    which is y's. scale (n,) float32 takes no gradient."""
    if scale is not None and scale.requires_grad:
        raise ValueError("scale takes no gradient")
    return _LowRankFn.apply(x, a, b, plan, scale, base)


def block_circulant_many(x: torch.Tensor, c: torch.Tensor, p: int, plan: _b.AdapterPlan,
                         base: torch.Tensor | None = None) -> torch.Tensor:
    """y_t = base_t + W(c_k) x_t; c (n, q, q, p) float32, base used in x's dtype, which is y's."""
    return _CirculantManyFn.apply(x, c, p, plan, base)


class LowRankAdapters(torch.nn.Module):
    """n low-rank adapters in_features -> out_features of rank r, scaled by alpha / r (the buffer
    `scale`, one value per adapter, fp32 whatever dtype the module is converted to).

    a is initialised i.i.d. N(0, 1/in_features), b to zero (each adapter starts as no change).
    r is a multiple of 8 up to 128."""

    def __init__(self, n: int, in_features: int, out_features: int, r: int, alpha: float | None = None, device=None,
                 generator: torch.Generator | None = None):
        super().__init__()
        if r % 8 or not 8 <= r <= 128 or in_features % 8 or out_features % 8:
            raise ValueError("r must be a multiple of 8 up to 128, the features multiples of 8")
        a = torch.randn(n, r, in_features, device=device, dtype=torch.float32, generator=generator)
        self.a = torch.nn.Parameter(a / math.sqrt(in_features))
        self.b = torch.nn.Parameter(torch.zeros(n, out_features, r, device=device, dtype=torch.float32))
        self.register_buffer("scale", torch.full((n,), (r if alpha is None else alpha) / r, dtype=torch.float32,
                                                 device=device))

    def _apply(self, fn, recurse=True):
        # .to(dtype) and the like move the scale with the parameters but leave it fp32: rounded to
        # bf16 it would change every output by up to 2^-9
        scale = self.scale
        super()._apply(fn, recurse)
        if self.scale.dtype != torch.float32:
            self.scale = scale.to(self.scale.device)
        return self

    def forward(self, x: torch.Tensor, plan: _b.AdapterPlan, base: torch.Tensor | None = None) -> torch.Tensor:
        return low_rank_many(x, self.a, self.b, plan, self.scale.float(), base)

    def extra_repr(self) -> str:
        n, r, K = self.a.shape
        return f"n={n}, in_features={K}, out_features={self.b.shape[1]}, r={r}"


class BlockCirculantAdapters(torch.nn.Module):
    """n block-circulant adapters D -> D with block size p (BlockCirculantLinear's parameters,
    one set per adapter)."""

    def __init__(self, n: int, features: int, block: int, device=None, generator: torch.Generator | None = None):
        super().__init__()
        if block < 64 or block & (block - 1) or features % block:
            raise ValueError("block must be a power of two >= 64 dividing features")
        q = features // block
        c = torch.randn(n, q, q, block, device=device, dtype=torch.float32, generator=generator)
        self.c = torch.nn.Parameter(c / math.sqrt(features))
        self.block = block

    def forward(self, x: torch.Tensor, plan: _b.AdapterPlan, base: torch.Tensor | None = None) -> torch.Tensor:
        return block_circulant_many(x, self.c, self.block, plan, base)

    def extra_repr(self) -> str:
        return f"n={self.c.shape[0]}, features={self.c.shape[1] * self.block}, block={self.block}"
