"""One MoE layer in its place on the residual stream (orchestration only).

    n = norm(x) * w_pre             the layer's input
    b = layer(n)
    y = x + alpha * gate_t * post(b)    post(b) = norm(b) * w_post, or b

The layer trains its quantizer scales (AngelSlim mcore_qad article, section 一); the
norms' weights are frozen with the rest unless ``learn_norms``. ``forward`` and
``backward`` are the training step around the layer's own, ``forward_int8`` is the
served w8a8 form, where the input norm leaves int8 codes that the layer's products
read. All buffers are allocated once; y, dx and db are the block's own, overwritten
by its next call.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (FQ_OP_NORM, fq_norm_residual_bwd, fq_norm_residual_fwd, fq_workspace_bytes)
from .layer import MoEFakeQuantLayer


def _at(t: torch.Tensor) -> int:
    return t.untyped_storage().data_ptr()


def _in(t: torch.Tensor, *buffers: torch.Tensor) -> bool:
    return any(_at(t) == _at(b) for b in buffers)


def _shifted(t: torch.Tensor, buffer: torch.Tensor) -> bool:
    """Rows of the buffer, but not its first ones: written in place, each would land on another."""
    return _in(t, buffer) and t.data_ptr() != buffer.data_ptr()


class MoEFakeQuantBlock:
    def __init__(self, layer: MoEFakeQuantLayer, w_pre: torch.Tensor,
                 w_post: Optional[torch.Tensor] = None, alpha: float = 1.0, eps: float = 1e-6,
                 learn_norms: bool = False):
        """w_pre, w_post [H] bf16. learn_norms: the backward also gives dw_pre (and
        dw_post), fp32 [H]."""
        H, T = layer.H, layer.T_max
        for name, w in (("w_pre", w_pre), ("w_post", w_post)):
            if w is not None and (w.shape != (H,) or w.dtype != torch.bfloat16):
                raise ValueError(f"{name} must be bf16 [{H}]")
        self.layer, self.w_pre, self.w_post = layer, w_pre, w_post
        self.alpha, self.eps = alpha, eps
        bf = dict(dtype=torch.bfloat16, device=layer.dev)
        f32 = dict(dtype=torch.float32, device=layer.dev)
        self.n = torch.empty(T, H, **bf)
        self.y = torch.empty(T, H, **bf)
        self.dx = torch.empty(T, H, **bf)
        self.db = torch.empty(T, H, **bf)
        # the layer's output lives in buffers that layers share: kept here where the
        # backward needs it
        self.b = torch.empty(T, H, **bf)
        self.dgate = torch.empty(T, **f32)
        self.dw_pre = torch.empty(H, **f32) if learn_norms else None
        self.dw_post = torch.empty(H, **f32) if learn_norms and w_post is not None else None
        n = max(256, fq_workspace_bytes(FQ_OP_NORM, (1, T, H), 0, 0)) if learn_norms else 256
        self.ws = torch.empty(n, dtype=torch.uint8, device=layer.dev)
        self.x = self.gate = None

    def _check(self, x: torch.Tensor, gate: Optional[torch.Tensor]) -> int:
        T = x.shape[0]
        if x.shape != (T, self.layer.H) or x.dtype != torch.bfloat16 or T > self.layer.T_max:
            raise ValueError(f"x must be bf16 [T <= {self.layer.T_max}, {self.layer.H}]")
        if gate is not None and (gate.shape != (T,) or gate.dtype != torch.float32):
            raise ValueError(f"gate must be float32 [{T}]")
        if gate is not None and _in(gate, self.dgate):
            raise ValueError("gate lies in the block's dgate, which the backward overwrites")
        return T

    def _join(self, x, b, gate, T):
        fq_norm_residual_fwd(x, b, gate, self.alpha, self.w_post, None, self.eps, T, self.layer.H,
                             self.y[:T])
        return self.y[:T]

    def forward(self, x: torch.Tensor, expert_ids: torch.Tensor, probs: torch.Tensor,
                gate: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y [T, H]. x is kept by reference for the backward, and gate; neither may be
        changed before it, nor may x lie in a buffer that the layer or the block overwrites."""
        T = self._check(x, gate)
        if _in(x, self.y, self.n, self.b, self.db, self.dx) or _at(x) in self.layer._scratch_at:
            raise ValueError("x lies in a buffer that the layer or the block overwrites before the "
                             "backward")
        fq_norm_residual_fwd(x, None, None, 1.0, None, self.w_pre, self.eps, T, self.layer.H, None,
                             self.n[:T])
        b = self.layer.forward(self.n[:T], expert_ids, probs)
        if self.w_post is not None or gate is not None:
            self.b[:T].copy_(b)
        self.x, self.gate = x, gate
        return self._join(x, b, gate, T)

    def backward(self, probs: torch.Tensor, dy: torch.Tensor):
        """dx, and the layer's scale gradients (ds_gu, ds_d); dgate [T], dw_pre and dw_post
        are the block's where they exist. dy may be the block's own dx, from its first row on."""
        if self.x is None:
            raise ValueError("backward needs a forward")
        T, H = self.x.shape[0], self.layer.H
        if dy.shape != (T, H) or dy.dtype != torch.bfloat16:
            raise ValueError(f"dy must be bf16 [{T}, {H}]")
        if _in(dy, self.db) or _shifted(dy, self.dx) or _at(dy) in self.layer._scratch_at:
            raise ValueError("dy lies in a buffer that the layer's backward overwrites")
        fq_norm_residual_bwd(dy, None, None, self.b[:T], self.gate, self.alpha, self.w_post, None,
                             self.eps, T, H, None, self.db[:T],
                             None if self.gate is None else self.dgate[:T], self.dw_post, None, self.ws)
        dn, ds_gu, ds_d = self.layer.backward(self.n[:T], probs, self.db[:T])
        fq_norm_residual_bwd(dy, dn, self.x, None, None, 1.0, None, self.w_pre, self.eps, T, H,
                             self.dx[:T], None, None, None, self.dw_pre, self.ws)
        return self.dx[:T], ds_gu, ds_d

    def forward_int8(self, x: torch.Tensor, expert_ids: torch.Tensor, probs: torch.Tensor,
                     gate: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y over the layer's exported int8 stacks: the norm's output goes to the products
        as codes with a scale a token and is never stored in bf16. x may be the block's own
        y, from its first row on."""
        T = self._check(x, gate)
        self.layer._check_int8()
        if _in(x, *(self.layer.i8[k] for k in ("a", "o", "out"))) or _shifted(x, self.y):
            raise ValueError("x lies in a buffer that the layer's steps overwrite, or in other rows of y")
        codes, scale = self.layer.i8["x_codes"], self.layer.i8["x_scale"]
        fq_norm_residual_fwd(x, None, None, 1.0, None, self.w_pre, self.eps, T, self.layer.H, None, None,
                             codes, scale)
        b = self.layer.forward_int8_codes(codes, scale, T, expert_ids, probs)
        return self._join(x, b, gate, T)
