"""The MoE layer on 8-bit expert weights (e4m3, one scale per 128 x 128 block).

The layer of moe.forward for serving, at half the weight bytes: the router
stays as it is, the experts' weights are quantised once when the layer is made.
Up to 8 tokens the layer is one call (moe.forward_few, whose activations stay
16-bit: a token's result is within 1.8e-3 of 64 bits on the same 8-bit weights,
as a norm); above that it is the following steps, whose activations are 8-bit
(4.4e-2 on the same weights).  Against the layer on 16-bit weights the two are
4.7e-2 and 6.4e-2 off: a token's result depends on the size of its batch.

  1. dispatch   route and copy each chosen (token, expert) row into expert order
  2. quantise   rows to 8 bits, one scale per 128 columns
  3. gate/up    8-bit grouped product, bf16 rows
  4. SwiGLU     and back to 8 bits, each row's gate weight in its scales
  5. down       8-bit grouped product: the weighted expert rows, bf16
  6. combine    y[t] = shared experts(x_t) + the token's k rows, in top-k order

with steps 2-5 once more for the shared experts, on all tokens.

What it is for: half the memory, and decode.  At d 2048, inter 1536, 64 + 4
experts it takes 36 us at 1 token, 86 at 8, 171 at 64 and 294 at 1024, where
moe.forward on 16-bit weights takes 80, 144, 228 and 326.  A prefill of 4096
tokens is slower, 750 to 800 us against 730: the 8-bit product with arbitrary
fp32 scales runs no faster than the 16-bit one (its sums leave the tensor core
every 128 columns), and the rows have to be made 8-bit.

Every computing step is a call into the CUDA library; this module only holds
the weights and passes buffers on.  There is no CPU fallback.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import moe


def _weights(name: str, W: torch.Tensor, shape, like: torch.Tensor) -> None:
    """W is of a type that moe.quantize_weight takes, of this shape, contiguous
    and on the device of `like`."""
    moe._dt(W)
    moe._want(name, W, shape, W.dtype, like)


class Fp8MoE:
    """One layer on 8-bit expert weights.

    W_router [E, d] (bfloat16) and expert_bias (float32 [E] or None) stay as
    given; W_gate_up [E, 2 inter, d], W_down [E, d, inter] and W_shared
    (moe.forward's layouts, bfloat16 or float32) are quantised here and not
    kept.  x is bfloat16 [T, d] on the weights' device, d a multiple of 256,
    inter of 16.
    Other types, shapes and devices are refused (TypeError, ValueError): the
    library sees only addresses.
    """

    def __init__(self, W_router, W_gate_up, W_down, W_shared, k: int, n_group: int,
                 topk_group: int, inter: int, n_shared: int,
                 out_dtype: torch.dtype = torch.float32, gate: str = "sigmoid",
                 expert_bias: Optional[torch.Tensor] = None):
        if W_router.dim() != 2 or W_router.shape[1] % 256:
            raise ValueError("W_router must be [E, d] with d a multiple of 256, got "
                             f"{tuple(W_router.shape)}")
        self.W_router = W_router
        self.E, self.d = E, d = W_router.shape
        moe._want("W_router", W_router, (E, d), torch.bfloat16, W_router)
        if expert_bias is not None:
            moe._want("expert_bias", expert_bias, (E,), torch.float32, W_router)
        SI = n_shared * inter
        if (n_shared > 0) != (W_shared is not None):
            raise ValueError("W_shared is given exactly when there are shared experts")
        if n_shared:
            if W_shared.numel() != 3 * SI * d:
                raise ValueError(f"W_shared must hold {3 * SI * d} values, got {W_shared.numel()}")
            _weights("W_shared", W_shared, W_shared.shape, W_router)
        _weights("W_gate_up", W_gate_up, (E, 2 * inter, d), W_router)
        _weights("W_down", W_down, (E, d, inter), W_router)
        self.k, self.n_group, self.topk_group = k, n_group, topk_group
        self.inter, self.n_shared = inter, n_shared
        self.out_dtype, self.gate, self.expert_bias = out_dtype, gate, expert_bias
        self.W_gate_up, self.s_gate_up = moe.quantize_weight(W_gate_up)
        self.W_down, self.s_down = moe.quantize_weight(W_down)
        self.W_shared = self.s_shared = None
        if n_shared:
            W_shared = W_shared.view(-1)
            n_gu = 2 * SI * d
            self.W_shared = torch.empty(W_shared.numel(), dtype=moe.E4M3, device=W_shared.device)
            s_gu, s_dn = (moe._blocks(2 * SI), d // 128), (d // 128, moe._blocks(SI))
            n_s = s_gu[0] * s_gu[1]
            self.s_shared = torch.empty(n_s + s_dn[0] * s_dn[1], dtype=torch.float32,
                                        device=W_shared.device)
            self.shared_gate_up = (self.W_shared[:n_gu].view(2 * SI, d),
                                   self.s_shared[:n_s].view(s_gu))
            self.shared_down = (self.W_shared[n_gu:].view(d, SI), self.s_shared[n_s:].view(s_dn))
            moe.quantize_weight(W_shared[:n_gu].view(2 * SI, d), *self.shared_gate_up)
            moe.quantize_weight(W_shared[n_gu:].view(d, SI), *self.shared_down)
        # 16 tokens take 164 us in the one call and 145 in steps, 8 tokens 86 and 113:
        # measured on one layer, that of the docstring above; `few` may be set lower
        # (0: always the steps) where another layer's figures cross elsewhere
        self.few = min(8, moe.few_max_tokens(self.d, self.E, k, inter, n_shared))

    def workspace_bytes(self, T: int) -> int:
        """A workspace for any batch of up to T tokens."""
        few = min(T, self.few)
        return max(moe.lib().moe_dispatch_workspace_bytes(T, self.E, self.k), 256,
                   moe.few_workspace_bytes(few, self.d, self.E, self.k, self.inter,
                                           self.n_shared) if few else 0)

    def shared(self, x: torch.Tensor,
               status_ws: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
        """The shared experts' sum, fp32 [T, d] (None without shared experts)."""
        if not self.n_shared:
            return None
        gate_up = moe.matmul_fp8(*moe.quantize_rows(x), *self.shared_gate_up, status_ws=status_ws)
        return moe.matmul_fp8(*moe.swiglu_quantize_rows(gate_up), *self.shared_down,
                              out_dtype=torch.float32, status_ws=status_ws)

    def experts(self, rows: torch.Tensor, w: torch.Tensor, counts: torch.Tensor,
                status_ws: Optional[torch.Tensor] = None) -> torch.Tensor:
        """w[r] * expert of row r, bfloat16; rows in expert order, counts[e] of
        expert e.  status_ws as moe.matmul_fp8's."""
        gate_up = moe.matmul_fp8(*moe.quantize_rows(rows), self.W_gate_up, self.s_gate_up, counts,
                                 status_ws=status_ws)
        return moe.matmul_fp8(*moe.swiglu_quantize_rows(gate_up, w), self.W_down, self.s_down,
                              counts, status_ws=status_ws)

    def forward(self, x: torch.Tensor, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y [T, d].  workspace: uint8, workspace_bytes(T), 256-byte aligned;
        moe.device_status(workspace) then gives the first device error of the
        call's steps, if any (without tokens nothing is queued and it stays as
        it was).  Calls that overlap in time need workspaces of their own."""
        if x.dim() != 2 or x.shape[1] != self.d:
            raise ValueError(f"x must be [T, {self.d}], got {tuple(x.shape)}")
        moe._want("x", x, x.shape, torch.bfloat16, self.W_router)
        moe._on_current("x", x, None)
        T = x.shape[0]
        if workspace is not None:
            moe._want("workspace", workspace, workspace.shape, torch.uint8, x)
        if T == 0:
            return torch.empty((0, self.d), dtype=self.out_dtype, device=x.device)
        if T <= self.few:
            return moe.forward_few(x, self.W_router, self.W_gate_up, self.W_down, self.W_shared,
                                   self.k, self.n_group, self.topk_group, self.inter,
                                   self.n_shared, scales=(self.s_gate_up, self.s_down,
                                                          self.s_shared),
                                   out_dtype=self.out_dtype, gate=self.gate,
                                   expert_bias=self.expert_bias, workspace=workspace)
        # dispatch clears the workspace's status words, the other steps set them
        disp = moe.dispatch(x, self.W_router, self.k, self.n_group, self.topk_group,
                            gate=self.gate, expert_bias=self.expert_bias, workspace=workspace)
        y_shared = self.shared(x, workspace)
        rows = self.experts(disp.x_perm, disp.w_perm, disp.counts, workspace)
        return moe.combine(rows, disp.slot_row, y_shared, T, self.k, self.out_dtype,
                           status_ws=workspace)

    __call__ = forward
