"""Training of the routed adapters, built from this library's entry points.

One router decision per token serves every adapted projection (decide once), in
training as in decoding.  A step, per batch of T tokens:

  forward   logits = x_r W_r (a library product), dlm_route: every token's top 2 of
            E experts and their weights, then the grouped SGMM: for every
            projection y += s sum_k g_k (x A_k^T) B_k^T on top of what the base
            product left in y;
  backward  (the caller has put dLoss/dy into every dy) the SGMM's gradients: dx is
            joined in place, dA and dB, and dg, the gradient of the gates, summed
            over the projections; dlm_route_backward takes dg to the logits, and two
            library products take it to W_r and to the router's input;
  step      one AdamW step over every A and B bank and W_r, in one launch, or one step
            of orthogonalised momentum (Muon) over their matrices, then the repack of the
            banks' copies that the forward pass reads.

With a base in 8 bits the step holds the base product too: forward writes its share of
every y before the adapters', backward its share of every dx.  With a balance loss the
forward pass leaves it in `loss`, and backward adds its gradient to the logits'.

The base weights are not touched.  Nothing here computes the method's steps: the
class holds buffers and issues the calls in order on one stream.
"""
from __future__ import annotations

import torch

from . import (DLM_OK, AdamW, Int8Group, Muon, SgmmGroup, _clean, balance, balance_backward, balance_workspace_size, route,
               route_backward, sgmm_status)


class AdapterTraining:
    """The adapters of a list of projections that share one router.

    projections: [(x [T][d_in], A [E][r][d_in], B [E][d_out][r], y [T][d_out])],
                 fixed buffers of one dtype (bf16 or fp32); A and B are trained.  Buffers
                 may hold more rows than x_r: the others are left as they are.
    router:      (x_r [T][d], W_r [d][E]) in the same dtype; W_r is trained.
    dys / dxs:   per projection dLoss/dy (filled by the caller) and dLoss/dx (added
                 to; None, or an entry None, where it is not wanted).
    dx_r:        optional [T][d] buffer the router's share of dLoss/dx_r is added to.
    score, renorm, bias, counts: the routing, as dlm_route takes them.
    masters:     keep fp32 copies of bf16 banks and router weight; state_bits,
                 betas, weight_decay, seed: AdamW's.
    base:        per projection the frozen base weight in 8 bits, (W [d_out][d_in] int8,
                 w_scale [d_out]): forward() then writes the base product to y, and
                 backward() its gradient to dx (written, problems that share a dx summed),
                 under the adapters' shares.
    optimizer:   "adamw" or "muon" (momentum, muon_scale: Muon's, "shape" with the outputs and
                 inputs of each map, W_r's too; state_bits 32).
    alpha, zeta, offsets: the balance loss over the sequences that offsets cut the rows
                 into (balance()'s arguments); none where both are 0.  Its value is `loss`."""

    def __init__(self, projections, router, dys, dxs, E: int, r: int, scale: float, dx_r=None, score: str = "softmax",
                 renorm: bool = True, bias=None, counts=None, masters: bool = True, state_bits: int = 32,
                 beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01, seed: int = 0,
                 base=None, optimizer: str = "adamw", momentum: float = 0.95, muon_scale="rms", alpha: float = 0.0,
                 zeta: float = 0.0, offsets=None):
        if optimizer not in ("adamw", "muon"):
            raise ValueError(f"optimizer is 'adamw' or 'muon', got {optimizer!r}")
        if optimizer == "muon" and state_bits != 32:
            raise ValueError("muon's momentum has 32 bits")
        self.projections, dys = list(projections), list(dys)
        dxs = None if dxs is None else list(dxs)
        self.x_r, self.W_r = router
        dev, T = self.x_r.device, self.x_r.shape[0]
        f32 = dict(dtype=torch.float32, device=dev)
        self.score, self.renorm, self.bias, self.counts, self.dx_r = score, renorm, bias, counts, dx_r
        self.group = SgmmGroup(self.projections, E, r, scale)
        self.base = None
        if base is not None:
            base = list(base)
            if len(base) != len(self.projections):
                raise ValueError("one base weight (W, w_scale) per projection")
            self.base = Int8Group([(x, W, ws, y) for (x, _, _, y), (W, ws) in zip(self.projections, base)])
            self.base.bind_grads(dys, dxs)
            self.ws_base, self.ws_base_backward = self.base.workspace(T), self.base.backward_workspace(T)
        self.dA = [torch.zeros(A.shape, **f32) for _, A, _, _ in self.projections]
        self.dB = [torch.zeros(B.shape, **f32) for _, _, B, _ in self.projections]
        self.dW_r = torch.zeros(self.W_r.shape, **f32)
        self.group.bind_grads(dys, dxs, self.dA, self.dB)
        self.logits = torch.empty((T, E), **f32)
        self.idx = torch.empty((T, 2), dtype=torch.int32, device=dev)
        self.g, self.dg = torch.empty((T, 2), **f32), torch.empty((T, 2), **f32)
        # status() may be asked before the first backward()
        self.ws_forward = _clean(self.group.workspace(T, dev))
        self.ws_backward = _clean(self.group.backward_workspace(T))
        params = [t for _, A, B, _ in self.projections for t in (A, B)] + [self.W_r]
        grads = [t for pair in zip(self.dA, self.dB) for t in pair] + [self.dW_r]
        keep = masters and self.W_r.dtype != torch.float32
        self.masters = [p.float() for p in params] if keep else None
        if optimizer == "muon":
            scales = list(muon_scale) if isinstance(muon_scale, (list, tuple)) else [muon_scale] * len(params)
            if len(scales) == len(params) and scales[-1] == "shape":  # W_r has its inputs first
                scales[-1] = max(1.0, E / self.W_r.shape[0]) ** 0.5
            self.opt = Muon(params, grads, masters=self.masters, momentum=momentum, weight_decay=weight_decay, scale=scales)
        else:
            self.opt = AdamW(params, grads, masters=self.masters, state_bits=state_bits, beta1=beta1, beta2=beta2, eps=eps,
                             weight_decay=weight_decay, seed=seed)
        self.balance, self.loss = None, None
        if alpha or zeta:
            self.balance = dict(score=score, alpha=alpha, zeta=zeta, offsets=offsets)
            S = 1 if offsets is None else offsets.shape[0] - 1
            self.loss, self.probs = torch.empty(2, **f32), torch.empty((S, E), **f32)
            self.slots = torch.empty((S, E), dtype=torch.int32, device=dev)
            self.rows = torch.empty(S, dtype=torch.int32, device=dev)
            self.ws_balance = torch.empty(balance_workspace_size(T, E, S), dtype=torch.uint8, device=dev)

    def forward(self):
        """Route every token and add its adapters to every y; returns (idx, g)."""
        torch.mm(self.x_r.float(), self.W_r.float(), out=self.logits)
        route(self.logits, 2, score=self.score, bias=self.bias, renorm=self.renorm, counts=self.counts, idx=self.idx,
              g=self.g)
        if self.balance:
            balance(self.logits, self.idx, loss=self.loss, counts=self.slots, rows=self.rows, probs=self.probs,
                    workspace=self.ws_balance, **self.balance)
        if self.base:
            self.base.run(T=self.x_r.shape[0], workspace=self.ws_base)
        self.group.run(self.idx, self.g, workspace=self.ws_forward)
        return self.idx, self.g

    def backward(self):
        """Gradients of the last forward() from the dys: dxs (with a base, written) and
        dx_r added to, dA, dB and dW_r written."""
        if self.base:
            self.base.backward(T=self.x_r.shape[0], workspace=self.ws_base_backward)
        self.group.backward(self.idx, self.g, self.dg, workspace=self.ws_backward)
        dl = route_backward(self.logits, self.idx, self.dg, score=self.score, renorm=self.renorm)
        if self.balance:
            balance_backward(self.logits, self.slots, self.rows, 2, dlogits=dl, accumulate=True, **self.balance)
        torch.mm(self.x_r.float().t(), dl, out=self.dW_r)
        if self.dx_r is not None:
            self.dx_r.add_((dl @ self.W_r.float().t()).to(self.dx_r.dtype))

    def step(self, lr: float):
        """The optimizer over every bank and the router's weight, then the banks' copies."""
        self.opt.step(lr)
        self.group.repack()

    def status(self) -> int:
        """DLM_OK, or DLM_EDEVICE if a routed set was rejected or a gradient was not finite (clears both)."""
        opt = self.opt.status()
        codes = [sgmm_status(self.ws_forward), sgmm_status(self.ws_backward), opt if isinstance(opt, int) else opt[1]]
        return next((c for c in codes if c != DLM_OK), DLM_OK)

    def close(self):
        self.group.close()
        self.opt.close()
        if self.base:
            self.base.close()
