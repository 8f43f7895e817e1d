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
  step      one AdamW step over every A and B bank and W_r, in one launch, then the
            repack of the banks' copies that the forward pass reads.

The base weights are not touched.  Nothing here computes the method's steps: the
class holds buffers and issues the calls in order on one stream.
"""
from __future__ import annotations

import torch

from . import DLM_OK, AdamW, SgmmGroup, _clean, route, route_backward, sgmm_status


class AdapterTraining:
    """The adapters of a list of projections that share one router.

    projections: [(x [T][d_in], A [E][r][d_in], B [E][d_out][r], y [T][d_out])],
                 fixed buffers of one dtype (bf16 or fp32); A and B are trained.
    router:      (x_r [T][d], W_r [d][E]) in the same dtype; W_r is trained.
    dys / dxs:   per projection dLoss/dy (filled by the caller) and dLoss/dx (added
                 to; None where it is not wanted).
    dx_r:        optional [T][d] buffer the router's share of dLoss/dx_r is added to.
    score, renorm, bias, counts: the routing, as dlm_route takes them.
    masters:     keep fp32 copies of bf16 banks and router weight; state_bits,
                 betas, weight_decay, seed: AdamW's."""

    def __init__(self, projections, router, dys, dxs, E: int, r: int, scale: float, dx_r=None, score: str = "softmax",
                 renorm: bool = True, bias=None, counts=None, masters: bool = True, state_bits: int = 32,
                 beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01, seed: int = 0):
        self.projections = list(projections)
        self.x_r, self.W_r = router
        dev, T = self.x_r.device, self.x_r.shape[0]
        self.score, self.renorm, self.bias, self.counts, self.dx_r = score, renorm, bias, counts, dx_r
        self.group = SgmmGroup(self.projections, E, r, scale)
        self.dA = [torch.zeros(A.shape, device=dev) for _, A, _, _ in self.projections]
        self.dB = [torch.zeros(B.shape, device=dev) for _, _, B, _ in self.projections]
        self.dW_r = torch.zeros(self.W_r.shape, device=dev)
        self.group.bind_grads(dys, dxs, self.dA, self.dB)
        self.logits = torch.empty((T, E), device=dev)
        self.idx = torch.empty((T, 2), dtype=torch.int32, device=dev)
        self.g, self.dg = torch.empty((T, 2), device=dev), torch.empty((T, 2), device=dev)
        # status() may be asked before the first backward()
        self.ws_forward = _clean(self.group.workspace(T, dev))
        self.ws_backward = _clean(self.group.backward_workspace(T))
        params = [t for _, A, B, _ in self.projections for t in (A, B)] + [self.W_r]
        grads = [t for pair in zip(self.dA, self.dB) for t in pair] + [self.dW_r]
        keep = masters and self.W_r.dtype != torch.float32
        self.masters = [p.float() for p in params] if keep else None
        self.opt = AdamW(params, grads, masters=self.masters, state_bits=state_bits, beta1=beta1, beta2=beta2, eps=eps,
                         weight_decay=weight_decay, seed=seed)

    def forward(self):
        """Route every token and add its adapters to every y; returns (idx, g)."""
        torch.mm(self.x_r.float(), self.W_r.float(), out=self.logits)
        route(self.logits, 2, score=self.score, bias=self.bias, renorm=self.renorm, counts=self.counts, idx=self.idx,
              g=self.g)
        self.group.run(self.idx, self.g, workspace=self.ws_forward)
        return self.idx, self.g

    def backward(self):
        """Gradients of the last forward() from the dys: dxs and dx_r added to, dA, dB
        and dW_r written."""
        self.group.backward(self.idx, self.g, self.dg, workspace=self.ws_backward)
        dl = route_backward(self.logits, self.idx, self.dg, score=self.score, renorm=self.renorm)
        torch.mm(self.x_r.float().t(), dl, out=self.dW_r)
        if self.dx_r is not None:
            self.dx_r.add_((dl @ self.W_r.float().t()).to(self.dx_r.dtype))

    def step(self, lr: float):
        """AdamW over every bank and the router's weight, then the banks' copies."""
        self.opt.step(lr)
        self.group.repack()

    def status(self) -> int:
        """DLM_OK, or DLM_EDEVICE if a routed set was rejected or a gradient was not finite (clears both)."""
        codes = [sgmm_status(self.ws_forward), sgmm_status(self.ws_backward), self.opt.status()[1]]
        return next((c for c in codes if c != DLM_OK), DLM_OK)

    def close(self):
        self.group.close()
        self.opt.close()
