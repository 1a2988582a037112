"""Optimizer state for a list of parameters: allocates the moments (with torch, on the parameters'
device) and calls mok_grad_sumsq, mok_adamw and mok_muon. Argument marshalling only."""
from __future__ import annotations

from typing import Optional

import torch

from . import adamw_plan, mok_adamw, mok_grad_sumsq, mok_muon, muon_plan, sumsq_plan


class MokAdamW:
    """AdamW over parameters updated in place from gradients that stay in the given tensors.

    params: float32 masters or bfloat16; grads: float32 or bfloat16 (each list of one type); copies:
    bfloat16 copies of float32 masters, written by every step (the layer's weights; None in the place of
    a master without one). state: "float32" or "mxfp8" moments. max_norm clips by the norm of all
    gradients, which stays on the device; with check_finite (or max_norm) a step whose norm is not finite
    changes nothing."""

    def __init__(self, params, grads, copies=None, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.0, max_norm: Optional[float] = None, check_finite: bool = False,
                 state: str = "float32", seed: int = 0):
        if state not in ("float32", "mxfp8"):
            raise ValueError("state is float32 or mxfp8")
        self.params, self.grads, self.copies = list(params), list(grads), copies
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.max_norm, self.seed, self.steps = max_norm, seed, 0
        flat = [p.numel() for p in self.params]
        new = lambda dtype, sizes: [torch.zeros(n, dtype=dtype, device=p.device)
                                    for n, p in zip(sizes, self.params)]
        kind = torch.float32 if state == "float32" else torch.uint8
        self.m, self.v = new(kind, flat), new(kind, flat)
        runs = [-(-n // 32) for n in flat]
        self.m_scale, self.v_scale = (None, None) if state == "float32" else (new(kind, runs), new(kind, runs))
        self.plan = adamw_plan(self.params, self.grads, self.m, self.v, copies, self.m_scale, self.v_scale)
        self.sumsq = None
        if max_norm is not None or check_finite:
            if len({g.dtype for g in self.grads}) > 1:
                raise ValueError("gradients of one call have one type")
            self.sumsq_plan = sumsq_plan(self.grads)
            self.sumsq = torch.zeros(1, dtype=torch.float64, device=self.params[0].device)

    def step(self, lr: Optional[float] = None):
        """One step; `lr` replaces the rate given at the start, for this step. Rate and step count are
        the host's, which a graph would keep: to capture a step call mok_adamw on this object's
        plan with both on the device. A step that the device leaves out because its norm is not
        finite counts, too, as the host does not read the norm."""
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a captured step takes its number from the device: see mok_adamw")
        step = self.steps + 1
        if self.sumsq is not None:
            mok_grad_sumsq(self.sumsq_plan, self.sumsq)
        mok_adamw(self.plan, lr=self.lr if lr is None else lr, step=step, beta1=self.betas[0],
                  beta2=self.betas[1], eps=self.eps, weight_decay=self.weight_decay,
                  seed=self.seed + step, sumsq=self.sumsq, max_norm=self.max_norm)
        self.steps = step   # (a refused call is no step)


class MokMuon:
    """Muon over matrices [..][rows][cols] updated in place from gradients that stay in the given tensors: momentum,
    orthogonalised by Newton-Schulz steps.

    params: float32 masters; grads: float32 or bfloat16 (one type); copies: bfloat16 copies, written by every step (None in
    the place of a master without one). adjust: "rms" gives updates AdamW's size, so both can share a rate; "spectral",
    "none". max_norm and check_finite as for MokAdamW."""

    def __init__(self, params, grads, copies=None, lr: float = 1e-3, momentum: float = 0.95, nesterov: bool = True,
                 weight_decay: float = 0.0, eps: float = 1e-7, adjust: str = "rms", max_norm: Optional[float] = None,
                 check_finite: bool = False):
        self.params, self.grads, self.copies, self.lr = list(params), list(grads), copies, lr
        self.hyper = dict(momentum=momentum, nesterov=nesterov, weight_decay=weight_decay, eps=eps, adjust=adjust)
        self.max_norm = max_norm
        self.m = [torch.zeros_like(p) for p in self.params]
        self.plan = muon_plan(self.params, self.grads, self.m, copies)
        self.sumsq = None
        if max_norm is not None or check_finite:
            self.sumsq_plan = sumsq_plan(self.grads)
            self.sumsq = torch.zeros(1, dtype=torch.float64, device=self.params[0].device)

    def step(self, lr=None):
        """One step; `lr` replaces the rate given at the start, for this step, and may be a device tensor (float64 [1]),
        which a captured step reads when it runs."""
        if self.sumsq is not None:
            mok_grad_sumsq(self.sumsq_plan, self.sumsq)
        mok_muon(self.plan, lr=self.lr if lr is None else lr, sumsq=self.sumsq, max_norm=self.max_norm, **self.hyper)
