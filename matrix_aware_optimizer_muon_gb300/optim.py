"""Stateful wrapper: momentum buffers, workspace and step counter around muon_periodic_step."""
from __future__ import annotations

from typing import Dict, List, Optional, Sequence

import torch

from . import _lib
from .clip import alloc_clip_workspace, muon_clip_grad_norm
from .head import AdamW8, _on


def _write_back(to: torch.Tensor, values: torch.Tensor) -> None:
    """values into a tensor of their shape, each element of a broadcast one once."""
    for d in range(to.dim()):
        if to.stride(d) == 0 and to.shape[d] > 1:
            to, values = to.narrow(d, 0, 1), values.narrow(d, 0, 1)
    with torch.no_grad():
        to.copy_(values)


class PeriodicMuon:
    """Periodic Row-wise Muon over a list of 2-D weight tensors (K = 1 is vanilla Muon).

    State is the fp32 momentum of every matrix and the integer step, which decides
    the branch (Newton-Schulz refresh when step % K == 0, RowNorm otherwise).
    """

    def __init__(self, params: Sequence[torch.Tensor], K: int = 3, gamma: float = 0.15, mu: float = 0.95,
                 eta: float = 0.02, lam: float = 0.01, ns5_mode: str = "bf16",
                 aux_params: Sequence[torch.Tensor] = (), aux_lr: float = 1e-4, betas=(0.9, 0.999),
                 eps: float = 1e-8, aux_bits: int = 32, aux_seed: int = 0, max_grad_norm: Optional[float] = None):
        """aux_params: parameters Muon does not take (biases, norms, out-of-block weights);
        they are updated by AdamW with learning rate aux_lr and the shared weight decay lam.
        aux_bits: 32, or 8 to hold AdamW's moments in 8 bits (aux_seed seeds their rounding).
        max_grad_norm: every step first scales all gradients, the auxiliary ones among them, in
        place so that their global norm is at most this; the norm before that is
        self.grad_norm, one number on the device."""
        self.params: List[torch.Tensor] = list(params)
        self.aux = list(aux_params)
        self.aux_lr, self.betas, self.eps = aux_lr, betas, eps
        if aux_bits not in (8, 32):
            raise ValueError("aux_bits is 8 or 32")
        self.aux8 = None
        if aux_bits == 8 and self.aux:
            self.aux8 = AdamW8(self.aux, aux_lr, betas, eps, lam, aux_seed)
        wide = [] if aux_bits == 8 else self.aux
        self.aux_m = [torch.zeros(p.numel(), dtype=torch.float32, device=p.device) for p in wide]
        self.aux_v = [torch.zeros(p.numel(), dtype=torch.float32, device=p.device) for p in wide]
        if not self.params:
            raise ValueError("no parameters")
        self.K, self.gamma, self.mu, self.eta, self.lam, self.ns5_mode = K, gamma, mu, eta, lam, ns5_mode
        dev = self.params[0].device
        self.M = [torch.zeros(p.shape, dtype=torch.float32, device=dev) for p in self.params]
        self.ws = _lib.alloc_workspace([tuple(p.shape) for p in self.params], ns5_mode, device=dev)
        # (made here, like ws: a step may run on another stream than the one that is current, whose
        # memory, freed but still in use there, a workspace made in the step could be)
        self.max_grad_norm, self.grad_norm, self._clip_ws = max_grad_norm, None, alloc_clip_workspace(dev)
        self.step_count = 0
        # W and M never move, so the C matrix array is built once; each step only
        # points it at that step's gradients (after checking them like the array build does).
        self._arr, self._n = _lib.make_matrices(self.M, self.params, self.params)
        self._gdt = None

    def step(self, grads: Sequence[torch.Tensor], aux_grads: Sequence[torch.Tensor] = (), stream=None) -> int:
        if len(grads) != self._n:
            raise ValueError("one gradient per matrix")
        for i, (g, p) in enumerate(zip(grads, self.params)):
            if g.shape != p.shape:
                raise ValueError("W, G and M must have the same shape")
            self._arr[i].G = _lib._ptr(g)
            self._arr[i].g_dtype = _lib._dt(g)
        # what cannot be read is refused before anything is enqueued
        given = aux_grads
        if self.aux:
            if len(aux_grads) != len(self.aux):
                raise ValueError("one gradient per auxiliary parameter")
            # copied on the stream that reads them: in its order, and in its share of the allocator
            with _on(stream):
                aux_grads = [g.contiguous() for g in aux_grads]
            if self.aux8 is not None:
                self.aux8._point(aux_grads)
            else:
                if len({(p.dtype, g.dtype) for p, g in zip(self.aux, aux_grads)}) != 1:
                    raise ValueError("auxiliary parameters, and their gradients, are of one dtype")
                aux = _lib.adamw_array(self.aux, aux_grads, self.aux_m, self.aux_v)
        if self.max_grad_norm is not None:
            self.grad_norm = muon_clip_grad_norm([*grads, *(aux_grads if self.aux else ())], self.max_grad_norm,
                                                 self._clip_ws, stream=stream)
            with _on(stream):
                for g, copy in zip(given, aux_grads if self.aux else ()):
                    if copy is not g:
                        _write_back(g, copy)
        br = _lib.periodic_step_prepared(self._arr, self._n, self.step_count, self.ws, self.K, self.gamma, self.mu,
                                         self.eta, self.lam, self.ns5_mode, stream=stream)
        if self.aux8 is not None:
            # the schedule of learning rate and decay is the caller's, as for 32 bits
            self.aux8.lr, self.aux8.betas, self.aux8.eps, self.aux8.weight_decay = self.aux_lr, self.betas, self.eps, self.lam
            self.aux8.step_count = self.step_count
            self.aux8._launch(stream)
        elif self.aux:
            _lib.adamw_step_prepared(aux, self.step_count + 1, self.aux_lr, self.betas[0], self.betas[1], self.eps,
                                     self.lam, stream=stream)
        self.step_count += 1
        return br

    def check(self, stream=None) -> int:
        return _lib.muon_check_status(self.ws, stream)

    def state_dict(self) -> Dict:
        return {"step": self.step_count, "M": [m.detach().clone() for m in self.M],
                "aux_m": [m.detach().clone() for m in self.aux_m], "aux_v": [v.detach().clone() for v in self.aux_v],
                "aux8": None if self.aux8 is None else self.aux8.state_dict(),
                "hyper": dict(K=self.K, gamma=self.gamma, mu=self.mu, eta=self.eta, lam=self.lam,
                              ns5_mode=self.ns5_mode)}

    def load_state_dict(self, sd: Dict) -> None:
        """Restores the momentum, the AdamW moments and the step.  The schedule period K
        and the NS5 mode must match the saved ones (they change which branch a step takes
        and its arithmetic); learning rate, weight decay and gamma may differ."""
        hyper = sd.get("hyper", {})
        for key in ("K", "ns5_mode"):
            if key in hyper and hyper[key] != getattr(self, key):
                raise ValueError(f"state was saved with {key}={hyper[key]!r}, this optimizer has {getattr(self, key)!r}")
        if len(sd["M"]) != len(self.M):
            raise ValueError("state has a different number of matrices")
        aux_m, aux_v = sd.get("aux_m", []), sd.get("aux_v", [])
        if len(aux_m) != len(self.aux_m) or len(aux_v) != len(self.aux_v):
            raise ValueError("state has a different number of auxiliary parameters")
        if (sd.get("aux8") is None) != (self.aux8 is None):
            raise ValueError("state was saved with another aux_bits")
        pairs = list(zip(self.M + self.aux_m + self.aux_v, list(sd["M"]) + list(aux_m) + list(aux_v)))
        if any(tuple(dst.shape) != tuple(src.shape) for dst, src in pairs):
            raise ValueError("state shape mismatch")
        if self.aux8 is not None:   # refused before anything is copied
            self.aux8._saved(sd["aux8"])
        for dst, src in pairs:
            dst.copy_(src)
        if self.aux8 is not None:
            self.aux8.load_state_dict(sd["aux8"])
        self.step_count = int(sd["step"])
