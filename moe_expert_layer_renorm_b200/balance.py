"""The router's balance loss, per-expert counts and the gradient of its logits:
torch buffers around ft_moe_balance and ft_moe_route_backward."""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .layer import _ptr, _stream


class RouterBalance:
    """Buffers and calls for batches of T tokens routed to k of E experts.

    loss = coef * E / (Tv k) * sum_e counts[e] * (1 / Tv) sum_t p[t, e] over the Tv valid tokens, p = softmax(logits).
    forward() leaves ``counts`` int32 [E], ``n_valid`` int32 [1] and ``loss`` fp32 [1]; backward() writes ``dlogits``.
    The buffers belong to this object: one batch is in flight at a time."""

    def __init__(self, T: int, E: int, k: int, coef: float, device="cuda"):
        self.T, self.E, self.k, self.coef = T, E, k, float(coef)
        self.dev = torch.device(device)
        self.counts = torch.empty(E, dtype=torch.int32, device=self.dev)
        self.n_valid = torch.empty(1, dtype=torch.int32, device=self.dev)
        self.loss = torch.empty(1, dtype=torch.float32, device=self.dev)
        self.dlogits = torch.empty((T, E), dtype=torch.float32, device=self.dev)
        self.ws_bytes = _lib.balance_workspace_size(T, E)
        self._ws = torch.empty(max(self.ws_bytes, 16), dtype=torch.uint8, device=self.dev)

    def _check(self, logits, ids, valid) -> None:
        assert logits.dtype == torch.float32 and logits.shape == (self.T, self.E) and logits.is_cuda
        assert self.E == 1 or logits.stride(1) == 1
        assert ids.dtype == torch.int32 and ids.shape == (self.T, self.k) and ids.is_contiguous()
        assert valid is None or (valid.dtype in (torch.bool, torch.uint8) and valid.shape == (self.T,) and
                                 valid.is_contiguous())
        here = torch.cuda.current_device()
        assert logits.get_device() == here and self.counts.get_device() == here and ids.get_device() == here and \
            (valid is None or valid.get_device() == here), "a tensor is not on the current device"

    def _pitch(self, t: torch.Tensor) -> int:
        return t.stride(0) if self.T > 1 else max(t.stride(0), self.E)

    def forward(self, logits: torch.Tensor, ids: torch.Tensor, valid: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """Counts and loss of one batch: logits fp32 [T, E], ids int32 [T, k] from the router, valid bool [T] or None."""
        self._check(logits, ids, valid)
        _lib.balance(logits.data_ptr(), self._pitch(logits), ids.data_ptr(), _ptr(valid), self.T, self.E, self.k,
                     self.coef, self.counts.data_ptr(), self.n_valid.data_ptr(), self.loss.data_ptr(),
                     self._ws.data_ptr(), self.ws_bytes, _stream(stream))
        return self.loss

    def backward(self, logits: torch.Tensor, ids: torch.Tensor, dloss: Optional[torch.Tensor] = None,
                 w: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                 valid: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """dlogits of the last forward()'s loss (times dloss, fp32 [1]; None: 1), plus that of the router's
        weights w with the gradient dw (both fp32 [T, k]) where they are given."""
        self._check(logits, ids, valid)
        assert dloss is None or (dloss.dtype == torch.float32 and dloss.numel() == 1 and
                                 dloss.get_device() == logits.get_device())
        assert (w is None) == (dw is None)
        for t in (w, dw):
            assert t is None or (t.dtype == torch.float32 and t.shape == (self.T, self.k) and t.is_contiguous() and
                                 t.get_device() == logits.get_device())
        _lib.route_backward(logits.data_ptr(), self._pitch(logits), ids.data_ptr(), _ptr(w), _ptr(dw), _ptr(valid),
                            self.T, self.E, self.k, self.coef, self.counts.data_ptr(), self.n_valid.data_ptr(),
                            _ptr(dloss), self.dlogits.data_ptr(), self.E, _stream(stream))
        return self.dlogits
