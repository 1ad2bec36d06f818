"""A trained layer for decode steps: ``FewTokenPass`` binds the parameters
once and runs the whole layer (router, gate, experts, combine, residual) on up
to ``ops.FEW_MAX_TOKENS`` tokens a call with ``moe_layer_few``.

``forward`` launches work on the current CUDA stream and neither allocates nor
synchronises, so a decode loop can capture it in a CUDA graph.  Longer inputs
(prompts) are ``layer.LayerPass``'s.  This module does no arithmetic of its
own.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import ops


class FewTokenPass:
    """Parameters: T the most tokens of one call (1 to ops.FEW_MAX_TOKENS); Wg
    [E,d], W1 [E,f,d], b1 [E,f], W2 [E,d,f], b2 [E,d] (b1, b2 or None) in bf16
    or fp32; k experts per token; renorm; beta [E] fp32 or None.  The tensors
    are read at every call, so weights updated in place take effect.

    ``y``, the workspace and the status word are this object's, on the weights'
    device, whichever is current: calls of one object run in order on one stream
    (use an object per stream), the current one of that device."""

    def __init__(self, T: int, Wg, W1, b1, W2, b2, k: int, renorm: int,
                 beta: Optional[torch.Tensor] = None):
        E, f, d = W1.shape
        for n, t, shape in (("Wg", Wg, (E, d)), ("b1", b1, (E, f)), ("W2", W2, (E, d, f)),
                            ("b2", b2, (E, d)), ("beta", beta, (E,))):
            if t is not None and tuple(t.shape) != shape:
                raise ValueError(f"{n} has shape {tuple(t.shape)}, expected {shape}")
        if W1.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"weights are {W1.dtype}, expected bfloat16 or float32")
        if not 1 <= T <= ops.FEW_MAX_TOKENS:
            raise ValueError(f"T is {T}, expected 1 to {ops.FEW_MAX_TOKENS}")
        self.T, self.d, self.dtype = T, d, W1.dtype
        self.shape = ops.make_shape(T, d, f, E, k, W1.dtype, renorm)
        self._weights = (Wg, beta, W1, b1, W2, b2)   # kept alive
        self.params = ops.make_layer_params(self.shape, *self._weights)
        dev = W1.device
        with torch.cuda.device(dev):
            n = ops.moe_layer_few_workspace_size(self.shape)
        if n == 0:
            raise ValueError("the layer's shape is not one that moe_layer_few takes")
        self.ws = torch.empty(n, dtype=torch.uint8, device=dev)
        self.y = torch.empty(T, d, dtype=W1.dtype, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._device = self.y.device.index
        self._owned = (self.ws.data_ptr(), self.status.data_ptr())

    def forward(self, x, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None):
        """x [t,d], t <= T; residual [t,d] or None; returns y [t,d] in ``out``
        (which may be residual) or in a buffer owned by this object."""
        size = x.shape
        y = self.y if out is None else out
        if size != y.shape:
            if len(size) != 2 or size[1] != self.d or size[0] > self.T:
                raise ValueError(f"x is {tuple(size)}, expected [t, {self.d}] with t <= {self.T}")
            if out is not None:
                raise ValueError(f"out is {tuple(out.shape)}, expected {tuple(size)}")
            y = self.y[:size[0]]
        elif out is not None and (len(size) != 2 or size[1] != self.d or size[0] > self.T):
            raise ValueError(f"x is {tuple(size)}, expected [t, {self.d}] with t <= {self.T}")
        if residual is not None and residual.shape != size:
            raise ValueError(f"residual is {tuple(residual.shape)}, expected {tuple(size)}")
        for t in (x, residual, out):
            if t is not None and t.get_device() != self._device:
                raise ops.MoEError("moe_layer_few", ops.MOE_ERR_INVALID,
                                   f"tensor on {t.device}, the weights on cuda:{self._device}")
        self.shape.T = size[0]
        if torch.cuda.current_device() == self._device:
            self._launch(x, residual, y)
        else:
            with torch.cuda.device(self._device):
                self._launch(x, residual, y)
        return y

    def _launch(self, x, residual, y):
        ops.moe_layer_few(self.shape, self.params, x, residual, y, *self._owned,
                          stream=ops.raw_stream(self._device))

    def check_status(self):
        """Synchronises and raises if one of the calls since the last check
        reported a device-side error (the first of them)."""
        ops.take_status(self.status)
