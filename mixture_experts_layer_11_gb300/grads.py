"""The end of a training step: the global norm of a list of gradients, and
clipping by it, over ``moe_grad_norm`` / ``moe_grad_clip``.

    clip = GradClip([lp.dWg, lp.dW1, lp.db1, lp.dW2, lp.db2])
    ...
    lp.backward(dy)
    norm = clip.clip(1.0)          # the gradients, in place; a device scalar

Calls launch work on the current CUDA stream and neither allocate nor
synchronise.  This module does no arithmetic of its own.
"""
from __future__ import annotations

import torch

from . import ops


class GradClip:
    """tensors: the gradients (on one CUDA device, whichever is current;
    contiguous, fp32 or bf16; any sizes, views of flat buffers included, none
    twice); outs: for each a tensor of its size and type that ``clip`` writes, or
    None for all: in place.  The norm, the workspace and the status word are this
    object's: calls of one object run in order on one stream, the current one of
    the gradients' device."""

    def __init__(self, tensors, outs=None):
        self._tensors = (list(tensors), None if outs is None else list(outs))   # kept alive
        self.grads = ops.make_grads(*self._tensors)
        dev = self._tensors[0][0].device if self._tensors[0] else torch.device("cuda")
        with torch.cuda.device(dev):
            n = ops.moe_grad_workspace_size(len(self.grads))
        self.ws = torch.empty(n, dtype=torch.uint8, device=dev)
        self.total = torch.zeros((), dtype=torch.float32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._device = self.total.device.index
        self._owned = (self.total.data_ptr(), self.ws.data_ptr(), self.status.data_ptr())

    def norm(self) -> torch.Tensor:
        """The norm of all gradients (a fp32 scalar owned by this object); sets
        ``status`` to MOE_ERR_NONFINITE when it is infinite or NaN."""
        return self._launch(ops.moe_grad_norm, self.grads)

    def clip(self, max_norm: float) -> torch.Tensor:
        """Scale the gradients by max_norm / norm if norm > max_norm (else, and
        with a norm that is not finite, they stay or are copied to outs as they
        are).  Returns the norm before."""
        return self._launch(ops.moe_grad_clip, self.grads, max_norm)

    def _launch(self, call, *args):
        if torch.cuda.current_device() == self._device:
            call(*args, *self._owned, stream=ops.raw_stream(self._device))
        else:
            with torch.cuda.device(self._device):
                call(*args, *self._owned, stream=ops.raw_stream(self._device))
        return self.total

    def check_status(self):
        """Synchronises and raises if one of the calls since the last check
        reported a device-side error (the first of them)."""
        ops.take_status(self.status)
