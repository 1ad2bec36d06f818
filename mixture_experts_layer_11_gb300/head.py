"""The loss between a model's last hidden states and its training signal, over a
vocabulary head whose logits are never kept: ``HeadLoss`` binds the head once and
runs ``moe_head_ce`` / ``moe_head_distill``.

    head = HeadLoss(T, W)                                  # W [V,d]
    loss, lse, dx, dW = head.cross_entropy(x, target, mean=True)
    lp.backward(dx, ...)                                   # dx is the layer's dy

    scores = HeadLoss(64, W, backward=False)
    loss, lse = scores.score(x, token)                     # -log p(token), per row

Calls launch work on the current CUDA stream and neither allocate nor
synchronise, so they can be captured in a CUDA graph.  This module does no
arithmetic of its own.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import ops


class HeadLoss:
    """Parameters: T the most tokens of one call; W [V,d] the head, bf16 or fp32,
    contiguous, d a multiple of 8, read at every call, so that weights updated in
    place, or given other memory, take effect; entries the most of a teacher's list a token (1 to
    ops.HEAD_MAX_ENTRIES); backward False for scores alone.  With backward: want_dx,
    want_dW which gradients (neither: the calls are scores); dW [V,d] the buffer for the head's (W's type or fp32),
    whose memory is bound here, None for one of W's type made here; piece the tokens whose probabilities are held
    at a time (0: as many as 2 GiB hold); more are worked on in rounds.  Scores hold
    no probabilities, but up to 65536 rows of x: an object with a small piece has a
    workspace for them too.

    The results, the workspace and the status word are this object's, on the head's
    device, whichever is current: calls of one object run in order on one stream
    (use an object per stream), the current one of that device, and the next call
    overwrites what one returned."""

    def __init__(self, T: int, W, entries: int = 1, backward: bool = True,
                 dW: Optional[torch.Tensor] = None, want_dx: bool = True, want_dW: bool = True,
                 piece: int = 0):
        if W.dim() != 2:
            raise ValueError(f"W has shape {tuple(W.shape)}, expected [V, d]")
        if W.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"W is {W.dtype}, expected bfloat16 or float32")
        if T < 0 or piece < 0:
            raise ValueError(f"T {T}, piece {piece}: expected no negative number")
        if not 1 <= entries <= ops.HEAD_MAX_ENTRIES:
            raise ValueError(f"entries is {entries}, expected 1 to {ops.HEAD_MAX_ENTRIES}")
        if dW is not None:
            if not (backward and want_dW):
                raise ValueError("dW given, but no gradient of the head is wanted")
            if dW.shape != W.shape or dW.dtype not in (W.dtype, torch.float32):
                raise ValueError(f"dW is {dW.dtype} {tuple(dW.shape)}, expected {W.dtype} or "
                                 f"torch.float32 {tuple(W.shape)}")
        ops.one_device("HeadLoss", W, dW)
        V, d = W.shape
        dev = W.device
        if not W.is_contiguous():
            raise ops.MoEError("HeadLoss", ops.MOE_ERR_INVALID, "W is not contiguous")
        self.T, self.W, self.entries = T, W, entries
        self.head = ops.make_head(T, V, d, W.dtype, entries, piece)
        self.grad = None
        self.dx = self.dW = None
        if backward:
            if want_dx:
                self.dx = torch.empty(T, d, dtype=W.dtype, device=dev)
            if want_dW:
                self.dW = torch.empty_like(W) if dW is None else dW
            if want_dx or want_dW:
                self.grad = ops.make_head_grad(self.dx, self.dW, W.dtype)
        self._backward = bool(backward)
        with torch.cuda.device(dev):
            n = ops.moe_head_workspace_size(self.head, self.grad)
        if n == 0:
            raise ValueError("the head's shape is not one that moe_head_ce takes")
        self.ws = torch.empty(n, dtype=torch.uint8, device=dev)
        self.loss = torch.empty(T, dtype=torch.float32, device=dev)
        self.lse = torch.empty(T, dtype=torch.float32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._device = self.loss.device.index
        self._results = (self.loss, self.lse, self.dx, self.dW)
        self._size = (T, d)
        self._shape = W.shape
        self._losses = (self.loss.data_ptr(), self.lse.data_ptr())
        self._owned = (self.ws.data_ptr(), self.status.data_ptr())

    def score(self, x, target):
        """x [t,d] of W's type, t <= T; target [t] int64, below 0 for none.  Returns
        (loss, lse), fp32 [t]: loss = lse - logit of the target = -log p(target)."""
        return self._call(x, target, None, 1.0, None)[:2]

    def cross_entropy(self, x, target, weight=None, scale: float = 1.0, mean: bool = False,
                      accumulate: bool = False):
        """Returns (loss, lse, dx, dW): the scores, not weighted, and the gradients
        (None: not wanted) of  scale * sum_t weight[t] loss[t], divided by the number
        of tokens with a target if ``mean``.  weight [t] fp32 or None; accumulate adds
        to an fp32 dW."""
        return self._call(x, target, None, 1.0, self._grad(x, weight, scale, mean, accumulate))

    def distill(self, x, idx, logits, temperature: float = 1.0, weight=None, scale: float = 1.0,
                mean: bool = False, accumulate: bool = False):
        """idx [t,n] int64 and logits [t,n] fp32, n <= entries: the teacher's entries,
        absent where idx is below 0 or the logit -inf.  Returns (loss, lse, dx, dW): loss
        = temperature^2 * KL(softmax of the entries present || student), lse that of the
        student's logits / temperature, gradients as in ``cross_entropy`` (None for an
        object without backward)."""
        if idx.dim() != 2 or idx.shape != logits.shape:
            raise ValueError(f"idx is {tuple(idx.shape)}, logits {tuple(logits.shape)}")
        if not 1 <= idx.shape[1] <= self.entries:
            raise ValueError(f"{idx.shape[1]} entries, expected 1 to {self.entries}")
        g = self._grad(x, weight, scale, mean, accumulate) if self._backward else None
        return self._call(x, idx, logits, temperature, g)

    def _grad(self, x, weight, scale, mean, accumulate):
        if not self._backward:
            raise ValueError("gradients of an object made with backward=False")
        if weight is not None:
            if tuple(weight.shape) != (x.shape[0],):
                raise ValueError(f"weight is {tuple(weight.shape)}, expected [{x.shape[0]}]")
            self._on_device("weight", weight)
        g = self.grad
        if accumulate and self.dW is not None and self.dW.dtype != torch.float32:
            raise ValueError(f"accumulate takes a float32 dW, this one is {self.dW.dtype}")
        address = ops._ptr(weight, torch.float32)
        if g is None:
            return None
        g.weight = address
        g.scale, g.mean, g.accumulate = float(scale), int(bool(mean)), int(bool(accumulate))
        return g

    def _on_device(self, name, t):
        if t.get_device() != self._device:
            raise ops.MoEError("moe_head", ops.MOE_ERR_INVALID,
                               f"{name} on {t.device}, the head on cuda:{self._device}")

    def _call(self, x, idx, logits, temperature, grad):
        size, d = x.shape, self._size[1]
        if size != self._size and (len(size) != 2 or size[1] != d or size[0] > self.T):
            raise ValueError(f"x is {tuple(size)}, expected [t, {d}] with t <= {self.T}")
        t, lists = size[0], idx.shape
        if (lists != (t,)) if logits is None else (lists[0] != t):
            raise ValueError(f"targets are {tuple(lists)} for {t} tokens")
        if self.W.shape != self._shape:
            raise ValueError(f"W is {tuple(self.W.shape)} now, was {tuple(self._shape)}")
        self._on_device("W", self.W)
        self._on_device("x", x)
        self._on_device("targets", idx)
        h = self.head
        h.T = t
        if logits is None:
            h.entries = 1
        else:
            self._on_device("logits", logits)
            h.entries = lists[1]
        if torch.cuda.current_device() == self._device:
            self._launch(x, idx, logits, temperature, grad)
        else:
            with torch.cuda.device(self._device):
                self._launch(x, idx, logits, temperature, grad)
        loss, lse, dx, dW = self._results
        if t != self.T:
            loss, lse = loss[:t], lse[:t]
            dx = None if dx is None else dx[:t]
        return (loss, lse, None, None) if grad is None else (loss, lse, dx, dW)

    def _launch(self, x, idx, logits, temperature, grad):
        stream = ops.raw_stream(self._device)
        if logits is None:
            ops.moe_head_ce(self.head, x, self.W, idx, *self._losses, grad, *self._owned, stream=stream)
        else:
            ops.moe_head_distill(self.head, x, self.W, idx, logits, temperature, *self._losses, grad,
                                 *self._owned, stream=stream)

    def check_status(self):
        """Synchronises and raises if one of the calls since the last check
        reported a device-side error (the first of them)."""
        ops.take_status(self.status)
