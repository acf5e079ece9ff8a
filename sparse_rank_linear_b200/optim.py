"""AdamW over many tensors in one kernel launch (salr_adamw of include/salr.h).

The class owns the moments (and the fp32 master copies, where asked for); parameters and
gradients are the caller's tensors.  Like the rest of the binding it only marshals
arguments: the step is one call of the CUDA library.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np

from .binding import AdamwConfig, AdamwTensor, _check, _on_device, _stream_ptr, load_library

BLOCK = 256  # elements that share a scale of the 8-bit moments
_TYPES = {"torch.bfloat16": 0, "torch.float32": 1}


class AdamW:
    """AdamW with decoupled weight decay over ``params``, a list of contiguous CUDA tensors
    of one type (bfloat16 or float32) on one device, updated in place.

    ``state_bits``: 32 holds the moments in fp32; 8 holds m and sqrt(v) as e4m3 values times
    one fp32 scale per 256 elements.  ``master``: bf16 parameters get fp32 master copies,
    made from them here, which the step updates; the parameters then receive their rounding.

    State, open to the caller for saving and loading (all zero, step 0, at the start).  Every
    tensor starts on a multiple of 256 elements of the flat buffers; ``slices[i]`` is the
    slice of parameter i:

    * ``exp_avg``, ``exp_avg_sq``: fp32 m and v, or float8_e4m3fn codes of m and sqrt(v);
    * ``exp_avg_scale``, ``exp_avg_sq_scale``: the codes' scales (None with 32 bits);
    * ``master``: fp32 (None without); ``step_count``: int64 scalar, the steps done.

    Steps are stream-ordered and allocate nothing, so a step can be captured into a CUDA
    graph: a replay takes the step count, and ``lr`` and ``grad_scale`` given as tensors, as
    they are then.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state_bits=32, master=False):
        import torch
        self.params = list(params)
        if not self.params:
            raise ValueError("params is empty")
        first = self.params[0]
        if str(first.dtype) not in _TYPES:
            raise TypeError("params must be bfloat16 or float32")
        for i, p in enumerate(self.params):
            if p.dtype != first.dtype:
                raise TypeError("params must have one type")
            if not p.is_contiguous():
                raise ValueError(f"params[{i}] must be contiguous")
            if not p.is_cuda:
                raise ValueError(f"params[{i}] must be a CUDA tensor")
            if p.device != first.device:
                raise ValueError("params must be on one device")
        spans = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size())
                       for p in self.params if p.numel())
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("params must not overlap (the same tensor twice?)")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if master and first.dtype != torch.bfloat16:
            raise ValueError("master copies are for bfloat16 params")
        beta1, beta2 = betas
        if not (0 <= beta1 < 1 and 0 <= beta2 < 1):
            raise ValueError("betas must be in [0, 1)")
        if not (math.isfinite(eps) and eps >= 0):
            raise ValueError("eps must be finite and not negative")
        self.device = first.device
        self.lr, self.betas, self.eps, self.weight_decay = lr, (beta1, beta2), eps, weight_decay
        self.state_bits = state_bits
        self.slices, total = [], 0
        for p in self.params:
            self.slices.append(slice(total, total + p.numel()))
            total += -(-p.numel() // BLOCK) * BLOCK
        kind = torch.float8_e4m3fn if state_bits == 8 else torch.float32
        self.exp_avg = torch.zeros(total, dtype=kind, device=self.device)
        self.exp_avg_sq = torch.zeros(total, dtype=kind, device=self.device)
        self.exp_avg_scale = self.exp_avg_sq_scale = self.master = None
        if state_bits == 8:
            self.exp_avg_scale = torch.zeros(total // BLOCK, device=self.device)
            self.exp_avg_sq_scale = torch.zeros(total // BLOCK, device=self.device)
        if master:
            self.master = torch.zeros(total, device=self.device)
            for p, s in zip(self.params, self.slices):
                self.master[s].copy_(p.detach().reshape(-1))
        self._step = torch.zeros(2, dtype=torch.int64, device=self.device)
        self.step_count = self._step[0]
        self._numel = [p.numel() for p in self.params]
        self._table = (AdamwTensor * len(self.params))()
        for t, p, s in zip(self._table, self.params, self.slices):
            t.param = p.data_ptr()
            t.exp_avg = self.exp_avg.data_ptr() + s.start * self.exp_avg.element_size()
            t.exp_avg_sq = self.exp_avg_sq.data_ptr() + s.start * self.exp_avg_sq.element_size()
            if state_bits == 8:
                t.exp_avg_scale = self.exp_avg_scale.data_ptr() + s.start // BLOCK * 4
                t.exp_avg_sq_scale = self.exp_avg_sq_scale.data_ptr() + s.start // BLOCK * 4
            if master:
                t.master = self.master.data_ptr() + s.start * 4
            t.n = p.numel()
        # the gradients' pointers in the table, as one strided array
        self._grads = np.frombuffer(self._table, dtype=np.uint64).reshape(len(self._table), -1)[
            :, AdamwTensor.grad.offset // 8]
        self._index = self._step.get_device()
        self._config = AdamwConfig(beta1=beta1, beta2=beta2, eps=eps, step=self._step.data_ptr(),
                                   param_type=_TYPES[str(first.dtype)], state_bits=state_bits,
                                   master=1 if master else 0)

    def _scalar(self, x, name):
        import torch
        if x.dtype != torch.float32 or x.numel() != 1 or x.device != self.device:
            raise ValueError(f"{name} must be one float32 on {self.device}")
        return x.data_ptr()

    def step(self, grads, lr=None, grad_scale=None, stream=None):
        """One step with ``grads``, one contiguous tensor (all of one type, bfloat16 or
        float32) or None per parameter; None leaves its parameter and moments as they are.

        ``lr``: a number or a one-element float32 CUDA tensor in place of ``self.lr``.
        ``grad_scale``: a one-element float32 CUDA tensor that multiplies every gradient (the
        factor of gradient clipping, or of undoing a loss scale)."""
        import torch
        T = torch.Tensor
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} params")
        if type(grads) is not list:
            grads = list(grads)
        # whole-list passes: a loop over hundreds of gradients would take longer than the step
        given = grads
        try:
            pointers = list(map(T.data_ptr, grads))
            numel = self._numel
        except TypeError:  # None among them
            given = [g for g in grads if g is not None]
            pointers = [0 if g is None else g.data_ptr() for g in grads]
            numel = [n for n, g in zip(self._numel, grads) if g is not None]
        kinds = set(map(T.dtype.__get__, given))
        kind = kinds.pop() if kinds else None
        if kinds or (kind is not None and str(kind) not in _TYPES):
            raise TypeError("grads must have one type, bfloat16 or float32")
        if (list(map(T.numel, given)) != numel or not all(map(T.is_contiguous, given)) or
                any(i != self._index for i in set(map(T.get_device, given)))):
            raise ValueError(f"each gradient must be contiguous, as large as its parameter and "
                             f"on {self.device}")
        self._grads[:] = pointers
        c = self._config
        c.grad_type = 0 if kind is None else _TYPES[str(kind)]
        c.lr, c.lr_dev = 0.0, None
        if lr is None:
            lr = self.lr
        if torch.is_tensor(lr):
            c.lr_dev = self._scalar(lr, "lr")
        else:
            c.lr = lr
        c.weight_decay = self.weight_decay
        c.grad_scale = None if grad_scale is None else self._scalar(grad_scale, "grad_scale")
        with _on_device(self._step):
            _check("salr_adamw", load_library().salr_adamw(self._table, len(self._table), ctypes.byref(c),
                                                           _stream_ptr(stream)))
