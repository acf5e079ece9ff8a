"""AdamW over many tensors in one kernel launch (salr_adamw of include/salr.h).

The class owns the moments (and the fp32 master copies, where asked for); parameters and
gradients are the caller's tensors.  Like the rest of the binding it only marshals
arguments: the step is one call of the CUDA library.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np

from .binding import AdamwConfig, AdamwTensor, _check, _on_device, _stream_ptr, _written, load_library

BLOCK = 256  # elements that share a scale of the 8-bit moments
_TYPES = {"torch.bfloat16": 0, "torch.float32": 1}


def _held(name):
    """Attribute for a buffer that may be changed in place (``x += y`` too) but not replaced."""
    def put(self, value):
        if value is not getattr(self, name):
            raise AttributeError(f"{name[1:]} cannot be replaced: copy into it")
    return property(lambda self: getattr(self, name), put)


class _Watch:
    """Whether a list of tensors has the types, devices, shapes and strides that it had when it
    was checked.  torch's guards compare a whole list in one call (17 us for 300 tensors, where
    the checks one by one take 110); without them the answer is no, and the checks run."""

    def __init__(self):
        self._guards = None

    def learn(self, tensors):
        import torch
        try:
            self._guards = torch._C._dynamo.guards.TensorGuards(
                *tensors, dynamic_dims_sizes=[list(t.shape) for t in tensors],
                dynamic_dims_strides=[list(t.stride()) for t in tensors])
        except Exception:
            self._guards = None

    def same(self, tensors):
        return self._guards is not None and self._guards.check(*tensors)


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

    ``lr``, ``betas``, ``eps`` and ``weight_decay`` are attributes that the next step takes as
    they are then (the library refuses values outside their ranges).

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
        self._refuse_overlap()
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
        self._kind = first.dtype
        self.lr, self.betas, self.eps, self.weight_decay = lr, (beta1, beta2), eps, weight_decay
        self.state_bits = state_bits
        self.slices, total = [], 0
        for p in self.params:
            self.slices.append(slice(total, total + p.numel()))
            total += -(-p.numel() // BLOCK) * BLOCK
        kind = torch.float8_e4m3fn if state_bits == 8 else torch.float32
        # held for as long as the table below points into them: read-only attributes
        m = self._exp_avg = torch.zeros(total, dtype=kind, device=self.device)
        v = self._exp_avg_sq = torch.zeros(total, dtype=kind, device=self.device)
        self._exp_avg_scale = self._exp_avg_sq_scale = self._master = None
        if state_bits == 8:
            self._exp_avg_scale = torch.zeros(total // BLOCK, device=self.device)
            self._exp_avg_sq_scale = torch.zeros(total // BLOCK, device=self.device)
        if master:
            self._master = torch.zeros(total, device=self.device)
            for p, s in zip(self.params, self.slices):
                self._master[s].copy_(p.detach().reshape(-1))
        self._step = torch.zeros(2, dtype=torch.int64, device=self.device)
        self._shapes = [p.shape for p in self.params]
        self._grads_seen, self._params_seen = _Watch(), _Watch()
        self._table = (AdamwTensor * len(self.params))()
        for t, p, s in zip(self._table, self.params, self.slices):
            t.exp_avg = m.data_ptr() + s.start * m.element_size()
            t.exp_avg_sq = v.data_ptr() + s.start * v.element_size()
            if state_bits == 8:
                t.exp_avg_scale = self._exp_avg_scale.data_ptr() + s.start // BLOCK * 4
                t.exp_avg_sq_scale = self._exp_avg_sq_scale.data_ptr() + s.start // BLOCK * 4
            if master:
                t.master = self._master.data_ptr() + s.start * 4
            t.n = p.numel()
        # columns of the table as strided arrays: every step writes both anew
        words = np.frombuffer(self._table, dtype=np.uint64).reshape(len(self._table), -1)
        self._grads = words[:, AdamwTensor.grad.offset // 8]
        self._params = words[:, AdamwTensor.param.offset // 8]
        self._index = self._step.get_device()
        self._at = None  # the parameters' addresses in the table
        self._config = AdamwConfig(step=self._step.data_ptr(), param_type=_TYPES[str(first.dtype)],
                                   state_bits=state_bits, master=1 if master else 0)

    exp_avg = _held("_exp_avg")
    exp_avg_sq = _held("_exp_avg_sq")
    exp_avg_scale = _held("_exp_avg_scale")
    exp_avg_sq_scale = _held("_exp_avg_sq_scale")
    master = _held("_master")
    step_count = property(lambda self: self._step[0])

    def _pointers(self, tensors, shapes, what):
        """Their addresses, after checks in whole-list passes (a loop over hundreds of tensors
        would take longer than the step), and their type (None for an empty list)."""
        import torch
        T = torch.Tensor
        pointers = list(map(T.data_ptr, tensors))
        kinds = set(map(T.dtype.__get__, tensors))
        kind = kinds.pop() if kinds else None
        if kinds or (kind is not None and str(kind) not in _TYPES):
            raise TypeError(f"{what} must have one type, bfloat16 or float32")
        if (list(map(T.size, tensors)) != shapes or not all(map(T.is_contiguous, tensors)) or
                any(i != self._index for i in set(map(T.get_device, tensors)))):
            raise ValueError(f"{what} must be contiguous, of the parameters' shapes and on {self.device}")
        return pointers, kind

    def _refuse_overlap(self):
        spans = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size())
                       for p in self.params if p.numel())
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("params must not overlap (the same tensor twice?)")

    def _scalar(self, x, name):
        import torch
        if x.dtype != torch.float32 or x.numel() != 1 or x.device != self.device:
            raise ValueError(f"{name} must be one float32 on {self.device}")
        return x.data_ptr()

    def step(self, grads, lr=None, grad_scale=None, stream=None):
        """One step with ``grads``, one contiguous tensor of the parameter's shape (all of one
        type, bfloat16 or float32) or None per parameter; None leaves its parameter and
        moments as they are.

        ``lr``: a number or a one-element float32 CUDA tensor in place of ``self.lr``.
        ``grad_scale``: a one-element float32 CUDA tensor that multiplies every gradient (the
        factor of gradient clipping, or of undoing a loss scale)."""
        import torch
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} params")
        changed = self.params
        if self._grads_seen.same(grads):
            pointers, kind = list(map(torch.Tensor.data_ptr, grads)), grads[0].dtype
        else:
            given = [g for g in grads if g is not None]
            shapes = [n for n, g in zip(self._shapes, grads) if g is not None]
            some, kind = self._pointers(given, shapes, "grads")
            if len(given) == len(grads):
                self._grads_seen.learn(grads)
            else:
                changed = [p for p, g in zip(self.params, grads) if g is not None]
            some = iter(some)
            pointers = [0 if g is None else next(some) for g in grads]
        # the parameters may have moved since the last step, or be another view of their
        # memory (p.data = ...)
        at = list(map(torch.Tensor.data_ptr, self.params))
        if at != self._at or not self._params_seen.same(self.params):
            at, now = self._pointers(self.params, self._shapes, "params")
            if now != self._kind:
                raise TypeError("params must keep their type")
            self._refuse_overlap()
            self._at = at
            self._params[:] = at
            self._params_seen.learn(self.params)
            # kept alive: while they are, an unchanged address means unchanged memory
            self._kept = [p.detach() for p in self.params]
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
        c.beta1, c.beta2 = self.betas
        c.eps, c.weight_decay = self.eps, self.weight_decay
        c.grad_scale = None if grad_scale is None else self._scalar(grad_scale, "grad_scale")
        with _on_device(self._step):
            _check("salr_adamw", load_library().salr_adamw(self._table, len(self._table), ctypes.byref(c),
                                                           _stream_ptr(stream)))
        _written(changed)
