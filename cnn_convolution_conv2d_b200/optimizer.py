"""AdamW over many tensors at once, a thin binding of ``include/optimizer_b200.h``.

``AdamWB200`` owns the states of a list of weights (of any layers: a gradient has its
weight's layout) and updates all of them in a few launches.
"""
from __future__ import annotations

import ctypes

from . import _check, _dtype_code, load
from .sequence import _on

_I, _P, _L, _D = ctypes.c_int, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_double


class AdamWTensor(ctypes.Structure):
    """adamw_tensor_t"""
    _fields_ = [("param", _P), ("master", _P), ("grad", _P), ("exp_avg", _P), ("exp_avg_sq", _P),
                ("exp_avg_scale", _P), ("exp_avg_sq_scale", _P), ("numel", _L)]


SIGNATURES = {
    "adamw_step": ([ctypes.POINTER(AdamWTensor), _I, _I, _I, _I, _D, _D, _D, _D, _D, _L, _P, _P, ctypes.c_uint, _P], _I),
    "adamw_describe_plan": ([ctypes.POINTER(AdamWTensor), _I, _I, _I, _I, ctypes.c_char_p, ctypes.c_size_t], _I),
}


def adamw_describe_plan(table, dtype, state_bits, sms) -> dict:
    """The launches of a step over ``table`` (an array of AdamWTensor) as a dict."""
    import json
    buf = ctypes.create_string_buffer(256 + 64 * len(table))
    _check(load().adamw_describe_plan(table, len(table), dtype, state_bits, int(sms), buf, ctypes.sizeof(buf)))
    return json.loads(buf.value.decode())


ADAMW_QUANT = 256  # elements that share a scale in an 8-bit state


def _overlap(tensors):
    """Whether two of the (contiguous) tensors share memory."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors if t.numel())
    return any(b[0] < a[1] for a, b in zip(spans, spans[1:]))


def _facts(tensors):
    """What decides whether tensors can be used, a list each: addresses (which tell the device), sizes, types, contiguity.  One
    loop for each, not for each tensor, since most of a step of many small tensors is spent here."""
    import torch
    t = torch.Tensor
    return [list(map(t.data_ptr, tensors)), list(map(t.numel, tensors)), [v.dtype for v in tensors],
            list(map(t.is_contiguous, tensors))]


class AdamWB200:
    """AdamW for ``params``: contiguous, 16-byte aligned CUDA tensors of one dtype (bf16 or fp32) on one device.

    ``state_bits``: 32 (fp32 states) or 8 (e4m3 and e5m2 codes with a power of two for each 256 elements, rounded by
    chance from ``seed``).  ``masters``: for bf16 weights, None (the weights themselves are updated, rounded to nearest),
    True (fp32 copies are made), or a list of fp32 tensors.  ``step_device``: an int64 CUDA tensor of one element that
    holds the number of the step to come, for steps captured into a graph; the caller counts it up (below 1 a
    step changes nothing, and ``conv2d_sync_status`` reports it).  Otherwise
    ``step_count`` counts the steps taken.

    The states lie in one buffer each, a tensor at a multiple of 256 elements: ``flat["m"]``, ``flat["v"]`` and, with 8
    bits, ``flat["m_scale"]``, ``flat["v_scale"]``; ``exp_avg`` and ``exp_avg_sq`` are views of them for each tensor.  Saving
    and restoring ``flat`` and ``step_count`` saves and restores the optimizer.

    A step works on the memory that ``params``, ``masters`` and ``flat`` have then: a weight's ``data`` may be replaced, and an
    entry of these by another tensor of its size and type.  (A captured step keeps the memory of its capture.)"""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, state_bits=32, masters=None,
                 seed=0, step_device=None):
        import torch
        self.params = list(params)
        if not self.params:
            raise ValueError("there are no weights")
        first = self.params[0]
        self.device, self.torch_dtype, self.dtype = first.device, first.dtype, _dtype_code(first.dtype)
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        self._sizes = [p.numel() for p in self.params]
        if masters is not None and first.dtype != torch.bfloat16:
            raise ValueError("fp32 weights are their own master weights")
        if masters is True:
            masters = [p.detach().float() for p in self.params]
        self.masters = None if masters is None else list(masters)
        self._check_weights()
        if step_device is not None and (step_device.dtype != torch.int64 or step_device.numel() != 1 or
                                        step_device.device != self.device):
            raise ValueError(f"step_device must be one int64 element on {self.device}")
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.state_bits, self.seed, self.step_device, self.step_count = state_bits, seed, step_device, 0
        at, starts = 0, []
        for n in self._sizes:
            starts.append(at)
            at += -(-n // ADAMW_QUANT) * ADAMW_QUANT
        new = lambda n, dtype: torch.zeros(n, dtype=torch.uint8 if dtype != torch.float32 else dtype,  # noqa: E731
                                           device=self.device).view(dtype)
        m_type, v_type = (torch.float8_e4m3fn, torch.float8_e5m2) if state_bits == 8 else (torch.float32, torch.float32)
        self.flat = {"m": new(at, m_type), "v": new(at, v_type)}
        if state_bits == 8:
            for name in ("m_scale", "v_scale"):
                self.flat[name] = torch.ones(at // ADAMW_QUANT, dtype=torch.float32, device=self.device)
        self._starts, self._flat_like = starts, {name: (t.dtype, t.numel()) for name, t in self.flat.items()}
        self._table = (AdamWTensor * len(self.params))()
        self._entries = list(self._table)  # (views: an index into the array makes one each time)
        self._known = None  # what the tensors in the table were
        self._grad_addresses, self._grad_devices = None, [self.device.index] * len(self.params)
        self._fill_table()

    def _views(self, name):
        return [self.flat[name][s:s + n] for s, n in zip(self._starts, self._sizes)]

    @property
    def exp_avg(self):
        return self._views("m")

    @property
    def exp_avg_sq(self):
        return self._views("v")

    def _check_weights(self):
        import torch
        for p in self.params:
            self._like(p, "a weight", self.torch_dtype)
        if [p.numel() for p in self.params] != self._sizes:
            raise ValueError("the weights have other sizes than their states")
        if self.masters is not None:
            if [m.numel() for m in self.masters] != self._sizes:
                raise ValueError("masters must have the weights' sizes")
            for m in self.masters:
                self._like(m, "a master weight", torch.float32)
        if _overlap(self.params + (self.masters or [])):
            raise ValueError("two weights share memory")

    def _fill_table(self):
        """Brings the table's addresses up to date; only where a tensor has changed are they looked at again."""
        masters = self.masters or []
        known = (_facts(self.params), masters and _facts(masters),
                 [(name, t.data_ptr(), t.dtype, t.shape, t.is_contiguous()) for name, t in self.flat.items()])
        if known == self._known:
            return
        self._check_weights()
        if self.flat.keys() != self._flat_like.keys():
            raise ValueError(f"flat must hold {', '.join(self._flat_like)}")
        for name, t in self.flat.items():
            self._like(t, f"flat[{name!r}]", self._flat_like[name][0])
            if t.dim() != 1 or t.numel() != self._flat_like[name][1]:
                raise ValueError(f"flat[{name!r}] must have {self._flat_like[name][1]} elements in one dimension")
        at = {name: t.data_ptr() for name, t in self.flat.items()}
        size = 1 if self.state_bits == 8 else 4
        for i, (e, p, n, start) in enumerate(zip(self._entries, self.params, self._sizes, self._starts)):
            e.param, e.numel = p.data_ptr(), n
            e.master = masters[i].data_ptr() if masters else None
            e.exp_avg, e.exp_avg_sq = at["m"] + start * size, at["v"] + start * size
            if self.state_bits == 8:
                e.exp_avg_scale = at["m_scale"] + 4 * (start // ADAMW_QUANT)
                e.exp_avg_sq_scale = at["v_scale"] + 4 * (start // ADAMW_QUANT)
        self._known = known

    def _like(self, t, what, dtype):
        if not t.is_cuda or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous CUDA tensor on {self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{what} must be {dtype}, not {t.dtype}")

    def step(self, grads, lr=None, grad_scale=None, stream=None):
        """One step with ``grads``, a gradient (bf16 or fp32, one dtype) for each weight.  ``grad_scale``: a
        one-element fp32 CUDA tensor that multiplies them; where it is not finite or not above zero nothing
        changes (the step is counted all the same).  ``lr``: this step's rate instead of the optimizer's."""
        import torch
        if len(grads) != len(self.params):
            raise ValueError(f"{len(self.params)} gradients are wanted, {len(grads)} given")
        self._fill_table()
        dtype, device, table = grads[0].dtype, self.device, self._table
        code = _dtype_code(dtype)
        count = len(grads)
        addresses, *facts = _facts(grads)
        moved = addresses != self._grad_addresses
        # (devices share one range of addresses, so the same ones as at the last step are where they were; the first one is looked
        # at all the same)
        devices = list(map(torch.Tensor.get_device, grads)) if moved or grads[0].device != device else self._grad_devices
        if facts != [self._sizes, [dtype] * count, [True] * count] or devices != self._grad_devices:
            i = next(i for i, f in enumerate(zip(*facts, devices)) if f != (self._sizes[i], dtype, True, device.index))
            raise ValueError(f"gradient {i} must be a contiguous {dtype} tensor of {self._sizes[i]} elements on {device}")
        if moved:
            for e, address in zip(self._entries, addresses):
                e.grad = address
            self._grad_addresses = addresses
        scale = None
        if grad_scale is not None:
            if grad_scale.dtype != torch.float32 or grad_scale.numel() != 1 or grad_scale.device != device:
                raise ValueError(f"grad_scale must be one fp32 element on {device}")
            scale = grad_scale.data_ptr()
        counter = None if self.step_device is None else self.step_device.data_ptr()
        _on(self.params[0], stream, lambda s: _check(load().adamw_step(
            table, len(table), self.dtype, code, self.state_bits, self.lr if lr is None else lr, self.betas[0],
            self.betas[1], self.eps, self.weight_decay, self.step_count + 1, counter, scale, self.seed & 0xFFFFFFFF, s)))
        self.step_count += 1
