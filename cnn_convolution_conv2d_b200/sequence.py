"""Operators over sequences: the causal depthwise convolution over time and the gated
linear recurrence, a thin binding of ``include/sequence_b200.h``.

Tensors over sequences are (B, T, C), or (rows, C) with ``offsets`` (B + 1 int32 values on the
device): sequences of their own lengths packed one behind the other.  Channels are contiguous
and rows a fixed distance apart, so a slice ``z[..., :C]`` of a wider projection is taken as it is.

``CausalConv1dB200`` and ``GatedRecurrenceB200`` hold a layer's weights; a call is the forward
pass, ``backward`` its gradients, ``step`` one token for each of a batch of sequences.  Scratch is
allocated for each call on the call's stream, so calls on several streams, and graphs captured
from them, share none.
"""
from __future__ import annotations

import ctypes
import functools

from . import _check, _dtype_code, load

CONV_ACT_NONE = 0
CONV_ACT_SILU = 1

_I, _P, _S, _L, _F = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_float
_SEQ = [_P, _I, _I, _L, _I]  # offsets, nseq, T, rows, C
SIGNATURES = {
    "conv1d_causal_forward": ([_P] * 6 + _SEQ + [_I, _I, _L, _L, _I, _P], _I),
    "conv1d_causal_backward_workspace_size": ([_L, _I, _I, ctypes.POINTER(_S)], _I),
    "conv1d_causal_backward": ([_P] * 10 + _SEQ + [_I, _I, _L, _L, _L, _I, _P, _S, _P], _I),
    "conv1d_causal_step": ([_P] * 6 + [_I] * 5 + [_L, _L, _I, _P], _I),
    "gated_recurrence_saved_size": ([_I, _I, _L, _I, _I, ctypes.POINTER(_S)], _I),
    "gated_recurrence_workspace_size": ([_I, _I, _L, _I, _I, ctypes.POINTER(_S)], _I),
    "gated_recurrence_backward_workspace_size": ([_I, _I, _L, _I, _I, ctypes.POINTER(_S)], _I),
    "gated_recurrence_forward": ([_P] * 4 + [_F] + [_P] * 4 + _SEQ + [_L] * 4 + [_I, _P, _S, _P], _I),
    "gated_recurrence_backward": ([_P] * 4 + [_F] + [_P] * 9 + _SEQ + [_L] * 7 + [_I, _P, _S, _P], _I),
    "gated_recurrence_step": ([_P] * 4 + [_F] + [_P] * 3 + [_I] * 3 + [_L] * 4 + [_I, _P], _I),
}


def _size(fn, *args) -> int:
    out = ctypes.c_size_t(0)
    _check(fn(*args, ctypes.byref(out)))
    return out.value


def conv1d_causal_backward_workspace_size(rows, C, K) -> int:
    return _size(load().conv1d_causal_backward_workspace_size, rows, C, K)


@functools.lru_cache(maxsize=4096)
def _conv_scratch_bytes(index, rows, C, K) -> int:
    """conv1d_causal_backward_workspace_size on device `index`, the current one, on which it depends besides."""
    return conv1d_causal_backward_workspace_size(rows, C, K)


# These three depend on their arguments alone: asked once for each.
@functools.lru_cache(maxsize=4096)
def gated_recurrence_saved_size(nseq, T, rows, C, dtype) -> int:
    return _size(load().gated_recurrence_saved_size, nseq, T, rows, C, dtype)


@functools.lru_cache(maxsize=4096)
def gated_recurrence_workspace_size(nseq, T, rows, C, dtype) -> int:
    return _size(load().gated_recurrence_workspace_size, nseq, T, rows, C, dtype)


@functools.lru_cache(maxsize=4096)
def gated_recurrence_backward_workspace_size(nseq, T, rows, C, dtype) -> int:
    return _size(load().gated_recurrence_backward_workspace_size, nseq, T, rows, C, dtype)


# ------------------------------------------------------------ argument checks ---
def _rows(name, t, like):
    """(pointer, row stride) of a tensor over rows: on `like`'s device, of `like`'s shape and dtype."""
    if t is not like:
        if t.device != like.device:
            raise ValueError(f"{name} must be on {like.device}, not on {t.device}")
        if t.dtype != like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, not {t.dtype}")
        if t.shape != like.shape:
            raise ValueError(f"{name} must have the shape {tuple(like.shape)}, not {tuple(t.shape)}")
    sizes = t.shape
    if t.is_contiguous():
        return t.data_ptr(), sizes[-1]
    stride = t.stride()
    if sizes[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    if len(sizes) == 2:
        return t.data_ptr(), stride[0] if sizes[0] > 1 else max(stride[0], sizes[1])
    B, T, C = sizes
    if T > 1:
        if B > 1 and stride[0] != T * stride[1]:
            raise ValueError(f"the rows of {name} must lie a fixed distance apart; use {name}.contiguous()")
        return t.data_ptr(), stride[1]
    return t.data_ptr(), stride[0] if B > 1 else max(stride[0], C)


def _new(x):
    """An uninitialised tensor like x, contiguous."""
    import torch
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _out(name, t, like):
    """(tensor, pointer, row stride) of an output over rows: t, or where there is none a new one like `like`, which needs no checks."""
    if t is None:
        t = _new(like)
        return t, t.data_ptr(), like.shape[-1]
    return (t, *_rows(name, t, like))


def _kind(t):
    """What of a tensor decides whether it can still be used as it was: compared at each call, for less than _whole costs."""
    return None if t is None else (t.data_ptr(), t.dtype, t.shape, t.is_contiguous())


def _whole(name, t, shape, dtype, device):
    """Pointer of a contiguous tensor of exactly this shape and type (None: no tensor)."""
    if t is None:
        return None
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.data_ptr()


def _sequences(x, offsets):
    """(offsets pointer, number of sequences, T, rows, C) of an input over sequences."""
    import torch
    if offsets is None:
        if x.dim() != 3:
            raise ValueError("without offsets, x must be (B, T, C)")
        B, T, C = x.shape
        return None, B, T, B * T, C
    if x.dim() != 2:
        raise ValueError("with offsets, x must be (rows, C)")
    if offsets.dim() != 1 or offsets.numel() < 2 or offsets.dtype != torch.int32:
        raise ValueError("offsets must hold one int32 value more than there are sequences")
    if offsets.device != x.device or not offsets.is_contiguous():
        raise ValueError(f"offsets must be a contiguous tensor on {x.device}")
    return offsets.data_ptr(), offsets.numel() - 1, 0, x.shape[0], x.shape[1]


def _current_stream(index):
    """The handle of a device's current stream: without the stream object, whose making costs more than a launch, where
    this torch offers that."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _on(x, stream, call):
    """call(raw stream) with x's device current, and `stream` (a torch stream or a handle) where
    one is given, so that what the call allocates belongs to the stream it is used on."""
    import torch
    if not x.is_cuda:
        raise ValueError("tensors passed to the library must be CUDA tensors")
    index = x.device.index
    if stream is None and torch.cuda.current_device() == index:
        return call(_current_stream(index))
    with torch.cuda.device(x.device):
        if stream is None:
            return call(torch.cuda.current_stream().cuda_stream)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=x.device) if stream else torch.cuda.default_stream(x.device)
        if stream.device != x.device:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to {x.device}")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _slots(slots, B, device):
    import torch
    return _whole("slots", slots, (B,), torch.int32, device)


def _scratch(nbytes, device):
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


# ----------------------------------------------------------------- convolution ---
class CausalConv1dB200:
    """A causal depthwise convolution over time: y[t] = act(bias + sum_k w[:, k] x[t-K+1+k]).

    ``w`` is (C, K) with 2 <= K <= 8, ``bias`` (C,) or None, both bf16 or fp32 on one CUDA device;
    ``activation`` is None or "silu".  The layer reads the tensors it was given: updating
    them in place (``AdamWB200`` does) updates the layer, and their ``data`` may be replaced by one of the same size and type."""

    def __init__(self, w, bias=None, activation=None):
        if w.dim() != 2:
            raise ValueError("w must be (C, K)")
        if not 2 <= w.shape[1] <= 8:
            raise ValueError("K must lie in 2 .. 8")
        if activation not in (None, "silu"):
            raise ValueError(f"unknown activation {activation!r}; use None or 'silu'")
        self.C, self.K = int(w.shape[0]), int(w.shape[1])
        self.dtype = _dtype_code(w.dtype)
        self.torch_dtype, self.device = w.dtype, w.device
        self.w, self.bias, self._known = w, bias, None
        self._weights()
        self.act = CONV_ACT_SILU if activation == "silu" else CONV_ACT_NONE

    def _input(self, x):
        if x.shape[-1] != self.C:
            raise ValueError(f"x has {x.shape[-1]} channels, the layer {self.C}")
        if x.dtype != self.torch_dtype:
            raise TypeError(f"x must be {self.torch_dtype}, not {x.dtype}")
        if x.device != self.device:
            raise ValueError(f"x must be on {self.device}, not on {x.device}")

    def __call__(self, x, y=None, offsets=None, initial_state=None, final_state=None, stream=None):
        """y for x (B, T, C), or (rows, C) with offsets.  ``initial_state`` (B, K-1, C): the rows before each
        sequence; ``final_state``: a buffer of that shape that receives its last K-1 rows."""
        self._input(x)
        seq = _sequences(x, offsets)
        window = (seq[1], self.K - 1, self.C)
        px, ldx = _rows("x", x, x)
        state = _whole("initial_state", initial_state, window, x.dtype, x.device)
        final = _whole("final_state", final_state, window, x.dtype, x.device)
        weights = self._weights()

        def call(s):
            out, py, ldy = _out("y", y, x)
            _check(load().conv1d_causal_forward(px, *weights, py, state, final, *seq, self.K,
                                                self.act, ldx, ldy, self.dtype, s))
            return out
        return _on(x, stream, call)

    def _weights(self):
        """The pointers of w and the bias, which are looked at again where they are not what they were at the last call."""
        known = w, bias = _kind(self.w), _kind(self.bias)
        if known != self._known:
            _whole("w", self.w, (self.C, self.K), self.torch_dtype, self.device)
            _whole("bias", self.bias, (self.C,), self.torch_dtype, self.device)
            self._known = known
        return w[0], bias and bias[0]

    def backward(self, x, dy, offsets=None, initial_state=None, d_final_state=None, dx=None, dw=None, db=None,
                 d_initial_state=None, stream=None):
        """(dx, dw, db, d_initial_state) for the forward pass's arguments and dy; db without a bias and
        d_initial_state without an initial state are None."""
        self._input(x)
        seq = _sequences(x, offsets)
        window = (seq[1], self.K - 1, self.C)
        px, ldx = _rows("x", x, x)
        pdy, lddy = _rows("dy", dy, x)
        state = _whole("initial_state", initial_state, window, x.dtype, x.device)
        dfinal = _whole("d_final_state", d_final_state, window, x.dtype, x.device)
        weights = self._weights()

        def call(s):
            gx, pgx, ldgx = _out("dx", dx, x)
            gw = _new(self.w) if dw is None else dw
            gb = _new(self.bias) if db is None and self.bias is not None else db
            gs = _new(initial_state) if d_initial_state is None and initial_state is not None else d_initial_state
            ws = _scratch(_conv_scratch_bytes(x.device.index, seq[3], self.C, self.K), x.device)
            _check(load().conv1d_causal_backward(
                px, *weights, pdy, state, dfinal, pgx,
                _whole("dw", gw, (self.C, self.K), x.dtype, x.device), _whole("db", gb, (self.C,), x.dtype, x.device),
                _whole("d_initial_state", gs, window, x.dtype, x.device), *seq, self.K, self.act, ldx, lddy, ldgx,
                self.dtype, None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), s))
            return gx, gw, gb, gs
        return _on(x, stream, call)

    def step(self, x, state, slots=None, y=None, stream=None):
        """One token for each of B sequences: y (B, C) for x (B, C), and the windows in ``state`` (pool, K-1, C)
        moved on in place.  Row b's window is state[slots[b]] (int32; outside the pool: no sequence, y's row stays
        as it was), or state[b] without slots."""
        self._input(x)
        if x.dim() != 2:
            raise ValueError("x must be (B, C)")
        B = x.shape[0]
        px, ldx = _rows("x", x, x)
        ps = _whole("state", state, (state.shape[0], self.K - 1, self.C), x.dtype, x.device)
        pslots = _slots(slots, B, x.device)
        weights = self._weights()

        def call(s):
            out, py, ldy = _out("y", y, x)
            _check(load().conv1d_causal_step(px, *weights, py, ps, pslots, B, state.shape[0],
                                             self.C, self.K, self.act, ldx, ldy, self.dtype, s))
            return out
        return _on(x, stream, call)


# ------------------------------------------------------------------ recurrence ---
class GatedRecurrenceB200:
    """The gated linear recurrence h[t] = a h[t-1] + sqrt(1 - a^2) sigmoid(gate_x) x with
    a = exp(-kappa softplus(decay) sigmoid(gate_a)), each channel by itself.

    ``decay`` is (C,) fp32; x and the gates are bf16 or fp32 of one shape; states are fp32.  The
    layer reads the ``decay`` it was given: updating it in place updates the layer, and its ``data`` may be replaced by one of
    the same size and type."""

    def __init__(self, decay, kappa=8.0):
        if decay.dim() != 1:
            raise ValueError("decay must be (C,)")
        self.decay, self.kappa, self.C, self.device = decay, float(kappa), int(decay.shape[0]), decay.device
        self._known = None
        self._decay()

    def _decay(self):
        """decay's pointer; decay is looked at again where it is not what it was at the last call."""
        import torch
        known = _kind(self.decay)
        if known != self._known:
            _whole("decay", self.decay, (self.C,), torch.float32, self.device)
            self._known = known
        return known[0]

    def _input(self, x):
        if x.shape[-1] != self.C:
            raise ValueError(f"x has {x.shape[-1]} channels, the layer {self.C}")
        if x.device != self.device:
            raise ValueError(f"x must be on {self.device}, not on {x.device}")
        return _dtype_code(x.dtype)

    def _saved_floats(self, x, code):
        packed = x.dim() == 2  # the size depends on the rows alone then, not on how they are cut
        nseq, T, rows = (1, 0, x.shape[0]) if packed else (x.shape[0], x.shape[1], x.shape[0] * x.shape[1])
        return gated_recurrence_saved_size(nseq, T, rows, self.C, code) // 4

    def saved_states(self, x):
        """A buffer for the states that the forward pass over x saves for its backward pass."""
        import torch
        return torch.empty(self._saved_floats(x, _dtype_code(x.dtype)), dtype=torch.float32, device=x.device)

    def _saved(self, saved, x, code):
        import torch
        return _whole("saved", saved, (self._saved_floats(x, code),), torch.float32, x.device)

    def __call__(self, x, gate_a, gate_x, y=None, offsets=None, initial_state=None, final_state=None, saved=None,
                 stream=None):
        """y = h for x (B, T, C), or (rows, C) with offsets.  ``initial_state`` (B, C): h before each sequence;
        ``final_state``: a buffer of that shape that receives its last h; ``saved``: ``saved_states(x)``, filled for
        ``backward``."""
        import torch
        code = self._input(x)
        seq = _sequences(x, offsets)
        (px, ldx), (pa, lda), (pg, ldg) = _rows("x", x, x), _rows("gate_a", gate_a, x), _rows("gate_x", gate_x, x)
        state = _whole("initial_state", initial_state, (seq[1], self.C), torch.float32, x.device)
        final = _whole("final_state", final_state, (seq[1], self.C), torch.float32, x.device)
        psaved = None if saved is None else self._saved(saved, x, code)
        pdecay = self._decay()

        def call(s):
            out, py, ldy = _out("y", y, x)
            ws = _scratch(gated_recurrence_workspace_size(*seq[1:], code), x.device)
            _check(load().gated_recurrence_forward(
                px, pa, pg, pdecay, self.kappa, py, state, final, psaved, *seq, ldx, lda, ldg, ldy, code,
                None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), s))
            return out
        return _on(x, stream, call)

    def backward(self, x, gate_a, gate_x, dy, saved, offsets=None, initial_state=None, d_final_state=None, dx=None,
                 d_gate_a=None, d_gate_x=None, d_decay=None, d_initial_state=None, stream=None):
        """(dx, d_gate_a, d_gate_x, d_decay, d_initial_state) for the forward pass's arguments, the ``saved`` it
        filled, and dy; d_initial_state is None without an initial state."""
        import torch
        code = self._input(x)
        seq = _sequences(x, offsets)
        (px, ldx), (pa, lda), (pg, ldg) = _rows("x", x, x), _rows("gate_a", gate_a, x), _rows("gate_x", gate_x, x)
        pdy, lddy = _rows("dy", dy, x)
        f32 = torch.float32
        state = _whole("initial_state", initial_state, (seq[1], self.C), f32, x.device)
        dfinal = _whole("d_final_state", d_final_state, (seq[1], self.C), f32, x.device)
        psaved = self._saved(saved, x, code)
        pdecay = self._decay()

        def call(s):
            gx, pgx, ldgx = _out("dx", dx, x)
            ga, pga, ldga = _out("d_gate_a", d_gate_a, x)
            gg, pgg, ldgg = _out("d_gate_x", d_gate_x, x)
            gd = _new(self.decay) if d_decay is None else d_decay
            gs = _new(initial_state) if d_initial_state is None and initial_state is not None else d_initial_state
            ws = _scratch(gated_recurrence_backward_workspace_size(*seq[1:], code), x.device)
            _check(load().gated_recurrence_backward(
                px, pa, pg, pdecay, self.kappa, pdy, psaved, state, dfinal, pgx, pga, pgg,
                _whole("d_decay", gd, (self.C,), f32, x.device),
                _whole("d_initial_state", gs, (seq[1], self.C), f32, x.device), *seq, ldx, lda, ldg, lddy, ldgx, ldga,
                ldgg, code, ws.data_ptr(), ws.numel(), s))
            return gx, ga, gg, gd, gs
        return _on(x, stream, call)

    def step(self, x, gate_a, gate_x, state, slots=None, y=None, stream=None):
        """One token for each of B sequences: y (B, C) for x and the gates (B, C); ``state`` (pool, C) fp32 is updated
        in place, slots as in ``CausalConv1dB200.step``."""
        import torch
        code = self._input(x)
        if x.dim() != 2:
            raise ValueError("x must be (B, C)")
        B = x.shape[0]
        (px, ldx), (pa, lda), (pg, ldg) = _rows("x", x, x), _rows("gate_a", gate_a, x), _rows("gate_x", gate_x, x)
        ps = _whole("state", state, (state.shape[0], self.C), torch.float32, x.device)
        pslots = _slots(slots, B, x.device)
        pdecay = self._decay()

        def call(s):
            out, py, ldy = _out("y", y, x)
            _check(load().gated_recurrence_step(px, pa, pg, pdecay, self.kappa, py, ps, pslots, B,
                                                state.shape[0], self.C, ldx, lda, ldg, ldy, code, s))
            return out
        return _on(x, stream, call)
