"""Training-step operators: products grouped by expert, gradient clipping, the
clipped policy loss (ctypes binding of include/conv_bwd_train.h).

Argument checks and marshalling only, as in ``binding``: every step of the
computation runs in the CUDA library.  Tensors are torch CUDA tensors; shapes,
types and strides are checked here (ValueError), addresses and the rest by the
library (ConvBwdError).  A plan belongs to the device that was current when it
was made: its tensors lie there, and that device is current in every call.
Outputs that are not passed in are allocated on the call's stream.  A plan owns a
workspace that its calls share: calls of one plan must not overlap on the GPU, so
keep one plan per stream.  The results carry no gradient functions; a tensor that
a call writes in place (``out``, the gradients of ``clip``) counts a new version, so
that autograd refuses a backward pass that had saved its old values.
"""
from __future__ import annotations

import array
import ctypes
import operator

import torch
from torch.autograd.graph import increment_version as _written  # what the library wrote in place, autograd may have saved

from . import binding as _b
from .binding import ConvBwdError, BF16, F32, OK  # noqa: F401  (part of this module's interface)

_TORCH = {F32: torch.float32, BF16: torch.bfloat16}
_NAMES = {"f32": F32, "bf16": BF16, torch.float32: F32, torch.bfloat16: BF16, F32: F32, BF16: BF16}
_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float

EXPORTED = [
    "conv_bwd_experts_create", "conv_bwd_experts_destroy", "conv_bwd_experts_forward", "conv_bwd_experts_data",
    "conv_bwd_experts_weight", "conv_bwd_experts_get_status", "conv_bwd_clip_create", "conv_bwd_clip_destroy",
    "conv_bwd_clip_norm", "conv_bwd_clip_run", "conv_bwd_clip_get_status", "conv_bwd_policy_create", "conv_bwd_policy_destroy",
    "conv_bwd_policy_forward", "conv_bwd_policy_backward", "conv_bwd_policy_forward_backward",
    "conv_bwd_policy_get_status",
]


class ExpertsDesc(ctypes.Structure):
    _fields_ = [("experts", _i64), ("K", _i64), ("N", _i64), ("dtype", _i32)]


class PolicyDesc(ctypes.Structure):
    _fields_ = [("vocab", _i64), ("dtype", _i32), ("clip_low", _f32), ("clip_high", _f32), ("kl", _f32),
                ("scale", _f32)]


def _declare():
    lib = _b.lib()
    P = ctypes.POINTER
    sig = {
        "conv_bwd_experts_create": [P(ExpertsDesc), P(_vp)],
        "conv_bwd_experts_destroy": [_vp],
        "conv_bwd_experts_forward": [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp],
        "conv_bwd_experts_data": [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp],
        "conv_bwd_experts_weight": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _vp],
        "conv_bwd_experts_get_status": [_vp, _vp, P(_i32)],
        "conv_bwd_clip_create": [_i32, P(_i64), P(_i32), P(_vp)],
        "conv_bwd_clip_destroy": [_vp],
        "conv_bwd_clip_norm": [_vp, _vp, _vp, _vp],
        "conv_bwd_clip_run": [_vp, _vp, _vp, _f32, _vp, _vp, _vp],
        "conv_bwd_clip_get_status": [_vp, _vp, P(_i32)],
        "conv_bwd_policy_create": [P(PolicyDesc), P(_vp)],
        "conv_bwd_policy_destroy": [_vp],
        "conv_bwd_policy_forward": [_vp, _i64, _vp, _i64] + [_vp] * 10,
        "conv_bwd_policy_backward": [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp],
        "conv_bwd_policy_forward_backward": [_vp, _i64, _vp, _i64] + [_vp] * 8 + [_i64, _vp],
        "conv_bwd_policy_get_status": [_vp, _vp, P(_i32)],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    return lib


_lib = _declare()


def _dtype(d):
    try:
        return _NAMES[d]
    except (KeyError, TypeError):
        raise ValueError(f"dtype {d!r}: f32 or bf16 wanted") from None


def _check(status, what):
    if status != OK:
        raise ConvBwdError(status, what)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # 0.1 us instead of 3 for a Stream object


def _stream(stream, device):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """A new tensor whose memory belongs to the call's stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=device)


# (a tensor's device as a number: -1 on the CPU; a plan made without a device has one that no tensor has)
_NOWHERE = -2


def _on(device):
    return f"on cuda:{device}" if device >= 0 else "on the plan's CUDA device"


def _rows(t, width, dtype, device, what):
    """Checks a matrix of rows with unit column stride; returns (rows, row stride)."""
    shape = t.shape
    if t.dtype != dtype or len(shape) != 2 or shape[1] != width or t.get_device() != device:
        raise ValueError(f"{what}: a {dtype} matrix with {width} columns {_on(device)} wanted, got {t.dtype} {tuple(shape)} on {t.device}")
    rows = shape[0]
    ld, unit = t.stride()
    if (unit != 1 and width > 1) or (ld < width and rows > 1):
        raise ValueError(f"{what}: unit column stride and rows that do not overlap wanted, got strides {t.stride()}")
    return rows, ld if ld > width else width


def _vector(t, n, dtype, device, what):
    if t.dtype != dtype or t.shape != (n,) or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous {dtype} vector of {n} {_on(device)} wanted, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


class _Plan:
    _destroy = None
    _h = None

    def __init__(self):
        self._device_index = torch.cuda.current_device() if torch.cuda.is_available() else _NOWHERE

    def close(self):
        h, self._h = self._h, None
        if h:
            self._destroy(h)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _status(call, handle, stream):
    det = _i32()
    device = torch.device("cuda", torch.cuda.current_device())
    return call(handle, _stream(stream, device), ctypes.byref(det)), det.value


class Experts(_Plan):
    """Matrix products grouped by expert with ragged sizes.

    Rows are sorted by expert; ``offsets`` (int32 CUDA tensor of experts + 1) says where each expert's rows begin, and
    stays on the GPU.  ``w`` is [experts, n, k].  Rows of no expert give zero rows.
    """
    _destroy = staticmethod(_lib.conv_bwd_experts_destroy)

    def __init__(self, experts, k, n, dtype="bf16"):
        super().__init__()
        self.experts, self.k, self.n = int(experts), int(k), int(n)
        self._code = _dtype(dtype)
        self.dtype = _TORCH[self._code]
        self._shape = (self.experts, self.n, self.k)
        desc, h = ExpertsDesc(self.experts, self.k, self.n, self._code), _vp()
        _check(_lib.conv_bwd_experts_create(ctypes.byref(desc), ctypes.byref(h)), "conv_bwd_experts_create")
        self._h = h.value

    def _product(self, call, name, what, a, wa, w, offsets, out, wo, stream):
        at = self._device_index
        rows, lda = _rows(a, wa, self.dtype, at, what)
        off = _vector(offsets, self.experts + 1, torch.int32, at, "offsets")
        if w.dtype != self.dtype or w.shape != self._shape or not w.is_contiguous() or w.get_device() != at:
            raise ValueError(f"w: a contiguous {self.dtype} tensor {list(self._shape)} {_on(at)} wanted, got {w.dtype} {tuple(w.shape)} on {w.device}")
        device, given = a.device, out
        if out is None:
            out = _empty((rows, wo), self.dtype, device, stream)
            ldo = wo
        else:
            r, ldo = _rows(out, wo, self.dtype, at, "out")
            if r != rows:
                raise ValueError(f"out: {rows} rows wanted, got {r}")
        st = call(self._h, rows, a.data_ptr(), lda, w.data_ptr(), off, out.data_ptr(), ldo, _stream(stream, device))
        if st != OK:
            raise ConvBwdError(st, name)
        if given is not None:
            _written(given)
        return out

    def forward(self, x, w, offsets, out=None, stream=None):
        """y[i] = w[e] x[i] for the rows i of every expert e; x [rows, k] -> y [rows, n]."""
        return self._product(_lib.conv_bwd_experts_forward, "conv_bwd_experts_forward", "x", x, self.k, w, offsets, out, self.n, stream)

    def backward_data(self, dy, w, offsets, out=None, stream=None):
        """dx[i] = w[e]^T dy[i]; dy [rows, n] -> dx [rows, k]."""
        return self._product(_lib.conv_bwd_experts_data, "conv_bwd_experts_data", "dy", dy, self.n, w, offsets, out, self.k, stream)

    def backward_weight(self, dy, x, offsets, out=None, accumulate=False, stream=None):
        """dw[e] = sum of dy[i] x[i]^T over the rows of e, in fp32 [experts, n, k]; added to ``out`` with ``accumulate``."""
        at = self._device_index
        rows, lddy = _rows(dy, self.n, self.dtype, at, "dy")
        r, ldx = _rows(x, self.k, self.dtype, at, "x")
        if r != rows:
            raise ValueError(f"x: {rows} rows wanted as in dy, got {r}")
        off = _vector(offsets, self.experts + 1, torch.int32, at, "offsets")
        given = out
        if out is None:
            if accumulate:
                raise ValueError("accumulate wants the gradients to add to in out")
            out = _empty(self._shape, torch.float32, dy.device, stream)
        elif out.dtype != torch.float32 or out.shape != self._shape or not out.is_contiguous() or out.get_device() != at:
            raise ValueError(f"out: a contiguous fp32 tensor {list(self._shape)} {_on(at)} wanted, got {out.dtype} {tuple(out.shape)} on {out.device}")
        _check(_lib.conv_bwd_experts_weight(self._h, rows, dy.data_ptr(), lddy, x.data_ptr(), ldx, off, out.data_ptr(),
                                            1 if accumulate else 0, _stream(stream, dy.device)), "conv_bwd_experts_weight")
        if given is not None:
            _written(given)
        return out

    def status(self, stream=None):
        """(status, detail) of the calls since the last one; synchronises the stream."""
        return _status(_lib.conv_bwd_experts_get_status, self._h, stream)


# (over hundreds of tensors a call, mapped in C)
_numel, _contiguous, _data_ptr, _get_device = torch.Tensor.numel, torch.Tensor.is_contiguous, torch.Tensor.data_ptr, torch.Tensor.get_device
_type = operator.attrgetter("dtype")


class GradClip(_Plan):
    """Global L2 norm over many tensors, and clipping.

    ``sizes`` and ``dtypes`` list the tensors' element counts and types; each call passes the tensors (contiguous, any
    shape) in that order.
    """
    _destroy = staticmethod(_lib.conv_bwd_clip_destroy)

    def __init__(self, sizes, dtypes):
        super().__init__()
        sizes = [int(n) for n in sizes]
        codes = [_dtype(d) for d in dtypes]
        if len(sizes) != len(codes):
            raise ValueError(f"{len(sizes)} sizes and {len(codes)} dtypes")
        self._sizes, self._types, self._devices = sizes, [_TORCH[c] for c in codes], [self._device_index] * len(sizes)
        self.count = n = len(sizes)
        h = _vp()
        _check(_lib.conv_bwd_clip_create(n, (_i64 * max(n, 1))(*sizes), (_i32 * max(n, 1))(*codes), ctypes.byref(h)), "conv_bwd_clip_create")
        self._h = h.value

    @classmethod
    def like(cls, tensors):
        """A plan for tensors of these sizes and types."""
        return cls([t.numel() for t in tensors], [t.dtype for t in tensors])

    def _pointers(self, tensors, what):
        if (list(map(_numel, tensors)) != self._sizes or list(map(_type, tensors)) != self._types
                or list(map(_get_device, tensors)) != self._devices or not all(map(_contiguous, tensors))):
            if len(tensors) != self.count:
                raise ValueError(f"{what}: {self.count} tensors wanted, got {len(tensors)}")
            for i, t in enumerate(tensors):
                if t.numel() != self._sizes[i] or t.dtype != self._types[i] or t.get_device() != self._device_index or not t.is_contiguous():
                    raise ValueError(f"{what}[{i}]: a contiguous {self._types[i]} tensor of {self._sizes[i]} elements {_on(self._device_index)} wanted, got {t.dtype} {tuple(t.shape)} on {t.device}")
        return array.array("Q", map(_data_ptr, tensors))

    def _device(self, grads):
        return grads[0].device if grads else torch.device("cuda", torch.cuda.current_device())

    def norm(self, grads, stream=None):
        """The norm as a CUDA fp32 tensor [1]."""
        g = self._pointers(grads, "grads")
        device = self._device(grads)
        norm = _empty((1,), torch.float32, device, stream)
        _check(_lib.conv_bwd_clip_norm(self._h, g.buffer_info()[0], norm.data_ptr(), _stream(stream, device)), "conv_bwd_clip_norm")
        return norm

    def clip(self, grads, max_norm, out=None, stream=None):
        """Scales ``grads`` by coef = min(1, max_norm / (norm + 1e-6)), in place or into ``out``; returns (norm, coef)."""
        max_norm = float(max_norm)
        if not max_norm >= 0:
            raise ValueError(f"max_norm {max_norm}: a number >= 0 wanted")
        g = self._pointers(grads, "grads")
        o = g if out is None else self._pointers(out, "out")
        device = self._device(grads)
        norm, coef = _empty((1,), torch.float32, device, stream), _empty((1,), torch.float32, device, stream)
        _check(_lib.conv_bwd_clip_run(self._h, g.buffer_info()[0], o.buffer_info()[0], max_norm, norm.data_ptr(), coef.data_ptr(), _stream(stream, device)), "conv_bwd_clip_run")
        _written(grads if out is None else out)
        return norm, coef

    def status(self, stream=None):
        """(status, detail) of the calls since the last one; synchronises the stream."""
        return _status(_lib.conv_bwd_clip_get_status, self._h, stream)


class PolicyLoss(_Plan):
    """Clipped policy loss with a KL term, from logits.

    loss = sum_t weight_t (-min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A) + kl (exp(d) - d - 1)) with
    r = exp(logp - old_logp), d = ref_logp - logp and logp the log-probability of the chosen token under
    softmax(scale * logits).  Tokens with weight 0 or a negative action are masked.
    """
    _destroy = staticmethod(_lib.conv_bwd_policy_destroy)

    def __init__(self, vocab, dtype="bf16", clip_low=0.2, clip_high=0.2, kl=0.0, scale=1.0):
        super().__init__()
        self.vocab = int(vocab)
        self._code = _dtype(dtype)
        self.dtype = _TORCH[self._code]
        desc, h = PolicyDesc(self.vocab, self._code, clip_low, clip_high, kl, scale), _vp()
        _check(_lib.conv_bwd_policy_create(ctypes.byref(desc), ctypes.byref(h)), "conv_bwd_policy_create")
        self._h = h.value

    def _inputs(self, logits, actions, advantage, weight, old_logp, ref_logp):
        at = self._device_index
        t, ld = _rows(logits, self.vocab, self.dtype, at, "logits")
        f = torch.float32
        return t, (self._h, t, logits.data_ptr(), ld, _vector(actions, t, torch.int32, at, "actions"),
                   _vector(advantage, t, f, at, "advantage"), _vector(weight, t, f, at, "weight"),
                   None if old_logp is None else _vector(old_logp, t, f, at, "old_logp"),
                   None if ref_logp is None else _vector(ref_logp, t, f, at, "ref_logp"))

    def _grad_out(self, logits, t, out, stream):
        if out is None:
            return _empty((t, self.vocab), self.dtype, logits.device, stream), self.vocab
        r, ld = _rows(out, self.vocab, self.dtype, self._device_index, "out")
        if r != t:
            raise ValueError(f"out: {t} rows wanted, got {r}")
        return out, ld

    def forward(self, logits, actions, advantage, weight, old_logp=None, ref_logp=None, stream=None):
        """(loss [1], logp, lse, coef [tokens]); lse and coef are what ``backward`` needs."""
        t, args = self._inputs(logits, actions, advantage, weight, old_logp, ref_logp)
        device = logits.device
        # (four tensors: views of one that is new cost more than its memory)
        logp, lse, coef = (_empty((t,), torch.float32, device, stream) for _ in range(3))
        loss = _empty((1,), torch.float32, device, stream)
        _check(_lib.conv_bwd_policy_forward(*args, loss.data_ptr(), logp.data_ptr(), lse.data_ptr(), coef.data_ptr(), _stream(stream, device)), "conv_bwd_policy_forward")
        return loss, logp, lse, coef

    def backward(self, logits, actions, lse, coef, grad=None, out=None, stream=None):
        """dlogits from the forward's lse and coef; ``grad`` [1] is the loss's upstream gradient; ``out`` may be logits."""
        at = self._device_index
        t, ld = _rows(logits, self.vocab, self.dtype, at, "logits")
        f = torch.float32
        args = (self._h, t, logits.data_ptr(), ld, _vector(actions, t, torch.int32, at, "actions"), _vector(lse, t, f, at, "lse"),
                _vector(coef, t, f, at, "coef"), None if grad is None else _vector(grad, 1, f, at, "grad"))
        given = out
        out, ldd = self._grad_out(logits, t, out, stream)
        _check(_lib.conv_bwd_policy_backward(*args, out.data_ptr(), ldd, _stream(stream, logits.device)), "conv_bwd_policy_backward")
        if given is not None:
            _written(given)
        return out

    def forward_backward(self, logits, actions, advantage, weight, old_logp=None, ref_logp=None, out=None, stream=None):
        """(loss [1], logp [tokens], dlogits) in one launch; ``out`` may be logits."""
        t, args = self._inputs(logits, actions, advantage, weight, old_logp, ref_logp)
        given = out
        out, ldd = self._grad_out(logits, t, out, stream)
        device = logits.device
        logp = _empty((t,), torch.float32, device, stream)
        loss = _empty((1,), torch.float32, device, stream)
        _check(_lib.conv_bwd_policy_forward_backward(*args, loss.data_ptr(), logp.data_ptr(), out.data_ptr(), ldd, _stream(stream, device)), "conv_bwd_policy_forward_backward")
        if given is not None:
            _written(given)
        return loss, logp, out

    def status(self, stream=None):
        """(status, detail) of the calls since the last one; synchronises the stream."""
        return _status(_lib.conv_bwd_policy_get_status, self._h, stream)
