"""The operators of a language model around its low-bit layers, on torch CUDA tensors.

:class:`QuantFC` is a layer object like the binary ones; :func:`block_norm` and
:func:`token_logprobs` (and their ``_backward``) are functions.  They only marshal: they check
types, shapes and devices, allocate outputs and workspaces with torch and call the C entry points on
the current stream of the tensors' device.  Activations are float32, bfloat16 or float16; inputs
whose last dimension (or, where rows have to be packed, whose rows) are not contiguous are
copied.  Scalars are numbers; a one-element tensor given for one is read at the call, which waits for it.
Gradients are explicit calls; nothing here records for autograd.
"""
from __future__ import annotations

import ctypes
import functools
import operator
from typing import NamedTuple

import torch

from . import _native as nat
from .layers import _Owner

_DTYPES = {torch.float32: nat.DTYPE_F32, torch.bfloat16: nat.DTYPE_BF16, torch.float16: nat.DTYPE_F16}
_NAMED = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _dtype(t) -> torch.dtype:
    t = _NAMED.get(t, t)
    if t not in _DTYPES:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, got {t}")
    return t


# The calls below are as short as the kernels they launch, so the checks are few and cheap: integers instead of
# torch.device objects, the C functions directly.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_empty_like = torch.empty_like
_F32 = torch.float32


def _call(name, device, *args):
    """A C entry point on the current stream of the device."""
    fn = _FUNCTIONS.get(name)
    if fn is None:
        fn = _FUNCTIONS[name] = getattr(nat.load_library(), name)
    if device == _current_device():
        status = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device))
    if status:
        raise nat.BconvError(status, name)


_FUNCTIONS: dict = {}


def _activation(x, name):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if x.dtype not in _DTYPES:
        raise TypeError(f"{name}: expected float32, bfloat16 or float16, got {x.dtype}")
    return x


def _like(t, device, dtype, shape, name):
    """t as a contiguous tensor, checked against a device, a dtype and a shape."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise TypeError(f"{name}: expected a tensor on cuda:{device}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t if t.is_contiguous() else t.contiguous()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _number(v, name):
    """v as it is now: a one-element tensor is read (which waits for it), not kept."""
    if type(v) is float:
        return v
    if isinstance(v, (str, bytes)):
        raise TypeError(f"{name}: expected a number, got {v!r}")
    return float(v.item() if isinstance(v, torch.Tensor) else v)


def _rows(x):
    """(tensor, rows, row stride) of x as a matrix over its last dimension; copied if it is none."""
    if x.dim() == 2:
        stride = x.stride()
        if stride[1] == 1 and stride[0] >= x.shape[1]:
            return x, x.shape[0], stride[0]
    x = x.contiguous()
    width = x.shape[-1]
    return x, x.numel() // width if width else 0, width


class QuantFC(_Owner):
    """A fully-connected layer with 4-bit weights and group scales on the current CUDA device.

    ``W[c][f] = scale[c][f // group_size] * (code[c][f] - zero[c][f // group_size])``.

    codes: uint8 0..15 [out_channels, in_channels], or ``packed`` uint8 [out_channels,
    ceil(in_channels / 2)], channel f in the low (f even) or high four bits of byte f // 2.  scale: float32
    [out_channels, groups]; zero: uint8 of the same shape (None: 8); bias: float32 [out_channels].  All
    may be numpy arrays or torch tensors on the host or the device; they are copied.
    group_size: 32, 64, a multiple of 128, or at least in_channels.

    ``layer(x)`` takes [..., in_channels] of ``dtype`` and returns [..., out_channels] of
    ``out_dtype`` (default: dtype).  A layer may be used on several streams at once.
    """

    _destroy = staticmethod(nat.bfc_quant_destroy)

    def __init__(self, in_channels, out_channels, *, codes=None, packed=None, scale, zero=None, bias=None,
                 group_size=128, relu=False, dtype=torch.bfloat16, out_dtype=None):
        self.handle = None
        self.in_channels, self.out_channels = int(in_channels), int(out_channels)
        self.dtype = _dtype(dtype)
        self.out_dtype = _dtype(out_dtype) if out_dtype is not None else self.dtype
        if group_size < 1 or in_channels < 1 or out_channels < 1:
            raise ValueError("in_channels, out_channels and group_size must be positive")
        groups = -(-self.in_channels // group_size)
        if packed is None:
            if codes is None:
                raise ValueError("give codes or packed")
            packed = self.pack(self._array(codes, torch.uint8, (self.out_channels, self.in_channels), "codes"))
        packed = self._array(packed, torch.uint8, (self.out_channels, (self.in_channels + 1) // 2), "packed")
        scale = self._array(scale, torch.float32, (self.out_channels, groups), "scale")
        zero = self._array(zero, torch.uint8, (self.out_channels, groups), "zero")
        bias = self._array(bias, torch.float32, (self.out_channels,), "bias")
        for t in (packed, scale, zero, bias):
            if t is not None and t.is_cuda:
                torch.cuda.current_stream(t.device).synchronize()  # the layout kernels run on another stream
        desc = nat.bfc_quant_desc_t(self.in_channels, self.out_channels, int(group_size),
                                    nat.NEURON_RELU if relu else nat.NEURON_NONE, _DTYPES[self.dtype],
                                    _DTYPES[self.out_dtype])
        self.handle = nat.bfc_quant_create(desc, _ptr(packed), _ptr(scale), _ptr(zero), _ptr(bias))
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._device = self.device.index
        lib = nat.load_library()
        self._forward, self._workspace_bytes = lib.bfc_quant_forward, lib.bfc_quant_workspace_bytes

    @staticmethod
    def _array(a, dtype, shape, name):
        if a is None:
            return None
        t = torch.as_tensor(a)
        if t.dtype != dtype:
            if dtype == torch.uint8 or not t.dtype.is_floating_point:
                raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
            t = t.to(dtype)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
        return t.contiguous()

    @staticmethod
    def pack(codes):
        """uint8 codes [..., n] -> packed uint8 [..., ceil(n / 2)]."""
        codes = torch.as_tensor(codes) & 15
        if codes.shape[-1] % 2:
            codes = torch.nn.functional.pad(codes, (0, 1))
        return codes[..., 0::2] | (codes[..., 1::2] << 4)

    @property
    def input_feature_channels(self) -> int:
        return nat.bfc_quant_input_feature_channels(self.handle)

    @property
    def output_feature_channels(self) -> int:
        return nat.bfc_quant_output_feature_channels(self.handle)

    def forward_into(self, x, out):
        """x [..., in_channels] into out [..., out_channels] (the rows of out may be strided)."""
        handle, device = self.handle, self._device
        if handle is None:
            raise ValueError("the layer is closed")
        if (not isinstance(x, torch.Tensor) or not isinstance(out, torch.Tensor) or x.get_device() != device
                or out.get_device() != device):
            raise TypeError(f"expected tensors on {self.device}")
        if x.dtype != self.dtype or out.dtype != self.out_dtype:
            raise TypeError(f"expected {self.dtype} -> {self.out_dtype}, got {x.dtype} -> {out.dtype}")
        if x.shape[-1] != self.in_channels or out.shape != x.shape[:-1] + (self.out_channels,):
            raise ValueError(f"expected [..., {self.in_channels}] -> [..., {self.out_channels}], got "
                             f"{tuple(x.shape)} -> {tuple(out.shape)}")
        x, rows, in_stride = _rows(x)
        to, _, out_stride = _rows(out)
        if to is not out and to.data_ptr() != out.data_ptr():
            raise ValueError("out must have contiguous channels, and rows without gaps unless it is a matrix")
        at = x.data_ptr()
        need = self._workspace_bytes(handle, at, in_stride, rows)
        ws = x.new_empty(need, dtype=torch.uint8) if need > 0 else None
        # (the library makes the layer's device current itself)
        status = self._forward(handle, at, in_stride, rows, to.data_ptr(), out_stride, _ptr(ws), _raw_stream(device))
        if status:
            raise nat.BconvError(status, "bfc_quant_forward")
        return out

    def __call__(self, x):
        if not isinstance(x, torch.Tensor) or not x.is_cuda:
            raise TypeError("expected a CUDA tensor")
        if x.dim() < 1:
            raise ValueError("expected [..., in_channels]")
        out = x.new_empty(x.shape[:-1] + (self.out_channels,), dtype=self.out_dtype)
        return self.forward_into(x, out)

    def sync_status(self):
        """Waits for the current stream of the layer's device and raises if a kernel of the layer gave up a wait."""
        nat.bfc_quant_sync_status(self.handle, _raw_stream(self._device))


class BlockNorm(NamedTuple):
    residual_out: torch.Tensor
    normed: torch.Tensor | None


class BlockNormGrad(NamedTuple):
    d_residual: torch.Tensor
    d_block: torch.Tensor | None
    d_pre_weight: torch.Tensor | None
    d_post_weight: torch.Tensor | None
    d_gate: torch.Tensor | None


def _norm_desc(device, rows, per, width, dtype, residual_scale, eps):
    """The C descriptor (by reference, and kept alive by its first item) and the backward's workspace on this device."""
    return _norm_desc_of(device, rows, per, width, dtype, _number(residual_scale, "residual_scale"), _number(eps, "eps"))


@functools.lru_cache(maxsize=256)  # (of plain numbers, which do not change behind its back)
def _norm_desc_of(device, rows, per, width, dtype, residual_scale, eps):
    desc = nat.bconv_block_norm_desc_t(rows, per, width, _DTYPES[dtype], residual_scale, eps)
    with torch.cuda.device(device):
        need = nat.load_library().bconv_block_norm_workspace_bytes(desc)
    return desc, ctypes.byref(desc), need


def _block_norm_args(residual, block, pre_weight, post_weight, gate, rows_per_gate, residual_scale, eps):
    residual = _activation(residual, "residual")
    if not residual.is_contiguous():
        residual = residual.contiguous()
    shape, dtype, device = residual.shape, residual.dtype, residual.get_device()
    if not shape or shape[-1] == 0:
        raise ValueError("residual: expected [..., width]")
    width = shape[-1]
    rows = residual.numel() // width
    if block is not None:
        block = _like(block, device, dtype, shape, "block")
    elif gate is not None or post_weight is not None:
        raise ValueError("gate and post_weight belong to a block")
    if pre_weight is not None:
        pre_weight = _like(pre_weight, device, _F32, (width,), "pre_weight")
    if post_weight is not None:
        post_weight = _like(post_weight, device, _F32, (width,), "post_weight")
    per = 1
    if gate is not None:
        if not isinstance(gate, torch.Tensor) or gate.dim() < 1 or gate.shape[-1] != width:
            raise ValueError(f"gate: expected [..., {width}]")
        gates = gate.numel() // width
        if rows_per_gate is not None:
            per = operator.index(rows_per_gate)
        elif rows:
            per = rows // max(gates, 1)
        if per < 1:
            raise ValueError("rows_per_gate must be positive, and there are not more gates than rows")
        if gates != -(-rows // per):
            raise ValueError(f"{gates} gate rows of {per} rows each do not fit {rows} rows")
        gate = _like(gate, device, dtype, gate.shape, "gate")
    return residual, block, pre_weight, post_weight, gate, device, (device, rows, per, width, dtype, residual_scale, eps)


def block_norm(residual, block=None, *, pre_weight=None, post_weight=None, gate=None, rows_per_gate=None,
               residual_scale=1.0, eps=1e-6) -> BlockNorm:
    """The norm behind a block, its gate and residual scale, the residual sum and the next norm.

    ``p = block * rsqrt(mean(block^2) + eps) * post_weight`` (``post_weight=None``: p = block),
    ``residual_out = residual + residual_scale * gate * p`` and ``normed = residual_out *
    rsqrt(mean(residual_out^2) + eps) * pre_weight`` (``pre_weight=None``: no ``normed``), over
    rows of the last dimension.  residual, block and gate have one dtype, the weights are float32.
    gate [..., width]: its row g holds for ``rows_per_gate`` consecutive rows (default: rows / gate
    rows).  ``block=None`` (the norm before the first block) returns residual itself.
    """
    if block is None and pre_weight is None:
        raise ValueError("without a block there is only the norm: give pre_weight")
    given = residual
    residual, block, pre_weight, post_weight, gate, device, args = _block_norm_args(
        residual, block, pre_weight, post_weight, gate, rows_per_gate, residual_scale, eps)
    out = _empty_like(residual) if block is not None else None
    normed = _empty_like(residual) if pre_weight is not None else None
    _call("bconv_block_norm_forward", device, _norm_desc(*args)[1], residual.data_ptr(), _ptr(block), _ptr(gate),
          _ptr(post_weight), _ptr(pre_weight), _ptr(out), _ptr(normed))
    return BlockNorm(given if out is None else out, normed)


def block_norm_backward(residual_out, block=None, *, pre_weight=None, post_weight=None, gate=None,
                        rows_per_gate=None, residual_scale=1.0, eps=1e-6, d_residual_out=None,
                        d_normed=None) -> BlockNormGrad:
    """The gradient of :func:`block_norm` at the residual it returned and the block it was given.

    Takes the gradients of residual_out and normed (either may be None) and returns those of
    residual, block, the weights and the gate (None where the forward had none); the sums
    over rows are float32.
    """
    residual_out, block, pre_weight, post_weight, gate, device, args = _block_norm_args(
        residual_out, block, pre_weight, post_weight, gate, rows_per_gate, residual_scale, eps)
    shape, dtype = residual_out.shape, residual_out.dtype
    if d_residual_out is not None:
        d_residual_out = _like(d_residual_out, device, dtype, shape, "d_residual_out")
    if d_normed is not None:
        d_normed = _like(d_normed, device, dtype, shape, "d_normed")
        if pre_weight is None:
            raise ValueError("d_normed needs pre_weight")
    g = BlockNormGrad(_empty_like(residual_out), None if block is None else _empty_like(block),
                      None if pre_weight is None else _empty_like(pre_weight),
                      None if post_weight is None else _empty_like(post_weight),
                      None if gate is None else _empty_like(gate, dtype=_F32))
    _, desc, need = _norm_desc(*args)
    ws = residual_out.new_empty(max(need, 1), dtype=torch.uint8)
    _call("bconv_block_norm_backward", device, desc, residual_out.data_ptr(), _ptr(block), _ptr(gate),
          _ptr(post_weight), _ptr(pre_weight), _ptr(d_residual_out), _ptr(d_normed), g.d_residual.data_ptr(),
          _ptr(g.d_block), _ptr(g.d_pre_weight), _ptr(g.d_post_weight), _ptr(g.d_gate), ws.data_ptr())
    return g


class TokenLogprobs(NamedTuple):
    logprob: torch.Tensor | None
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logprob: torch.Tensor | None
    top_index: torch.Tensor | None


def _token_desc(rows, stride, vocab, dtype, top, temperature):
    """The C descriptor by reference (kept alive by the first item)."""
    return _token_desc_of(rows, stride, vocab, dtype, operator.index(top), _number(temperature, "temperature"))


@functools.lru_cache(maxsize=256)  # (of plain numbers, as above)
def _token_desc_of(rows, stride, vocab, dtype, top, temperature):
    desc = nat.bconv_token_desc_t(rows, stride, vocab, _DTYPES[dtype], top, temperature)
    return desc, ctypes.byref(desc)


def _logits(logits):
    _activation(logits, "logits")
    if logits.dim() < 1 or logits.shape[-1] == 0:
        raise ValueError("logits: expected [..., vocab]")
    return _rows(logits)


def token_logprobs(logits, tokens=None, *, top=0, temperature=1.0) -> TokenLogprobs:
    """Log probabilities of given tokens, entropy, log-sum-exp and the top alternatives of logits / temperature.

    logits [..., vocab]; tokens int64 [...] (a negative one: the row has no token, its logprob is 0;
    one outside the vocabulary: NaN).  Returns float32 [...] (``top_logprob`` float32 and ``top_index``
    int32 [..., top], in descending order of the logits, equal ones by ascending index).
    """
    x, rows, stride = _logits(logits)
    lead, device = logits.shape[:-1], x.get_device()
    if tokens is not None:
        tokens = _like(tokens, device, torch.int64, lead, "tokens")
    desc = _token_desc(rows, stride, x.shape[-1], x.dtype, top, temperature)[1]
    # (one allocation for the statistics of a row)
    if tokens is not None:
        logprob, entropy, lse = x.new_empty((3,) + lead, dtype=_F32).unbind(0)
    else:
        logprob, (entropy, lse) = None, x.new_empty((2,) + lead, dtype=_F32).unbind(0)
    top_logprob = top_index = None
    if top > 0:
        top_logprob = x.new_empty(lead + (top,), dtype=_F32)
        top_index = x.new_empty(lead + (top,), dtype=torch.int32)
    _call("bconv_token_logprobs_forward", device, desc, x.data_ptr(), _ptr(tokens), _ptr(logprob), entropy.data_ptr(),
          lse.data_ptr(), _ptr(top_logprob), _ptr(top_index))
    return TokenLogprobs(logprob, entropy, lse, top_logprob, top_index)


def token_logprobs_backward(logits, tokens, lse, entropy, *, d_logprob=None, d_entropy=None, temperature=1.0):
    """The gradient of the logits from those of logprob and entropy (either may be None).

    lse and entropy are what :func:`token_logprobs` returned for these logits; the result has
    the logits' dtype.  entropy may be None without d_entropy, tokens without d_logprob.
    """
    x, rows, stride = _logits(logits)
    lead, device, vocab = logits.shape[:-1], x.get_device(), x.shape[-1]
    if lse is None or (d_logprob is not None and tokens is None) or (d_entropy is not None and entropy is None):
        raise ValueError("lse is needed, tokens with d_logprob, entropy with d_entropy")
    if tokens is not None:
        tokens = _like(tokens, device, torch.int64, lead, "tokens")
    lse = _like(lse, device, _F32, lead, "lse")
    if entropy is not None:
        entropy = _like(entropy, device, _F32, lead, "entropy")
    if d_logprob is not None:
        d_logprob = _like(d_logprob, device, _F32, lead, "d_logprob")
    if d_entropy is not None:
        d_entropy = _like(d_entropy, device, _F32, lead, "d_entropy")
    out = x.new_empty(logits.shape)
    _call("bconv_token_logprobs_backward", device, _token_desc(rows, stride, vocab, x.dtype, 0, temperature)[1],
          x.data_ptr(), _ptr(tokens), lse.data_ptr(), _ptr(entropy), _ptr(d_logprob), _ptr(d_entropy), out.data_ptr(),
          vocab)
    return out
