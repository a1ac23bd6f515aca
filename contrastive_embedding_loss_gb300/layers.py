"""The operators around the loss: Python binding of ``include/uf_layers.h``.

RMS norm with the residual's addition, linear projections and the gated feed-forward block,
forward and backward, and the AdamW step.  A native module (``csrc/layers_binding.cpp``) checks
the tensors, takes outputs and scratch from torch's allocator (device memory only) and makes one
C call on the current stream (or ``stream``, a ``torch.cuda.Stream``); what is wrong raises
``UfError``, TypeError or ValueError, and there is no fallback.

The functions return dicts, as ``binding.contrastive_fwd_bwd`` does.  Matrices are 2-D CUDA
tensors whose rows may be strided (a stride of 1 within a row).  ``workspace`` may be a
preallocated uint8 CUDA tensor of at least the C entry point's workspace size, ``device_status`` an
int32 one that a kernel sets to ``binding.UF_DEVICE_TIMEOUT`` if a bounded wait in it ran out.

A call on another ``stream`` than the current one does not wait for the current one: the caller
orders the streams, as for any torch work on another stream.  Inputs may be freed right after the
call; its outputs belong to ``stream`` (``Tensor.record_stream`` before they are freed while a
third stream uses them).

Nothing here is recorded by autograd: outputs have no gradient function, whatever the inputs
require; the backward functions are called by the program.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import binding
from . import build as _build

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
STATE_BLOCK = 256  # elements that share a scale in AdamW's 8-bit states

_P, _I64, _I32, _F32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ENTRY_POINTS = {
    "uf_rmsnorm_fwd": (_I32, [_P, _I64, _I32, _P, _I64, _I32, _P, _I32, _I64, _I32, _F32, _P, _I64, _I32, _P, _P, _I64, _P,
                              _P]),
    "uf_rmsnorm_bwd_workspace": (_SZ, [_I64, _I32]),
    "uf_rmsnorm_bwd": (_I32, [_P, _I64, _I32, _P, _I64, _I32, _P, _I32, _P, _P, _I64, _I64, _I32, _P, _I64, _P, _P, _SZ, _P]),
    "uf_linear_fwd_workspace": (_SZ, [_I64, _I32, _I32, _I32]),
    "uf_linear_fwd": (_I32, [_P, _I64, _P, _I64, _I32, _P, _P, _P, _I32, _P, _I64, _I32, _I64, _I32, _I32, _P, _I64, _P, _I64,
                             _P, _SZ, _P, _P]),
    "uf_linear_bwd_workspace": (_SZ, [_I64, _I32, _I32]),
    "uf_linear_bwd": (_I32, [_P, _I64, _I32, _P, _I64, _P, _I64, _P, _I64, _I32, _I64, _I32, _I32, _P, _I64, _P, _I64, _P, _P,
                             _SZ, _P, _P]),
    "uf_gated_fwd_workspace": (_SZ, [_I64, _I32, _I32]),
    "uf_gated_fwd": (_I32, [_P, _I64, _P, _I64, _I32, _I64, _I32, _I32, _P, _I64, _P, _I64, _P, _SZ, _P, _P]),
    "uf_gated_bwd_workspace": (_SZ, [_I64, _I32, _I32]),
    "uf_gated_bwd": (_I32, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I32, _I64, _I32, _I32, _P, _I64, _P, _I64, _P, _SZ, _P,
                            _P]),
    "uf_adamw_step": (_I32, [_I32, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _F32, _P, ctypes.c_double,
                             ctypes.c_double, _F32, _F32, _I64, _P, ctypes.c_uint32, _P, _P]),
}
_lib = None


def _load() -> ctypes.CDLL:
    """The library with the entry points of uf_layers.h declared: raw calls, as in ``binding``."""
    global _lib
    if _lib is None:
        lib = binding.load()
        for name, (restype, argtypes) in _ENTRY_POINTS.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = restype, argtypes
        _lib = lib
    return _lib


def _load_native():
    path = _build.native_path()
    if not os.path.exists(path):
        raise ImportError(f"the native binding is not built for this torch ({path} is missing); "
                          "run `python -c 'import __graft_entry__ as g; g.build()'`")
    loader = importlib.machinery.ExtensionFileLoader("_layers_native", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_layers_native", loader))
    loader.exec_module(module)
    lib = _load()
    module.bind(binding.UfError, {name: ctypes.cast(getattr(lib, name), _P).value for name in _ENTRY_POINTS})
    return module


_native = _load_native()


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, not {act!r}")
    return ACTS[act]


def _sequence(tensors):
    """A list or tuple as it is, other iterables (a generator, read once) as a list."""
    return tensors if tensors is None or isinstance(tensors, (list, tuple)) else list(tensors)


def _asked(need, names):
    if any(k not in names for k in need):
        raise ValueError(f"need names {', '.join(names[:-1])} or {names[-1]}")
    return [k in need for k in names]


# ---- RMS norm ----------------------------------------------------------------------------

def rmsnorm_fwd(x, weight, residual=None, eps=1e-6, out="bf16", stream=None):
    """RMS norm of ``s = x + residual`` (or of x) times ``weight``, statistics in fp32.

    x: rows x width, bf16 (or fp32 without a residual); residual: bf16 or fp32 (the residual
    stream's type); weight: [width] fp32 or bf16.  Returns ``y`` (bf16, or with ``out="e4m3"``
    float8_e4m3fn with the fp32 row scales ``scale``), ``rstd`` [rows] and, with a residual,
    ``stream``: s in the residual's type."""
    if out not in ("bf16", "e4m3"):
        raise ValueError(f"out must be 'bf16' or 'e4m3', not {out!r}")
    return _native.rmsnorm_fwd(x, weight, residual, eps, out == "e4m3", stream)


def rmsnorm_bwd(dy, s, weight, rstd, d_stream=None, weight_grad=True, workspace=None, stream=None):
    """Backward of ``rmsnorm_fwd``: ``dx``, the gradient of s (hence of x and of the residual) in
    s's type, and ``dweight`` (fp32).  s: the forward's ``stream`` (its x, without a residual);
    d_stream: the gradient that reaches s past the norm, in s's type."""
    return _native.rmsnorm_bwd(dy, s, weight, rstd, d_stream, weight_grad, workspace, stream)


# ---- linear projection -------------------------------------------------------------------

def linear_fwd(x, W, bias=None, act="none", residual=None, x_scale=None, w_scale=None, keep_pre=False, workspace=None,
               device_status=None, stream=None):
    """``y = act(x W^T + bias) + residual`` (bf16) of x (rows x inner) and W (outer x inner), both
    bf16, or both float8_e4m3fn with fp32 scales ``x_scale`` [rows] and ``w_scale`` [outer].
    ``keep_pre``: also return ``pre``, the activation's input in bf16, for the backward."""
    return _native.linear_fwd(x, W, bias, _act(act), residual, x_scale, w_scale, keep_pre, workspace, device_status, stream)


def linear_bwd(dy, x, W, pre=None, act="none", need=("dx", "dW", "dbias"), workspace=None, device_status=None, stream=None):
    """Backward of ``linear_fwd`` (bf16 operands): the asked ones of ``dx`` and ``dW`` (bf16) and
    ``dbias`` (fp32).  dy: rows x outer, bf16 or fp32; pre: the forward's ``pre``, needed with an
    activation.  The residual's gradient is dy."""
    return _native.linear_bwd(dy, x, W, pre, _act(act), *_asked(need, ("dx", "dW", "dbias")), workspace, device_status, stream)


# ---- gated feed-forward ------------------------------------------------------------------

def gated_fwd(x, W, act="silu", keep_pre=False, workspace=None, device_status=None, stream=None):
    """Gated feed-forward block: ``h = act(g) * u`` with ``[g | u] = x W^T`` (bf16).  W holds the
    gate's ``outer`` rows, then the up projection's.  ``keep_pre``: also return ``pre`` = [g | u]."""
    return _native.gated_fwd(x, W, _act(act), keep_pre, workspace, device_status, stream)


def gated_bwd(dh, x, W, pre, act="silu", need=("dx", "dW"), workspace=None, device_status=None, stream=None):
    """Backward of ``gated_fwd``: ``dx`` and ``dW`` (bf16).  dh: rows x outer bf16; pre: the
    forward's ``pre``."""
    return _native.gated_bwd(dh, x, W, pre, _act(act), *_asked(need, ("dx", "dW")), workspace, device_status, stream)


# ---- AdamW -------------------------------------------------------------------------------

class AdamW:
    """AdamW over a list of parameters, one kernel launch a step (per 256 tensors), in place.

    params: contiguous CUDA tensors, all fp32 or all bf16 (bf16: stochastic rounding).  m, v: the
    states in the same order, fp32, or float8_e4m3fn codes of m and sqrt(v) with fp32 scales
    ``m_scale`` / ``v_scale`` for blocks of 256 elements; ``new_states`` makes them.  copies:
    bf16 tensors that receive the new fp32 parameters (the operands of the next forward).
    step: steps already taken.

    The lists are the attributes ``params``, ``m``, ``v``, ``m_scale``, ``v_scale`` and ``copies``.
    Every step reads and checks them anew, so entries may be replaced between steps (a loaded
    checkpoint) and tensors may get other storage (``p.data = ...``, a state moved away and back);
    a captured step keeps the addresses that it was captured with."""

    def __init__(self, params, m, v, m_scale=None, v_scale=None, copies=None, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=0.01, step=0):
        lists = tuple(_sequence(t) for t in (params, m, v, m_scale, v_scale, copies))
        self.params, self.m, self.v, self.m_scale, self.v_scale, self.copies = lists
        self.betas, self.eps, self.weight_decay, self.t = betas, eps, weight_decay, step
        _native.adamw_check(*lists)

    @staticmethod
    def new_states(params, bits=32):
        """Zero states for ``params``: (m, v) of fp32, or (m, v, m_scale, v_scale) in 8 bits."""
        if bits not in (32, 8):
            raise ValueError("states have 32 or 8 bits")
        if bits == 32:
            return tuple([torch.zeros(p.shape, dtype=torch.float32, device=p.device) for p in params] for _ in range(2))
        codes = tuple([torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(torch.float8_e4m3fn) for p in params]
                      for _ in range(2))
        return codes + tuple([torch.zeros(-(-p.numel() // STATE_BLOCK), dtype=torch.float32, device=p.device)
                              for p in params] for _ in range(2))

    def step(self, grads, lr, seed=None, grad_scale=None, step_dev=None, stream=None):
        """One step.  grads: contiguous CUDA tensors, all fp32 or all bf16.  lr: a float, or a
        one-element fp32 CUDA tensor that the kernel reads.  seed: of the stochastic rounding (default:
        the step's number).  grad_scale: a one-element fp32 CUDA tensor that multiplies the gradients.
        step_dev: a one-element int64 CUDA tensor with the step's number, read by the kernel (and
        added to the seed), for captured graphs."""
        t = self.t + 1
        if seed is None:
            seed = 0 if step_dev is not None else t
        _native.adamw_step(self.params, self.m, self.v, self.m_scale, self.v_scale, self.copies, _sequence(grads), lr,
                           *self.betas, self.eps, self.weight_decay, t, step_dev, seed & 0xFFFFFFFF, grad_scale, stream)
        self.t = t
