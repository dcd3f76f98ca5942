"""What a layer computes around its recurrence, on CUDA tensors.

  conv, conv_step    short causal convolution with SiLU, the L2 norm of the
                     query and key heads, and the carried inputs of every slot
  ssm, ssm_step      selective state space scan over prompts, and one token
  gated_norm         norm and gate of every head's output
  add_norm           residual sum and the norm before the next block

Marshalling of the dl_conv, dl_ssm, dl_ssm_step, dl_gated_norm and dl_add_norm
calls (include/deltalog.h says what each computes); every step runs in the
library's kernels, on torch's current stream.  Calls are asynchronous and can
be captured into a CUDA graph; outputs and workspaces come from torch's
allocator.  Inference only: a tensor that asks for a gradient is refused.

Tokens of ``n`` rows (sequences) are laid out
  token-major  [T, n, ...]: with ``lengths``, row i has its first lengths[i]
               tokens (outputs past them are not written);
  packed       [total, ...] with ``lengths``: the rows one after the other;
  one a row    [n, ...] in the *_step calls.
Strides between tokens and rows are free; what belongs to one token is
contiguous.  ``slots``, ``lengths`` and ``fresh`` live on the host (lists or
numpy arrays; int32 arrays are used as they are).  ``state`` is a pool with one
entry a slot; row i reads and updates entry slots[i].  ``fresh`` (one flag, or
one for each row) starts rows from an empty state.
"""
import ctypes
import struct
import threading

import numpy as np
import torch

from . import deltalog as _dl

_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_ACT = {None: 0, "none": 0, "silu": 1, "sigmoid": 2}
_KIND = {"rms": 0, "layer": 1}
_ERR = 256
_local = threading.local()

# The C structs, every member eight bytes (see the header for their order).
_CONV = struct.Struct("=8q8qd3q3q12q4q")
_SSM = struct.Struct("=8q7q15q5qq")
_GATED = struct.Struct("=9qd5q3q")
_ADD = struct.Struct("=6q2d8q4q")


def _signatures(lib):
    for name in ("dl_conv", "dl_ssm", "dl_ssm_step", "dl_gated_norm", "dl_add_norm"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.c_char_p, ctypes.c_void_p, ctypes.c_char_p, ctypes.c_int32]
        fn.restype = ctypes.c_int32
    lib.dl_mixer_sync.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.c_char_p, ctypes.c_int32]
    lib.dl_mixer_sync.restype = ctypes.c_int32
    lib.dl_ssm_workspace.argtypes = [ctypes.c_char_p]
    lib.dl_ssm_workspace.restype = ctypes.c_int64
    return lib


_lib = _signatures(_dl.library())


def _call(fn, args, device):
    err = getattr(_local, "err", None)
    if err is None:
        err = _local.err = ctypes.create_string_buffer(_ERR)
    rc = fn(args, torch.cuda.current_stream(device).cuda_stream, err, _ERR)
    if rc:
        raise _dl.DeltaLogError(rc, err.value.decode())


def _cuda(name, t, dtype, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, x on %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise ValueError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError("%s requires a gradient: these operators have no backward" % name)


def _x(t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    if t.dtype not in _DTYPE:
        raise ValueError("x: %s is not supported" % t.dtype)
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError("x requires a gradient: these operators have no backward")
    return t.device


def _dense(name, t, inner):
    """The last `inner` dimensions are contiguous."""
    want = 1
    for size, stride in zip(t.shape[:-inner - 1:-1], t.stride()[:-inner - 1:-1]):
        if size != 1 and stride != want:
            raise ValueError("%s: the last %d dimension(s) must be contiguous" % (name, inner))
        want *= size


def _vector(name, t, shape, dtypes, device):
    """A dense parameter; returns its address."""
    if t is None:
        return 0
    _cuda(name, t, t.dtype if t.dtype in dtypes else dtypes[0], device)
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError("%s: expected contiguous %s, got %s" % (name, shape, tuple(t.shape)))
    return t.data_ptr()


def _strides(t, lead):
    """(data, stride between tokens, stride between rows)"""
    if lead == 2:
        return t.data_ptr(), t.stride(0), t.stride(1)
    return t.data_ptr(), t.stride(0), 0


def _host(a, dtype, n, name):
    a = np.ascontiguousarray(a, dtype=dtype)
    if a.shape != (n,):
        raise ValueError("%s: expected %d entries, got %s" % (name, n, a.shape))
    return a


def sync(device=None):
    """Wait for the current stream and report a kernel's error since the last call."""
    err = ctypes.create_string_buffer(_ERR)
    rc = _lib.dl_mixer_sync(torch.cuda.current_stream(device).cuda_stream, None, err, _ERR)
    if rc:
        raise _dl.DeltaLogError(rc, err.value.decode())


class _Rows:
    """The dl_tokens of a call: checks the lists against the tensors' layout."""
    __slots__ = ("lead", "keep", "fields")

    def __init__(self, lead_shape, step, slots, lengths, fresh, state, device, state_shape, state_dtype):
        self.keep = []
        packed = 0
        if step:
            n, T, self.lead = lead_shape[0], 1, 1
        elif len(lead_shape) == 2:
            (T, n), self.lead = lead_shape, 2
        else:
            if lengths is None:
                raise ValueError("packed tokens need lengths")
            packed, self.lead = 1, 1
            lengths = np.ascontiguousarray(lengths, dtype=np.int32).reshape(-1)
            n, T = lengths.size, int(lengths.max()) if lengths.size else 0
            if int(lengths.sum(dtype=np.int64)) != lead_shape[0]:
                raise ValueError("lengths add up to %d, x has %d tokens" % (int(lengths.sum(dtype=np.int64)), lead_shape[0]))
        num_slots = 0
        if state is not None:
            _cuda("state", state, state_dtype, device)
            if tuple(state.shape[1:]) != state_shape or not state.is_contiguous():
                raise ValueError("state: expected contiguous [slots, %s], got %s"
                                 % (", ".join(map(str, state_shape)), tuple(state.shape)))
            if slots is None:
                raise ValueError("a state pool needs slots")
            num_slots = state.shape[0]
            slots = _host(slots, np.int32, n, "slots")
        elif slots is not None:
            raise ValueError("slots need a state pool")
        ptrs = [0, 0, 0]
        if slots is not None:
            ptrs[0] = slots.__array_interface__["data"][0]
        if lengths is not None:
            lengths = _host(lengths, np.int32, n, "lengths")
            ptrs[1] = lengths.__array_interface__["data"][0]
        if fresh is True or fresh is False:
            fresh_all = int(fresh)
        else:
            fresh_all = 0
            fresh = _host(fresh, np.uint8, n, "fresh")
            ptrs[2] = fresh.__array_interface__["data"][0]
        self.keep = (slots, lengths, fresh)       # alive until the call has read them
        self.fields = (ptrs[0], ptrs[1], ptrs[2], fresh_all, n, T, packed, num_slots)

    def of(self, t, step):
        """A tensor's (data, stride_t, stride_n)."""
        if step:
            return t.data_ptr(), 0, t.stride(0)
        return _strides(t, self.lead)


def _conv(x, weight, bias, slots, state, lengths, fresh, activation, l2_channels, head_dim, eps, split, out, step):
    dev = _x(x)
    if x.dim() not in ((2,) if step else (2, 3)):
        raise ValueError("x: expected %s, got %s" % ("[n, C]" if step else "[T, n, C] or [total, C]", tuple(x.shape)))
    _dense("x", x, 1)
    dt, lead = x.dtype, tuple(x.shape[:-1])
    C, W = x.shape[-1], weight.shape[-1]
    rows = _Rows(lead, step, slots, lengths, fresh, state, dev, (W - 1, C), dt)
    wp = _vector("weight", weight, (C, W), (dt, torch.float32), dev)
    bp = _vector("bias", bias, (C,), (weight.dtype,), dev)
    parts = (C,) if split is None else tuple(split)
    if out is None:
        outs = [torch.empty(lead + (c,), dtype=dt, device=dev) for c in parts]
    else:
        outs = [out] if split is None else list(out)
        if len(outs) != len(parts):
            raise ValueError("out: expected %d tensors" % len(parts))
        for t, c in zip(outs, parts):
            _cuda("out", t, dt, dev)
            if tuple(t.shape) != lead + (c,):
                raise ValueError("out: expected %s, got %s" % (lead + (c,), tuple(t.shape)))
            _dense("out", t, 1)
    if not 1 <= len(parts) <= 4:
        raise ValueError("split: 1 to 4 ranges")
    views, pad = [], 4 - len(parts)
    for t in outs:
        views += rows.of(t, step)
    _call(_lib.dl_conv, _CONV.pack(*rows.fields, _DTYPE[dt], int(weight.dtype == torch.float32), C, W,
                                   _ACT[activation], l2_channels, head_dim, len(parts), eps, *rows.of(x, step),
                                   wp, bp, 0 if state is None else state.data_ptr(),
                                   *views, *([0] * (3 * pad)), *parts, *([0] * pad)), dev)
    return outs[0] if split is None else tuple(outs)


def conv(x, weight, bias=None, *, slots=None, state=None, lengths=None, fresh=False, activation="silu",
         l2_channels=0, head_dim=0, eps=1e-6, split=None, out=None):
    """Causal convolution of x [T, n, C] (or packed [total, C]) over time.

    weight [C, W] (W = 2, 3, 4; the last tap is the current token) and bias [C]
    are of x's type or fp32; state [num_slots, W - 1, C] is of x's type and
    holds every slot's last inputs, oldest first.  The first ``l2_channels``
    channels are heads of ``head_dim``, each divided by its L2 norm (eps inside
    the root).  ``split`` gives the widths of consecutive channel ranges that
    come back as tensors of their own, for example q, k and v."""
    return _conv(x, weight, bias, slots, state, lengths, fresh, activation, l2_channels, head_dim, eps, split,
                 out, False)


def conv_step(x, weight, bias=None, *, slots, state, activation="silu", l2_channels=0, head_dim=0, eps=1e-6,
              split=None, out=None):
    """``conv`` of one token a row: x [n, C]."""
    return _conv(x, weight, bias, slots, state, None, False, activation, l2_channels, head_dim, eps, split,
                 out, True)


def _ssm(fn, x, dt, A, B, C, D, dt_bias, dt_softplus, slots, state, lengths, fresh, out, step):
    dev = _x(x)
    lead_dims = x.dim() - 2
    if lead_dims not in ((1,) if step else (1, 2)):
        raise ValueError("x: expected %s, got %s"
                         % ("[n, H, P]" if step else "[T, n, H, P] or [total, H, P]", tuple(x.shape)))
    lead, (H, P) = tuple(x.shape[:-2]), x.shape[-2:]
    G, N = B.shape[-2:]
    for name, t, shape in (("dt", dt, (H,)), ("B", B, (G, N)), ("C", C, (G, N))):
        _cuda(name, t, torch.float32 if name == "dt" and t.dtype == torch.float32 else x.dtype, dev)
        if tuple(t.shape) != lead + shape:
            raise ValueError("%s: expected %s, got %s" % (name, lead + shape, tuple(t.shape)))
        _dense(name, t, len(shape))
    _dense("x", x, 2)
    rows = _Rows(lead, step, slots, lengths, fresh, state, dev, (H, P, N), torch.float32)
    f32 = (torch.float32,)
    if out is None:
        out = torch.empty(lead + (H, P), dtype=x.dtype, device=dev)
    else:
        _cuda("out", out, x.dtype, dev)
        if out.shape != x.shape:
            raise ValueError("out: expected %s, got %s" % (tuple(x.shape), tuple(out.shape)))
        _dense("out", out, 2)
    head = rows.fields + (_DTYPE[x.dtype], int(dt.dtype == torch.float32), int(dt_softplus), H, G, P, N,
                          *rows.of(x, step), *rows.of(dt, step), *rows.of(B, step), *rows.of(C, step),
                          *rows.of(out, step), _vector("A", A, (H,), f32, dev), _vector("D", D, (H,), f32, dev),
                          _vector("dt_bias", dt_bias, (H,), f32, dev), 0 if state is None else state.data_ptr())
    if A is None:
        raise TypeError("A must be a CUDA tensor")
    workspace, size = None, 0
    if not step:
        size = _lib.dl_ssm_workspace(_SSM.pack(*head, 0, 0))
        if size > 0:
            workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    _call(fn, _SSM.pack(*head, 0 if workspace is None else workspace.data_ptr(), max(size, 0)), dev)
    return out


def ssm(x, dt, A, B, C, D=None, *, dt_bias=None, dt_softplus=True, slots=None, state=None, lengths=None,
        fresh=False, out=None):
    """State space scan of x [T, n, H, P] (or packed [total, H, P]); returns y like x.

    dt [..., H] (x's type or fp32) is the step size before its bias and
    softplus, A [H] the decay rates (negative), B and C [..., G, N] the input
    and output maps shared by H / G consecutive heads, D [H] the skip.
    A, D and dt_bias are fp32.  state [num_slots, H, P, N] fp32."""
    return _ssm(_lib.dl_ssm, x, dt, A, B, C, D, dt_bias, dt_softplus, slots, state, lengths, fresh, out, False)


def ssm_step(x, dt, A, B, C, D=None, *, dt_bias=None, dt_softplus=True, slots, state, out=None):
    """``ssm`` of one token a row: x [n, H, P], dt [n, H], B and C [n, G, N]."""
    return _ssm(_lib.dl_ssm_step, x, dt, A, B, C, D, dt_bias, dt_softplus, slots, state, None, False, out, True)


def _rows_of(name, t, shape, dtype, dev, inner):
    _cuda(name, t, dtype, dev)
    if tuple(t.shape) != shape:
        raise ValueError("%s: expected %s, got %s" % (name, shape, tuple(t.shape)))
    _dense(name, t, inner)
    return t.data_ptr()


def gated_norm(x, weight, gate=None, *, bias=None, kind="rms", activation="silu", gate_first=False, eps=1e-5,
               out=None):
    """Norm and gate of every head of x [rows, H, d]: (norm(x) weight + bias) act(gate),
    or norm(x act(gate)) weight + bias with ``gate_first``.

    weight and bias are [d] or [H, d], of x's type or fp32; the gate has x's
    shape and type.  ``out`` may be x or the gate."""
    dev = _x(x)
    if x.dim() != 3:
        raise ValueError("x: expected [rows, H, d], got %s" % (tuple(x.shape),))
    shape, dt = tuple(x.shape), x.dtype
    _dense("x", x, 2)
    wshape = shape[1:] if weight.dim() == 2 else shape[2:]
    wp = _vector("weight", weight, wshape, (dt, torch.float32), dev)
    bp = _vector("bias", bias, wshape, (weight.dtype,), dev)
    gp = 0 if gate is None else _rows_of("gate", gate, shape, dt, dev, 2)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=dev)
    op = _rows_of("out", out, shape, dt, dev, 2)
    _call(_lib.dl_gated_norm, _GATED.pack(_DTYPE[dt], int(weight.dtype == torch.float32), int(weight.dim() == 2),
                                          *shape, _KIND[kind], _ACT[activation], int(gate_first), eps, x.data_ptr(),
                                          gp, wp, bp, op, x.stride(0), 0 if gate is None else gate.stride(0),
                                          out.stride(0)), dev)
    return out


def add_norm(x, residual, weight, *, bias=None, scale=None, alpha=1.0, post_weight=None, kind="rms", eps=1e-5,
             out=None, out_residual=None):
    """h = residual + alpha * scale * x' and y = norm(h) weight + bias; returns (y, h).

    x [rows, D] is the block's output, x' = norm(x) post_weight where that is
    given and x otherwise; residual [rows, D] (x's type or fp32; None: zero)
    is the stream h continues, in its type.  weight, bias, scale and
    post_weight are [D], all of x's type or all fp32.  ``out`` may be x,
    ``out_residual`` the residual."""
    dev = _x(x)
    if x.dim() != 2:
        raise ValueError("x: expected [rows, D], got %s" % (tuple(x.shape),))
    shape, dt = tuple(x.shape), x.dtype
    _dense("x", x, 1)
    wp = _vector("weight", weight, shape[1:], (dt, torch.float32), dev)
    more = [_vector(name, t, shape[1:], (weight.dtype,), dev)
            for name, t in (("bias", bias), ("scale", scale), ("post_weight", post_weight))]
    rt = dt if residual is None and out_residual is None else (out_residual if residual is None else residual).dtype
    if rt not in (dt, torch.float32):
        raise ValueError("residual: expected %s or fp32, got %s" % (dt, rt))
    rp = 0 if residual is None else _rows_of("residual", residual, shape, rt, dev, 1)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=dev)
    if out_residual is None:
        out_residual = torch.empty(shape, dtype=rt, device=dev)
    op = _rows_of("out", out, shape, dt, dev, 1)
    hp = _rows_of("out_residual", out_residual, shape, rt, dev, 1)
    _call(_lib.dl_add_norm, _ADD.pack(_DTYPE[dt], int(rt == torch.float32), int(weight.dtype == torch.float32),
                                      *shape, _KIND[kind], eps, alpha, x.data_ptr(), rp, wp, *more, op, hp,
                                      x.stride(0), 0 if residual is None else residual.stride(0), out.stride(0),
                                      out_residual.stride(0)), dev)
    return out, out_residual
