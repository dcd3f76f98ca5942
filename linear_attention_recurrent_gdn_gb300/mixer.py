"""What a layer computes around its recurrence, on CUDA tensors.

  conv, conv_step    short causal convolution with SiLU, the L2 norm of the
                     query and key heads, and the carried inputs of every slot
  ssm, ssm_step      selective state space scan over prompts, and one token
  gated_norm         norm and gate of every head's output
  add_norm           residual sum and the norm before the next block

Marshalling of the dl_conv, dl_ssm, dl_ssm_step, dl_gated_norm and dl_add_norm
calls (include/deltalog.h says what each computes); every step runs in the
library's kernels, on the current stream of the tensors' device.  Calls are
asynchronous and can be captured into a CUDA graph; outputs and workspaces come
from torch's allocator.  Inference only: a tensor that asks for a gradient, or
carries a forward-mode tangent, is refused.

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
from torch.autograd import forward_ad as _fwd

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
        fn.argtypes = [ctypes.c_char_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32]
        fn.restype = ctypes.c_int32
    lib.dl_mixer_sync.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.c_char_p, ctypes.c_int32]
    lib.dl_mixer_sync.restype = ctypes.c_int32
    lib.dl_ssm_workspace.argtypes = [ctypes.c_char_p]
    lib.dl_ssm_workspace.restype = ctypes.c_int64
    return lib


_lib = _signatures(_dl.library())
_raw_stream = torch._C._cuda_getCurrentRawStream     # the current stream's handle, without an object around it
_device = torch._C._cuda_getDevice                   # the current device's number
_F32 = torch.float32


def _on(dev, fn, *args):
    """fn(*args) with ``dev`` as the current device: the library's calls launch on that one, whatever their stream."""
    if dev == _device():
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _call(fn, args, dev):
    try:
        err, at = _local.err
    except AttributeError:
        err = ctypes.create_string_buffer(_ERR)
        err, at = _local.err = err, ctypes.addressof(err)
    if dev == _device():
        rc = fn(args, _raw_stream(dev), at, _ERR)
    else:
        rc = _on(dev, fn, args, _raw_stream(dev), at, _ERR)
    if rc:
        raise _dl.DeltaLogError(rc, err.value.decode())


def sync(device=None):
    """Wait for the device's current stream and report an error of its kernels since the last call."""
    stream = torch.cuda.current_stream(device)
    err = ctypes.create_string_buffer(_ERR)
    rc = _on(stream.device_index, _lib.dl_mixer_sync, stream.cuda_stream, None, err, _ERR)
    if rc:
        raise _dl.DeltaLogError(rc, err.value.decode())


# The checks below are written for few Python steps: in a decode loop they are
# the cost of a call.  A CPU tensor's device number is -1.

def _differentiated(t):
    """Whether the tensor asks for a gradient or, inside a forward-mode level, carries a tangent."""
    return t.requires_grad and torch.is_grad_enabled() or \
        _fwd._current_level >= 0 and _fwd.unpack_dual(t).tangent is not None


def _bad(name, t, dtype, dev):
    """Says what is wrong with a tensor that failed a check."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if _differentiated(t):
        raise ValueError("%s is being differentiated: these operators have no derivatives" % name)
    raise ValueError("%s: expected %s on device %s, got %s on %s" % (name, dtype, dev, t.dtype, t.device))


def _x(t):
    """The first tensor of a call; returns its device's number."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    if t.dtype not in _DTYPE:
        raise ValueError("x: %s is not supported" % t.dtype)
    if (t.requires_grad or _fwd._current_level >= 0) and _differentiated(t):
        _bad("x", t, t.dtype, t.get_device())
    return t.get_device()


def _check(name, t, shape, dtype, dev):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or \
            (t.requires_grad or _fwd._current_level >= 0) and _differentiated(t):
        _bad(name, t, dtype, dev)
    if t.shape != shape:
        raise ValueError("%s: expected %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _param(name, t, shape, dtype, dev):
    """A contiguous parameter; returns its address (0 for None)."""
    if t is None:
        return 0
    _check(name, t, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _dense(name, t, inner, stride):
    """The last `inner` dimensions are contiguous (dimensions of one entry have no stride)."""
    want = 1
    shape = t.shape
    for k in range(-1, -1 - inner, -1):
        if stride[k] != want and shape[k] != 1:
            raise ValueError("%s: the last %d dimension(s) must be contiguous" % (name, inner))
        want *= shape[k]


def _one_of(names, name, what):
    """The number of an activation or a norm."""
    try:
        return names[name]
    except (KeyError, TypeError):
        raise ValueError("%s: expected one of %s, got %r" % (what, ", ".join(map(repr, names)), name)) from None


def _tokens(name, t, shape, dtype, dev, inner, lead):
    """A per-token tensor: checks it and returns (data, stride between tokens, between rows)."""
    _check(name, t, shape, dtype, dev)
    stride = t.stride()
    if not t.is_contiguous():
        _dense(name, t, inner, stride)
    if lead == 0:                          # one token a row
        return t.data_ptr(), 0, stride[0]
    if lead == 1:                          # packed
        return t.data_ptr(), stride[0], 0
    return t.data_ptr(), stride[0], stride[1]


def _host(a, dtype, n, name):
    """A host list as an array and its address.  Whole numbers only, and none that `dtype` cannot hold."""
    if type(a) is not np.ndarray or a.dtype != dtype or not a.flags.c_contiguous:
        given = np.asarray(a)
        if given.dtype.kind not in "iub" and given.size:
            raise ValueError("%s: whole numbers wanted, got %s" % (name, given.dtype))
        a = np.ascontiguousarray(given, dtype=dtype)
        if (a != given).any():
            raise ValueError("%s: a number does not fit into %s" % (name, a.dtype))
    if a.shape != (n,):
        raise ValueError("%s: expected %d entries, got %s" % (name, n, a.shape))
    return a, a.__array_interface__["data"][0]


def _rows(lead_shape, step, slots, lengths, fresh, state, dev, state_shape, state_dtype):
    """The dl_tokens of a call, checked against the tensors' layout.  Returns
    its fields, the state's address, the layout (0: one token a row, 1: packed,
    2: token-major) and the arrays to keep until the call has read them."""
    packed, plen, pfresh = 0, 0, 0
    if step:
        n, T, lead = lead_shape[0], 1, 0
    elif len(lead_shape) == 2:
        (T, n), lead = lead_shape, 2
        if lengths is not None:
            lengths, plen = _host(lengths, np.int32, n, "lengths")
    else:
        if lengths is None:
            raise ValueError("packed tokens need lengths")
        packed, lead, n = 1, 1, len(lengths)
        lengths, plen = _host(lengths, np.int32, n, "lengths")
        T = int(lengths.max()) if n else 0
        if int(lengths.sum(dtype=np.int64)) != lead_shape[0]:
            raise ValueError("lengths add up to %d, x has %d tokens" % (lengths.sum(dtype=np.int64), lead_shape[0]))
    if state is None:
        if slots is not None:
            raise ValueError("slots need a state pool")
        pool = pslots = num_slots = 0
    else:
        num_slots = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() else 0
        pool = _param("state", state, (num_slots,) + state_shape, state_dtype, dev)
        if slots is None:
            raise ValueError("a state pool needs slots")
        slots, pslots = _host(slots, np.int32, n, "slots")
    if fresh is not True and fresh is not False:
        fresh, pfresh = _host(fresh, np.uint8, n, "fresh")
    return (pslots, plen, pfresh, fresh is True, n, T, packed, num_slots), pool, lead, (slots, lengths, fresh)


def _conv(x, weight, bias, slots, state, lengths, fresh, activation, l2_channels, head_dim, eps, split, out, step):
    dev, dt, shape = _x(x), x.dtype, x.shape
    if len(shape) != 2 and (step or len(shape) != 3):
        raise ValueError("x: expected %s, got %s" % ("[n, C]" if step else "[T, n, C] or [total, C]", tuple(shape)))
    lead_shape, C = shape[:-1], shape[-1]
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise TypeError("weight must be a CUDA tensor [C, W]")
    W, wt = weight.shape[1], _F32 if weight.dtype is _F32 else dt
    wp = _param("weight", weight, (C, W), wt, dev)
    bp = _param("bias", bias, (C,), wt, dev)
    fields, pool, lead, keep = _rows(lead_shape, step, slots, lengths, fresh, state, dev, (W - 1, C), dt)
    xv = _tokens("x", x, shape, dt, dev, 1, lead)
    parts = (C,) if split is None else tuple(split)
    if not 1 <= len(parts) <= 4:
        raise ValueError("split: 1 to 4 ranges")
    views = []
    if out is None:
        outs, place = [], x.device
        for c in parts:
            t = torch.empty(lead_shape + (c,), dtype=dt, device=place)
            outs.append(t)
            views += (t.data_ptr(), 0, c) if lead == 0 else (t.data_ptr(), c, 0) if lead == 1 else \
                (t.data_ptr(), c * shape[1], c)
    else:
        outs = [out] if split is None else list(out)
        if len(outs) != len(parts):
            raise ValueError("out: expected %d tensors" % len(parts))
        for t, c in zip(outs, parts):
            views += _tokens("out", t, lead_shape + (c,), dt, dev, 1, lead)
    pad = 4 - len(parts)
    act = _one_of(_ACT, activation, "activation")
    _call(_lib.dl_conv, _CONV.pack(*fields, _DTYPE[dt], wt is _F32, C, W, act, l2_channels, head_dim,
                                   len(parts), eps, *xv, wp, bp, pool, *views, *_ZEROS[:3 * pad], *parts,
                                   *_ZEROS[:pad]), dev)
    return outs[0] if split is None else tuple(outs)


_ZEROS = (0,) * 12


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
    dev, xt, shape = _x(x), x.dtype, x.shape
    if len(shape) != 3 and (step or len(shape) != 4):
        raise ValueError("x: expected %s, got %s"
                         % ("[n, H, P]" if step else "[T, n, H, P] or [total, H, P]", tuple(shape)))
    if A is None or not isinstance(B, torch.Tensor) or B.dim() != len(shape) or not isinstance(dt, torch.Tensor):
        raise TypeError("dt, A and B must be CUDA tensors, B with x's leading dimensions")
    lead_shape, H, P = shape[:-2], shape[-2], shape[-1]
    G, N = B.shape[-2:]
    fields, pool, lead, keep = _rows(lead_shape, step, slots, lengths, fresh, state, dev, (H, P, N), _F32)
    maps, dtt = lead_shape + (G, N), _F32 if dt.dtype is _F32 else xt
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    head = fields + (_DTYPE[xt], dtt is _F32, bool(dt_softplus), H, G, P, N) \
        + _tokens("x", x, shape, xt, dev, 2, lead) + _tokens("dt", dt, lead_shape + (H,), dtt, dev, 1, lead) \
        + _tokens("B", B, maps, xt, dev, 2, lead) + _tokens("C", C, maps, xt, dev, 2, lead) \
        + _tokens("out", out, shape, xt, dev, 2, lead) \
        + (_param("A", A, (H,), _F32, dev), _param("D", D, (H,), _F32, dev),
           _param("dt_bias", dt_bias, (H,), _F32, dev), pool)
    args = _SSM.pack(*head, 0, 0)
    if not step:
        size = _on(dev, _lib.dl_ssm_workspace, args)
        if size > 0:
            workspace = torch.empty(size, dtype=torch.uint8, device=x.device)
            args = _SSM.pack(*head, workspace.data_ptr(), size)
    _call(fn, args, dev)
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


def _matrix(name, t, shape, dtype, dev, inner):
    """A tensor of rows: checks it and returns its address and the stride between rows."""
    _check(name, t, shape, dtype, dev)
    stride = t.stride()
    if not t.is_contiguous():
        _dense(name, t, inner, stride)
    return t.data_ptr(), stride[0]


def gated_norm(x, weight, gate=None, *, bias=None, kind="rms", activation="silu", gate_first=False, eps=1e-5,
               out=None):
    """Norm and gate of every head of x [rows, H, d]: (norm(x) weight + bias) act(gate),
    or norm(x act(gate)) weight + bias with ``gate_first``.

    weight and bias are [d] or [H, d], of x's type or fp32; the gate has x's
    shape and type.  ``out`` may be x or the gate."""
    dev, dt, shape = _x(x), x.dtype, x.shape
    if len(shape) != 3:
        raise ValueError("x: expected [rows, H, d], got %s" % (tuple(shape),))
    if not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a CUDA tensor")
    heads, wt = weight.dim() == 2, _F32 if weight.dtype is _F32 else dt
    wshape = shape[1:] if heads else shape[2:]
    wp = _param("weight", weight, wshape, wt, dev)
    bp = _param("bias", bias, wshape, wt, dev)
    xp, xs = _matrix("x", x, shape, dt, dev, 2)
    gp, gs = (0, 0) if gate is None else _matrix("gate", gate, shape, dt, dev, 2)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        op, os = out.data_ptr(), shape[1] * shape[2]
    else:
        op, os = _matrix("out", out, shape, dt, dev, 2)
    act, kind = _one_of(_ACT, activation, "activation"), _one_of(_KIND, kind, "kind")
    _call(_lib.dl_gated_norm, _GATED.pack(_DTYPE[dt], wt is _F32, heads, *shape, kind, act, bool(gate_first), eps,
                                          xp, gp, wp, bp, op, xs, gs, os), dev)
    return out


def add_norm(x, residual, weight, *, bias=None, scale=None, alpha=1.0, post_weight=None, kind="rms", eps=1e-5,
             out=None, out_residual=None):
    """h = residual + alpha * scale * x' and y = norm(h) weight + bias; returns (y, h).

    x [rows, D] is the block's output, x' = norm(x) post_weight where that is
    given and x otherwise; residual [rows, D] (x's type or fp32; None: zero)
    is the stream h continues, in its type.  weight, bias, scale and
    post_weight are [D], all of x's type or all fp32.  ``out`` may be x,
    ``out_residual`` the residual."""
    dev, dt, shape = _x(x), x.dtype, x.shape
    if len(shape) != 2:
        raise ValueError("x: expected [rows, D], got %s" % (tuple(shape),))
    if not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a CUDA tensor")
    wt, wshape = _F32 if weight.dtype is _F32 else dt, shape[1:]
    wp = _param("weight", weight, wshape, wt, dev)
    bp = _param("bias", bias, wshape, wt, dev)
    sp = _param("scale", scale, wshape, wt, dev)
    pp = _param("post_weight", post_weight, wshape, wt, dev)
    stream = out_residual if residual is None else residual
    rt = _F32 if isinstance(stream, torch.Tensor) and stream.dtype is _F32 else dt
    xp, xs = _matrix("x", x, shape, dt, dev, 1)
    rp, rs = (0, 0) if residual is None else _matrix("residual", residual, shape, rt, dev, 1)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        op, os = out.data_ptr(), shape[1]
    else:
        op, os = _matrix("out", out, shape, dt, dev, 1)
    if out_residual is None:
        out_residual = torch.empty_like(x if rt is dt else residual, memory_format=torch.contiguous_format)
        hp, hs = out_residual.data_ptr(), shape[1]
    else:
        hp, hs = _matrix("out_residual", out_residual, shape, rt, dev, 1)
    _call(_lib.dl_add_norm, _ADD.pack(_DTYPE[dt], rt is _F32, wt is _F32, *shape, _one_of(_KIND, kind, "kind"), eps,
                                      alpha, xp, rp, wp, bp, sp, pp, op, hp, xs, rs, os, hs), dev)
    return out, out_residual
