"""Softmax attention beside the recurrent layers, on CUDA tensors.

  new_tables                an empty block table, its lengths and free pages
  extend, truncate          pages and places for new tokens; pages given back
  append                    the new tokens' keys and values into their pages
  attend, attend_step       attention of prompts (or later pieces of them), and
                            of one token a row, over the pages

Marshalling of the dl_pages_*, dl_kv_append and dl_attend* calls
(include/deltalog.h says what each computes); every step runs in the library's
kernels, on the current stream of the tensors' device.  Calls are asynchronous
and can be captured into a CUDA graph; outputs and workspaces come from torch's
allocator.  Inference only: a tensor that asks for a gradient, or carries a
forward-mode tangent, is refused.

Keys and values live in pools ``k_pages`` and ``v_pages`` [num_pages, G,
page_size, d] with any strides but a contiguous last dimension (a transposed
[num_pages, page_size, G, d] will do); page_size is a power of two from 16 to
256.  ``table`` [num_slots, max_pages], ``lengths`` [num_slots] and ``free``
[1 + num_pages] (how many pages are free, then a stack of them), ``slots``
[n <= 1024] and numbers of tokens [n] are int32 tensors on the device: a
captured step follows them from replay to replay.  One table serves the pools
of every layer.

What the host cannot see there is checked on the device: a call that meets a
slot, length, number of tokens or page out of range, or runs out of pages, does
not follow it, and ``sync`` raises.

Tokens of n rows are token-major [T, n, ...], packed [total, ...] one row after
the other, or one a row [n, ...].
"""
import ctypes
import struct

import torch

from . import deltalog as _dl
from .mixer import _ERR, _DTYPE, _bad, _call, _check, _device, _differentiated, _lib, _on, _tokens

# The C structs, every member eight bytes (see the header for their order).
_PAGES = struct.Struct("=9q8q")
_APPEND = struct.Struct("=7q6q8qq")
_ATTEND = struct.Struct("=13qd6q8q2q4q")          # and the workspace
_WORKSPACE = struct.Struct("=2q")
_NO_WORKSPACE = _WORKSPACE.pack(0, 0)
_I32 = torch.int32


def _signatures(lib):
    for name in ("dl_pages_extend", "dl_pages_truncate", "dl_kv_append", "dl_attend", "dl_attend_step"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.c_char_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32]
        fn.restype = ctypes.c_int32
    lib.dl_attend_sync.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.c_char_p, ctypes.c_int32]
    lib.dl_attend_sync.restype = ctypes.c_int32
    lib.dl_attend_workspace.argtypes = [ctypes.c_char_p]
    lib.dl_attend_workspace.restype = ctypes.c_int64


_signatures(_lib)


def sync(device=None):
    """Wait for the device's current stream and report an error of its attention kernels since the last call."""
    stream = torch.cuda.current_stream(device)
    err = ctypes.create_string_buffer(_ERR)
    rc = _on(stream.device_index, _lib.dl_attend_sync, stream.cuda_stream, None, err, _ERR)
    if rc:
        raise _dl.DeltaLogError(rc, err.value.decode())


def _ints(name, t, shape, dev):
    """A contiguous int32 tensor; returns its address."""
    _check(name, t, shape, _I32, dev)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _first(name, t, dim):
    """The first tensor of a call; returns its device's number."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dim() != dim:
        raise ValueError("%s: expected %d dimensions, got %s" % (name, dim, tuple(t.shape)))
    return t.get_device()


def _table(table, lengths, dev):
    """(address, stride, num_slots, max_pages, lengths' address)"""
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise TypeError("table must be a CUDA tensor [num_slots, max_pages]")
    shape = table.shape
    _check("table", table, shape, _I32, dev)
    stride = table.stride()
    if stride[1] != 1 and shape[1] != 1:
        raise ValueError("table: rows must be contiguous")
    return table.data_ptr(), stride[0], shape[0], shape[1], _ints("lengths", lengths, shape[:1], dev)


def new_tables(num_slots, max_pages, num_pages, device="cuda"):
    """(table, lengths, free) of num_slots empty slots of at most max_pages pages; all of num_pages pages are free."""
    free = torch.arange(num_pages, -1, -1, dtype=_I32, device=device)      # how many, then N - 1 ... 0
    return (torch.zeros(num_slots, max_pages, dtype=_I32, device=device),
            torch.zeros(num_slots, dtype=_I32, device=device), free)


def _pages(slots, tokens, table, lengths, free, dev):
    n = slots.shape[0]
    at, stride, num_slots, max_pages, lens = _table(table, lengths, dev)
    if not isinstance(free, torch.Tensor) or free.dim() != 1:
        raise TypeError("free must be a CUDA tensor [1 + num_pages]")
    head = (_ints("slots", slots, (n,), dev), 0 if tokens is None else _ints("tokens", tokens, (n,), dev), at, lens,
            _ints("free", free, free.shape, dev))
    return head, stride, num_slots, max_pages, free.shape[0] - 1


def extend(slots, tokens, size, table, lengths, free, *, page_size):
    """Pages and places for tokens[i] new tokens of slot slots[i]; returns (starts, where, positions).

    tokens [n] None: one each.  ``size`` lays the maps out: None [n], at most
    one token a row; (T, n) token-major; a number of entries for packed tokens
    (at least as many as there are).  where holds every token's place in the
    pools and positions its position in its row, -1 where there is no token;
    starts [n + 1] the tokens before each row.  table, lengths and free are
    updated.  A call that cannot be done (see ``sync``) changes nothing,
    and gives empty rows."""
    dev = _first("slots", slots, 1)
    n = slots.shape[0]
    head, stride, num_slots, max_pages, num_pages = _pages(slots, tokens, table, lengths, free, dev)
    if size is None:
        T, shape = 1, (n,)
    elif isinstance(size, int):
        T, shape = 0, (size,)
    else:
        T, rows = shape = tuple(size)
        if rows != n or T < 1:
            raise ValueError("size: expected (T, %d), got %s" % (n, shape))
    if n == 0:
        raise ValueError("slots: no rows")
    entries = shape[0] if T == 0 else T * n
    place, empty = slots.device, torch.empty
    starts, work = empty(n + 1, dtype=_I32, device=place), empty(2 * n + 2, dtype=_I32, device=place)
    where, positions = empty(shape, dtype=_I32, device=place), empty(shape, dtype=_I32, device=place)
    _call(_lib.dl_pages_extend, _PAGES.pack(*head, starts.data_ptr(), where.data_ptr(), positions.data_ptr(),
                                            work.data_ptr(), stride, entries, n, T, num_slots, max_pages, num_pages,
                                            page_size), dev)
    return starts, where, positions


def truncate(slots, keep, table, lengths, free, *, page_size):
    """Cut slot slots[i] to its first keep[i] tokens (None: none); pages behind them become free again."""
    dev = _first("slots", slots, 1)
    head, stride, num_slots, max_pages, num_pages = _pages(slots, keep, table, lengths, free, dev)
    _call(_lib.dl_pages_truncate, _PAGES.pack(*head, 0, 0, 0, 0, stride, 0, slots.shape[0], 0, num_slots, max_pages,
                                              num_pages, page_size), dev)


def _pools(k_pages, v_pages, dtype, dev):
    """Two pools of pages alike; returns their addresses and strides."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise TypeError("k_pages must be a CUDA tensor [num_pages, G, page_size, d]")
    shape = k_pages.shape
    _check("k_pages", k_pages, shape, dtype, dev)
    _check("v_pages", v_pages, shape, dtype, dev)
    k, v = k_pages.stride(), v_pages.stride()
    if (k[3] != 1 or v[3] != 1) and shape[3] != 1:
        raise ValueError("k_pages, v_pages: the last dimension must be contiguous")
    return k_pages.data_ptr(), k[0], k[1], k[2], v_pages.data_ptr(), v[0], v[1], v[2]


def _lead(name, t, least, most):
    """The first per-token tensor of a call, of `least` to `most` dimensions; returns its device's number and type."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if not least <= t.dim() <= most:
        raise ValueError("%s: expected %s dimensions, got %s"
                         % (name, least if least == most else "%d or %d" % (least, most), tuple(t.shape)))
    dtype = t.dtype
    if dtype not in _DTYPE:
        raise ValueError("%s: %s is not supported" % (name, dtype))
    if _differentiated(t):
        _bad(name, t, dtype, t.get_device())
    return t.get_device(), dtype


def append(k, v, k_pages, v_pages, where):
    """Keys and values of new tokens, k and v [..., G, d], to the places ``where`` [...] that ``extend`` gave.

    Leading dimensions are [T, n], [total] or [n], as the call of ``extend``
    laid its maps out; negative places are left out, the others are distinct."""
    dev, dt = _lead("k", k, 3, 4)
    pools = _pools(k_pages, v_pages, dt, dev)
    num_pages, G, page_size, d = k_pages.shape
    if 0 in pools and any(s == 0 and c > 1 for p in (k_pages, v_pages) for s, c in zip(p.stride(), p.shape)):
        raise ValueError("k_pages, v_pages: an expanded tensor cannot be written")
    lead = k.shape[:-2]
    T, n = lead if len(lead) == 2 else (lead[0], 1)
    shape = lead + (G, d)
    _call(_lib.dl_kv_append, _APPEND.pack(_DTYPE[dt], T, n, G, d, page_size, num_pages,
                                          *_tokens("k", k, shape, dt, dev, 2, len(lead)),
                                          *_tokens("v", v, shape, dt, dev, 2, len(lead)), *pools,
                                          _ints("where", where, lead, dev)), dev)


def _attend(fn, q, k_pages, v_pages, table, lengths, slots, starts, tokens, window, sinks, scale, out, step):
    dev, dt = _lead("q", q, 3, 3 if step else 4)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise TypeError("slots must be a CUDA tensor [n]")
    shape, n = q.shape, slots.shape[0]
    H, d = shape[-2:]
    pools = _pools(k_pages, v_pages, dt, dev)
    num_pages, G, page_size, dk = k_pages.shape
    if dk != d:
        raise ValueError("k_pages: heads of %d, q has heads of %d" % (dk, d))
    at, stride, num_slots, max_pages, lens = _table(table, lengths, dev)
    packed = pstarts = ptokens = 0
    T = shape[0]
    if step:
        if T != n:
            raise ValueError("q: expected %d rows, got %d" % (n, T))
        T, kind, o_st, o_sn = 1, 0, 0, H * d
    elif len(shape) == 3:
        if starts is None or tokens is not None:
            raise ValueError("packed tokens need starts, and no tokens")
        packed, kind, o_st, o_sn = 1, 1, H * d, 0
        pstarts = _ints("starts", starts, (n + 1,), dev)
    else:
        kind, o_st, o_sn = 2, n * H * d, H * d
        if shape[1] != n:
            raise ValueError("q: expected %d rows, got %d" % (n, shape[1]))
        if starts is not None:
            raise ValueError("starts are for packed tokens")
        if tokens is not None:
            ptokens = _ints("tokens", tokens, (n,), dev)
    if window is None:
        window = 0
    elif window < 1:
        raise ValueError("window: at least 1, or None")
    if out is None:
        out = torch.empty(shape, dtype=dt, device=q.device)
        view = out.data_ptr(), o_st, o_sn
    else:
        view = _tokens("out", out, shape, dt, dev, 2, kind)
    args = _ATTEND.pack(_DTYPE[dt], n, T, packed, H, G, d, page_size, max_pages, num_slots, num_pages, window, sinks,
                        d ** -0.5 if scale is None else scale, *_tokens("q", q, shape, dt, dev, 2, kind), *view,
                        *pools, at, stride, lens, _ints("slots", slots, (n,), dev), pstarts, ptokens)
    size = _lib.dl_attend_workspace(args + _NO_WORKSPACE) if dev == _device() else \
        _on(dev, _lib.dl_attend_workspace, args + _NO_WORKSPACE)
    if size > 0:
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
        args += _WORKSPACE.pack(workspace.data_ptr(), size)
    else:
        args += _NO_WORKSPACE
    _call(fn, args, dev)
    return out


def attend(q, k_pages, v_pages, table, lengths, slots, *, starts=None, tokens=None, window=None, sinks=0, scale=None,
           out=None):
    """Attention of the last tokens of every slot: q [T, n, H, d], or packed [total, H, d] with ``starts`` [n + 1].

    tokens [n]: how many of the T tokens row i has (None: T each); the slot
    of a row that has none may be anything.  H / G
    consecutive query heads share a head of keys and values.  A token sees its
    own position and those before it; with ``window`` only the last ``window``
    of them and the row's first ``sinks``.  scale: 1 / sqrt(d) unless given.
    out: like q, with any strides whose tokens share no elements.
    The tokens' own keys and values have to be in the pages already."""
    return _attend(_lib.dl_attend, q, k_pages, v_pages, table, lengths, slots, starts, tokens, window, sinks, scale, out,
                   False)


def attend_step(q, k_pages, v_pages, table, lengths, slots, *, window=None, sinks=0, scale=None, out=None):
    """``attend`` of one token a row, its slot's last: q [n, H, d].  A slot of length 0 gives zero."""
    return _attend(_lib.dl_attend_step, q, k_pages, v_pages, table, lengths, slots, None, None, window, sinks, scale,
                   out, True)
