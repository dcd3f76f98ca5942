"""Host-side checks of the mixer calls (no GPU needed): struct layouts and
refusals.  Pointers are fake device addresses that no call gets far enough to
use: every call is invalid in exactly one way, or has no rows."""
import ctypes

import numpy as np
import pytest

from linear_attention_recurrent_gdn_gb300 import build

I64, P = ctypes.c_int64, ctypes.c_void_p
BASE = 0x7f0000000000


class Tokens(ctypes.Structure):
    _fields_ = [("slots", P), ("lengths", P), ("fresh", P), ("fresh_all", I64), ("n", I64), ("T", I64),
                ("packed", I64), ("num_slots", I64)]


class View(ctypes.Structure):
    _fields_ = [("data", P), ("stride_t", I64), ("stride_n", I64)]


class Conv(ctypes.Structure):
    _fields_ = [("tokens", Tokens)] + [(k, I64) for k in ("dtype", "weight_f32", "C", "W", "act", "l2_channels",
                                                         "head_dim", "n_parts")] + \
        [("eps", ctypes.c_double), ("x", View), ("weight", P), ("bias", P), ("state", P), ("y", View * 4),
         ("part_channels", I64 * 4)]


class Ssm(ctypes.Structure):
    _fields_ = [("tokens", Tokens)] + [(k, I64) for k in ("dtype", "dt_f32", "softplus", "H", "G", "P", "N")] + \
        [(k, View) for k in ("x", "dt", "B", "C", "y")] + \
        [(k, P) for k in ("A", "D", "dt_bias", "state", "workspace")] + [("workspace_bytes", I64)]


class Gated(ctypes.Structure):
    _fields_ = [(k, I64) for k in ("dtype", "weight_f32", "weight_heads", "rows", "H", "d", "kind", "act",
                                   "gate_first")] + [("eps", ctypes.c_double)] + \
        [(k, P) for k in ("x", "gate", "weight", "bias", "y")] + \
        [(k, I64) for k in ("x_stride", "gate_stride", "y_stride")]


class Add(ctypes.Structure):
    _fields_ = [(k, I64) for k in ("dtype", "residual_f32", "weight_f32", "rows", "D", "kind")] + \
        [("eps", ctypes.c_double), ("alpha", ctypes.c_double)] + \
        [(k, P) for k in ("x", "residual", "weight", "bias", "scale", "post", "y", "h")] + \
        [(k, I64) for k in ("x_stride", "residual_stride", "y_stride", "h_stride")]


@pytest.fixture(scope="module")
def mx():
    build.build()
    from linear_attention_recurrent_gdn_gb300 import mixer
    return mixer


_KEEP = []      # host lists that the structs point to


def _fake():
    return iter(range(BASE, BASE + 64 * (1 << 20), 1 << 20))


def _tokens(n=3, T=5, num_slots=8):
    slots = np.arange(n, dtype=np.int32)
    t = Tokens(slots.ctypes.data, 0, 0, 0, n, T, 0, num_slots)
    _KEEP.append(slots)
    return t


def _conv():
    a = _fake()
    q = Conv(_tokens(), 1, 0, 192, 4, 1, 128, 64, 2, 1e-6, View(next(a), 576, 192), next(a), next(a), next(a))
    q.y[0], q.y[1] = View(next(a), 384, 128), View(next(a), 192, 64)
    q.part_channels[0], q.part_channels[1] = 128, 64
    return q


def _ssm(T=5):
    a = _fake()
    v = lambda w: View(next(a), 3 * w, w)  # noqa: E731
    return Ssm(_tokens(T=T), 1, 0, 1, 4, 2, 64, 64, v(256), v(4), v(128), v(128), v(256), next(a), next(a), next(a),
               next(a), 0, 0)


def _gated():
    a = _fake()
    return Gated(1, 0, 0, 7, 4, 64, 0, 1, 0, 1e-5, next(a), next(a), next(a), next(a), next(a), 256, 256, 256)


def _add():
    a = _fake()
    return Add(1, 0, 0, 7, 256, 0, 1e-5, 1.0, *[next(a) for _ in range(8)], 256, 256, 256, 256)


MAKE = dict(dl_conv=_conv, dl_ssm=_ssm, dl_ssm_step=lambda: _ssm(1), dl_gated_norm=_gated, dl_add_norm=_add)


def _call(mx, fn, q):
    err = ctypes.create_string_buffer(256)
    return getattr(mx._lib, fn)(ctypes.string_at(ctypes.addressof(q), ctypes.sizeof(q)), None, err, 256), \
        err.value.decode()


def _set(q, path, value):
    *most, last = path.split(".")
    for k in most:
        q = q[int(k)] if k.isdigit() else getattr(q, k)
    if last.isdigit():
        q[int(last)] = value
    else:
        setattr(q, last, value)


def test_struct_sizes_match_the_binding(mx):
    assert ctypes.sizeof(Conv) == mx._CONV.size and ctypes.sizeof(Ssm) == mx._SSM.size
    assert ctypes.sizeof(Gated) == mx._GATED.size and ctypes.sizeof(Add) == mx._ADD.size


@pytest.mark.parametrize("fn,changes", [
    ("dl_conv", {"tokens.n": 0}), ("dl_ssm", {"tokens.n": 0}), ("dl_ssm_step", {"tokens.n": 0}),
    ("dl_gated_norm", {"rows": 0}), ("dl_add_norm", {"rows": 0}),
    ("dl_conv", {"tokens.n": 0, "x.data": 0}),
])
def test_no_rows_is_fine(mx, fn, changes):
    q = MAKE[fn]()
    for k, v in changes.items():
        _set(q, k, v)
    assert _call(mx, fn, q) == (0, "")


@pytest.mark.parametrize("fn,path,value,status,word", [
    ("dl_conv", "dtype", 3, "EINVAL", "dtype"),
    ("dl_conv", "W", 5, "EUNSUPPORTED", "width"),
    ("dl_conv", "W", 1, "EUNSUPPORTED", "width"),
    ("dl_conv", "C", 0, "EINVAL", "channels"),
    ("dl_conv", "act", 2, "EINVAL", "activation"),
    ("dl_conv", "n_parts", 5, "EINVAL", "ranges"),
    ("dl_conv", "n_parts", 1, "EINVAL", "add up"),
    ("dl_conv", "part_channels.1", 65, "EINVAL", "add up"),
    ("dl_conv", "part_channels.0", 0, "EINVAL", "add up"),
    ("dl_conv", "head_dim", 48, "EUNSUPPORTED", "power of two"),
    ("dl_conv", "head_dim", 512, "EUNSUPPORTED", "power of two"),
    ("dl_conv", "l2_channels", 96, "EINVAL", "whole heads"),
    ("dl_conv", "l2_channels", 256, "EINVAL", "normalised"),
    ("dl_conv", "eps", -1.0, "EINVAL", "eps"),
    ("dl_conv", "eps", float("nan"), "EINVAL", "eps"),
    ("dl_conv", "x.data", 0, "EINVAL", "NULL"),
    ("dl_conv", "y.1.data", 0, "EINVAL", "NULL"),
    ("dl_conv", "weight", 0, "EINVAL", "NULL"),
    ("dl_conv", "x.data", BASE + 1, "EINVAL", "misaligned"),
    ("dl_conv", "state", BASE + 1, "EINVAL", "misaligned"),
    ("dl_conv", "tokens.n", 1025, "EINVAL", "1024"),
    ("dl_conv", "tokens.n", -1, "EINVAL", "rows"),
    ("dl_conv", "tokens.T", -1, "EINVAL", "tokens"),
    ("dl_conv", "tokens.packed", 1, "EINVAL", "lengths"),
    ("dl_conv", "tokens.slots", 0, "EINVAL", "slots"),
    ("dl_conv", "tokens.num_slots", 2, "EINVAL", "not in"),
    ("dl_conv", "tokens.num_slots", 0, "EINVAL", "slots"),
    ("dl_ssm", "H", 5, "EINVAL", "groups"),
    ("dl_ssm", "G", 0, "EINVAL", "groups"),
    ("dl_ssm", "N", 257, "EUNSUPPORTED", "256"),
    ("dl_ssm", "P", 0, "EINVAL", "state"),
    ("dl_ssm", "A", 0, "EINVAL", "NULL"),
    ("dl_ssm", "dt.data", 0, "EINVAL", "NULL"),
    ("dl_ssm", "state", BASE + 2, "EINVAL", "misaligned"),
    ("dl_ssm", "B.data", BASE + 1, "EINVAL", "misaligned"),
    ("dl_ssm_step", "state", 0, "EINVAL", "state pool"),
    ("dl_ssm_step", "tokens.T", 2, "EINVAL", "one token"),
    ("dl_gated_norm", "d", 16385, "EUNSUPPORTED", "16384"),
    ("dl_gated_norm", "kind", 2, "EINVAL", "norm"),
    ("dl_gated_norm", "act", 3, "EINVAL", "activation"),
    ("dl_gated_norm", "rows", -1, "EINVAL", "rows"),
    ("dl_gated_norm", "weight", 0, "EINVAL", "NULL"),
    ("dl_gated_norm", "gate", BASE + 1, "EINVAL", "misaligned"),
    ("dl_add_norm", "D", 16385, "EUNSUPPORTED", "16384"),
    ("dl_add_norm", "D", 0, "EINVAL", "rows"),
    ("dl_add_norm", "y", 0, "EINVAL", "NULL"),
    ("dl_add_norm", "residual", BASE + 1, "EINVAL", "misaligned"),
    ("dl_add_norm", "dtype", -1, "EINVAL", "dtype"),
])
def test_refusals(mx, fn, path, value, status, word):
    from linear_attention_recurrent_gdn_gb300 import deltalog as dl
    q = MAKE[fn]()
    _set(q, path, value)
    rc, msg = _call(mx, fn, q)
    assert rc == getattr(dl, status) and word in msg, (rc, msg)


@pytest.mark.parametrize("slots", [[0, 1, 0], [-1, 0, 1], [0, 8, 1], [7, 3, 7]])
def test_slot_lists(mx, slots):
    q, s = _conv(), np.array(slots, np.int32)
    q.tokens.slots = s.ctypes.data
    rc, msg = _call(mx, "dl_conv", q)
    assert rc == 1 and ("twice" in msg or "not in" in msg), msg


def test_many_slots_with_one_repeated(mx):
    s = np.random.RandomState(0).permutation(1 << 20)[:1024].astype(np.int32)
    s[1023] = s[511]
    q = _conv()
    q.tokens.slots, q.tokens.n, q.tokens.num_slots = s.ctypes.data, 1024, 1 << 20
    rc, msg = _call(mx, "dl_conv", q)
    assert rc == 1 and "slot %d appears twice" % s[511] in msg


@pytest.mark.parametrize("lengths", [[5, 6, 0], [5, -1, 0]])
def test_lengths(mx, lengths):
    q, v = _ssm(), np.array(lengths, np.int32)
    q.tokens.lengths = v.ctypes.data
    rc, msg = _call(mx, "dl_ssm", q)
    assert rc == 1 and "tokens" in msg


def test_null_arguments_and_no_buffer(mx):
    for fn in MAKE:
        assert getattr(mx._lib, fn)(None, None, None, 0) == 1
    q = _conv()
    q.dtype = 9
    assert mx._lib.dl_conv(ctypes.string_at(ctypes.addressof(q), ctypes.sizeof(q)), None, None, 0) == 1


def test_workspace_refuses_bad_sizes(mx):
    q = _ssm()
    size = lambda: mx._lib.dl_ssm_workspace(ctypes.string_at(ctypes.addressof(q), ctypes.sizeof(q)))  # noqa: E731
    assert size() >= 0
    q.N = 300
    assert size() == -1
