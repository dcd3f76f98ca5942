"""Outputs whose tokens share elements are refused, before any CUDA call.  Pointers are fake device addresses, and every
call lacks its lengths: one that is not refused for its output is refused for that."""
import itertools

import pytest

from test_attention_cpu import MAKE, _call, at  # noqa: F401  (the module fixture)


def _strided(fn, T, n, st, sn, packed=0):
    q = MAKE[fn]()
    q.T, q.n, q.packed, q.o.stride_t, q.o.stride_n = T, n, packed, st, sn
    q.starts = q.slots if packed else None
    q.lengths = None
    return q


def _shares(w, T, n, st, sn):
    """Whether two tokens' ranges of w elements meet, by looking at all pairs."""
    at = sorted(t * st + i * sn for t, i in itertools.product(range(T), range(n)))
    return any(b - a < w for a, b in zip(at, at[1:]))


W = 8 * 128          # a token of _attend's calls
STRIDES = [0, 1, 8, W - 8, W, W + 8, 2 * W - 8, 2 * W, 3 * W, 3 * W + 8, 5 * W, 7 * W - 8, 7 * W, 1 << 40]


@pytest.mark.parametrize("T,n", [(1, 1), (1, 3), (4, 1), (2, 3), (3, 2), (5, 3), (4, 4)])
def test_token_major_outputs(at, T, n):  # noqa: F811
    for st, sn in itertools.product(STRIDES, STRIDES):
        rc, msg = _call(at, "dl_attend", _strided("dl_attend", T, n, st, sn))
        assert rc == at._dl.EINVAL
        assert ("share" in msg) == _shares(W, T, n, st, sn), (st, sn, msg)


@pytest.mark.parametrize("T", [1, 2, 50])
def test_packed_outputs(at, T):  # noqa: F811
    for st in STRIDES:
        rc, msg = _call(at, "dl_attend", _strided("dl_attend", T, 3, st, 0, packed=1))
        assert rc == at._dl.EINVAL and ("share" in msg) == _shares(W, T, 1, st, 0)


@pytest.mark.parametrize("n", [1, 2, 50])
def test_outputs_of_a_step(at, n):  # noqa: F811
    for sn in STRIDES:
        rc, msg = _call(at, "dl_attend_step", _strided("dl_attend_step", 1, n, 0, sn))
        assert rc == at._dl.EINVAL and ("share" in msg) == _shares(W, 1, n, 0, sn)


def test_many_rows_between_long_rows(at):  # noqa: F811
    """Neither stride spans the other dimension: 1000 rows of 600 tokens in turns, and one token that meets another."""
    for n, T, st, sn in ((1000, 600, 1000 * W, W), (1000, 600, W, 600 * W)):
        assert "share" not in _call(at, "dl_attend", _strided("dl_attend", T, n, st, sn))[1]
        assert "share" in _call(at, "dl_attend", _strided("dl_attend", T, n, max(st, W) - (st > W) * 8, sn - (sn > W) * 8))[1]
    # token 599 of row 0 and token 0 of row 999, and nobody else
    sn = 599 * 1000 * W // 999 // 8 * 8
    assert _shares(W, 600, 1000, 1000 * W, sn) == ("share" in _call(at, "dl_attend", _strided("dl_attend", 600, 1000, 1000 * W, sn))[1])
