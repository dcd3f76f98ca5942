"""Scales at the ends of what 32 bits hold."""
import pytest
import torch

from attention_helpers import Setup, check_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def at():
    from linear_attention_recurrent_gdn_gb300 import build
    build.build()
    from linear_attention_recurrent_gdn_gb300 import attention
    attention.sync()
    return attention


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp16", 128), ("bf16", 256), ("bf16", 20), ("fp32", 64)])
@pytest.mark.parametrize("scale", [1e-300, 1e-46, 1e-44, 1e-40, 1e-38, 1e-30])
@pytest.mark.parametrize("window,sinks", [(None, 0), (30, 3)])
def test_scales_that_vanish(at, dtype, d, scale, window, sinks):
    """A scale that is zero in 32 bits: every key that a token sees counts the same, and the others do not count (a
    masked score of -inf times zero would be a NaN).  Below the normal numbers a scale is off by half of 2^-149 at most,
    which moves a score of these inputs by 2^-138."""
    s = Setup([150], 1, d, 16, dtype, seed=d)
    q, host = s.queries((150,), 2)
    o = at.attend(q, *s.args(), starts=s.dev([0, 150]), window=window, sinks=sinks, scale=scale)
    last = at.attend_step(q[149:], *s.args(), window=window, sinks=sinks, scale=scale)
    at.sync()
    check_rows(s, host, o.cpu(), [150], [0], window, sinks, scale)
    check_rows(s, host[149:], last.cpu(), [1], [0], window, sinks, scale)
