"""Outputs: expanded ones are refused, and those that interleave with other tensors are written as they are."""
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


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_expanded_outputs_are_refused(at, dtype):
    s = Setup([9, 30], 1, 64, 16, dtype, seed=1)
    q, _ = s.queries((4, 2), 2)
    for shape in ((1, 2, 2, 64), (4, 1, 2, 64)):
        out = torch.zeros(shape, dtype=s.dt, device="cuda")
        with pytest.raises(RuntimeError, match="share"):
            at.attend(q, *s.args(), out=out.expand(4, 2, 2, 64))
        assert not out.any()
    one = torch.zeros(1, 2, 64, dtype=s.dt, device="cuda")
    with pytest.raises(RuntimeError, match="share"):
        at.attend(q[:, 0], *s.args(), starts=s.dev([0, 2, 4]), out=one.expand(4, 2, 64))
    with pytest.raises(RuntimeError, match="share"):
        at.attend_step(q[0], *s.args(), out=one.expand(2, 2, 64))
    at.sync()
    assert not one.any()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 20), ("fp32", 64)])
def test_rows_first_and_in_turns(at, dtype, d):
    """Rows outside, tokens outside, and both in steps of a wider tensor."""
    s = Setup([70, 5], 1, d, 16, dtype, seed=2)
    q, host = s.queries((4, 2), 2)
    new = lambda *shape: torch.full(shape, 7.0, dtype=s.dt, device="cuda")  # noqa: E731
    wide = new(3, 8, 5, d)
    for out in (new(4, 2, 2, d), new(2, 4, 2, d).transpose(0, 1), wide[:2, ::2, 1:3].transpose(0, 1)):
        o = at.attend(q, *s.args(), out=out)
        at.sync()
        for i in range(2):
            one = Setup.__new__(Setup)
            one.__dict__.update(s.__dict__, after=[s.after[i]], k=[s.k[i]], v=[s.v[i]])
            check_rows(one, host[:, i], o[:, i].cpu(), [4], [0], None, 0)
    wide[:2, ::2, 1:3] = 7
    assert (wide == 7).all()
