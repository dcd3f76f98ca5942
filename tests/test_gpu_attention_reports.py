"""What the attention calls report, and what they do not: the same whatever kernel a call's size and type choose."""
import itertools

import pytest
import torch

from attention_helpers import Setup, bound, check, check_rows
from oracle import attention_model as model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def at():
    from linear_attention_recurrent_gdn_gb300 import build
    build.build()
    from linear_attention_recurrent_gdn_gb300 import attention
    attention.sync()
    return attention


# Prompts on the tensor cores with keys split over the GPU (few tiles, at most 64 rows) and not, and on the FP32 cores.
KINDS = [("bf16", 64, 5), ("bf16", 256, 5), ("bf16", 64, 70), ("bf16", 128, 64), ("fp32", 64, 5), ("bf16", 20, 5)]


@pytest.mark.parametrize("dtype,d,n", KINDS)
@pytest.mark.parametrize("layout", ["packed", "major"])
def test_rows_without_tokens_are_not_looked_at(at, layout, dtype, d, n):
    """Padding rows: no token, and a slot out of range or of an impossible length."""
    counts = [0 if i % 5 in (1, 3) else 1 + i % 4 for i in range(n)]
    s = Setup([c + 30 + i for i, c in enumerate(counts)], 1, d, 16, dtype, seed=n + d)
    k, v, table, lengths, slots = s.args()
    for i, c in enumerate(counts):
        if c == 0 and i % 5 == 1:
            slots[i] = -1 if i % 2 else 1 << 30
        elif c == 0:
            lengths[s.slots[i]] = -5 if i % 2 else s.max_pages * 16 + 1
    starts = list(itertools.accumulate([0] + counts))
    if layout == "packed":
        q, host = s.queries((starts[-1],), 2)
        o = at.attend(q, k, v, table, lengths, slots, starts=s.dev(starts))
    else:
        q, rows = s.queries((4, n), 2)
        o = at.attend(q, k, v, table, lengths, slots, tokens=s.dev(counts))
        o = torch.cat([o[:c, i] for i, c in enumerate(counts)])
        host = torch.cat([rows[:c, i] for i, c in enumerate(counts)])
    at.sync()
    check_rows(s, host, o.cpu(), counts, starts, None, 0)


@pytest.mark.parametrize("dtype,d,n", KINDS)
@pytest.mark.parametrize("number", [-1, -(1 << 31), 5, 0x7fffffff])
def test_numbers_of_tokens_out_of_range_are_reported(at, number, dtype, d, n):
    """A row with a negative number of tokens has none, one with more than T has T; both are reported."""
    T = 4
    s = Setup([50 + i for i in range(n)], 1, d, 16, dtype, seed=n + d)
    q, host = s.queries((T, n), 2)
    tokens = s.dev([T - i % 2 for i in range(n)])
    tokens[n - 2] = number
    out = torch.full_like(q, 7.0)
    at.attend(q, *s.args(), tokens=tokens, out=out)
    with pytest.raises(Exception, match="tokens"):
        at.sync()
    for i in range(n):
        t = min(max(int(tokens[i]), 0), T)
        ref, mag, big = model.attend_row(host[:t, i], s.k[i], s.v[i], torch.arange(s.after[i] - t, s.after[i]))
        check(out[:t, i], ref, bound(ref, mag, big, s.dt, d, s.after[i]), "row %d" % i)
        assert (out[t:, i] == 7).all()
    for good in (0, T):
        tokens[n - 2] = good
        at.attend(q, *s.args(), tokens=tokens, out=out)
        at.sync()
