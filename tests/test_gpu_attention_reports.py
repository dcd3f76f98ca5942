"""What the attention calls report, and what they do not: the same whatever kernel a call's size and type choose."""
import itertools

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
