"""Which kernel a call of prompts takes, and whether its keys are split, where only the result's bits or a report tell."""
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


def test_many_tokens_and_heads_run_on_the_tensor_cores(at, monkeypatch):
    """2^26 pairs of tokens and heads: 262 thousand items of the tensor-core kernel.  Its test-only stall shows that it ran."""
    T, H, G, d = 4100, 16384, 128, 64
    s = Setup([T], G, d, 64, "bf16", seed=3, spare=0)
    gen = torch.Generator(device="cuda").manual_seed(3)
    # queries whose tokens share their memory: what is written is of full size
    q = torch.as_strided(torch.randn(T * d + H * d, generator=gen, device="cuda").to(torch.bfloat16), (T, H, d), (d, d, 1))
    run = lambda: at.attend(q, *s.args(), starts=s.dev([0, T]), window=40)  # noqa: E731
    out = run()
    at.sync()
    for t in (0, 39, 40, 2047, 4098, 4099):
        ref, mag, big = model.attend_row(q[t:t + 1].cpu(), s.k[0], s.v[0], [t], 40)
        check(out[t:t + 1], ref, bound(ref, mag, big, torch.bfloat16, d, T), "token %d" % t)
    monkeypatch.setenv("DL_TEST_STALL", "1")
    monkeypatch.setenv("DL_TEST_WAIT_MS", "40")
    run()
    monkeypatch.delenv("DL_TEST_STALL")
    monkeypatch.delenv("DL_TEST_WAIT_MS")
    with pytest.raises(Exception, match="status 5"):
        at.sync()
    at.sync()


@pytest.mark.parametrize("tokens,before,H,G,d", [(4, 300, 32, 8, 128), (16, 300, 16, 2, 128), (64, 300, 32, 8, 128), (4, 300, 8, 1, 64),
                                                 (300, 0, 8, 1, 64)])
def test_short_calls_stay_whole(at, tokens, before, H, G, d):
    """Where a join costs more than it gives, a row's bits are those it has among 70 rows, whose keys are never split."""
    s = Setup([tokens + before], G, d, 64, "bf16", seed=tokens + d)
    k, v, table, lengths, slots = s.args()
    q, host = s.queries((tokens,), H)
    one = at.attend(q, k, v, table, lengths, slots, starts=s.dev([0, tokens]))
    many = at.attend(q.repeat(70, 1, 1), k, v, table, lengths, slots.repeat(70), starts=s.dev([tokens * i for i in range(71)]))
    at.sync()
    check_rows(s, host, one.cpu(), [tokens], [0], None, 0)
    assert torch.equal(one, many[:tokens]) and torch.equal(one, many[-tokens:])


@pytest.mark.parametrize("keys", [1000, 20000])
def test_longer_calls_are_split(at, keys):
    """The other side: one row of few tokens behind more keys does not walk them in one item a head."""
    s = Setup([keys], 1, 64, 64, "bf16", seed=2)
    k, v, table, lengths, slots = s.args()
    q, host = s.queries((4,), 8)
    one = at.attend(q, k, v, table, lengths, slots, starts=s.dev([0, 4]))
    many = at.attend(q.repeat(70, 1, 1), k, v, table, lengths, slots.repeat(70), starts=s.dev([4 * i for i in range(71)]))
    at.sync()
    check_rows(s, host, one.cpu(), [4], [0], None, 0)
    check_rows(s, host, many[:4].cpu(), [4], [0], None, 0)
    assert not torch.equal(one, many[:4])
