"""Which kernel a call of prompts takes, where only a report tells."""
import pytest
import torch

from attention_helpers import Setup, bound, check
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
