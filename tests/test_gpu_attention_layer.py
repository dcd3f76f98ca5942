"""The example's attention layer: the attention calls together, prompts against single tokens."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def layers():
    from linear_attention_recurrent_gdn_gb300 import build
    build.build()
    import mixer_layer
    return mixer_layer


# A layer rounds to bf16 in the norm, the projection, the weights of the values, the attention's output and the output
# projection.  Prompt and step differ in those roundings at most: five of 2^-8 each of the values that go in.  The
# cached keys and values see the first two.
OUT_TOL, STATE_TOL = 5 * 2.0 ** -8, 2 * 2.0 ** -8


@pytest.mark.parametrize("slots,tokens,steps", [(1, 1, 3), (4, 96, 8), (3, 33, 20)])
@pytest.mark.parametrize("d,window,sinks", [(64, None, 0), (128, 20, 2)])
def test_attn_layer(layers, slots, tokens, steps, d, window, sinks):
    make = lambda: layers.AttnLayer(4, d, slots, tokens + steps, kv_heads=2, window=window, sinks=sinks)  # noqa: E731
    out, state = layers.compare(make, slots, tokens, steps)
    assert out <= OUT_TOL and state <= STATE_TOL


def test_command(layers, capsys):
    out, state = layers.main(["--layer", "attn", "--slots", "2", "--tokens", "40", "--steps", "4"])
    assert out <= OUT_TOL and state <= STATE_TOL
    assert "attn layer" in capsys.readouterr().out
