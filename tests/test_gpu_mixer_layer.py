"""The example layers: the mixer calls together, prompts against single tokens."""
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


# A layer rounds to bf16 in the projection, the convolution, the recurrence, the
# gated norm and the output projection.  Prompt and step differ in those
# roundings at most: five of 2^-8 each of the values that go in, and a value of
# the output sums many of them.  States see the first two.
OUT_TOL, STATE_TOL = 5 * 2.0 ** -8, 2 * 2.0 ** -8


@pytest.mark.parametrize("slots,tokens,steps", [(1, 1, 3), (4, 96, 8), (3, 33, 20)])
def test_gdn_layer(layers, slots, tokens, steps):
    out, state = layers.compare(lambda: layers.GdnLayer(4, 64, slots), slots, tokens, steps)
    assert out <= OUT_TOL and state <= STATE_TOL


@pytest.mark.parametrize("slots,tokens,steps", [(1, 1, 3), (4, 130, 6), (3, 33, 20)])
@pytest.mark.parametrize("groups", [1, 2])
def test_ssm_layer(layers, slots, tokens, steps, groups):
    out, state = layers.compare(lambda: layers.SsmLayer(4, 64, 64, slots, groups), slots, tokens, steps)
    assert out <= OUT_TOL and state <= STATE_TOL


def test_command(layers, capsys):
    for layer in ("gdn", "ssm"):
        out, state = layers.main(["--layer", layer, "--slots", "2", "--tokens", "40", "--steps", "4"])
        assert out <= OUT_TOL and state <= STATE_TOL
        assert "%s layer" % layer in capsys.readouterr().out
