"""Head dimensions between those that the tensor-core kernels are made for: the rest of a tile is zero, and is not written."""
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


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [8, 24, 56, 72, 120, 136, 200, 248])
@pytest.mark.parametrize("H,G,page", [(6, 2, 16), (40, 1, 128)])
def test_dimensions(at, d, dtype, H, G, page):
    """Whole and split prompts, and single tokens, into a wider tensor whose other values stay."""
    for tokens, before in (([3, 40, 0, 130], [0, 77, 5, 300]), ([4], [3000])):
        s = Setup([t + b for t, b in zip(tokens, before)], G, d, page, dtype, seed=d + H)
        starts = list(itertools.accumulate([0] + tokens))
        q, host = s.queries((starts[-1],), H)
        wide = torch.full((starts[-1] + 1, H + 2, d), 7.0, dtype=s.dt, device="cuda")
        o = at.attend(q, *s.args(), starts=s.dev(starts), out=wide[:-1, 1:-1])
        at.sync()
        check_rows(s, host, o.cpu(), tokens, starts, None, 0)
        o.fill_(7)
        assert (wide == 7).all()
        q, host = s.queries((len(tokens),), H)
        wide = torch.full((len(tokens) + 1, H + 2, d), 7.0, dtype=s.dt, device="cuda")
        o = at.attend_step(q, *s.args(), window=200, sinks=3, out=wide[:-1, 1:-1])
        at.sync()
        check_rows(s, host, o.cpu(), [1] * len(tokens), range(len(tokens)), 200, 3)
        o.fill_(7)
        assert (wide == 7).all()
