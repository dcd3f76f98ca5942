"""The state space scan on given inputs, against its 64-bit definition.

Tolerances count roundings.  A state element is a chain of multiply-adds in 32
bits, `steps` of them with the steps of its decays (an exponent that is a sum
of logs of one sign is off by a few 2^-24 of its size s, and s e^-s < 1), so it
is off by at most steps 2^-24 of the sum of its terms' absolute values; an
output sums N of those and is rounded once to its own type.  The tensor-core
scan (bf16, N <= 128, a row of 32 tokens or more) rounds one factor of each of
an output's terms, the pair weight or the state, to bf16 besides: half a step
of the sum of the terms' absolute values.
"""
import numpy as np
import pytest
import torch

from oracle import mixer_model as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def mx():
    from linear_attention_recurrent_gdn_gb300 import build
    build.build()
    from linear_attention_recurrent_gdn_gb300 import mixer
    return mixer


def half(t):
    return torch.finfo(t).eps / 2


def rnd(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, generator=g)).to(dtype)


def run_packed(mx, rows, A, D=None, state=None, slots=None, fresh=False, softplus=False):
    """rows: one (x, dt, B, C) a row, [t, ...] each.  Returns the rows' outputs and the pool."""
    lengths = [r[0].shape[0] for r in rows]
    dev = [torch.cat([r[k] for r in rows]).cuda() for k in range(4)]
    pool = None if state is None else state.cuda()
    y = mx.ssm(dev[0], dev[1], A.cuda(), dev[2], dev[3], None if D is None else D.cuda(), dt_softplus=softplus,
               slots=slots, state=pool, lengths=lengths, fresh=fresh)
    return torch.split(y.cpu(), lengths), None if pool is None else pool.cpu()


def check_packed(mx, rows, A, D=None, softplus=False, mma=False, S0=None):
    """Every row against the definition, outputs and states."""
    H, P, N = rows[0][0].shape[1], rows[0][0].shape[2], rows[0][2].shape[2]
    dt = rows[0][0].dtype
    state = torch.zeros(len(rows), H, P, N) if S0 is None else S0
    ys, pool = run_packed(mx, rows, A, D, state, list(range(len(rows))), S0 is None, softplus)
    for i, r in enumerate(rows):
        want, S, ymag, Smag = ref.ssm_row(r[0], r[1], A, r[2], r[3], D, state[i], None, softplus)
        steps = 3 * r[0].shape[0] + 16
        tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
        tol = half(dt) * want.abs() + tiny + ((steps + N) * U + (1.01 * half(dt) if mma else 0)) * ymag
        top = torch.finfo(dt).max                 # past its type's range an output is an infinity
        off = (ys[i].double().clamp(-top, top) - want.clamp(-top, top)).abs()
        assert (off <= tol).all(), \
            "y of row %d: %.3g times what is allowed" % (i, float((off / tol).max()))
        soff, stol = (pool[i].double() - S).abs(), steps * U * Smag + 1e-30
        assert (soff <= stol).all(), \
            "state of row %d: %.3g times what is allowed" % (i, float((soff / stol).max()))


# ------------------------------------------------------------------- decays --
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("big", [100.0, 1e3, 1e4])
@pytest.mark.parametrize("positive", [False, True])
def test_strong_decays_among_weak_ones(mx, dtype, big, positive):
    """Tokens that forget everything before them leave the weights of the tokens after them alone: few of them,
    at places all over the chunk, its blocks of 32 and their halves, among steps of 0.01.  With positive inputs
    an output is as large as the sum of its terms, and a weight's error shows in full."""
    g = torch.Generator().manual_seed(int(big))
    H, P, N, dt = 2, 64, 64, DT[dtype]
    rows = []
    for at in ((0, 40), (3, 16, 127), (31, 95, 96, 190), (64, 65, 66), (15, 47, 111)):
        t = 100 + at[-1] % 60
        step = torch.full((t, H), 0.01)
        for k in at:
            if k < t:
                step[k] = torch.tensor([big, 0.01])       # one head forgets, the other one does not
        xbc = [rnd(g, t, *s, dtype=dt) for s in ((H, P), (1, N), (1, N))]
        if positive:
            xbc = [v.abs() for v in xbc]
        rows.append((xbc[0], step, xbc[1], xbc[2]))
    check_packed(mx, rows, torch.tensor([-16.0, -16.0]), mma=dtype == "bf16")


@pytest.mark.parametrize("seed", range(4))
def test_every_step_a_strong_decay(mx, seed):
    """A = -50 and steps of 0 to 40 or so: sums over a chunk of a hundred thousand, pairs next to one another."""
    g = torch.Generator().manual_seed(seed)
    H, P, N, t = 4, 64, 64, 250
    rows = [(rnd(g, t, H, P, dtype=torch.bfloat16), rnd(g, t, H, scale=40.0), rnd(g, t, 1, N, dtype=torch.bfloat16),
             rnd(g, t, 1, N, dtype=torch.bfloat16))]
    check_packed(mx, rows, -1 - 49 * torch.rand(H, generator=g), softplus=True, mma=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decays_that_overflow(mx, dtype):
    """dt A = -inf is a decay to zero, not a NaN."""
    g = torch.Generator().manual_seed(0)
    H, P, N, dt, t = 1, 16, 24, DT[dtype], 140
    step = torch.full((t, H), 1e-28)
    step[[5, 6, 70, 127, 128]] = 1e12
    rows = [(rnd(g, t, H, P, dtype=dt), step, rnd(g, t, 1, N, dtype=dt), rnd(g, t, 1, N, dtype=dt))]
    assert torch.isinf(step[5] * -1e28).all()
    check_packed(mx, rows, torch.tensor([-1e28]), mma=dtype == "bf16", S0=rnd(g, 1, H, P, N))


# ------------------------------------------------------ a wait that runs out --
def scan_inputs(g, T, n, H, P, N):
    x, B, C = (rnd(g, T, n, *s, dtype=torch.bfloat16).cuda() for s in ((H, P), (1, N), (1, N)))
    return x, rnd(g, T, n, H, dtype=torch.bfloat16).cuda(), -torch.rand(H, generator=g).cuda() - 0.1, B, C


@pytest.mark.parametrize("P,N", [(64, 64), (128, 128), (36, 20)])      # tensor copies, and values one by one
def test_a_wait_that_runs_out_is_reported_and_leaves_no_results(mx, monkeypatch, P, N):
    """DL_TEST_STALL makes one thread of the first CTA wait, for 25 ms, on a barrier that nothing arrives on.  No fault
    is involved: the CTA lets its copies and products land and leaves, and the calls after the report run as ever."""
    from linear_attention_recurrent_gdn_gb300 import deltalog as dl
    g = torch.Generator().manual_seed(P)
    T, n, H = 250, 3, 2
    args = scan_inputs(g, T, n, H, P, N)
    start = rnd(g, n, H, P, N).cuda()
    good = start.clone()
    want = mx.ssm(*args, slots=[0, 1, 2], state=good)
    mx.sync()
    pool, out = start.clone(), torch.full_like(want, 7.0)
    monkeypatch.setenv("DL_TEST_WAIT_MS", "50")
    monkeypatch.setenv("DL_TEST_STALL", "1")
    mx.ssm(*args, slots=[0, 1, 2], state=pool, out=out)
    monkeypatch.delenv("DL_TEST_STALL")
    monkeypatch.delenv("DL_TEST_WAIT_MS")
    with pytest.raises(dl.DeltaLogError) as e:
        mx.sync()
    assert e.value.status == dl.EDEVICE and "device status %d" % dl.DEV_TEST_STALL in str(e.value)
    # the first CTA had 64 state rows of row 0's first head: none of its results; everything else
    p = min(P, 64)
    assert (out[:, 0, 0, :p] == 7).all() and torch.equal(pool[0, 0, :p], start[0, 0, :p])
    out[:, 0, 0, :p], pool[0, 0, :p] = want[:, 0, 0, :p], good[0, 0, :p]
    assert torch.equal(out, want) and torch.equal(pool, good)
    mx.sync()                                                          # reported once
    pool = start.clone()
    assert torch.equal(mx.ssm(*args, slots=[0, 1, 2], state=pool), want) and torch.equal(pool, good)
    mx.sync()


def test_launches_after_a_wait_that_ran_out(mx, monkeypatch):
    """Segments: the launches after the first find the error and may leave early, and every one of them ends."""
    from linear_attention_recurrent_gdn_gb300 import deltalog as dl
    g = torch.Generator().manual_seed(0)
    args = scan_inputs(g, 1200, 2, 4, 64, 128)
    want = mx.ssm(*args)
    mx.sync()
    monkeypatch.setenv("DL_TEST_WAIT_MS", "50")
    monkeypatch.setenv("DL_TEST_STALL", "1")
    mx.ssm(*args)
    monkeypatch.delenv("DL_TEST_STALL")
    monkeypatch.delenv("DL_TEST_WAIT_MS")
    for _ in range(3):
        mx.ssm(*args)
    with pytest.raises(dl.DeltaLogError) as e:
        mx.sync()
    assert e.value.status == dl.EDEVICE
    assert torch.equal(mx.ssm(*args), want)
    mx.sync()


# ------------------------------------------------------- infinities and NaN --
INF, NAN = float("inf"), float("nan")
# which input, at which token, and its value there (one head, group, channel or state column of it)
ODD = [("x", 3, INF), ("x", 77, NAN), ("x", 31, -INF), ("B", 64, INF), ("B", 5, NAN), ("C", 33, INF), ("C", 90, NAN),
       ("dt", 10, INF), ("dt", 95, NAN), ("x", 127, INF), ("x", 128, INF), ("state", 0, INF)]


@pytest.mark.parametrize("dtype,P,N", [("bf16", 64, 64), ("bf16", 72, 40), ("bf16", 40, 24), ("bf16", 20, 13),
                                       ("fp16", 40, 24), ("fp32", 64, 64), ("fp32", 20, 13)])
@pytest.mark.parametrize("lengths", [[140, 131], [700]])       # whole rows, and a row in segments
@pytest.mark.parametrize("what,at,value", ODD)
def test_infinities_and_nan_reach_what_follows_from_them(mx, dtype, P, N, lengths, what, at, value):
    """Tokens before them, other rows, heads, channels and state columns are as without them; an output that
    depends on one is not finite, and the state is as it is defined: an infinity of its sign, or a NaN."""
    g = torch.Generator().manual_seed(at)
    dt, H = DT[dtype], 2
    rows = []
    for t in lengths:
        rows.append([rnd(g, t, H, P, dtype=dt), rnd(g, t, H) * 0.01 + 0.02, rnd(g, t, 1, N, dtype=dt),
                     rnd(g, t, 1, N, dtype=dt)])
    S0 = rnd(g, len(rows), H, P, N)
    index = {"x": (at, 1, P // 2), "dt": (at, 1), "B": (at, 0, N // 3), "C": (at, 0, N // 3)}
    if what == "state":
        S0[0, 1, P // 2, N // 3] = value
    else:
        rows[0][("x", "dt", "B", "C").index(what)][index[what]] = value
    A = torch.tensor([-1.0, -0.5])
    D = rnd(g, H)
    ys, pool = run_packed(mx, rows, A, D, S0, list(range(len(rows))))
    for i, r in enumerate(rows):
        want, S, ymag, Smag = ref.ssm_row(r[0], r[1], A, r[2], r[3], D, S0[i], None, False)
        steps = 3 * r[0].shape[0] + 16
        fine, sfine = torch.isfinite(want), torch.isfinite(S)
        assert fine.any() and sfine.any()
        assert torch.equal(torch.isfinite(ys[i]), fine), "y of row %d: not finite in other places" % i
        off = (ys[i].double() - want).abs()[fine]
        tol = half(dt) * want.abs() + 1e-30 + ((steps + N) * U + (1.01 * half(dt) if dtype == "bf16" else 0)) * ymag
        if dtype == "fp16":
            tol = tol + 2.0 ** -24
        assert (off <= tol[fine]).all(), "y of row %d" % i
        got = pool[i].double()
        assert torch.equal(torch.isnan(got), torch.isnan(S)), "state of row %d: NaN in other places" % i
        assert torch.equal(got[torch.isinf(S)], S[torch.isinf(S)]), "state of row %d: infinities" % i
        assert ((got - S).abs()[sfine] <= (steps * U * Smag + 1e-30)[sfine]).all(), "state of row %d" % i
