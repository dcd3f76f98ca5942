"""Attention over pages against its definition in 64 bits."""
import itertools

import pytest
import torch

from attention_helpers import DT, Setup, bound, check, check_rows
from oracle import attention_model as model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def at():
    from linear_attention_recurrent_gdn_gb300 import build
    build.build()
    from linear_attention_recurrent_gdn_gb300 import attention
    return attention


def _starts(tokens):
    return list(itertools.accumulate([0] + list(tokens)))


# ------------------------------------------------------------------ one token --
STEP = [
    # after, H, G, d, page, window, sinks
    ([1], 1, 1, 64, 16, None, 0),
    ([0, 1, 2, 15, 16, 17, 63, 64, 65], 8, 2, 128, 16, None, 0),
    ([127, 128, 129, 500, 0, 1000], 32, 8, 128, 64, None, 0),
    ([33, 700, 64], 40, 8, 64, 16, 50, 4),
    ([33, 700, 64, 0, 1], 14, 2, 128, 32, 1, 0),
    ([300, 1000], 4, 4, 128, 128, 300, 130),
    ([257, 90], 32, 1, 256, 256, None, 0),
    ([257, 90, 31], 24, 8, 256, 64, 40, 1),
    ([70, 300], 16, 1, 96, 16, None, 0),
    ([70, 300], 34, 2, 80, 16, 100, 3),
    ([70, 130], 6, 3, 20, 16, None, 0),
    ([70, 130, 5], 4, 2, 33, 16, 20, 2),
    ([3000], 8, 1, 64, 64, None, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("after,H,G,d,page,window,sinks", STEP)
def test_step(at, after, H, G, d, page, window, sinks, dtype):
    s = Setup(after, G, d, page, dtype, seed=len(after) + d)
    q, host = s.queries((len(after),), H)
    o = at.attend_step(q, *s.args(), window=window, sinks=sinks)
    at.sync()
    check_rows(s, host, o.cpu(), [1] * len(after), range(len(after)), window, sinks)
    assert not o[[i for i, a in enumerate(after) if a == 0]].any()


@pytest.mark.parametrize("pool", ["tokens_first", "odd"])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("fp32", 64)])
def test_step_strides(at, pool, dtype, d):
    after = [40, 513, 1, 200]
    s = Setup(after, 2, d, 16, dtype, seed=5, pool=pool)
    q, host = s.queries((4,), 6, fused=3)
    wide = torch.full((4, 9, d), 7.0, dtype=s.dt, device="cuda")
    o = at.attend_step(q, *s.args(), window=400, sinks=2, out=wide[:, 1:7])
    at.sync()
    assert o.data_ptr() == wide[:, 1:7].data_ptr()
    check_rows(s, host, o.cpu(), [1] * 4, range(4), 400, 2)
    assert (wide[:, 0] == 7).all() and (wide[:, 7:] == 7).all()


def test_step_many_rows(at):
    after = [(i * 37) % 301 for i in range(1024)]
    s = Setup(after, 1, 64, 16, "bf16", seed=3)
    q, host = s.queries((1024,), 2)
    o = at.attend_step(q, *s.args())
    at.sync()
    check_rows(s, host, o.cpu(), [1] * 1024, range(1024), None, 0)


def test_step_scale(at):
    s = Setup([200, 77], 2, 128, 32, "bf16", seed=9)
    q, host = s.queries((2,), 8, scale=1.0)
    o = at.attend_step(q, *s.args(), scale=0.3)
    check_rows(s, host, o.cpu(), [1, 1], range(2), None, 0, 0.3)


# -------------------------------------------------------------------- prompts --
PROMPT = [
    # tokens, before, H, G, d, page, window, sinks
    ([1], [0], 1, 1, 64, 16, None, 0),
    ([5, 3], [0, 0], 8, 2, 128, 16, None, 0),
    ([130, 0, 257, 1, 64], [0, 9, 0, 300, 0], 8, 2, 128, 64, None, 0),
    ([300], [0], 32, 8, 128, 64, None, 0),
    ([129, 200], [500, 77], 10, 2, 64, 16, 100, 4),
    ([129, 200], [500, 0], 14, 2, 128, 32, 1, 0),
    ([260, 20], [30, 700], 4, 4, 128, 128, 129, 130),
    ([140, 33], [0, 200], 8, 2, 256, 64, None, 0),
    ([140, 33], [0, 200], 16, 1, 256, 16, 70, 3),
    ([70, 65], [40, 0], 6, 2, 80, 16, 100, 3),
    ([70, 65], [40, 0], 6, 2, 96, 32, None, 0),
    ([70, 33], [0, 5], 6, 3, 20, 16, 30, 0),
    ([40, 33], [0, 50], 2, 1, 33, 16, None, 0),
    ([7], [2900], 16, 2, 128, 64, None, 0),
    ([40, 3], [0, 100], 80, 1, 64, 16, None, 0),
    ([3, 2], [10, 0], 200, 1, 128, 16, None, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,before,H,G,d,page,window,sinks", PROMPT)
def test_packed(at, tokens, before, H, G, d, page, window, sinks, dtype):
    s = Setup([t + b for t, b in zip(tokens, before)], G, d, page, dtype, seed=sum(tokens) + d)
    starts = _starts(tokens)
    q, host = s.queries((starts[-1] + 3,), H)
    out = torch.full_like(q, 7.0)
    o = at.attend(q, *s.args(), starts=s.dev(starts), window=window, sinks=sinks, out=out)
    at.sync()
    check_rows(s, host, o.cpu(), tokens, starts, window, sinks)
    assert (o[starts[-1]:] == 7).all()                   # behind the last row


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("T,n,H,G,d,window", [(1, 3, 4, 2, 128, None), (150, 3, 8, 2, 128, None), (70, 2, 10, 2, 64, 33),
                                              (70, 2, 4, 2, 256, None)])
def test_token_major(at, T, n, H, G, d, window, given, dtype):
    tokens = [(T * (i + 1) * 7) % (T + 1) for i in range(n)] if given else [T] * n
    s = Setup([t + 20 * i for i, t in enumerate(tokens)], G, d, 16, dtype, seed=T)
    q, host = s.queries((T, n), H, fused=2)
    out = torch.full((T, n, H, d), 7.0, dtype=s.dt, device="cuda")
    o = at.attend(q, *s.args(), tokens=s.dev(tokens) if given else None, window=window, out=out)
    at.sync()
    for i, t in enumerate(tokens):
        ref, mag, big = model.attend_row(host[:t, i], s.k[i], s.v[i], torch.arange(s.after[i] - t, s.after[i]), window)
        check(o[:t, i], ref, bound(ref, mag, big, s.dt, d, s.after[i]), "row %d" % i)
        assert (o[t:, i] == 7).all()


@pytest.mark.parametrize("pool", ["tokens_first", "odd"])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
def test_packed_strides(at, pool, dtype, d):
    tokens = [33, 150]
    s = Setup([40, 150], 2, d, 16, dtype, seed=8, pool=pool)
    q, host = s.queries((183,), 4, fused=1)
    o = at.attend(q, *s.args(), starts=s.dev([0, 33, 183]))
    at.sync()
    check_rows(s, host, o.cpu(), tokens, [0, 33], None, 0)


def test_tokens_ahead_of_their_slot_see_nothing(at):
    """A row with more tokens than its slot holds: those at negative positions are zero."""
    s = Setup([6], 2, 64, 16, "bf16", seed=1)
    q, host = s.queries((10,), 4)
    o = at.attend(q, *s.args(), starts=s.dev([0, 10])).cpu()
    at.sync()
    assert not o[:4].any()
    check_rows(s, host[4:], o[4:], [6], [0], None, 0)


# ------------------------------------------------- infinities, NaN, low scores --
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_what_is_not_seen_does_not_reach(at, dtype, bad, d):
    """Values that are not finite at key 100: tokens that do not see it are as they would be without it."""
    s = Setup([200], 2, d, 32, dtype, seed=d)
    q, host = s.queries((200,), 4)
    page, off = s.table[s.slots[0]][100 // 32], 100 % 32
    for pools in ((s.k_pages,), (s.v_pages,), (s.k_pages, s.v_pages)):
        saved = [p[page, :, off].clone() for p in pools]
        for p in pools:
            p[page, 1, off, 3] = bad
        for window, sinks in ((None, 0), (30, 0), (30, 101), (30, 100)):
            o = at.attend(q, *s.args(), starts=s.dev([0, 200]), window=window, sinks=sinks).cpu()
            at.sync()
            see = [100 <= p and (window is None or 100 > p - window or 100 < sinks) for p in range(200)]
            ref, mag, big = model.attend_row(host, s.k[0], s.v[0], torch.arange(200), window, sinks)
            tol = bound(ref, mag, big, s.dt, d, 200)
            blind = [p for p in range(200) if not see[p]]
            check(o[blind], ref[blind], tol[blind], "tokens that do not see it")
            check(o[:, :2], ref[:, :2], tol[:, :2], "the other head")
            if window is not None and sinks < 101:
                last = at.attend_step(q[199:], *s.args(), window=window, sinks=sinks).cpu()
                check(last, ref[199:], tol[199:], "the last token alone")
            elif pools[0] is s.v_pages and bad == bad:
                assert (o[see, 2:, 3] == bad).all()
            elif bad != bad:
                assert torch.isnan(o[see, 2:].float()).any(-1).all()
        for p, old in zip(pools, saved):
            p[page, :, off] = old


@pytest.mark.parametrize("dtype,low", [("bf16", torch.finfo(torch.bfloat16).min), ("fp32", torch.finfo(torch.float32).min / 2),
                                       ("fp16", -60000.0)])
def test_scores_at_the_type_s_end(at, dtype, low):
    """Scores as low as the type goes for some keys, and for all of them: weights come from their differences."""
    s = Setup([90], 1, 64, 16, dtype, seed=2)
    pages = s.table[s.slots[0]]
    for keys in (range(0, 90, 2), range(90)):
        for p in keys:
            s.k_pages[pages[p // 16], 0, p % 16] = 0
            s.k_pages[pages[p // 16], 0, p % 16, 0] = low
            s.k[0][p] = 0
            s.k[0][p, 0, 0] = low
        q, host = s.queries((90,), 2, scale=0.0)
        q[..., 0] = 1
        host[..., 0] = 1
        o = at.attend(q, *s.args(), starts=s.dev([0, 90])).cpu()
        last = at.attend_step(q[89:], *s.args()).cpu()
        at.sync()
        ref, mag, big = model.attend_row(host, s.k[0], s.v[0], torch.arange(90))
        tol = bound(ref, mag, big * 0, s.dt, 64, 90)     # products with 1 and 0: scores are exact but for their scaling
        check(o, ref, tol)
        check(last, ref[89:], tol[89:])


def test_scores_of_minus_infinity_alone_give_zero(at):
    s = Setup([20], 1, 64, 16, "bf16", seed=2)
    s.k_pages[:] = 0
    s.k_pages[..., 0] = float("-inf")
    q = torch.ones(20, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert not at.attend(q, *s.args(), starts=s.dev([0, 20])).any()
    assert not at.attend_step(q[19:], *s.args()).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_rising_and_falling_scores(at, dtype):
    """Scores that rise by far more than a weight's range, and fall again: the running maximum moves many times."""
    L, d = 700, 128
    s = Setup([L], 1, d, 64, dtype, seed=4)
    ramp = torch.cat([torch.linspace(-30, 30, 400), torch.linspace(30, -30, L - 400)])
    for p in range(L):
        s.k[0][p, 0, 0] = ramp[p].item()
        s.k_pages[s.table[s.slots[0]][p // 64], 0, p % 64, 0] = s.k[0][p, 0, 0].item()
    q, host = s.queries((L,), 4, scale=0.3)
    q[..., 0] = 20
    host[..., 0] = 20
    o = at.attend(q, *s.args(), starts=s.dev([0, L])).cpu()
    last = at.attend_step(q[L - 1:], *s.args()).cpu()
    at.sync()
    check_rows(s, host, o, [L], [0], None, 0)
    check_rows(s, host[L - 1:], last, [1], [0], None, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("level", [-400.0, 400.0])
@pytest.mark.parametrize("window,sinks", [(40, 0), (70, 3), (200, 0), (None, 0)])
def test_scores_far_from_zero_behind_keys_that_are_not_seen(at, dtype, level, window, sinks):
    """Rows that see nothing of their first blocks of keys, and then scores whose exponentials alone would be zero or
    infinite."""
    L, d = 500, 64
    s = Setup([L], 1, d, 16, dtype, seed=6)
    s.k[0][..., 0] = level / 20
    for p in range(L):
        s.k_pages[s.table[s.slots[0]][p // 16], 0, p % 16, 0] = level / 20
    q, host = s.queries((L,), 2, scale=0.5)
    q[..., 0] = 160
    host[..., 0] = 160
    o = at.attend(q, *s.args(), starts=s.dev([0, L]), window=window, sinks=sinks).cpu()
    last = at.attend_step(q[L - 1:], *s.args(), window=window, sinks=sinks).cpu()
    at.sync()
    check_rows(s, host, o, [L], [0], window, sinks)
    check_rows(s, host[L - 1:], last, [1], [0], window, sinks)


# ---------------------------------------------------------------- wrong tables --
def test_wrong_slots_lengths_and_pages_are_reported(at):
    from linear_attention_recurrent_gdn_gb300.deltalog import DeltaLogError
    s = Setup([40, 50], 2, 64, 16, "bf16", seed=1)
    q, _ = s.queries((2,), 4)
    k, v, table, lengths, slots = s.args()
    for j, value, word in ((0, 99, "slot"), (0, -1, "slot")):
        bad = slots.clone()
        bad[j] = value
        at.attend_step(q, k, v, table, lengths, bad)
        with pytest.raises(DeltaLogError, match=word):
            at.sync()
    for value in (-5, s.max_pages * 16 + 1):
        bad = lengths.clone()
        bad[s.slots[1]] = value
        at.attend_step(q, k, v, table, bad, slots)
        with pytest.raises(DeltaLogError, match="tokens"):
            at.sync()
    for value in (-1, s.num_pages, 0x7fffffff):
        bad = table.clone()
        bad[s.slots[0], 1] = value
        at.attend_step(q, k, v, bad, lengths, slots)
        with pytest.raises(DeltaLogError, match="page"):
            at.sync()
        at.attend(q, k, v, bad, lengths, slots, starts=s.dev([0, 1, 2]))
        with pytest.raises(DeltaLogError, match="page"):
            at.sync()
    for what, value, word in (("slots", 99, "slot"), ("slots", -1, "slot"), ("lengths", -5, "tokens"),
                              ("lengths", s.max_pages * 16 + 1, "tokens")):
        more = dict(lengths=lengths, slots=slots)
        bad = more[what].clone()
        bad[0 if what == "slots" else s.slots[1]] = value
        for x in (q, q.float()):                            # on the tensor cores, and not
            at.attend(x, k.to(x.dtype), v.to(x.dtype), table, **{**more, what: bad}, starts=s.dev([0, 1, 2]))
            with pytest.raises(DeltaLogError, match=word):
                at.sync()
    # starts that go backwards or past the tokens are held to them
    for starts in ([0, 5, 2], [-7, 1, 1 << 30], [2, 0, 1]):
        at.attend(q, k, v, table, lengths, slots, starts=s.dev(starts))
        torch.cuda.synchronize()
    at.sync()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("after,tokens,H,G", [([20000], [4], 8, 1), ([9000, 37, 1, 6000], [3, 2, 1, 5], 6, 2),
                                              ([30000, 12000], [1, 70], 4, 2)])
def test_few_tokens_behind_many_keys(at, d, after, tokens, H, G):
    """Keys split over all SMs: many parts of few rows to join, beside rows with one."""
    s = Setup(after, G, d, 64, "bf16", seed=d + len(after))
    starts = _starts(tokens)
    q, host = s.queries((sum(tokens),), H)
    out = at.attend(q, *s.args(), starts=s.dev(starts))
    check_rows(s, host, out.cpu(), tokens, starts[:-1], None, 0)
    assert torch.equal(out, at.attend(q, *s.args(), starts=s.dev(starts)))
    at.sync()


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("n", [32, 33, 64, 65, 100, 128, 129])
def test_many_rows_of_uneven_lengths(at, n, d):
    """Few tokens a row: up to 64 rows' keys are split by one plan; some rows are empty, a few long."""
    tokens = [(5 * i + 1) % 4 for i in range(n)]
    after = [t + (3000 + 7 * i if i % 31 == 5 else (37 * i) % 150) for i, t in enumerate(tokens)]
    s = Setup(after, 1, d, 64, "bf16", seed=n + d)
    starts = _starts(tokens)
    q, host = s.queries((sum(tokens),), 4)
    out = at.attend(q, *s.args(), starts=s.dev(starts))
    check_rows(s, host, out.cpu(), tokens, starts[:-1], None, 0)
    assert torch.equal(out, at.attend(q, *s.args(), starts=s.dev(starts)))
    at.sync()
