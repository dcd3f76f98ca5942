"""The attention calls beside their values: refusals on CUDA tensors, graphs, streams, waits that run out, offsets past
32 bits."""
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
    return attention


@pytest.fixture(scope="module")
def s():
    return Setup([40, 70], 2, 64, 16, "bf16", seed=1)


def test_refusals(at, s):
    k, v, table, lengths, slots = s.args()
    q, _ = s.queries((2,), 4)
    p, _ = s.queries((5, 2), 4)
    starts = s.dev([0, 3, 10])
    bad = [
        (ValueError, "dimensions", lambda: at.attend_step(q[0], k, v, table, lengths, slots)),
        (ValueError, "rows", lambda: at.attend_step(q[:1], k, v, table, lengths, slots)),
        (ValueError, "not supported", lambda: at.attend_step(q.double(), k, v, table, lengths, slots)),
        (ValueError, "k_pages", lambda: at.attend_step(q.half(), k, v, table, lengths, slots)),
        (ValueError, "heads of", lambda: at.attend_step(q[..., :32].contiguous(), k, v, table, lengths, slots)),
        (ValueError, "v_pages", lambda: at.attend_step(q, k, v[1:], table, lengths, slots)),
        (TypeError, "k_pages", lambda: at.attend_step(q, k[0], v, table, lengths, slots)),
        (ValueError, "contiguous", lambda: at.attend_step(q, k.transpose(2, 3), v.transpose(2, 3), table, lengths, slots)),
        (ValueError, "contiguous", lambda: at.attend_step(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, table, lengths, slots)),
        (ValueError, "table", lambda: at.attend_step(q, k, v, table.long(), lengths, slots)),
        (ValueError, "lengths", lambda: at.attend_step(q, k, v, table, lengths[1:], slots)),
        (TypeError, "slots", lambda: at.attend_step(q, k, v, table, lengths, slots.cpu())),
        (ValueError, "window", lambda: at.attend_step(q, k, v, table, lengths, slots, window=0)),
        (RuntimeError, "first tokens", lambda: at.attend_step(q, k, v, table, lengths, slots, window=3, sinks=-1)),
        (RuntimeError, "scale", lambda: at.attend_step(q, k, v, table, lengths, slots, scale=-1.0)),
        (RuntimeError, "heads", lambda: at.attend_step(q[:, :3], k, v, table, lengths, slots)),
        (ValueError, "out", lambda: at.attend_step(q, k, v, table, lengths, slots, out=q.float())),
        (ValueError, "starts", lambda: at.attend(q, k, v, table, lengths, slots)),
        (ValueError, "starts", lambda: at.attend(q, k, v, table, lengths, slots, starts=starts[1:])),
        (ValueError, "starts", lambda: at.attend(p, k, v, table, lengths, slots, starts=starts)),
        (ValueError, "tokens", lambda: at.attend(q, k, v, table, lengths, slots, starts=starts, tokens=slots)),
        (ValueError, "tokens", lambda: at.attend(p, k, v, table, lengths, slots, tokens=slots[:1])),
        (ValueError, "where", lambda: at.append(q[:1, :2], q[:1, :2], k, v, slots)),
        (ValueError, "expanded", lambda: at.append(q[:1, :2], q[:1, :2], k[:1].expand(3, -1, -1, -1),
                                                   v[:1].expand(3, -1, -1, -1), slots[:1])),
        (ValueError, "size", lambda: at.extend(slots, None, (3, 4), table, lengths, lengths, page_size=16)),
        (ValueError, "tokens", lambda: at.extend(slots, starts, 9, table, lengths, lengths, page_size=16)),
        (RuntimeError, "power of two", lambda: at.extend(slots, None, None, table, lengths, lengths, page_size=20)),
        (ValueError, "no rows", lambda: at.extend(slots[:0], None, None, table, lengths, lengths, page_size=16)),
        (ValueError, "differentiated", lambda: at.attend_step(q.clone().requires_grad_(), k, v, table, lengths, slots)),
        (ValueError, "differentiated", lambda: at.attend_step(q, k.clone().requires_grad_(), v, table, lengths, slots)),
    ]
    before = [t.clone() for t in (table, lengths)]
    for error, word, call in bad:
        with pytest.raises(error, match=word):
            call()
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(q, torch.ones_like(q))
        with pytest.raises(ValueError, match="differentiated"):
            at.attend_step(dual, k, v, table, lengths, slots)
    at.sync()
    assert torch.equal(before[0], table) and torch.equal(before[1], lengths)


def test_no_rows_and_no_tokens(at, s):
    k, v, table, lengths, slots = s.args()
    none = slots[:0]
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert at.attend_step(q, k, v, table, lengths, none).shape == q.shape
    assert at.attend(q, k, v, table, lengths, slots, starts=s.dev([0, 0, 0])).shape == q.shape
    assert at.attend(q[None], k, v, table, lengths, none).shape == (1, 0, 4, 64)
    at.append(q[:, :2], q[:, :2], k, v, none)
    at.truncate(none, None, table, lengths, lengths, page_size=16)
    at.sync()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 256), ("fp32", 64)])
def test_captured_prompts_follow_their_tables(at, dtype, d):
    """A graph of packed pieces, split over the keys, replayed for other rows, tokens and lengths."""
    a = Setup([900, 64, 300, 5], 2, d, 16, dtype, seed=d)
    k, v, table, lengths, slots = a.args()
    q, host = a.queries((90,), 4)
    starts = a.dev([0, 1, 2, 3, 4])
    graph = torch.cuda.CUDAGraph()
    at.attend(q, k, v, table, lengths, slots, starts=starts)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o = at.attend(q, k, v, table, lengths, slots, starts=starts)
    for tokens in ([90, 0, 0, 0], [1, 60, 20, 5], [0, 0, 90, 0], [3, 3, 3, 3]):
        begin = [0]
        for t in tokens:
            begin.append(begin[-1] + t)
        starts.copy_(a.dev(begin))
        graph.replay()
        check_rows(a, host, o.cpu(), tokens, begin, None, 0)
    at.sync()


def test_captured_maps_of_two_launches(at):
    state = at.new_tables(3, 2000, 4000)
    slots, tokens = torch.tensor([2, 0], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    at.extend(slots, tokens, 6000, *state, page_size=16)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        starts, where, positions = at.extend(slots, tokens, 6000, *state, page_size=16)
    t = model.Tables(*(x.tolist() for x in state), 16)
    for counts in ([3000, 3000], [5, 0], [0, 6000]):
        tokens.copy_(torch.tensor(counts))
        graph.replay()
        want = [c for row in t.extend([2, 0], counts) for c in row]
        n = len(want)
        assert where.tolist() == [c[0] for c in want] + [-1] * (6000 - n)
        assert positions.tolist() == [c[1] for c in want] + [-1] * (6000 - n) and starts.tolist() == [0, counts[0], n]
    at.sync()


def test_two_streams_at_once(at):
    """Calls on two streams keep apart: each has a workspace of its own."""
    sets = [Setup([3000 + 17 * i, 70], 2, 128, 64, "bf16", seed=i) for i in range(2)]
    qs = [x.queries((2,), 8) for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    args = [x.args() for x in sets]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(at.attend_step(qs[i][0], *args[i]))
                outs[i].append(at.attend(qs[i][0], *args[i], starts=sets[i].dev([0, 1, 2])))
    torch.cuda.synchronize()
    for x, (_, host), got in zip(sets, qs, outs):
        for o in got[::2]:
            assert torch.equal(o, got[0])
        for o in got[1::2]:
            assert torch.equal(o, got[1])
        check_rows(x, host, got[0].cpu(), [1, 1], [0, 1], None, 0)
        check_rows(x, host, got[1].cpu(), [1, 1], [0, 1], None, 0)
    at.sync()


def test_results_repeat(at):
    """The order of every sum is set by the sizes."""
    s = Setup([5000, 900, 33], 2, 64, 16, "fp16", seed=3)
    q, _ = s.queries((3,), 10)
    p, _ = s.queries((60,), 10)
    starts = s.dev([0, 20, 40, 60])
    one = [at.attend_step(q, *s.args(), window=700, sinks=3), at.attend(p, *s.args(), starts=starts)]
    for _ in range(5):
        two = [at.attend_step(q, *s.args(), window=700, sinks=3), at.attend(p, *s.args(), starts=starts)]
        assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_a_wait_that_runs_out_is_reported(at, monkeypatch):
    """The tensor-core kernel leaves without results, the report names it, and the next call is right."""
    s = Setup([200], 2, 128, 64, "bf16", seed=7)
    q, host = s.queries((200,), 8)
    run = lambda: at.attend(q, *s.args(), starts=s.dev([0, 200]))  # noqa: E731
    run()
    at.sync()
    monkeypatch.setenv("DL_TEST_STALL", "1")
    monkeypatch.setenv("DL_TEST_WAIT_MS", "40")
    run()
    with pytest.raises(Exception, match="status 5"):
        at.sync()
    monkeypatch.delenv("DL_TEST_STALL")
    monkeypatch.delenv("DL_TEST_WAIT_MS")
    at.sync()
    check_rows(s, host, run().cpu(), [200], [0], None, 0)
    at.sync()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_calls_behind_an_unread_report_end(at, monkeypatch, d):
    """Waits end early once one has run out; every role still ends its copies and products before its CTA leaves."""
    s = Setup([700, 90, 1], 2, d, 32, "bf16", seed=d)
    q, host = s.queries((120,), 8)
    run = lambda: at.attend(q, *s.args(), starts=s.dev([0, 70, 119, 120]))  # noqa: E731
    run()
    at.sync()
    monkeypatch.setenv("DL_TEST_STALL", "1")
    monkeypatch.setenv("DL_TEST_WAIT_MS", "20")
    run()
    monkeypatch.delenv("DL_TEST_STALL")
    monkeypatch.delenv("DL_TEST_WAIT_MS")
    for _ in range(20):
        run()
    with pytest.raises(Exception, match="status 5"):
        at.sync()
    check_rows(s, host, run().cpu(), [70, 49, 1], [0, 70, 119], None, 0)
    at.sync()


@pytest.mark.parametrize("total,reported", [(128, False), (1024, True)])
@pytest.mark.parametrize("d", [64, 256])
def test_starts_that_go_back_and_forth(at, d, total, reported):
    """16 rows that claim the same tokens: 16 ceil(total / tile) tiles, where total / tile + 32 are the most of a call
    (tiles of 128 tokens, and of 64 for heads of 256).  More are reported: the workspace has no room for their parts."""
    rows, tile = 32, 64 if d == 256 else 128
    assert (16 * (total // tile) > total // tile + rows) == reported
    s = Setup([4000] * rows, 1, d, 64, "bf16", seed=d)
    q, host = s.queries((total,), 2)
    out = at.attend(q, *s.args(), starts=s.dev([0, total] * 16 + [0]))
    if reported:
        with pytest.raises(Exception, match="tokens"):
            at.sync()
    else:
        at.sync()
    starts = list(range(0, total + 1, total // rows))
    at.attend(q, *s.args(), starts=s.dev(starts), out=out)
    at.sync()
    check_rows(s, host, out.cpu(), [total // rows] * rows, starts[:-1], None, 0)


@pytest.mark.parametrize("what", ["queries", "rows", "heads", "pages"])
def test_expanded_inputs(at, what):
    """Inputs whose entries share their memory are read like any others."""
    s = Setup([16, 16], 2, 64, 16, "bf16", seed=2, spare=0)
    k, v, table, lengths, slots = s.args()
    q, host = s.queries((3, 2), 4)
    if what == "queries":
        q, host = q[:1].expand(3, -1, -1, -1), host[:1].expand(3, -1, -1, -1)
    elif what == "rows":
        q, host = q[:, :1].expand(-1, 2, -1, -1), host[:, :1].expand(-1, 2, -1, -1)
    elif what == "heads":
        k, v = k[:, :1].expand(-1, 2, -1, -1), v[:, :1].expand(-1, 2, -1, -1)
        s.k, s.v = ([x[:, :1].expand(-1, 2, -1) for x in t] for t in (s.k, s.v))
    else:
        page = s.table[s.slots[0]][0]
        k, v = (t[page:page + 1].expand(2, -1, -1, -1) for t in (k, v))
        s.k, s.v = ([t[0], t[0]] for t in (s.k, s.v))
    o = at.attend(q, k, v, table, lengths, slots)
    last = at.attend_step(q[2], k, v, table, lengths, slots)
    at.sync()
    for i in range(2):
        ref, mag, big = model.attend_row(host[:, i], s.k[i], s.v[i], torch.arange(13, 16))
        tol = bound(ref, mag, big, s.dt, 64, 16)
        check(o[:, i], ref, tol)
        check(last[i:i + 1], ref[2:], tol[2:])


@pytest.mark.parametrize("kind", ["step", "attend", "simt"])
def test_offsets_past_32_bits(at, kind):
    """A slot's pages at both ends of pools of more than 2^31 elements."""
    G, page, d, num_pages = 8, 256, 128, 8300                   # 2.18e9 elements each
    dtype = torch.bfloat16
    k, v = (torch.zeros(num_pages, G, page, d, dtype=dtype, device="cuda") for _ in range(2))
    L = 700
    pages = [num_pages - 1, 0, num_pages - 2]
    gen = torch.Generator().manual_seed(4)
    kk, vv = (torch.randn(L, G, d, generator=gen).to(dtype) for _ in range(2))
    table = torch.tensor([pages], dtype=torch.int32, device="cuda")
    where = torch.tensor([pages[p // page] * page + p % page for p in range(L)], dtype=torch.int32, device="cuda")
    at.append(kk.cuda(), vv.cuda(), k, v, where)
    assert torch.equal(k[num_pages - 1, :, 3].cpu(), kk[3]) and torch.equal(v[num_pages - 2, :, 100].cpu(), vv[612])
    lengths, slots = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (L, 0))
    n = 1 if kind == "step" else 20
    q = torch.randn(n, 16, d, generator=gen).to(dtype)
    args = (k, v, table, lengths, slots)
    if kind == "step":
        o = at.attend_step(q.cuda(), *args)
    elif kind == "attend":
        o = at.attend(q.cuda(), *args, starts=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    else:
        wide = torch.zeros(n, 16, d + 1, dtype=dtype, device="cuda")[:, :, 1:]     # heads apart: no vectors
        odd = torch.zeros(n * 16 * d + 1, dtype=dtype, device="cuda")[1:].view(n, 16, d)
        assert wide.shape == odd.shape
        odd.copy_(q)
        o = at.attend(odd, *args, starts=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    at.sync()
    ref, mag, big = model.attend_row(q, kk, vv, torch.arange(L - n, L))
    check(o.cpu(), ref, bound(ref, mag, big, dtype, d, L))


def test_append_at_the_ends_of_an_int32_place(at):
    """Places up to 2^31 - 1 cannot be wrapped: negative ones are left out, those past the pool are reported."""
    pools = [torch.zeros(4, 1, 16, 64, device="cuda") for _ in range(2)]
    kv = torch.ones(3, 1, 64, device="cuda")
    at.append(kv, kv, *pools, torch.tensor([-2 ** 31, 2 ** 31 - 1, 63], dtype=torch.int32, device="cuda"))
    with pytest.raises(Exception, match="page"):
        at.sync()
    assert pools[0].sum() == 64 and (pools[1][3, 0, 15] == 1).all()
