"""Block tables, slot maps and the append against their integer model, and a decode run of all of them together."""
import random

import pytest
import torch

from attention_helpers import DT, bound, check
from oracle import attention_model as model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def at():
    from linear_attention_recurrent_gdn_gb300 import build
    build.build()
    from linear_attention_recurrent_gdn_gb300 import attention
    return attention


def _dev(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Both:
    """The device's tables and the model's, compared after every call."""

    def __init__(self, at, num_slots, max_pages, num_pages, page):
        self.at, self.page, self.num_pages = at, page, num_pages
        self.state = at.new_tables(num_slots, max_pages, num_pages)
        self.model = model.Tables(*(t.tolist() for t in self.state), page)

    def compare(self):
        table, lengths, free = (t.tolist() for t in self.state)
        assert lengths == self.model.lengths
        assert free[0] == len(self.model.stack) and free[1:1 + free[0]] == self.model.stack
        for s, L in enumerate(lengths):
            held = -(-L // self.page)
            assert table[s][:held] == self.model.table[s][:held]
        pages = [p for s, L in enumerate(lengths) for p in table[s][:-(-L // self.page)]] + self.model.stack
        assert sorted(pages) == list(range(self.num_pages))

    def extend(self, slots, tokens, size):
        before = [t.clone() for t in self.state]
        got = self.at.extend(_dev(slots), None if tokens is None else _dev(tokens), size, *self.state, page_size=self.page)
        starts, where, positions = (t.tolist() for t in got)
        want = self.model.extend(slots, [1] * len(slots) if tokens is None else tokens)
        if want is None:
            with pytest.raises(Exception, match="DL_EDEVICE"):
                self.at.sync()
            assert all(torch.equal(a, b) for a, b in zip(before, self.state))
            assert not any(starts) and (got[1] == -1).all() and (got[2] == -1).all()
            return False
        self.at.sync()
        if isinstance(size, tuple):
            flat = [[row[t] if t < len(row) else (-1, -1) for row in want] for t in range(size[0])]
            assert where == [[c[0] for c in r] for r in flat] and positions == [[c[1] for c in r] for r in flat]
        else:
            flat = [c for row in want for c in row] if size is not None else [row[0] if row else (-1, -1) for row in want]
            flat += [(-1, -1)] * (len(where) - len(flat))
            assert where == [c[0] for c in flat] and positions == [c[1] for c in flat]
        sums = [0]
        for row in want:
            sums.append(sums[-1] + len(row))
        assert starts == sums
        self.compare()
        return True

    def truncate(self, slots, keep):
        self.at.truncate(_dev(slots), None if keep is None else _dev(keep), *self.state, page_size=self.page)
        self.model.truncate(slots, [0] * len(slots) if keep is None else keep)
        self.at.sync()
        self.compare()


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("seed", range(4))
def test_random_runs(at, page, seed):
    rng = random.Random(100 * page + seed)
    num_slots = rng.choice([1, 7, 40])
    b = Both(at, num_slots, 12, rng.choice([5, 8 * num_slots, 12 * num_slots]), page)
    done = 0
    for _ in range(40):
        n = rng.randint(1, num_slots)
        slots = rng.sample(range(num_slots), n)
        kind = rng.random()
        if kind < 0.3:
            b.truncate(slots, [rng.randint(0, b.model.lengths[s]) for s in slots] if rng.random() < 0.8 else None)
        elif kind < 0.6:
            done += b.extend(slots, rng.choice([None, [rng.randint(0, 1) for _ in slots]]), None)
        else:
            tokens = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, 5 * page)]) for _ in slots]
            size = (max(tokens) + rng.randint(1, 5), n) if rng.random() < 0.5 else sum(tokens) + rng.randint(0, 9)
            done += b.extend(slots, tokens, size)
    assert done


@pytest.mark.parametrize("n,page,packed", [(1, 16, True), (1, 16, False), (1024, 16, True), (1024, 64, False), (3, 256, True)])
def test_large_maps(at, n, page, packed):
    """More entries than one block writes, up to the most rows, with empty rows among them."""
    tokens = [(i * 7919) % 23 if n == 1024 else 9000 + 13 * i for i in range(n)]
    tokens[n // 2] += 5000 if packed else 0
    cap = max(tokens) // page + 2
    b = Both(at, n + 5, cap, sum(-(-t // page) for t in tokens) + 2 * n, page)
    slots = random.Random(n).sample(range(n + 5), n)
    assert b.extend(slots, [t % 5 for t in tokens], sum(t % 5 for t in tokens) + 1)
    later = [t - t % 5 for t in tokens]
    assert b.extend(slots, later, sum(later) if packed else (max(later), n))
    b.truncate(slots, [t // 2 for t in tokens])
    b.truncate(slots, None)


def test_calls_that_cannot_be_done_change_nothing(at):
    b = Both(at, 4, 3, 6, 16)
    assert b.extend([2, 0], [17, 40], 60)
    assert not b.extend([1, 1], [1, 1], 2)                    # named twice
    assert not b.extend([4], [1], 1) and not b.extend([-1], [1], 1)
    assert not b.extend([0], [9], 9)                          # the row is full
    assert not b.extend([1, 3], [16, 16], (16, 2))            # one page is left
    assert not b.extend([1], [-1], 4)
    for size in (4, (4, 1)):                                  # more than the maps hold
        before = [t.clone() for t in b.state]
        starts, where, _ = at.extend(_dev([1]), _dev([5]), size, *b.state, page_size=16)
        with pytest.raises(Exception, match="tokens"):
            at.sync()
        assert not starts.any() and (where == -1).all()
        assert all(torch.equal(x, y) for x, y in zip(before, b.state))
    for slots, keep in (([2, 2], [1, 1]), ([7], [0]), ([2], [18]), ([2], [-1])):
        before = [t.clone() for t in b.state]
        at.truncate(_dev(slots), _dev(keep), *b.state, page_size=16)
        with pytest.raises(Exception, match="DL_EDEVICE"):
            at.sync()
        assert all(torch.equal(x, y) for x, y in zip(before, b.state))
    assert b.extend([1], [16], 16)
    b.truncate([0, 1, 2, 3], None)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 20), ("fp32", 64), ("fp32", 33), ("bf16", 7)])
@pytest.mark.parametrize("pool", ["pages_first", "tokens_first"])
@pytest.mark.parametrize("lead", [(5,), (300,), (40, 3)])
def test_append(at, dtype, d, pool, lead):
    G, page, num_pages = 3, 16, 40
    gen = torch.Generator(device="cuda").manual_seed(d)
    k, v = (torch.randn(*lead, 2 * G, d, generator=gen, device="cuda").to(DT[dtype])[..., G * i:G * i + G, :] for i in (0, 1))
    count = k[..., 0, 0].numel()
    where = torch.randperm(num_pages * page, generator=torch.Generator().manual_seed(d))[:count].int()
    where[::7] = -1
    pools = [torch.full((num_pages, G, page, d), 3.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    if pool == "tokens_first":
        pools = [p.transpose(1, 2).contiguous().transpose(1, 2) for p in pools]
    want = [p.clone() for p in pools]
    at.append(k, v, *pools, where.view(lead).cuda())
    at.sync()
    for w, new in zip(want, (k, v)):
        for j, (x, row) in enumerate(zip(where.tolist(), new.reshape(count, G, d))):
            if x >= 0:
                w[x // page, :, x % page] = row
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


def test_append_places_out_of_range_are_reported(at):
    pools = [torch.zeros(4, 1, 16, 64, device="cuda") for _ in range(2)]
    kv = torch.ones(2, 1, 64, device="cuda")
    at.append(kv, kv, *pools, _dev([64, 3]))
    with pytest.raises(Exception, match="page"):
        at.sync()
    assert pools[0].sum() == 64 and (pools[0][0, 0, 3] == 1).all()


@pytest.mark.parametrize("dtype,d,window,sinks", [("bf16", 128, None, 0), ("fp16", 64, 40, 4), ("fp32", 40, None, 0)])
def test_prompts_pieces_and_single_tokens_together(at, dtype, d, window, sinks):
    """Prompts, a later piece, single tokens, a row cut back and written again: every output is the whole row's."""
    H, G, page, slots = 4, 2, 16, [3, 0, 5]
    plan = [[70, 9, 33], [20, 50, 1], [1, 1, 1], [1, 1, 1], [1, 1, 1], [1, 1, 1]]
    gen = torch.Generator().manual_seed(d)
    total = [sum(p[i] for p in plan) for i in range(3)]
    data = [[torch.randn(t, h, d, generator=gen).to(DT[dtype]) for h in (H, G, G)] for t in total]
    state = at.new_tables(6, 40, 60)
    pools = [torch.full((60, G, page, d), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2)]
    more = dict(window=window, sinks=sinks)
    done, outs = [0, 0, 0], [[], [], []]

    def run(tokens):
        parts = [[x[a:a + t] for x in row] for row, a, t in zip(data, done, tokens)]
        q, k, v = (torch.cat([p[j] for p in parts]).cuda() for j in range(3))
        one = tokens == [1, 1, 1]
        starts, where, positions = at.extend(_dev(slots), None if one else _dev(tokens), None if one else len(q), *state,
                                             page_size=page)
        at.append(k, v, *pools, where)
        args = (q, *pools, *state[:2], _dev(slots))
        o = (at.attend_step(*args, **more) if one else at.attend(*args, starts=starts, **more)).cpu()
        assert positions.tolist() == [p for a, t in zip(done, tokens) for p in range(a, a + t)]
        for i, part in enumerate(o.split(tokens)):
            outs[i].append(part)
            done[i] += tokens[i]

    for tokens in plan[:4]:
        run(tokens)
    at.truncate(_dev([slots[1]]), _dev([done[1] - 2]), *state, page_size=page)
    done[1] -= 2
    outs[1] = [torch.cat(outs[1])[:-2]]
    for _ in range(2):
        run([1, 1, 1])
    at.sync()
    for i in range(3):
        q, k, v = (x[:done[i]] for x in data[i])
        o, mag, big = model.attend_row(q, k, v, torch.arange(done[i]), window, sinks)
        check(torch.cat(outs[i]), o, bound(o, mag, big, DT[dtype], d, done[i]), "row %d" % i)


def test_a_captured_step_follows_its_tables(at):
    """One graph of extend, append and attention, replayed for other slots, lengths and tokens."""
    H, G, d, page, n = 8, 2, 128, 16, 3
    state = at.new_tables(8, 30, 100)
    pools = [torch.zeros(100, G, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, G, G))
    slots, counts = _dev([0, 1, 2]), _dev([0, 0, 0])

    def step():
        _, where, _ = at.extend(slots, counts, None, *state, page_size=page)
        at.append(k, v, *pools, where)
        return at.attend_step(q, *pools, *state[:2], slots)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    rows = [([], []) for _ in range(8)]
    rng = random.Random(5)
    for _ in range(60):
        chosen = rng.sample(range(8), n)
        live = [rng.random() < 0.8 for _ in range(n)]
        hq, hk, hv = (torch.randn(n, h, d, generator=gen).to(torch.bfloat16) for h in (H, G, G))
        for dst, src in ((q, hq), (k, hk), (v, hv)):
            dst.copy_(src)
        slots.copy_(_dev(chosen))
        counts.copy_(_dev([int(x) for x in live]))
        graph.replay()
        got = out.cpu()
        for i, s in enumerate(chosen):
            if live[i]:
                rows[s][0].append(hk[i])
                rows[s][1].append(hv[i])
            if not rows[s][0]:
                assert not got[i].any()
                continue
            kk, vv = (torch.stack(x) for x in rows[s])
            o, mag, big = model.attend_row(hq[i:i + 1], kk, vv, [len(kk) - 1])
            check(got[i:i + 1], o, bound(o, mag, big, torch.bfloat16, d, len(kk)))
    at.sync()


def test_another_stream(at):
    """Calls go to the current stream, behind what it holds."""
    state = at.new_tables(4, 8, 20)
    other = torch.cuda.Stream()
    x = torch.ones(1 << 24, device="cuda")
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        for _ in range(20):
            x = x * 1.0001
        slots.fill_(3)
        starts, where, _ = at.extend(slots, None, None, *state, page_size=16)
    other.synchronize()
    assert state[1].tolist() == [0, 0, 0, 1] and where.tolist() == [state[0][3, 0].item() * 16]
