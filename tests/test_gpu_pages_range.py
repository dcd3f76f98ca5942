"""Page numbers out of range on the stack of free pages and in the block table: no call hands them out, writes through
them or gives them back."""
import pytest
import torch

from oracle import attention_model as model

pytestmark = pytest.mark.gpu

PAGE, NUM_PAGES = 16, 6000
# Below the range, its end, one whose place would wrap to page 3 in 32 bits, and the type's end.
BAD = [-1, NUM_PAGES, (1 << 28) + 3, 0x7fffffff]


@pytest.fixture(scope="module")
def at():
    from linear_attention_recurrent_gdn_gb300 import build
    build.build()
    from linear_attention_recurrent_gdn_gb300 import attention
    attention.sync()
    return attention


def _dev(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _refused(at, state, call):
    """The call reports a page and leaves the tables as they were."""
    before = [t.clone() for t in state]
    got = call()
    with pytest.raises(Exception, match="page"):
        at.sync()
    assert all(torch.equal(a, b) for a, b in zip(before, state))
    return got


# Rows of 0, 20 and 32 tokens.  New ones: a few pages, and more than a block has threads; maps that one launch writes
# (up to 2048 entries) and that take a second.
CALLS = [([1, 13, 17], "packed"), ([1, 13, 17], "major"), ([900, 0, 800], "packed"), ([30000, 5, 20000], "packed"),
         ([30000, 5, 20000], "major")]


def _state(at):
    state = at.new_tables(5, 4000, NUM_PAGES)
    at.extend(_dev([4, 0, 2]), _dev([0, 20, 32]), 52, *state, page_size=PAGE)
    at.sync()
    return state


def _extend(at, state, tokens, layout):
    size = sum(tokens) if layout == "packed" else (max(tokens), 3)
    return at.extend(_dev([4, 0, 2]), _dev(tokens), size, *state, page_size=PAGE)


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("tokens,layout", CALLS)
@pytest.mark.parametrize("depth", ["first", "last"])
def test_extend_takes_no_page_out_of_range(at, tokens, layout, depth, bad):
    """The first or last page that the call would take off the stack."""
    state = _state(at)
    free = state[2]
    height = int(free[0])
    taken = sum(-(-(a + t) // PAGE) - -(-a // PAGE) for a, t in zip([0, 20, 32], tokens))
    place = height - (0 if depth == "first" else taken - 1)
    was = int(free[place])
    free[place] = bad
    starts, where, positions = _refused(at, state, lambda: _extend(at, state, tokens, layout))
    assert not starts.any() and (where == -1).all() and (positions == -1).all()
    # with a good page the same call goes through, whatever lies below what it takes
    free[place] = was
    free[height - taken] = bad
    _, where, _ = _extend(at, state, tokens, layout)
    at.sync()
    assert int((where >= 0).sum()) == sum(tokens) and int(where.max()) < NUM_PAGES * PAGE


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("tokens,layout", CALLS)
def test_extend_follows_no_table_entry_out_of_range(at, tokens, layout, bad):
    """The half-filled page of slot 0; the full last page of slot 2 is not written to any more."""
    state = _state(at)
    table = state[0]
    table[2, 1] = bad
    t = model.Tables(*(x.tolist() for x in state), PAGE)
    was = int(table[0, 1])
    table[0, 1] = bad
    if tokens[1]:
        starts, where, positions = _refused(at, state, lambda: _extend(at, state, tokens, layout))
        assert not starts.any() and (where == -1).all() and (positions == -1).all()
        table[0, 1] = was
    _, where, _ = _extend(at, state, tokens, layout)
    at.sync()
    want = t.extend([4, 0, 2], tokens)
    flat = [c[0] for r in want for c in r]
    if layout == "packed":
        assert where.tolist() == flat
    else:
        assert sorted(where[where >= 0].tolist()) == sorted(flat)


def test_a_wrapped_place_is_not_written(at):
    """Pages of 16: number 2^28 + 3 times 16 is place 48 in 32 bits, the first of page 3, which another row holds."""
    state = at.new_tables(2, 4, 8)
    at.extend(_dev([0]), _dev([64]), 64, *state, page_size=PAGE)
    assert 3 in state[0][0].tolist()
    pools = [torch.zeros(8, 1, PAGE, 64, device="cuda") for _ in range(2)]
    state[2][int(state[2][0])] = (1 << 28) + 3
    kv = torch.ones(1, 1, 64, device="cuda")
    _, where, _ = at.extend(_dev([1]), None, None, *state, page_size=PAGE)
    at.append(kv, kv, *pools, where)
    with pytest.raises(Exception, match="page"):
        at.sync()
    assert not pools[0].any() and not pools[1].any()


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("column", [2, 9, 900, 2999])
def test_truncate_returns_no_page_out_of_range(at, column, bad):
    """Early and late among thousands of pages that go back; kept ones and those behind the row are not looked at."""
    state = at.new_tables(3, 3010, NUM_PAGES)
    counts = [16 * 3000, 16 * 2500 - 3, 7]
    at.extend(_dev([1, 2, 0]), _dev(counts), sum(counts), *state, page_size=PAGE)
    at.sync()
    table = state[0]
    was = int(table[1, column])
    table[1, column] = bad
    table[1, 1] = bad
    table[1, 3000:] = bad
    keep = [20, 0, 0]
    _refused(at, state, lambda: at.truncate(_dev([1, 2, 0]), _dev(keep), *state, page_size=PAGE))
    table[1, column] = was
    t = model.Tables(*(x.tolist() for x in state), PAGE)
    at.truncate(_dev([1, 2, 0]), _dev(keep), *state, page_size=PAGE)
    at.sync()
    t.truncate([1, 2, 0], keep)
    assert state[1].tolist() == t.lengths and state[2][1:1 + int(state[2][0])].tolist() == t.stack
