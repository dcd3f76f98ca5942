"""Host-side checks of the attention calls (no GPU needed): struct layouts and refusals.  Pointers are fake device
addresses that no call gets far enough to use: every call is invalid in exactly one way, or has nothing to do."""
import ctypes

import pytest
import torch

from linear_attention_recurrent_gdn_gb300 import build

I64, P = ctypes.c_int64, ctypes.c_void_p
BASE = 0x7f0000000000


class View(ctypes.Structure):
    _fields_ = [("data", P), ("stride_t", I64), ("stride_n", I64)]


class Pool(ctypes.Structure):
    _fields_ = [("data", P), ("stride_page", I64), ("stride_head", I64), ("stride_token", I64)]


class Pages(ctypes.Structure):
    _fields_ = [(k, P) for k in ("slots", "tokens", "table", "lengths", "free", "starts", "where", "positions", "work")] + \
        [(k, I64) for k in ("table_stride", "size", "n", "T", "num_slots", "max_pages", "num_pages", "page_size")]


class Append(ctypes.Structure):
    _fields_ = [(k, I64) for k in ("dtype", "T", "n", "G", "d", "page_size", "num_pages")] + \
        [("k", View), ("v", View), ("k_pages", Pool), ("v_pages", Pool), ("where", P)]


class Attend(ctypes.Structure):
    _fields_ = [(k, I64) for k in ("dtype", "n", "T", "packed", "H", "G", "d", "page_size", "max_pages", "num_slots",
                                   "num_pages", "window", "sinks")] + \
        [("scale", ctypes.c_double), ("q", View), ("o", View), ("k_pages", Pool), ("v_pages", Pool), ("table", P),
         ("table_stride", I64)] + [(k, P) for k in ("lengths", "slots", "starts", "tokens", "workspace")] + \
        [("workspace_bytes", I64)]


@pytest.fixture(scope="module")
def at():
    build.build()
    from linear_attention_recurrent_gdn_gb300 import attention
    return attention


def _fake():
    return iter(range(BASE, BASE + 64 * (1 << 20), 1 << 20))


def _pages():
    a = _fake()
    return Pages(*[next(a) for _ in range(9)], 12, 30, 3, 10, 8, 12, 40, 16)


def _append():
    a = _fake()
    v, p = lambda: View(next(a), 3 * 256, 256), lambda: Pool(next(a), 2 * 16 * 128, 16 * 128, 128)  # noqa: E731
    return Append(1, 5, 3, 2, 128, 16, 40, v(), v(), p(), p(), next(a))


def _attend(T=5, packed=0):
    a = _fake()
    v, p = lambda: View(next(a), 3 * 1024, 1024), lambda: Pool(next(a), 2 * 16 * 128, 16 * 128, 128)  # noqa: E731
    return Attend(1, 3, T, packed, 8, 2, 128, 16, 12, 8, 40, 0, 0, 0.1, v(), v(), p(), p(), next(a), 12, next(a),
                  next(a), next(a) if packed else 0, 0, 0, 0)


MAKE = dict(dl_pages_extend=_pages, dl_pages_truncate=_pages, dl_kv_append=_append, dl_attend=_attend,
            dl_attend_step=lambda: _attend(1))


def _call(at, fn, q):
    err = ctypes.create_string_buffer(256)
    return getattr(at._lib, fn)(ctypes.string_at(ctypes.addressof(q), ctypes.sizeof(q)), None, err, 256), \
        err.value.decode()


def _set(q, path, value):
    *most, last = path.split(".")
    for k in most:
        q = getattr(q, k)
    setattr(q, last, value)


def test_struct_sizes_match_the_binding(at):
    assert ctypes.sizeof(Pages) == at._PAGES.size and ctypes.sizeof(Append) == at._APPEND.size
    assert ctypes.sizeof(Attend) == at._ATTEND.size + at._WORKSPACE.size


@pytest.mark.parametrize("fn,changes", [
    ("dl_pages_truncate", {"n": 0}), ("dl_kv_append", {"n": 0}), ("dl_kv_append", {"T": 0}), ("dl_attend", {"n": 0}),
    ("dl_attend", {"T": 0}), ("dl_attend_step", {"n": 0}), ("dl_attend", {"n": 0, "q.data": 0}),
])
def test_nothing_to_do_is_fine(at, fn, changes):
    q = MAKE[fn]()
    for k, v in changes.items():
        _set(q, k, v)
    assert _call(at, fn, q) == (0, "")


TABLE = [("n", -1, "EINVAL", "rows"), ("n", 1025, "EINVAL", "rows"), ("num_slots", 0, "EINVAL", "slots"),
         ("num_slots", 2 ** 31, "EINVAL", "slots"), ("max_pages", 0, "EINVAL", "pages"),
         ("max_pages", 2 ** 27, "EINVAL", "pages"), ("table_stride", 11, "EINVAL", "overlap"),
         ("page_size", 8, "EUNSUPPORTED", "power of two"), ("page_size", 24, "EUNSUPPORTED", "power of two"),
         ("page_size", 512, "EUNSUPPORTED", "power of two"), ("num_pages", 0, "EINVAL", "pages"),
         ("num_pages", 2 ** 28, "EINVAL", "pages")]
HEADS = [("dtype", 3, "EINVAL", "dtype"), ("dtype", -1, "EINVAL", "dtype"), ("G", 0, "EINVAL", "heads"),
         ("d", 0, "EINVAL", "heads"), ("d", 257, "EUNSUPPORTED", "heads")]
ATTEND = TABLE + HEADS + [
    ("H", 0, "EINVAL", "heads"), ("H", 7, "EINVAL", "heads"), ("T", -1, "EINVAL", "tokens"), ("window", -1, "EINVAL", "window"),
    ("sinks", -1, "EINVAL", "first tokens"), ("scale", 0.0, "EINVAL", "scale"), ("scale", -1.0, "EINVAL", "scale"),
    ("scale", float("inf"), "EINVAL", "scale"), ("scale", float("nan"), "EINVAL", "scale"), ("scale", 1e300, "EINVAL", "scale"),
    ("q.data", 0, "EINVAL", "NULL"), ("o.data", 0, "EINVAL", "NULL"), ("k_pages.data", 0, "EINVAL", "NULL"),
    ("v_pages.data", 0, "EINVAL", "NULL"), ("table", 0, "EINVAL", "NULL"), ("lengths", 0, "EINVAL", "NULL"),
    ("slots", 0, "EINVAL", "NULL"), ("q.data", BASE + 1, "EINVAL", "alignment"), ("lengths", BASE + 2, "EINVAL", "alignment"),
    ("workspace", 0, "EINVAL", "workspace")]
REFUSALS = [("dl_pages_extend",) + r for r in TABLE + [
    ("n", 0, "EINVAL", "maps"), ("T", -1, "EINVAL", "maps"), ("size", -1, "EINVAL", "maps"), ("size", 29, "EINVAL", "maps"),
    ("slots", 0, "EINVAL", "NULL"), ("table", 0, "EINVAL", "NULL"), ("lengths", 0, "EINVAL", "NULL"),
    ("free", 0, "EINVAL", "NULL"), ("starts", 0, "EINVAL", "NULL"), ("where", 0, "EINVAL", "NULL"),
    ("work", 0, "EINVAL", "NULL"), ("where", BASE + 2, "EINVAL", "alignment")]] + \
    [("dl_pages_truncate",) + r for r in TABLE + [("slots", 0, "EINVAL", "NULL"), ("free", BASE + 1, "EINVAL", "alignment")]] + \
    [("dl_kv_append",) + r for r in HEADS + [
        ("T", -1, "EINVAL", "tokens"), ("n", -1, "EINVAL", "tokens"), ("T", 2 ** 30, "EINVAL", "tokens"),
        ("page_size", 17, "EUNSUPPORTED", "power of two"), ("k.data", 0, "EINVAL", "NULL"), ("v.data", 0, "EINVAL", "NULL"),
        ("k_pages.data", 0, "EINVAL", "NULL"), ("v_pages.data", 0, "EINVAL", "NULL"), ("where", 0, "EINVAL", "NULL"),
        ("where", BASE + 1, "EINVAL", "alignment"), ("v.data", BASE + 1, "EINVAL", "alignment")]] + \
    [("dl_attend",) + r for r in ATTEND] + [("dl_attend_step",) + r for r in ATTEND] + \
    [("dl_attend_step", "T", 2, "EINVAL", "one token"), ("dl_attend_step", "packed", 1, "EINVAL", "one token"),
     ("dl_attend_step", "tokens", BASE, "EINVAL", "one token"), ("dl_attend", "packed", 1, "EINVAL", "starts")]


@pytest.mark.parametrize("fn,path,value,status,word", REFUSALS)
def test_refusals(at, fn, path, value, status, word):
    q = MAKE[fn]()
    _set(q, path, value)
    rc, msg = _call(at, fn, q)
    assert at._dl.STATUS_NAMES[rc] == "DL_" + status and word in msg


def test_null_arguments(at):
    for fn in MAKE:
        assert getattr(at._lib, fn)(None, None, None, 0) == at._dl.EINVAL
    assert at._lib.dl_attend_workspace(None) == -1


@pytest.mark.parametrize("path,value", [("d", 0), ("H", 7), ("page_size", 8), ("window", -1)])
def test_workspace_of_invalid_sizes(at, path, value):
    q = _attend()
    _set(q, path, value)
    assert at._lib.dl_attend_workspace(ctypes.string_at(ctypes.addressof(q), ctypes.sizeof(q))) == -1


def _workspace(at, q):
    return at._lib.dl_attend_workspace(ctypes.string_at(ctypes.addressof(q), ctypes.sizeof(q)))


def test_workspace_does_not_grow_with_the_cache(at):
    """It is for the parts of split keys: by the GPU's size, not the contexts'."""
    for T, packed in ((1, 0), (5, 0), (7, 1)):
        sizes = []
        for max_pages in (12, 1000, 60000):
            q = _attend(T, packed)
            q.max_pages = q.table_stride = max_pages
            sizes.append(_workspace(at, q))
        assert sizes[0] == sizes[1] == sizes[2] > 0
    q = _attend(2048)
    q.n = 64
    assert _workspace(at, q) == 0        # enough work without splitting


# -------------------------------------------------------------------- binding --
def test_host_tensors_are_refused(at):
    x, i = torch.zeros(3, 4, 64), torch.zeros(3, dtype=torch.int32)
    pool, table = torch.zeros(8, 2, 16, 64), torch.zeros(8, 4, dtype=torch.int32)
    for call in (lambda: at.attend_step(x, pool, pool, table, i, i), lambda: at.attend(x, pool, pool, table, i, i, starts=i),
                 lambda: at.append(x, x, pool, pool, i), lambda: at.extend(i, None, None, table, i, i, page_size=16),
                 lambda: at.truncate(i, None, table, i, i, page_size=16)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()


def test_new_tables(at):
    table, lengths, free = at.new_tables(3, 5, 7, device="cpu")
    assert table.shape == (3, 5) and lengths.tolist() == [0, 0, 0] and free.tolist() == [7, 6, 5, 4, 3, 2, 1, 0]
    assert {t.dtype for t in (table, lengths, free)} == {torch.int32}
