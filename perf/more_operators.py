"""The attention layers beside a recurrence, as cases that can be timed and checked.

Hybrid models put a softmax attention layer between their recurrent ones.  Four
operators serve it, around one cache of keys and values in pages:

  pages   block tables and slot maps from request lengths: pages taken for new
          tokens, and given back when a request is cut to its old length
  append  the new tokens' keys and values into their pages
  step    attention of one new token a request over its pages
  attend  attention of prompts, also of their later pieces, over the pages

A request's token at position p sees the positions j <= p with j > p - window
(all without a window) and j < sinks.  ``run`` computes a case with elementary
torch operations in 32 bits, or, where ``own`` is true, with this package's
kernels.  ``exact`` is the definition in 64 bits, one request after the other.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
MOST_PAIRS = 1 << 28        # (head, query, key) triples that a plain form holds at a time


# ------------------------------------------------------------------- cases --
# n requests; T new tokens each (packed ones: up to T, one request after the
# other), ctx cached tokens each before them (ragged: up to ctx).  H query
# heads share G heads of keys and values; pages of `page` tokens.
def listed():
    return [
        # The tables of a decode step: one token for each of 256 requests, every 64th of which needs a page.
        dict(name="pages_step_256", op="pages", n=256, T=1, packed=False, ragged=True, ctx=4096, page=64),
        # 64 prompts of up to 2048 tokens that arrive together, small pages.
        dict(name="pages_prompt_64x2048", op="pages", n=64, T=2048, packed=True, ragged=True, ctx=0, page=16),
        # A decode step's keys and values of 256 requests, 8 heads of 128.
        dict(name="append_256x8x128", op="append", dtype="bf16", n=256, T=1, packed=False, ragged=True,
             ctx=2048, page=64, H=32, G=8, d=128),
        # The keys and values of 16 prompts of 512 tokens, token-major as the recurrent prefill takes them.
        dict(name="append_16x512x8x128", op="append", dtype="bf16", n=16, T=512, packed=False, ragged=False,
             ctx=0, page=64, H=32, G=8, d=128),
        # One request at a short context: a call's latency.
        dict(name="step_1x512", op="step", dtype="bf16", n=1, T=1, packed=False, ragged=False, ctx=512, page=64,
             H=32, G=8, d=128, window=0, sinks=0),
        # The serving batch of the decode workloads at 2048 tokens each.
        dict(name="step_256x2048", op="step", dtype="bf16", n=256, T=1, packed=False, ragged=False, ctx=2048,
             page=64, H=32, G=8, d=128, window=0, sinks=0),
        # One long document: all of the GPU for the keys of one request.
        dict(name="step_1x131072", op="step", dtype="bf16", n=1, T=1, packed=False, ragged=False, ctx=131072,
             page=64, H=32, G=8, d=128, window=0, sinks=0),
        # Ragged contexts under a window with its first tokens kept, five query heads to a head of keys, small pages.
        dict(name="step_37x5000_window", op="step", dtype="fp16", n=37, T=1, packed=False, ragged=True, ctx=5000,
             page=16, H=40, G=8, d=64, window=1000, sinks=4),
        # 16 contexts of 512 tokens, 32 heads of 128: the prompts of the chunked-prefill workload.
        dict(name="attend_16x512", op="attend", dtype="bf16", n=16, T=512, packed=False, ragged=False, ctx=0,
             page=64, H=32, G=8, d=128, window=0, sinks=0),
        # One long prompt.
        dict(name="attend_1x8192", op="attend", dtype="bf16", n=1, T=8192, packed=False, ragged=False, ctx=0,
             page=64, H=32, G=8, d=128, window=0, sinks=0),
        # Packed prompts under a window with its first tokens kept.
        dict(name="attend_7x4001_window", op="attend", dtype="fp16", n=7, T=4001, packed=True, ragged=True, ctx=0,
             page=16, H=40, G=8, d=64, window=1000, sinks=4),
        # Packed pieces of up to 200 tokens behind long cached contexts: few rows, a long axis.
        dict(name="attend_3x200_behind_30000", op="attend", dtype="bf16", n=3, T=200, packed=True, ragged=True,
             ctx=30000, page=64, H=32, G=8, d=128, window=0, sinks=0),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["pages", "append", "step", "step", "attend", "attend"])
    page = rng.choice([16, 16, 32, 64, 64, 128, 256])
    packed = rng.random() < 0.5
    case = dict(op=op, page=page, ragged=rng.random() < 0.6)
    if op == "pages":
        T = 1 if rng.random() < 0.4 else log_int(2, 4096)
        n = max(1, min(log_int(1, 1024), 64 * 2048 // T))
        return dict(case, n=n, T=T, packed=packed and T > 1, ctx=rng.choice([0, log_int(1, 8192)]))
    G, per = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16])
    d = rng.choice([64, 64, 128, 128, 128, 80, 96, 256, 20])
    case.update(H=G * per, G=G, d=d, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "append":
        T = 1 if rng.random() < 0.4 else log_int(2, 4096)
        n = max(1, min(log_int(1, 512), 16 * 512 * 1024 // (T * G * d)))
        return dict(case, n=n, T=T, packed=packed and T > 1, ctx=rng.choice([0, log_int(1, 2048)]))
    case["window"] = rng.choice([0, 0, log_int(1, 4096)])
    case["sinks"] = rng.choice([0, 1, 4, 130]) if case["window"] else 0
    if op == "step":
        ctx = log_int(1, 131072)
        n = max(1, min(log_int(1, 512), 256 * 2048 * 1024 // (ctx * G * d) // (BYTES[case["dtype"]] // 2)))
        return dict(case, n=n, T=1, packed=False, ctx=ctx)
    T = log_int(2, 4096)
    ctx = rng.choice([0, log_int(1, 16384)])
    most = 4096 * 8192 * 32 * 128 // (8 if case["dtype"] == "fp32" or d == 20 else 1)
    n = max(1, min(log_int(1, 64), most // (T * (T // 2 + ctx + 1) * case["H"] * max(d, 64))))
    while n == 1 and T * (T // 2 + ctx + 1) * case["H"] * max(d, 64) > most:
        T, ctx = (T + 1) // 2, ctx // 2
    return dict(case, n=n, T=T, packed=packed, ctx=ctx)


def _spread(n, most, ragged, salt):
    """n lengths: most each, or spread over 0 .. most with the first at most."""
    if not ragged:
        return np.full(n, most, np.int64)
    return np.array([most if i == 0 else (i * 7919 + salt * most + 13) % (most + 1) for i in range(n)], np.int64)


def _sizes(case):
    """New tokens and cached ones before them of every request."""
    tokens = _spread(case["n"], case["T"], case["ragged"] and case["packed"], 13)
    ctx = _spread(case["n"], case["ctx"], case["ragged"], 29)
    if case["op"] == "step":                 # ctx counts the new token
        ctx = np.maximum(ctx, 1) - 1
    return tokens, ctx


def _pages_of(lengths, page):
    return -(-lengths // page)


# ------------------------------------------------------------------ inputs --
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rs = np.random.RandomState(int(seed) % (1 << 32))
    tokens, ctx = _sizes(case)
    n, page, op = case["n"], case["page"], case["op"]
    total = int(tokens.sum())
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731

    num_slots = n + n // 8 + 1
    slots = rs.permutation(num_slots)[:n]
    after = ctx + tokens
    held = _pages_of(ctx if op == "pages" else after, page)       # pages that the requests hold before the call
    need = int(_pages_of(after, page).sum())
    num_pages = need + need // 8 + 1
    order = rs.permutation(num_pages)                             # pages in the order they were handed out
    max_pages = int(_pages_of(after, page).max()) + 1
    table = np.zeros((num_slots, max_pages), np.int64)
    lengths = np.zeros(num_slots, np.int64)
    lengths[slots] = ctx if op == "pages" else after
    at = 0
    for i in range(n):
        table[slots[i], :held[i]] = order[at:at + held[i]]
        at += held[i]
    free = np.zeros(num_pages + 1, np.int64)                      # how many, and a stack of them
    free[0] = num_pages - at
    free[1:1 + num_pages - at] = order[at:]
    s = dict(case=case, slots=dev(slots), table=dev(table), lengths=dev(lengths), free=dev(free),
             tokens=dev(tokens), total=total)
    if op == "pages":
        s["before"] = dev(ctx)
        return s

    H, G, d, dt = case["H"], case["G"], case["d"], DTYPES[case["dtype"]]
    lead = (n,) if case["T"] == 1 and not case["packed"] else (total,) if case["packed"] else (case["T"], n)
    # q, k and v as a projection leaves them, side by side
    fused = torch.randn(*lead, (H + 2 * G) * d, generator=gen, device="cuda")
    fused[..., :H * d] *= 2
    fused = fused.to(dt)
    q, k, v = fused.split((H * d, G * d, G * d), -1)
    s.update(q=q.unflatten(-1, (H, d)), k=k.unflatten(-1, (G, d)), v=v.unflatten(-1, (G, d)))
    for name in ("k_pages", "v_pages"):
        pool = torch.empty(num_pages, G, page, d, dtype=dt, device="cuda")
        for part in pool.split(max(1, (1 << 27) // (G * page * d))):
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
        s[name] = pool
    starts = np.concatenate([[0], np.cumsum(tokens)])
    s["starts"] = dev(starts)
    if op == "append":
        where = np.concatenate([table[slots[i], (ctx[i] + np.arange(tokens[i])) // page] * page
                                + (ctx[i] + np.arange(tokens[i])) % page for i in range(n)] + [np.zeros(0, np.int64)])
        if not case["packed"]:
            where = where.reshape(n, case["T"]).T.reshape(lead)
        s["where"] = dev(where)
    return s


# -------------------------------------------------------------- plain forms --
def _plain_pages(s):
    case, page = s["case"], s["case"]["page"]
    slots, tokens, table, lengths, free = (s[k].long() for k in ("slots", "tokens", "table", "lengths", "free"))
    n, T = case["n"], case["T"]
    old = lengths[slots]
    new = old + tokens
    have, want = (old + page - 1) // page, (new + page - 1) // page
    starts = torch.nn.functional.pad(tokens.cumsum(0), (1, 0))
    # every table entry that is new, and the page it gets: from the stack's top, request by request
    col = torch.arange(table.shape[1], device="cuda")
    fresh = (col >= have[:, None]) & (col < want[:, None])
    base = (want - have).cumsum(0) - (want - have)
    pick = free[0] - 1 - (base[:, None] + col - have[:, None])
    rows = torch.where(fresh, free[1 + pick.clamp(min=0, max=free.numel() - 2)], table[slots])
    if case["packed"]:
        at = torch.arange(s["total"], device="cuda")
        row = torch.searchsorted(starts, at, right=True) - 1
        pos = old[row] + at - starts[row]
    else:
        row = torch.arange(n, device="cuda").expand(T, n)
        pos = old + torch.arange(T, device="cuda")[:, None]
    where = rows[row, pos // page] * page + pos % page
    s["table"][slots] = rows.int()
    # back to the old lengths: the pages return to where they were, so the stack and its height are as before
    shape = (n,) if T == 1 and not case["packed"] else where.shape
    return dict(starts=starts.int(), where=where.int().view(shape), positions=pos.int().view(shape),
                table=s["table"], lengths=s["lengths"], free=s["free"])


def _plain_append(s):
    where, page = s["where"].long(), s["case"]["page"]
    s["k_pages"][where // page, :, where % page] = s["k"]
    s["v_pages"][where // page, :, where % page] = s["v"]
    return dict(k_pages=s["k_pages"], v_pages=s["v_pages"])


def _seen(case, pos, key):
    """Whether position pos sees position key."""
    near = key <= pos
    if not case["window"]:
        return near
    return near & ((key > pos - case["window"]) | (key < case["sinks"]))


def _softmax_sum(scores, seen, v):
    """Weighted sums of v [..., keys, d] under scores [..., rows, keys]; rows that see nothing: zero."""
    scores = scores.masked_fill(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = torch.exp(scores - top)
    return torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-38)


def _plain_step(s):
    case, page = s["case"], s["case"]["page"]
    n, H, G, d = case["n"], case["H"], case["G"], case["d"]
    lengths = s["lengths"][s["slots"].long()].long()
    table = s["table"][s["slots"].long()].long()
    longest = table.shape[1] * page
    out = torch.empty(n, H, d, dtype=s["q"].dtype, device="cuda")
    group = max(1, MOST_PAIRS // (longest * G * max(d, H // G)))
    key = torch.arange(longest, device="cuda")
    for r in range(0, n, group):
        k, v = (s[name][table[r:r + group]].float().transpose(1, 2).flatten(2, 3) for name in ("k_pages", "v_pages"))
        q = s["q"][r:r + group].float().unflatten(1, (G, H // G))
        scores = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
        seen = _seen(case, lengths[r:r + group, None] - 1, key)[:, None, None]
        out[r:r + group] = _softmax_sum(scores, seen, v).flatten(1, 2).to(out.dtype)
    return dict(o=out)


def _plain_attend(s):
    case, page = s["case"], s["case"]["page"]
    H, G, d = case["H"], case["G"], case["d"]
    tokens, ctx = _sizes(case)
    out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    begin = 0
    for i in range(case["n"]):
        t, L = int(tokens[i]), int(tokens[i] + ctx[i])
        q = s["q"][begin:begin + t] if case["packed"] else s["q"][:, i]
        o = out[begin:begin + t] if case["packed"] else out[:, i]
        begin += t
        if t == 0:
            continue
        ids = s["table"][s["slots"][i].long(), :-(-L // page)].long()
        k, v = (s[name][ids].transpose(0, 1).flatten(1, 2)[:, None, :L] for name in ("k_pages", "v_pages"))
        step = max(1, MOST_PAIRS // (L * H))
        for a in range(0, t, step):
            b = min(t, a + step)
            lo = 0 if not case["window"] or case["sinks"] else max(0, L - t + a - case["window"] + 1)
            hi = L - t + b
            key = torch.arange(lo, hi, device="cuda")
            pos = torch.arange(L - t + a, hi, device="cuda")
            qs = q[a:b].float().unflatten(1, (G, H // G)).permute(1, 2, 0, 3)      # [G, per, tokens, d]
            scores = torch.matmul(qs, k[:, :, lo:hi].float().transpose(-1, -2)) * d ** -0.5
            part = _softmax_sum(scores, _seen(case, pos[:, None], key), v[:, :, lo:hi].float())
            o[a:b] = part.permute(2, 0, 1, 3).flatten(1, 2).to(out.dtype)
    return dict(o=out)


# ------------------------------------------------------------ own kernels ----
def _own(s):
    from linear_attention_recurrent_gdn_gb300 import attention
    case, op = s["case"], s["case"]["op"]
    if op == "pages":
        state = (s["table"], s["lengths"], s["free"])
        one = case["T"] == 1 and not case["packed"]
        size = s["total"] if case["packed"] else None if one else (case["T"], case["n"])
        starts, where, positions = attention.extend(s["slots"], None if one else s["tokens"], size, *state,
                                                    page_size=case["page"])
        attention.truncate(s["slots"], s["before"], *state, page_size=case["page"])
        return dict(starts=starts, where=where, positions=positions, table=s["table"], lengths=s["lengths"],
                    free=s["free"])
    if op == "append":
        attention.append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["where"])
        return dict(k_pages=s["k_pages"], v_pages=s["v_pages"])
    args = (s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["slots"])
    more = dict(window=case["window"] or None, sinks=case["sinks"])
    if op == "step":
        return dict(o=attention.attend_step(*args, **more))
    return dict(o=attention.attend(*args, starts=s["starts"] if case["packed"] else None, **more))


def run(s):
    if own:
        return _own(s)
    plain = dict(pages=_plain_pages, append=_plain_append, step=_plain_step, attend=_plain_attend)
    return plain[s["case"]["op"]](s)


# -------------------------------------------------------------------- work --
def _visible(case, tokens, ctx):
    """(query, key) pairs that see each other, and keys that anyone sees."""
    pairs = keys = 0
    for t, c in zip(tokens.tolist(), ctx.tolist()):
        if t == 0:
            continue
        pos = np.arange(c, c + t)
        if not case["window"]:
            pairs, keys = pairs + int((pos + 1).sum()), keys + c + t
        else:
            w, k = case["window"], case["sinks"]
            low = np.maximum(pos - w + 1, 0)
            pairs += int((pos + 1 - low + np.minimum(low, k)).sum())
            keys += c + t - int(low[0]) + min(int(low[0]), k)
    return pairs, keys


def work(case):
    tokens, ctx = _sizes(case)
    total, n = int(tokens.sum()), case["n"]
    if case["op"] == "pages":
        fresh = int((_pages_of(ctx + tokens, case["page"]) - _pages_of(ctx, case["page"])).sum())
        # slots, counts and lengths; the maps; new pages from the stack into the table, and back
        return dict(bytes=4 * (7 * n + 2 * total + 4 * fresh), flops=0)
    e = BYTES[case["dtype"]]
    if case["op"] == "append":
        return dict(bytes=4 * total * case["G"] * case["d"] * e + 4 * total, flops=0)
    pairs, keys = _visible(case, tokens, ctx)
    return dict(bytes=e * case["d"] * 2 * (total * case["H"] + keys * case["G"]) + 4 * (keys // case["page"] + 2 * n),
                flops=4 * pairs * case["H"] * case["d"])


# ------------------------------------------------------------------- exact --
def _exact_pages(case, s):
    page, n = case["page"], case["n"]
    slots, tokens = s["slots"].tolist(), s["tokens"].tolist()
    table, lengths, free = (s[k].cpu().numpy().copy() for k in ("table", "lengths", "free"))
    stack = free[1:1 + free[0]].tolist()
    starts, maps = [0], []
    for slot, t in zip(slots, tokens):
        length, cells = int(lengths[slot]), []
        for p in range(length, length + t):
            if p % page == 0:
                table[slot, p // page] = stack.pop()
            cells.append((int(table[slot, p // page]) * page + p % page, p))
        maps.append(cells)
        starts.append(starts[-1] + t)
    if case["packed"]:
        flat = [c for cells in maps for c in cells]
    else:
        flat = [maps[i][t] for t in range(case["T"]) for i in range(n)]
    where, positions = np.array(flat, np.int64).reshape(-1, 2).T
    shape = (case["T"], n) if case["T"] > 1 and not case["packed"] else (-1,)
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    return dict(starts=put(starts), where=put(where.reshape(shape)), positions=put(positions.reshape(shape)),
                table=put(table), lengths=put(lengths), free=put(free))


def exact(case, seed):
    tokens, ctx = _sizes(case)
    if case["op"] in ("step", "attend"):
        pairs = _visible(dict(case, window=0), tokens, ctx)[0]
        if 4 * pairs * case["H"] * case["d"] > 8e12:
            return None
    s = prepare(case, seed)
    if case["op"] == "pages":
        return _exact_pages(case, s)
    page, per = case["page"], case["H"] // case["G"]
    if case["op"] == "append":
        pools = {}
        where = s["where"].flatten().long()
        for name, new in (("k_pages", s["k"]), ("v_pages", s["v"])):
            tokens_first = s[name].double().transpose(1, 2).flatten(0, 1)
            tokens_first[where] = new.double().reshape(-1, case["G"], case["d"])
            pools[name] = tokens_first.unflatten(0, (-1, page)).transpose(1, 2)
        return pools
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    slots, begin = s["slots"].tolist(), 0
    for i in range(case["n"]):
        t, L = int(tokens[i]), int(tokens[i] + ctx[i])
        rows = (slice(i, i + 1),) if case["op"] == "step" else (slice(begin, begin + t),) if case["packed"] \
            else (slice(None), i)
        begin += t
        if t == 0:
            continue
        p = torch.arange(L, device="cuda")
        cell = s["table"][slots[i]].long()[p // page]
        for g in range(case["G"]):
            k, v = s["k_pages"][cell, g, p % page].double(), s["v_pages"][cell, g, p % page].double()
            q = s["q"][rows][:, g * per:(g + 1) * per].double()
            o = torch.zeros(t, per, case["d"], dtype=torch.float64, device="cuda")
            for a in range(0, t, 512):
                z = torch.einsum("thd,kd->htk", q[a:a + 512], k) / case["d"] ** 0.5
                at = torch.arange(L - t + a, L - t + min(t, a + 512), device="cuda")
                hidden = p[None] > at[:, None]
                if case["window"]:
                    hidden |= (at[:, None] - p[None] >= case["window"]) & (p[None] >= case["sinks"])
                o[a:a + 512] = torch.einsum("htk,kd->thd", torch.softmax(z.masked_fill(hidden, -torch.inf), -1), v)
            out[rows][:, g * per:(g + 1) * per] = o
    return dict(o=out)
