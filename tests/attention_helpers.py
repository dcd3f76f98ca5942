"""Inputs, reference and error bounds of the attention tests."""
import numpy as np
import torch

from oracle import attention_model as model

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


class Setup:
    """n slots with `after` tokens each in pages of random order.  Places that hold no token are NaN."""

    def __init__(self, after, G, d, page, dtype, seed, pool="pages_first", spare=2, scale=1.0):
        gen = torch.Generator().manual_seed(seed)
        rs = np.random.RandomState(seed)
        n = len(after)
        self.after, self.page, self.G, self.d, self.dt = list(after), page, G, d, DT[dtype]
        counts = [-(-a // page) for a in after]
        self.num_slots, self.num_pages = n + 3, sum(counts) + spare
        self.max_pages = max(counts + [1]) + 1
        order = rs.permutation(self.num_pages).tolist()
        self.slots = rs.permutation(self.num_slots)[:n].tolist()
        self.table = [[0x7ffffff0] * self.max_pages for _ in range(self.num_slots)]    # no page is read from these
        self.lengths = [0] * self.num_slots
        for s, a, c in zip(self.slots, after, counts):
            self.table[s][:c] = [order.pop() for _ in range(c)]
            self.lengths[s] = a
        self.free = [len(order)] + order + [0] * (self.num_pages - len(order))
        self.k, self.v = [], []
        k_pages = torch.full((self.num_pages, G, page, d), float("nan"), dtype=self.dt)
        v_pages = k_pages.clone()
        for s, a in zip(self.slots, after):
            k, v = ((scale * torch.randn(a, G, d, generator=gen)).to(self.dt) for _ in range(2))
            self.k.append(k)
            self.v.append(v)
            for p in range(0, a, page):
                m = min(page, a - p)
                k_pages[self.table[s][p // page], :, :m] = k[p:p + m].transpose(0, 1)
                v_pages[self.table[s][p // page], :, :m] = v[p:p + m].transpose(0, 1)
        self.gen = gen
        self.k_pages, self.v_pages = self.place(k_pages, pool), self.place(v_pages, pool)

    def place(self, t, pool):
        """On the device: pages, heads, tokens; tokens before heads; or at an odd offset with padded rows."""
        if pool == "pages_first":
            return t.cuda()
        if pool == "tokens_first":
            return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        shape = t.shape[:3] + (self.d + 3,)
        wide = torch.full((t.numel() // self.d * (self.d + 3) + 1,), float("nan"), dtype=self.dt, device="cuda")
        view = wide[1:].view(shape)[..., :self.d]
        view.copy_(t)
        return view

    def dev(self, a):
        return torch.tensor(a, dtype=torch.int32, device="cuda")

    def args(self):
        return (self.k_pages, self.v_pages, self.dev(self.table), self.dev(self.lengths), self.dev(self.slots))

    def queries(self, lead, H, scale=1.5, fused=0):
        """q [*lead, H, d]; fused: the first heads of a wider tensor with `fused` heads more."""
        q = (scale * torch.randn(*lead, H + fused, self.d, generator=self.gen)).to(self.dt)
        return q.cuda()[..., :H, :], q[..., :H, :]


def bound(o, mag, big, dt, d, keys, tensor=True):
    """How far an output may be off.  u: half a step of the type (its rounding at the end, and the weights' on the
    tensor cores, where a weight is also 2^-25 off at most in fp16, below its normal range).  A score is off by its
    products' sum (d roundings of 2^-24), its scaling and its difference to the maximum (4 more of at most its size,
    each side), which the exponential turns into a relative error; exp2 adds 2^-21, sums over the keys 2^-24 each in
    numerator and denominator."""
    u = torch.finfo(dt).eps / 2
    score = 2 * (d + 8) * 2.0 ** -24 * big[..., None]
    rel = torch.expm1(score) * 2 + 2.0 ** -20 + 2 * keys * 2.0 ** -24
    if tensor and dt != torch.float32:
        rel = rel + u * 1.01
        if dt == torch.float16:
            rel = rel + keys * 2.0 ** -25
    tiny = torch.finfo(dt).tiny * torch.finfo(dt).eps
    return u * o.abs() * 1.01 + mag * rel * 1.01 + tiny


def check(got, want, tol, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    if got.numel() == 0:
        return
    assert torch.isfinite(want).all() and torch.isfinite(got).all(), "%s: not finite" % what
    off = (got - want).abs() - tol
    worst = int(off.argmax())
    assert off.max() <= 0, "%s: %d of %d outputs off; worst %g for %g, allowed %g" % (
        what, int((off > 0).sum()), off.numel(), got.flatten()[worst], want.flatten()[worst], tol.flatten()[worst])


def check_rows(s, q, got, tokens, begin, window, sinks, scale=None):
    """Every row's tokens of a packed q / got [total, H, d] (host), row i's from begin[i] on."""
    for i, t in enumerate(tokens):
        if t == 0:
            continue
        at = slice(begin[i], begin[i] + t)
        pos = torch.arange(s.after[i] - t, s.after[i])
        o, mag, big = model.attend_row(q[at], s.k[i], s.v[i], pos, window, sinks, scale)
        check(got[at], o, bound(o, mag, big, s.dt, s.d, max(s.after[i], 1)), "row %d" % i)
