"""Paged softmax attention and its block tables in 64 bits, one row at a time, from their definitions.

``attend_row`` also returns what rounding errors go by: for every output the
weighted sum of the absolute values, and for every token the largest sum of
absolute products in a score.  Test infrastructure; shares nothing with the
CUDA path.
"""
import torch

F64 = torch.float64


class Tables:
    """Slots, their pages and the stack of free ones, as Python lists."""

    def __init__(self, table, lengths, free, page):
        self.table, self.lengths, self.page = [list(r) for r in table], list(lengths), page
        self.stack = list(free[1:1 + free[0]])

    def extend(self, slots, tokens):
        """[(place, position)] of every row, or None where the call cannot be done."""
        old = [self.lengths[s] for s in slots] if all(0 <= s < len(self.lengths) for s in slots) else None
        if old is None or len(set(slots)) != len(slots) or min(tokens, default=0) < 0:
            return None
        need = sum(-(-(L + t) // self.page) - -(-L // self.page) for L, t in zip(old, tokens))
        if need > len(self.stack) or any(L + t > len(self.table[s]) * self.page for s, L, t in zip(slots, old, tokens)):
            return None
        out = []
        for s, L, t in zip(slots, old, tokens):
            row = []
            for p in range(L, L + t):
                if p % self.page == 0:
                    self.table[s][p // self.page] = self.stack.pop()
                row.append((self.table[s][p // self.page] * self.page + p % self.page, p))
            self.lengths[s] = L + t
            out.append(row)
        return out

    def truncate(self, slots, keep):
        for s, k in reversed(list(zip(slots, keep))):
            first, last = -(-k // self.page), -(-self.lengths[s] // self.page)
            self.stack += [self.table[s][c] for c in reversed(range(first, last))]
            self.lengths[s] = k


def attend_row(q, k, v, pos, window=None, sinks=0, scale=None):
    """q [t, H, d] at positions pos [t] over k, v [L, G, d].  Returns o, the sums of absolute weighted values, the
    largest sum of absolute products in a score [t, H].  Keys that a token does not see do not enter."""
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    t, H, d = q.shape
    G = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, mag, big = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(t, H, dtype=F64)
    key = torch.arange(k.shape[0])
    for i in range(t):
        p = int(pos[i])
        see = key <= p
        if window is not None:
            see &= (key > p - window) | (key < sinks)
        if not see.any():
            continue
        for g in range(G):
            ks, vs = k[see, g], v[see, g]
            qs = q[i, g * (H // G):(g + 1) * (H // G)]
            z = qs @ ks.T * scale
            top = z.amax(-1, keepdim=True)
            w = torch.exp(z - torch.where(torch.isneginf(top), torch.zeros_like(top), top))
            l = w.sum(-1, keepdim=True)
            w = torch.where(l == 0, torch.zeros_like(w), w / l)
            dead = (l == 0)
            at = slice(g * (H // G), (g + 1) * (H // G))
            o[i, at] = torch.where(dead, torch.zeros_like(qs), w @ vs)
            mag[i, at] = torch.where(dead, torch.zeros_like(qs), w @ vs.abs())
            big[i, at] = (qs.abs() @ ks.abs().T * scale).amax(-1)
    return o, mag, big
