"""Two token-mixing layers built from the library's calls, from prompts to single tokens.

  GdnLayer   residual sum and norm -> projection -> short convolution with the
             L2 norm of q and k -> Gated DeltaNet (DeltaLog) -> gated norm ->
             projection
  SsmLayer   the same around the selective state space scan

A layer holds random weights and the state of its slots.  ``prompt`` feeds T
tokens to the listed slots, ``step`` one token; both return the layer's output
and the residual stream.  The command runs a prompt and some single tokens
after it, and the same tokens as one prompt, and compares the two:

  python examples/mixer_layer.py --layer gdn --slots 4 --tokens 96 --steps 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_attention_recurrent_gdn_gb300 import deltalog as dl  # noqa: E402
from linear_attention_recurrent_gdn_gb300 import mixer  # noqa: E402

BF16 = torch.bfloat16


class _Layer:
    def __init__(self, hidden, width, conv_channels, slots, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.norm = self.weight(hidden, scale=0.1) + 1
        self.w_in = self.weight(hidden, width, scale=hidden ** -0.5)
        self.conv_w = self.weight(conv_channels, 4, scale=0.5)
        self.conv_pool = torch.zeros(slots, 3, conv_channels, dtype=BF16, device="cuda")

    def weight(self, *shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=self.gen, device="cuda")).to(BF16)

    def enter(self, x, residual):
        """The sum with the residual stream, its norm, and the input projection of [..., hidden] tokens."""
        lead = x.shape[:-1]
        y, h = mixer.add_norm(x.reshape(-1, x.shape[-1]), None if residual is None else residual.reshape(-1, x.shape[-1]),
                              self.norm)
        return (y @ self.w_in).unflatten(0, lead), h.view(x.shape)


class GdnLayer(_Layer):
    """Heads of d = 64 or 128; hidden = heads * d."""

    def __init__(self, heads, d, slots, merge_interval=8, seed=0):
        hd = heads * d
        super().__init__(hd, 4 * hd + 2 * heads, 3 * hd, slots, seed)
        self.H, self.d, self.hd = heads, d, hd
        self.decay = -torch.rand(heads, generator=self.gen, device="cuda")
        self.dt_bias = torch.randn(heads, generator=self.gen, device="cuda") - 2
        self.out_norm = self.weight(d, scale=0.1) + 1
        self.w_out = self.weight(hd, hd, scale=hd ** -0.5)
        self.ctx = dl.DeltaLog(dl.GDN, slots, heads, d, merge_interval=merge_interval, scale=d ** -0.5)
        self.ctx.set_state(list(range(slots)), torch.zeros(slots, heads, d, d, device="cuda"))

    def _mix(self, x, residual, conv, recur):
        z, h = self.enter(x, residual)
        hd, H, d = self.hd, self.H, self.d
        q, k, v = (t.unflatten(-1, (H, d)) for t in conv(z[..., :3 * hd]))
        a, b = z[..., 4 * hd:4 * hd + H].float(), z[..., 4 * hd + H:].float()
        g = (self.decay * torch.nn.functional.softplus(a + self.dt_bias)).contiguous()
        o = recur(q, k, v, g, torch.sigmoid(b).contiguous())
        gate = z[..., 3 * hd:4 * hd].flatten(0, -2).unflatten(-1, (H, d))
        y = mixer.gated_norm(o.reshape(-1, H, d), self.out_norm, gate)
        return (y.flatten(1) @ self.w_out).view(x.shape), h

    def prompt(self, x, residual, slots, fresh=True):
        """x [T, n, hidden] for the listed slots, which own their bases and have empty logs."""
        return self._mix(
            x, residual,
            lambda z: mixer.conv(z, self.conv_w, slots=slots, state=self.conv_pool, fresh=fresh,
                                 l2_channels=2 * self.hd, head_dim=self.d, split=(self.hd,) * 3),
            lambda q, k, v, g, b: self.ctx.prefill(slots, q, k, v, g, b))

    def step(self, x, residual, slots):
        """x [n, hidden]: one token of every listed slot."""
        return self._mix(
            x, residual,
            lambda z: mixer.conv_step(z, self.conv_w, slots=slots, state=self.conv_pool,
                                      l2_channels=2 * self.hd, head_dim=self.d, split=(self.hd,) * 3),
            lambda q, k, v, g, b: self.ctx.step(slots, q, k, v, g, b))

    def state(self, slots):
        return self.ctx.read_state(slots)


class SsmLayer(_Layer):
    """H heads of P channels over states of N, their maps shared in G groups; hidden = H * P."""

    def __init__(self, heads, P, N, slots, groups=1, seed=0):
        hp, gn = heads * P, groups * N
        super().__init__(hp, 2 * hp + 2 * gn + heads, hp + 2 * gn, slots, seed)
        self.H, self.P, self.N, self.G = heads, P, N, groups
        self.A = -1 - 15 * torch.rand(heads, generator=self.gen, device="cuda")
        self.D = torch.ones(heads, device="cuda")
        self.dt_bias = torch.randn(heads, generator=self.gen, device="cuda") - 4
        self.out_norm = self.weight(hp, scale=0.1) + 1
        self.w_out = self.weight(hp, hp, scale=hp ** -0.5)
        self.pool = torch.zeros(slots, heads, P, N, device="cuda")

    def _mix(self, x, residual, conv, scan):
        z, h = self.enter(x, residual)
        hp, gn = self.H * self.P, self.G * self.N
        u = conv(z[..., hp:2 * hp + 2 * gn])
        y = scan(u[..., :hp].unflatten(-1, (self.H, self.P)), z[..., 2 * hp + 2 * gn:],
                 u[..., hp:hp + gn].unflatten(-1, (self.G, self.N)), u[..., hp + gn:].unflatten(-1, (self.G, self.N)))
        y = mixer.gated_norm(y.reshape(-1, 1, hp), self.out_norm, z[..., :hp].reshape(-1, 1, hp), gate_first=True)
        return (y.flatten(1) @ self.w_out).view(x.shape), h

    def prompt(self, x, residual, slots, fresh=True):
        return self._mix(
            x, residual,
            lambda z: mixer.conv(z, self.conv_w, slots=slots, state=self.conv_pool, fresh=fresh),
            lambda u, dt, B, C: mixer.ssm(u, dt, self.A, B, C, self.D, dt_bias=self.dt_bias, slots=slots,
                                          state=self.pool, fresh=fresh))

    def step(self, x, residual, slots):
        return self._mix(
            x, residual,
            lambda z: mixer.conv_step(z, self.conv_w, slots=slots, state=self.conv_pool),
            lambda u, dt, B, C: mixer.ssm_step(u, dt, self.A, B, C, self.D, dt_bias=self.dt_bias, slots=slots,
                                               state=self.pool))

    def state(self, slots):
        return self.pool[slots]


def compare(make, slots, tokens, steps, seed=1):
    """Largest difference, relative to the largest value, of outputs and states between a prompt with single
    tokens after it and one prompt."""
    one, two = make(), make()
    hidden = one.norm.numel()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens + steps, slots, hidden, generator=gen, device="cuda").to(BF16)
    ids = list(range(slots))
    whole, stream = one.prompt(x, None, ids)
    first, _ = two.prompt(x[:tokens], None, ids)
    rest = [two.step(x[tokens + t], None, ids)[0] for t in range(steps)]
    parts = torch.cat([first] + [r[None] for r in rest])
    rel = lambda a, b: float((a.float() - b.float()).abs().max() / b.float().abs().max())  # noqa: E731
    mixer.sync()
    return rel(parts, whole), rel(two.state(ids), one.state(ids))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layer", choices=("gdn", "ssm"), default="gdn")
    ap.add_argument("--slots", type=int, default=4)
    ap.add_argument("--heads", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=96)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args(argv)
    make = {"gdn": lambda: GdnLayer(a.heads, 128, a.slots), "ssm": lambda: SsmLayer(a.heads, 64, 128, a.slots)}[a.layer]
    out, state = compare(make, a.slots, a.tokens, a.steps)
    print("%s layer, %d slots: %d prompt tokens and %d single ones against one prompt: outputs %.2e, states %.2e apart"
          % (a.layer, a.slots, a.tokens, a.steps, out, state))
    return out, state


if __name__ == "__main__":
    main()
