"""The mixer operators in 64 bits, one row at a time, from their definitions.

Every function also returns, for each output, the sum of the absolute values
of the terms that make it up: the scale that rounding errors in a sum go by.
Test infrastructure; shares nothing with the CUDA path.
"""
import torch

F64 = torch.float64


def _act(z, act):
    if act is None:
        return z
    return torch.sigmoid(z) * (z if act == "silu" else 1.0)


def conv_row(x, carried, w, b=None, act="silu", l2_channels=0, head_dim=0, eps=1e-6):
    """x [t, C], carried [W - 1, C], w [C, W].  Returns y, carried, abs(z terms)."""
    x, carried, w = x.to(F64), carried.to(F64), w.to(F64)
    W = w.shape[1]
    full = torch.cat([carried, x], 0)
    z = torch.zeros_like(x)
    mag = torch.zeros_like(x)
    for j in range(W):
        term = full[j:j + x.shape[0]] * w[:, j]
        z, mag = z + term, mag + term.abs()
    if b is not None:
        z, mag = z + b.to(F64), mag + b.to(F64).abs()
    y = _act(z, act)
    if l2_channels:
        heads = y[:, :l2_channels].reshape(x.shape[0], -1, head_dim)
        heads = heads / torch.sqrt((heads * heads).sum(-1, keepdim=True) + eps)
        y = torch.cat([heads.reshape(x.shape[0], l2_channels), y[:, l2_channels:]], 1)
    return y, full[full.shape[0] - (W - 1):], mag


def ssm_row(x, dt, A, B, C, D, S, dt_bias=None, softplus=True):
    """x [t, H, P], dt [t, H], B, C [t, G, N], S [H, P, N].  Returns y, S, and the sums of absolute terms of both."""
    x, dt, A, B, C, S = (v.to(F64) for v in (x, dt, A, B, C, S))
    H, per = x.shape[1], x.shape[1] // B.shape[1]
    if dt_bias is not None:
        dt = dt + dt_bias.to(F64)
    if softplus:
        dt = torch.logaddexp(dt, torch.zeros_like(dt))
    D = torch.zeros(H, dtype=F64) if D is None else D.to(F64)
    y, ymag, Smag = torch.empty_like(x), torch.empty_like(x), S.abs()
    S = S.clone()
    for t in range(x.shape[0]):
        Bt, Ct = B[t].repeat_interleave(per, 0), C[t].repeat_interleave(per, 0)
        dec = torch.exp(dt[t] * A)[:, None, None]
        add = (dt[t][:, None] * x[t])[:, :, None] * Bt[:, None]
        S, Smag = dec * S + add, dec * Smag + add.abs()
        y[t] = (S * Ct[:, None]).sum(-1) + D[:, None] * x[t]
        ymag[t] = (Smag * Ct.abs()[:, None]).sum(-1) + (D[:, None] * x[t]).abs()
    return y, S, ymag, Smag


def norm(x, kind, eps):
    x = x.to(F64)
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def gated_norm(x, w, gate=None, bias=None, kind="rms", act="silu", gate_first=False, eps=1e-5):
    g = 1.0 if gate is None else _act(gate.to(F64), act)
    x = x.to(F64)
    y = norm(x * g if gate_first else x, kind, eps) * w.to(F64)
    if bias is not None:
        y = y + bias.to(F64)
    return y if gate_first else y * g


def add_norm(x, residual, w, bias=None, scale=None, alpha=1.0, post=None, kind="rms", eps=1e-5):
    x = x.to(F64)
    if post is not None:
        x = norm(x, kind, eps) * post.to(F64)
    h = x * alpha * (1.0 if scale is None else scale.to(F64))
    if residual is not None:
        h = h + residual.to(F64)
    y = norm(h, kind, eps) * w.to(F64)
    return (y if bias is None else y + bias.to(F64)), h
