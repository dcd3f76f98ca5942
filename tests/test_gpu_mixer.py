"""The mixer operators against their 64-bit definitions.

Tolerances count roundings.  An output of type t is rounded once (half a step:
eps(t) / 2 of its value).  In 32 bits a sum of K terms is off by at most about
K steps of 2^-24 of the sum of its terms' absolute values; exp, the activation
and the roots add a few steps each (the fast 16-bit forms 2^-20, counted as 16).
"""
import numpy as np
import pytest
import torch

from oracle import mixer_model as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def mx():
    from linear_attention_recurrent_gdn_gb300 import build
    build.build()
    from linear_attention_recurrent_gdn_gb300 import mixer
    return mixer


def half(t):
    return torch.finfo(t).eps / 2


def near(got, want, tol, what):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, what
    off = (got - want).abs() - tol
    assert torch.isfinite(got).all() and not (off > 0).any(), \
        "%s: off by %.3g more than allowed" % (what, float(off.max()))


def rnd(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, generator=g)).to(dtype)


def place(rows, layout, T, dtype, fill=0.0):
    """Per-row [t, ...] tensors as one CUDA tensor of the layout (and its lengths)."""
    n = len(rows)
    inner = rows[0].shape[1:]
    if layout == "packed":
        return torch.cat(rows, 0).to(dtype).cuda()
    if layout == "step":
        return torch.cat(rows, 0).to(dtype).cuda()
    x = torch.full((T, n) + tuple(inner), fill, dtype=dtype)
    for i, r in enumerate(rows):
        x[:r.shape[0], i] = r
    if layout == "batch":                 # [n, T, ...] memory, seen token-major
        return x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    return x.cuda()


def take(y, lengths, layout):
    """The rows' [t, ...] of an output."""
    y = y.cpu()
    if layout in ("packed", "step"):
        return list(torch.split(y, list(lengths)))
    return [y[:n, i] for i, n in enumerate(lengths)]


# --------------------------------------------------------------------- conv --
def check_conv(mx, dtype, C, W, lengths, layout="token", bias=True, act="silu", l2=0, hd=0, split=None, fresh=False,
               pool=True, w32=False, seed=0, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    n, T = len(lengths), max(lengths)
    xs = [rnd(g, t, C, dtype=dt) for t in lengths]
    wt = torch.float32 if w32 else dt
    w = rnd(g, C, W, dtype=wt, scale=W ** -0.5)
    b = rnd(g, C, dtype=wt, scale=0.1) if bias else None
    num_slots = n + 3
    state = rnd(g, num_slots, W - 1, C, dtype=dt)
    slots = torch.randperm(num_slots, generator=g)[:n].numpy().astype(np.int32)
    x = place(xs, layout, T, dt, fill=float("nan"))
    if pad:                               # channels of a wider projection: a row stride, an odd start
        wide = torch.full(x.shape[:-1] + (C + pad,), float("nan"), dtype=dt, device="cuda")
        wide[..., shift:shift + C] = x
        x = wide[..., shift:shift + C]
    dev_state = state.cuda() if pool else None
    more = dict(activation=act, l2_channels=l2, head_dim=hd, split=split)
    if layout == "step":
        y = mx.conv_step(x, w.cuda(), b.cuda() if bias else None, slots=slots, state=dev_state, **more)
    else:
        y = mx.conv(x, w.cuda(), b.cuda() if bias else None, slots=slots if pool else None, state=dev_state,
                    lengths=lengths if layout == "packed" or min(lengths) < T else None, fresh=fresh, **more)
    parts = [take(p, lengths, layout) for p in (y if split else (y,))]
    want_state = state.clone()
    for i in range(n):
        zero = not pool or (fresh[i] if isinstance(fresh, (list, np.ndarray)) else fresh)
        carried = torch.zeros_like(state[0]) if zero else state[slots[i]]
        yr, cr, mag = ref.conv_row(xs[i], carried, w, b, act, l2, hd)
        got = torch.cat([p[i] for p in parts], -1)
        # |act'| <= 1.1; a head's norm divides by it and spreads the others' errors: twice that over the root
        tol32 = (2 * W + 16) * U * (1.1 * mag)
        if l2:
            heads = ref.conv_row(xs[i], carried, w, b, act)[0][:, :l2].reshape(lengths[i], -1, hd)
            root = torch.sqrt((heads * heads).sum(-1, keepdim=True) + 1e-6)
            spread = tol32[:, :l2].reshape(heads.shape).norm(dim=-1, keepdim=True)
            th = (tol32[:, :l2].reshape(heads.shape) + spread + (hd + 4) * U * root) / root
            tol32 = torch.cat([th.reshape(lengths[i], l2), tol32[:, l2:]], 1)
        tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
        near(got, yr, half(dt) * yr.abs() + tol32 + tiny, "y of row %d" % i)
        want_state[slots[i]] = cr.to(dt)
    if pool:
        assert torch.equal(dev_state.cpu(), want_state)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C", [1, 7, 64, 264, 1030])
def test_conv_sizes(mx, dtype, W, C):
    check_conv(mx, dtype, C, W, [1, 5, 0, 33, 64, 2, 3], "packed", seed=C + W)


@pytest.mark.parametrize("layout", ["token", "batch", "packed", "step"])
@pytest.mark.parametrize("fresh", [False, True, "some"])
def test_conv_layouts_and_carried_inputs(mx, layout, fresh):
    lengths = [1] * 5 if layout == "step" else [70, 0, 1, 31, 97]
    if layout == "step" and fresh:
        pytest.skip("a step continues its rows")
    check_conv(mx, "bf16", 200, 4, lengths, layout, fresh=[1, 0, 1, 0, 0] if fresh == "some" else fresh, seed=3)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("hd", [8, 64, 128, 256])
def test_conv_heads(mx, dtype, hd):
    check_conv(mx, dtype, 5 * hd, 4, [3, 40, 1], "packed", bias=False, l2=2 * hd, hd=hd, split=(hd, hd, 3 * hd), seed=hd)
    check_conv(mx, dtype, 3 * hd + 5, 3, [1] * 4, "step", l2=3 * hd, hd=hd, split=(hd, 2 * hd + 5), seed=hd + 1)


def test_conv_odd_ranges_strides_and_starts(mx):
    check_conv(mx, "bf16", 37, 4, [9, 40], "token", split=(3, 17, 1, 16), seed=1)
    check_conv(mx, "bf16", 64, 4, [9, 40], "token", pad=24, shift=8, seed=2)
    check_conv(mx, "bf16", 64, 4, [9, 40], "packed", pad=3, shift=1, seed=3)
    check_conv(mx, "fp32", 72, 2, [33, 8], "batch", pad=5, shift=5, act=None, w32=True, seed=4)
    check_conv(mx, "fp16", 72, 2, [1] * 9, "step", pad=8, shift=0, w32=True, seed=5)
    check_conv(mx, "bf16", 48, 3, [6, 6], "token", pool=False, seed=6)


def test_conv_prompt_equals_steps(mx):
    g = torch.Generator().manual_seed(0)
    x, w = rnd(g, 9, 3, 96, dtype=torch.bfloat16).cuda(), rnd(g, 96, 4, dtype=torch.bfloat16).cuda()
    s1, s2 = (torch.zeros(3, 3, 96, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    y = mx.conv(x, w, slots=[2, 0, 1], state=s1, fresh=True)
    z = torch.stack([mx.conv_step(x[t], w, slots=[2, 0, 1], state=s2) for t in range(9)])
    assert torch.equal(y, z) and torch.equal(s1, s2)


def test_conv_many_rows(mx):
    check_conv(mx, "bf16", 16, 4, [i % 5 for i in range(1024)], "packed", seed=9)


def test_conv_infinities_and_nan_stay_in_their_channel_and_window(mx):
    x = torch.zeros(40, 1, 16, device="cuda", dtype=torch.bfloat16)
    x[5, 0, 3], x[5, 0, 4] = float("nan"), float("inf")
    y = mx.conv(x, torch.ones(16, 4, device="cuda", dtype=torch.bfloat16), activation=None)
    bad = ~torch.isfinite(y[:, 0])
    assert bad[5:9, 3:5].all() and int(bad.sum()) == 8


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_conv_activation_of_extreme_values(mx, dtype):
    """Neighbouring channels do not touch each other, whatever their values."""
    top = 6e4 if dtype == "fp16" else 1e30
    row = torch.tensor([1.0, float("nan"), -2.0, float("inf"), 3.0, -top, 0.5, top, -1.0, -100.0, 30.0, -30.0,
                        0.0, -44.0, -0.0, 88.0], dtype=DT[dtype])
    x = row.repeat(1, 3, 1).cuda()          # one token of three rows: a zero weight times inf would be a NaN
    w = torch.zeros(16, 2, device="cuda", dtype=DT[dtype])
    w[:, 1] = 1
    y = mx.conv(x, w)[0].cpu().double()
    want = row.double() * torch.sigmoid(row.double())
    assert torch.isnan(y[:, 1]).all() and (y[:, 3] == float("inf")).all()
    ok = torch.isfinite(want) & torch.isfinite(row.double())
    # below -43 the 16-bit forms give -9e-18
    tol = half(DT[dtype]) * want.abs() + 64 * U * want.abs() + 1e-17 + tiny(DT[dtype])
    assert ((y[:, ok] - want[ok]).abs() <= tol[ok]).all()


# ---------------------------------------------------------------------- ssm --
def check_ssm(mx, dtype, H, G, P, N, lengths, layout="token", fresh=False, pool=True, D=True, bias=True, softplus=True,
              dt32=False, seed=0, decay=(1.0, 16.0), step_scale=1.0, gap=0, mma=False):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    n, T = len(lengths), max(lengths)
    per_row = [[rnd(g, t, H, P, dtype=dt), rnd(g, t, H, dtype=torch.float32 if dt32 else dt, scale=step_scale),
                rnd(g, t, G, N, dtype=dt), rnd(g, t, G, N, dtype=dt)] for t in lengths]
    if not softplus:
        for r in per_row:
            r[1] = (r[1].abs() * 0.1).to(r[1].dtype)
    A = -(decay[0] + (decay[1] - decay[0]) * torch.rand(H, generator=g))
    Dv = rnd(g, H) if D else None
    bv = torch.log(torch.expm1(torch.exp(np.log(1e-3) + np.log(100.0) * torch.rand(H, generator=g)))) if bias else None
    num_slots = n + 2
    state = rnd(g, num_slots, H, P, N, scale=0.3)
    slots = torch.randperm(num_slots, generator=g)[:n].numpy().astype(np.int32)
    dev = [place([r[k] for r in per_row], layout, T, per_row[0][k].dtype, fill=float("nan")) for k in range(4)]
    if gap:                               # x, B and C as slices of one wide tensor
        flat = [dev[k].flatten(-2) for k in (0, 2, 3)]
        wide = torch.cat([torch.zeros_like(flat[0][..., :gap])] + flat, -1)
        a, b = gap + H * P, gap + H * P + G * N
        dev[0] = wide[..., gap:a].unflatten(-1, (H, P))
        dev[2], dev[3] = wide[..., a:b].unflatten(-1, (G, N)), wide[..., b:].unflatten(-1, (G, N))
    pool_dev = state.cuda() if pool else None
    up = lambda v: None if v is None else v.cuda()  # noqa: E731
    args = (dev[0], dev[1], A.cuda(), dev[2], dev[3], up(Dv))
    if layout == "step":
        y = mx.ssm_step(*args, dt_bias=up(bv), dt_softplus=softplus, slots=slots, state=pool_dev)
    else:
        y = mx.ssm(*args, dt_bias=up(bv), dt_softplus=softplus, slots=slots if pool else None, state=pool_dev,
                   lengths=lengths if layout == "packed" or min(lengths) < T else None, fresh=fresh)
    ys = take(y, lengths, layout)
    got = pool_dev.cpu() if pool else None
    touched = set()
    for i in range(n):
        zero = not pool or (fresh[i] if isinstance(fresh, (list, np.ndarray)) else fresh)
        S0 = torch.zeros_like(state[0]) if zero else state[slots[i]]
        yr, Sr, ymag, Smag = ref.ssm_row(*[per_row[i][k] for k in (0, 1)], A, *per_row[i][2:], Dv, S0, bv, softplus)
        # A state element is a chain of at most `len` multiply-adds; its decays' exponents are off by a few
        # steps of their size (a term that has decayed by e^-s is off by 4 s U: at most 4 U s e^-s < 2 U of the
        # undecayed term, counted with the steps).  An output sums N of them.
        steps = 3 * lengths[i] + 16
        near(ys[i], yr, half(dt) * yr.abs() + tiny(dt) + ((steps + N) * U + (2 * half(dt) if mma else 0)) * ymag,
             "y of row %d" % i)
        if pool:
            near(got[slots[i]], Sr, steps * U * Smag + 1e-30, "state of row %d" % i)
            touched.add(int(slots[i]))
    if pool:
        for s in set(range(num_slots)) - touched:
            assert torch.equal(got[s], state[s])


def tiny(dt):
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("P,N", [(1, 1), (5, 16), (40, 24), (64, 64), (33, 72), (128, 128), (64, 200), (16, 256)])
def test_ssm_scan_sizes(mx, dtype, P, N):
    check_ssm(mx, dtype, 2, 1, P, N, [1, 0, 17, 40], "packed", seed=P + N, mma=dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("P,N", [(1, 1), (5, 16), (40, 24), (64, 64), (33, 71), (128, 128), (64, 200), (16, 256)])
def test_ssm_step_sizes(mx, dtype, P, N):
    check_ssm(mx, dtype, 6, 2, P, N, [1] * 5, "step", seed=P + N)


@pytest.mark.parametrize("layout", ["token", "batch", "packed"])
@pytest.mark.parametrize("fresh", [False, True, "some"])
def test_ssm_layouts_and_states(mx, layout, fresh):
    check_ssm(mx, "bf16", 4, 2, 64, 64, [70, 0, 1, 31, 97], layout,
              fresh=[1, 0, 1, 1, 0] if fresh == "some" else fresh, seed=5, mma=True)


@pytest.mark.parametrize("H,G", [(1, 1), (3, 3), (6, 2), (8, 1)])
def test_ssm_groups(mx, H, G):
    check_ssm(mx, "bf16", H, G, 64, 128, [130, 7], "packed", seed=H, mma=True)
    check_ssm(mx, "fp32", H, G, 24, 32, [30, 7], "packed", seed=H)


def test_calls_of_several_launches(mx):
    """More rows than one launch takes, in every layout."""
    check_conv(mx, "bf16", 24, 4, [1] * 600, "step", seed=1)
    check_conv(mx, "fp32", 24, 3, [(i * 7) % 11 for i in range(300)], "token", seed=2)
    check_ssm(mx, "bf16", 2, 1, 8, 16, [1] * 530, "step", seed=3)
    check_ssm(mx, "bf16", 2, 1, 8, 16, [33 + i % 9 for i in range(150)], "token", seed=4, mma=True)
    check_ssm(mx, "fp32", 2, 2, 8, 16, [i % 5 for i in range(300)], "packed", seed=5)


def test_ssm_options(mx):
    check_ssm(mx, "bf16", 4, 1, 64, 64, [50], D=False, bias=False, softplus=False, dt32=True, seed=1, mma=True)
    check_ssm(mx, "fp32", 4, 1, 64, 64, [50, 20], pool=False, seed=2)
    check_ssm(mx, "bf16", 4, 2, 64, 64, [150, 20], "packed", gap=8, seed=3, mma=True)
    check_ssm(mx, "bf16", 4, 2, 64, 64, [150, 20], "packed", gap=3, seed=4, mma=True)
    check_ssm(mx, "fp16", 4, 2, 16, 20, [1] * 3, "step", gap=5, dt32=True, seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("decay,step_scale", [((0.0, 0.001), 1.0), ((200.0, 4000.0), 1.0), ((1.0, 50.0), 40.0)])
def test_ssm_decays(mx, dtype, decay, step_scale):
    """From hardly any decay to states that vanish within a token (e^-x underflows)."""
    check_ssm(mx, dtype, 4, 1, 64, 64, [200], decay=decay, step_scale=step_scale, seed=6, mma=dtype == "bf16")


@pytest.mark.parametrize("n,T,H,P,N", [(1, 1500, 4, 64, 128), (2, 700, 3, 128, 64), (1, 2048, 2, 128, 128)])
def test_ssm_long(mx, n, T, H, P, N):
    check_ssm(mx, "bf16", H, 1, P, N, [T - 37 * i for i in range(n)], "packed", seed=T, mma=True)
    check_ssm(mx, "fp32", H, 1, P, N, [T - 37 * i for i in range(n)], "packed", seed=T)


def test_ssm_prompt_in_pieces_equals_steps(mx):
    g = torch.Generator().manual_seed(0)
    T, n, H, P, N = 12, 3, 4, 64, 64
    x, B, C = rnd(g, T, n, H, P).cuda(), rnd(g, T, n, 1, N).cuda(), rnd(g, T, n, 1, N).cuda()
    dt, A, D = rnd(g, T, n, H).cuda(), -torch.rand(H, generator=g).cuda() - 0.1, torch.ones(H).cuda()
    pools = [torch.zeros(n, H, P, N, device="cuda") for _ in range(2)]
    ys = [torch.cat([mx.ssm(x[a:b], dt[a:b], A, B[a:b], C[a:b], D, slots=[1, 2, 0], state=pools[0])
                     for a, b in ((0, 5), (5, 12))]),
          torch.stack([mx.ssm_step(x[t], dt[t], A, B[t], C[t], D, slots=[1, 2, 0], state=pools[1]) for t in range(T)])]
    for a, b in (ys, pools):
        assert (a - b).abs().max() <= 200 * U * b.abs().max() + 200 * U


def test_ssm_repeats_bitwise(mx):
    g = torch.Generator().manual_seed(1)
    args = [rnd(g, 700, 1, 4, 64, dtype=torch.bfloat16).cuda(), rnd(g, 700, 1, 4, dtype=torch.bfloat16).cuda(),
            -torch.rand(4, generator=g).cuda(), rnd(g, 700, 1, 1, 128, dtype=torch.bfloat16).cuda(),
            rnd(g, 700, 1, 1, 128, dtype=torch.bfloat16).cuda()]
    a, b = mx.ssm(*args), mx.ssm(*args)
    assert torch.equal(a, b)


# -------------------------------------------------------------------- norms --
def norm_tol(dt, w, n, r):
    """Of y = x / root * w: roundings of the mean, the root and the products, in 32 bits."""
    return half(dt) * r.abs() + (n ** 0.5 + 32) * U * (r.abs() + w.double().abs() * 4) + tiny(dt)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows,H,d", [(1, 1, 1), (3, 5, 7), (2, 40, 64), (9, 32, 128), (1, 2, 200), (4, 3, 256),
                                      (3, 1, 257), (2, 2, 1000), (2, 1, 4096), (3, 1, 16384), (2, 1, 12345)])
def test_gated_norm(mx, dtype, kind, rows, H, d):
    g = torch.Generator().manual_seed(d)
    dt = DT[dtype]
    x, gate = rnd(g, rows, H, d, dtype=dt), rnd(g, rows, H, d, dtype=dt, scale=3.0)
    for heads, bias, act, first, w32 in ((False, False, "silu", False, False), (True, True, "sigmoid", True, True),
                                         (True, False, "silu", True, False), (False, True, None, False, True)):
        wt = torch.float32 if w32 else dt
        shape = (H, d) if heads else (d,)
        w = rnd(g, *shape, dtype=wt) + 1
        b = rnd(g, *shape, dtype=wt) if bias else None
        gt = None if act is None else gate
        y = mx.gated_norm(x.cuda(), w.cuda(), None if gt is None else gt.cuda(), bias=b.cuda() if bias else None,
                          kind=kind, activation=act, gate_first=first)
        want = ref.gated_norm(x, w, gt, b, kind, act, first)
        scale = 1 if gt is None or first else 1 + gate.double().abs()
        # a layer norm of d values of a gate-first product: its mean cancels at most the largest value's size
        near(y, want, norm_tol(dt, (w.double().abs() + (b.double().abs() if bias else 0)) * scale, d, want),
             "y (%s)" % ((heads, bias, act, first),))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gates_of_extreme_values(mx, dtype, act):
    """Neighbouring values do not touch each other, whatever their gates."""
    top = 6e4 if dtype == "fp16" else 1e30
    gate = torch.tensor([1.0, float("nan"), -2.0, float("inf"), 3.0, -top, 0.5, top, -1.0, -100.0, 30.0, -30.0,
                         0.0, -44.0, -0.0, 88.0], dtype=DT[dtype])
    x = torch.ones(1, 1, 16, dtype=DT[dtype])
    y = mx.gated_norm(x.cuda(), torch.ones(16, device="cuda", dtype=DT[dtype]), gate.view(1, 1, 16).cuda(),
                      activation=act, eps=0.0)[0, 0].cpu().double()
    g = gate.double()
    want = torch.sigmoid(g) * (g if act == "silu" else 1.0)
    assert torch.isnan(y[1]) and y[3] == (float("inf") if act == "silu" else 1.0)
    ok = torch.isfinite(want)
    tol = half(DT[dtype]) * want.abs() + 64 * U * want.abs() + 1e-17 + tiny(DT[dtype])
    assert ((y[ok] - want[ok]).abs() <= tol[ok]).all()


def test_gated_norm_strides_starts_and_in_place(mx):
    g = torch.Generator().manual_seed(0)
    for shift, dt in ((8, torch.bfloat16), (3, torch.bfloat16), (1, torch.float32)):
        wide = rnd(g, 11, 3 * 4 * 64 + 16, dtype=dt)
        dev = wide.cuda()
        x, gate = (v[:, shift:shift + 256].unflatten(1, (4, 64)) for v in (wide, wide.flip(1)))
        xd, gd = (v[:, shift:shift + 256].unflatten(1, (4, 64)) for v in (dev, dev.flip(1)))
        w = rnd(g, 64, dtype=dt) + 1
        want = ref.gated_norm(x, w, gate)
        y = mx.gated_norm(xd, w.cuda(), gd)
        near(y, want, norm_tol(dt, w.double().abs() * (1 + gate.double().abs()), 64, want), "strided")
        z = mx.gated_norm(xd, w.cuda(), gd, out=xd)
        assert z is xd and torch.equal(z, y)


@pytest.mark.parametrize("dtype,res32", [("bf16", False), ("bf16", True), ("fp16", False), ("fp16", True), ("fp32", True)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows,D", [(1, 1), (5, 33), (3, 256), (2, 264), (7, 1000), (2, 4096), (3, 4099), (2, 16384), (1, 16383)])
def test_add_norm(mx, dtype, res32, kind, rows, D):
    g = torch.Generator().manual_seed(D + rows)
    dt = DT[dtype]
    rt = torch.float32 if res32 else dt
    x, res = rnd(g, rows, D, dtype=dt), rnd(g, rows, D, dtype=rt, scale=3.0)
    for post, scale, bias, alpha, w32 in ((False, False, False, 1.0, False), (True, True, True, 0.5, True),
                                          (True, False, False, -2.0, False), (False, True, True, 1.0, False)):
        wt = torch.float32 if w32 else dt
        w, p, s, b = (rnd(g, D, dtype=wt) + 1 for _ in range(4))
        up = lambda v, on: v.cuda() if on else None  # noqa: E731
        y, h = mx.add_norm(x.cuda(), res.cuda(), w.cuda(), bias=up(b, bias), scale=up(s, scale), alpha=alpha,
                           post_weight=up(p, post), kind=kind)
        opt = lambda v, on: v if on else None  # noqa: E731
        wy, wh = ref.add_norm(x, res, w, opt(b, bias), opt(s, scale), alpha, opt(p, post), kind)
        amp = abs(alpha) * (s.double().abs() if scale else 1) * (p.double().abs() if post else 1)
        htol = (D ** 0.5 + 32) * U * (wh.abs() + 4 * amp + res.double().abs())
        near(h, wh, half(rt) * wh.abs() + htol, "h")
        # y takes h in 32 bits: h's error over the root, and the norm's own roundings
        hc = wh - wh.mean(-1, keepdim=True) if kind == "layer" else wh
        root = torch.sqrt((hc * hc).mean(-1, keepdim=True) + 1e-5)
        spread = htol + htol.pow(2).mean(-1, keepdim=True).sqrt() * (1 + hc.abs() / root)
        near(y, wy, norm_tol(dt, w.double().abs() + (b.double().abs() if bias else 0), D, wy)
             + spread / root * w.double().abs() + 4 * (D ** 0.5 + 8) * U * wh.abs().mean(-1, keepdim=True) / root * w.double().abs(), "y")


def test_add_norm_without_residual_strides_and_in_place(mx):
    g = torch.Generator().manual_seed(0)
    x, w = rnd(g, 6, 300, dtype=torch.bfloat16), rnd(g, 256, dtype=torch.bfloat16)
    for shift in (0, 8, 5):
        v = x.cuda()[:, shift:shift + 256]
        y, h = mx.add_norm(v, None, w.cuda())
        assert torch.equal(h, v)
        r = v.clone()
        y2, h2 = mx.add_norm(v, r, w.cuda(), out=v, out_residual=r)
        wy, _ = ref.add_norm(h.cpu(), h.cpu(), w)
        assert y2 is v and h2 is r
        near(y2, wy, norm_tol(torch.bfloat16, w.double().abs(), 256, wy), "in place")


def test_norms_of_zero_rows_and_infinities(mx):
    w = torch.ones(128, device="cuda", dtype=torch.bfloat16)
    x = torch.zeros(3, 2, 128, device="cuda", dtype=torch.bfloat16)
    x[1, 0, 5] = float("nan")
    y = mx.gated_norm(x, w, torch.ones_like(x))
    assert torch.isnan(y[1, 0]).all() and int(torch.isnan(y).sum()) == 128 and (y[0] == 0).all()
    y, h = mx.add_norm(x[:, 0], torch.zeros_like(x[:, 0]), w)
    assert (y[0] == 0).all() and torch.isnan(y[1]).all() and (y[2] == 0).all()


# -------------------------------------------------- streams, graphs, errors --
def test_other_streams_and_graph_capture(mx):
    g = torch.Generator().manual_seed(0)
    n, H, P, N = 3, 4, 64, 64
    x, B, C = (rnd(g, n, *s, dtype=torch.bfloat16).cuda() for s in ((H, P), (1, N), (1, N)))
    dt, A = rnd(g, n, H, dtype=torch.bfloat16).cuda(), -torch.rand(H, generator=g).cuda()
    w, cw = torch.ones(P, device="cuda", dtype=torch.bfloat16), rnd(g, H * P, 4, dtype=torch.bfloat16).cuda()
    pools = [(torch.zeros(n, H, P, N, device="cuda"), torch.zeros(n, 3, H * P, device="cuda", dtype=torch.bfloat16))
             for _ in range(3)]

    def layer(pool):
        z = mx.conv_step(x.flatten(1), cw, slots=[0, 1, 2], state=pool[1]).unflatten(1, (H, P))
        y = mx.ssm_step(z, dt, A, B, C, slots=[0, 1, 2], state=pool[0])
        return mx.add_norm(mx.gated_norm(y, w, x).flatten(1), None, torch.ones(H * P, device="cuda", dtype=y.dtype))[0]

    want = [layer(pools[0]).clone() for _ in range(4)][-1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [layer(pools[1]) for _ in range(4)][-1]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    warm = tuple(p.clone() for p in pools[2])
    with torch.cuda.stream(side):
        layer(warm)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = layer(pools[2])
    for p in pools[2]:
        p.zero_()
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_binding_refusals(mx):
    from linear_attention_recurrent_gdn_gb300 import deltalog as dl
    x = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(64, 4, device="cuda", dtype=torch.bfloat16)
    st = torch.zeros(2, 3, 64, device="cuda", dtype=torch.bfloat16)
    bad = [lambda: mx.conv(x.cpu(), w), lambda: mx.conv(x.double(), w), lambda: mx.conv(x, w.half()),
           lambda: mx.conv(x, w[:32]), lambda: mx.conv(x, w, slots=[0, 1]), lambda: mx.conv(x, w, state=st),
           lambda: mx.conv(x, w, slots=[0], state=st), lambda: mx.conv(x, w, slots=[0, 1], state=st.float()),
           lambda: mx.conv(x, w, slots=[0, 1], state=st[:, :2]), lambda: mx.conv(x[:, 0], w),
           lambda: mx.conv(x[:, 0], w, lengths=[3]), lambda: mx.conv(x, w, out=x[:2]),
           lambda: mx.conv(x.transpose(1, 2), w), lambda: mx.conv(x, w, split=(32, 31)),
           lambda: mx.conv(x.requires_grad_(), w)]
    for call in bad:
        with pytest.raises((TypeError, ValueError, dl.DeltaLogError)):
            call()
    x = x.detach()
    with pytest.raises(dl.DeltaLogError) as e:
        mx.conv(x, w, slots=[1, 1], state=st)
    assert e.value.status == dl.EINVAL and "twice" in str(e.value)
    with pytest.raises(dl.DeltaLogError):
        mx.conv(x, w, lengths=[5, 1])
    h, f = torch.zeros(3, 4, 64, device="cuda"), torch.zeros(3, 1, 64, device="cuda")
    d, A, pool = torch.zeros(3, 4, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(3, 4, 64, 64, device="cuda")
    ok = lambda **k: mx.ssm_step(*[k.get(v, t) for v, t in (("x", h), ("dt", d), ("A", A), ("B", f), ("C", f))],  # noqa: E731
                                 slots=k.get("slots", [0, 1, 2]), state=k.get("state", pool))
    ok()
    for k in (dict(A=A[:3]), dict(A=None), dict(A=A.half()), dict(B=f[:2]), dict(dt=d[:, :3]), dict(state=pool.half()),
              dict(state=pool.transpose(2, 3)), dict(x=h.transpose(1, 2)), dict(slots=[0, 1]), dict(slots=[0, 1, 3])):
        with pytest.raises((TypeError, ValueError, dl.DeltaLogError)):
            ok(**k)
    with pytest.raises(ValueError):
        mx.gated_norm(h, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        mx.add_norm(h[:, 0], h[:, 0].half(), torch.ones(64, device="cuda"))


# ------------------------------------------------------ large offsets --------
def test_offsets_past_32_bits(mx):
    """The last slots, rows and tokens of tensors of more than 2^31 values, against the same ones alone."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    H, P, N = 16, 128, 128
    pool = torch.empty(8200, H, P, N, device="cuda")
    one = torch.randn(1, H, P, N, generator=g, device="cuda")
    pool[8199:] = one
    x, B, C, dt, A = rn(1, H, P), rn(1, 1, N), rn(1, 1, N), rn(1, H), -torch.rand(H, device="cuda")
    y = mx.ssm_step(x, dt, A, B, C, slots=[8199], state=pool)
    z = mx.ssm_step(x, dt, A, B, C, slots=[0], state=one)
    assert torch.equal(y, z) and torch.equal(pool[8199:], one)
    del pool
    T, K = 270000, 100
    x = torch.zeros(T, 8192, device="cuda", dtype=torch.bfloat16)
    x[-K:] = rn(K, 8192)
    w = rn(8192, 4)
    y = mx.conv(x, w, lengths=[T - K, K])
    assert torch.equal(y[-K:], mx.conv(x[-K:].clone(), w, lengths=[K]))
    del y
    h = x.view(T, 128, 64)
    B, C, dt, A = rn(T, 1, 64), rn(T, 1, 64), rn(T, 128), -torch.rand(128, device="cuda")
    y = mx.ssm(h, dt, A, B, C, lengths=[T - K, K])
    z = mx.ssm(h[-K:].clone(), dt[-K:].clone(), A, B[-K:].clone(), C[-K:].clone(), lengths=[K])
    assert torch.equal(y[-K:], z)
    del y
    w = rn(64)
    v = mx.gated_norm(h, w, h)
    assert torch.equal(v[-K:], mx.gated_norm(h[-K:].clone(), w, h[-K:].clone()))
    del v
    w = rn(8192)
    v, r = mx.add_norm(x, x, w)
    v1, r1 = mx.add_norm(x[-K:].clone(), x[-K:].clone(), w)
    assert torch.equal(v[-K:], v1) and torch.equal(r[-K:], r1)


def test_status_word_is_clean(mx):
    """No wait of the tensor-core scan ran out in the tests before."""
    mx.sync()
