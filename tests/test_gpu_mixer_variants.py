"""The variants of the mixer kernels that a call's size chooses, each against the 64-bit definition.

Each test says which variant its sizes reach.  Tolerances are those of
test_gpu_mixer.py, where they are derived.
"""
import threading

import pytest
import torch

from oracle import mixer_model as ref
from test_gpu_mixer import DT, U, check_conv, check_ssm, half, mx, norm_tol, rnd  # noqa: F401  (mx is a fixture)

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------- single tokens --
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("P,N", [(33, 71), (64, 72), (40, 16), (64, 200), (9, 256)])
def test_step_of_many_slots(mx, dtype, P, N):
    """Eight rows of the state a warp: 24 x 32 x P / (8 * 32 / lanes a row) >= 608 warps."""
    check_ssm(mx, dtype, 32, 4, P, N, [1] * 24, "step", seed=P + N)


# ---------------------------------------------------------------- convolution --
LENGTHS = [33 + (7 * i) % 23 for i in range(125)] + [1, 2, 3, 130]         # 5.6 thousand tokens, 129 rows


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["packed", "token"])
def test_convolution_tiles_longer_than_the_ring(mx, dtype, layout):
    """1040 channels are two blocks wide: tiles of 16 tokens, past the 12 (bf16) or 8 (fp32) places of the ring, with
    ragged tails and rows in two launches."""
    fresh = [i % 3 == 0 for i in range(len(LENGTHS))]
    check_conv(mx, dtype, 1040, 4, LENGTHS, layout, l2=640, hd=64, split=(320, 320, 400), fresh=fresh, seed=1)
    check_conv(mx, dtype, 1040, 3, LENGTHS + [0], layout, act=None, seed=2)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_convolution_tiles_of_64_tokens(mx, dtype):
    """4104 channels are five blocks wide: 7900 tokens make 124 tiles of 64, 620 blocks of the 608 wanted."""
    check_conv(mx, dtype, 4104, 2, [100] * 78 + [37, 65], "packed", bias=False, l2=256, hd=128, split=(4096, 8), seed=3)


def test_convolution_tiles_of_unaligned_channels(mx):
    """The same tiles where no vector divides the channels."""
    check_conv(mx, "bf16", 1037, 4, [0] + LENGTHS, "packed", seed=4)
    check_conv(mx, "fp32", 1037, 2, LENGTHS, "packed", l2=512, hd=256, seed=5)


# ----------------------------------------------------------------- prompt scan --
MIXED = [0, 1, 130, 128, 256, 300, 129, 31, 127, 257, 2, 200]


@pytest.mark.parametrize("layout", ["token", "batch", "packed"])
@pytest.mark.parametrize("gap", [0, 3])
def test_scan_of_more_units_than_ctas(mx, layout, gap):
    """24 rows of 8 heads of 72 state rows: 384 units of 64 rows, more than two CTAs an SM, so that CTAs go on to a
    second unit, with rows of 0 to 3 chunks (tensor copies; with a gap of 3 values, value by value)."""
    lengths = MIXED + [(37 * i) % 150 for i in range(12)]
    check_ssm(mx, "bf16", 8, 2, 72, 40, lengths, layout, fresh=[i % 4 == 1 for i in range(24)], gap=gap, seed=6, mma=True)


@pytest.mark.parametrize("layout", ["token", "batch", "packed"])
@pytest.mark.parametrize("P,N", [(40, 24), (64, 72), (128, 128), (96, 8)])
def test_scan_of_whole_chunks_in_every_layout(mx, layout, P, N):
    """Several rows of whole chunks, whose outputs leave as tensor copies, and sizes that do not fill a box of 64."""
    check_ssm(mx, "bf16", 3, 1, P, N, [260, 128, 256], layout, fresh=[0, 1, 0], seed=7, mma=True)


def test_scan_of_whole_chunks_in_several_launches(mx):
    """More rows than one launch takes, whole chunks and ragged ones."""
    check_ssm(mx, "bf16", 1, 1, 40, 24, [128 + i % 3 for i in range(131)], "token", seed=8, mma=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_scan_segments_of_rows_of_different_lengths(mx, dtype):
    """Rows with many segments, two, one, and without tokens, in one call."""
    check_ssm(mx, dtype, 2, 1, 40, 72, [1100, 0, 150, 64, 700, 33], "packed", fresh=[0, 1, 1, 0, 1, 0], seed=9,
              mma=dtype == "bf16")


# ----------------------------------------------------------------------- norms --
def on_gpu(g, *shape, dtype, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def compare(got, want, tol, what):
    off = (got.double() - want).abs() - tol
    assert torch.isfinite(got).all() and not (off > 0).any(), \
        "%s: off by %.3g more than allowed" % (what, float(off.max()))


# rows, heads, values: a warp with two pieces a lane (33 to 64 pieces of eight), with four (65 to 128); four rows of a
# head a thread (many short rows, their number no multiple of four), heads of 7 to 255 values in lanes of 1 to 32.
GATED = [(155, 2, 264), (155, 2, 265), (311, 1, 512), (155, 2, 520), (311, 1, 1024), (104, 3, 1021),
         (19461, 8, 64), (19461, 8, 56), (19462, 8, 60), (13003, 3, 255), (38915, 1, 256), (415063, 3, 7)]


@pytest.mark.parametrize("rows,H,d", GATED)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_gated_norm_of_many_rows(mx, dtype, rows, H, d):
    g = torch.Generator(device="cuda").manual_seed(d)
    dt = DT[dtype]
    x, gate = on_gpu(g, rows, H, d, dtype=dt), on_gpu(g, rows, H, d, dtype=dt, scale=3.0)
    for heads, bias, act, first, w32, kind in ((True, True, "silu", True, False, "layer"),
                                               (False, False, "sigmoid", False, True, "rms")):
        wt = torch.float32 if w32 else dt
        shape = (H, d) if heads else (d,)
        w = on_gpu(g, *shape, dtype=wt) + 1
        b = on_gpu(g, *shape, dtype=wt) if bias else None
        y = mx.gated_norm(x, w, gate, bias=b, kind=kind, activation=act, gate_first=first)
        want = ref.gated_norm(x, w, gate, b, kind, act, first)
        scale = 1 if first else 1 + gate.double().abs()
        tol = norm_tol(dt, (w.double().abs() + (b.double().abs() if bias else 0)) * scale, d, want)
        if first and kind == "layer":
            # v = x act(gate) is off by some 32 U |v|, its mean by sqrt(d) U of the mean |v|; both over the root, whose
            # own error is the rms of the first
            v = x.double() * gate.double() * torch.sigmoid(gate.double())
            c = v - v.mean(-1, keepdim=True)
            root = torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5)
            rms = (v * v).mean(-1, keepdim=True).sqrt()
            tol = tol + U / root * (w.double().abs() + 1) * ((d ** 0.5 + 32) * (v.abs() + v.abs().mean(-1, keepdim=True))
                                                             + 32 * c.abs() / root * rms)
        compare(y, want, tol, "y (%s)" % ((heads, bias, act, first),))


@pytest.mark.parametrize("rows,D", [(311, 264), (311, 271), (311, 520), (311, 1024), (311, 1003), (38915, 256),
                                    (38915, 200), (38914, 199), (155650, 61)])
@pytest.mark.parametrize("dtype,res32", [("bf16", True), ("bf16", False), ("fp16", True), ("fp32", True)])
def test_add_norm_of_many_rows(mx, dtype, res32, rows, D):
    g = torch.Generator(device="cuda").manual_seed(D)
    dt = DT[dtype]
    rt = torch.float32 if res32 else dt
    x, res = on_gpu(g, rows, D, dtype=dt), on_gpu(g, rows, D, dtype=rt, scale=3.0)
    for post, bias, kind, alpha in ((True, True, "layer", 0.5), (False, False, "rms", 1.0)):
        w, p, s, b = (on_gpu(g, D, dtype=dt) + 1 for _ in range(4))
        y, h = mx.add_norm(x, res, w, bias=b if bias else None, scale=s, alpha=alpha, post_weight=p if post else None,
                           kind=kind)
        wy, wh = ref.add_norm(x, res, w, b if bias else None, s, alpha, p if post else None, kind)
        amp = abs(alpha) * s.double().abs() * (p.double().abs() if post else 1)
        htol = (D ** 0.5 + 32) * U * (wh.abs() + 4 * amp + res.double().abs())
        compare(h, wh, half(rt) * wh.abs() + htol, "h")
        hc = wh - wh.mean(-1, keepdim=True) if kind == "layer" else wh
        root = torch.sqrt((hc * hc).mean(-1, keepdim=True) + 1e-5)
        spread = htol + htol.pow(2).mean(-1, keepdim=True).sqrt() * (1 + hc.abs() / root)
        compare(y, wy, norm_tol(dt, w.double().abs() + (b.double().abs() if bias else 0), D, wy)
                + spread / root * w.double().abs()
                + 4 * (D ** 0.5 + 8) * U * wh.abs().mean(-1, keepdim=True) / root * w.double().abs(), "y")


# --------------------------------------------------------------------- threads --
def test_calls_from_several_host_threads(mx):
    """Every thread has its own launch arguments: the same results from eight at once, each on its own stream."""
    g = torch.Generator().manual_seed(0)
    H, P, N, W = 4, 64, 64, 4
    jobs = []
    for k in range(8):
        T, n = 130 + k, 2 + k % 3
        x, B, C = (rnd(g, T, n, *s, dtype=torch.bfloat16).cuda() for s in ((H, P), (1, N), (1, N)))
        jobs.append((x, rnd(g, T, n, H, dtype=torch.bfloat16).cuda(), -torch.rand(H, generator=g).cuda(), B, C,
                     rnd(g, H * P, W, dtype=torch.bfloat16).cuda(), rnd(g, P, dtype=torch.bfloat16).cuda()))

    def run(job):
        x, dt, A, B, C, cw, w = job
        n = x.shape[1]
        pool = torch.zeros(n, H, P, N, device="cuda")
        z = mx.conv(x.flatten(2), cw).unflatten(2, (H, P))
        y = mx.ssm(z, dt, A, B, C, slots=list(range(n)), state=pool, fresh=True)
        for t in range(3):
            s = mx.ssm_step(z[t], dt[t], A, B[t], C[t], slots=list(range(n)), state=pool)
        return mx.gated_norm(y.flatten(0, 1), w), s, pool

    want = [run(job) for job in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                got = run(jobs[k])
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                    wrong.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# --------------------------------------------------------------------- outputs --
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [8, 3])            # vectors and tensor copies, and values one by one
def test_outputs_in_wider_tensors_and_past_the_rows(mx, dtype, shift):
    """Outputs that are ranges of wider tensors: what lies beside them and past each row's tokens is not written."""
    g = torch.Generator().manual_seed(shift)
    dt, lengths, T, H, P, N = DT[dtype], [300, 0, 128, 77], 300, 2, 64, 64
    n, mark = len(lengths), 7.0
    x, B, C = (rnd(g, T, n, *s, dtype=dt).cuda() for s in ((H, P), (1, N), (1, N)))
    step, A = rnd(g, T, n, H, dtype=dt).cuda(), -torch.rand(H, generator=g).cuda()
    w = rnd(g, H * P, 4, dtype=dt).cuda()
    live = torch.arange(T)[:, None] < torch.tensor(lengths)
    for call in (lambda out: mx.ssm(x, step, A, B, C, lengths=lengths, out=out),
                 lambda out: mx.conv(x.flatten(2), w, lengths=lengths, out=None if out is None else out.flatten(2))):
        want = call(None).view(T, n, H * P)
        wide = torch.full((T, n, H * P + 16), mark, dtype=dt, device="cuda")
        call(wide[..., shift:shift + H * P].unflatten(2, (H, P)))
        got = wide[..., shift:shift + H * P]
        assert torch.equal(got[live], want[live])
        assert (got[~live] == mark).all() and (wide[..., :shift] == mark).all() and (wide[..., shift + H * P:] == mark).all()
    y = wide[:, 0, shift:shift + H * P]
    h = torch.full_like(wide[:, 0], mark)[:, shift:shift + H * P]
    weight = rnd(g, H * P, dtype=dt).cuda()
    a, b = mx.add_norm(x[:, 0].flatten(1), None, weight)
    mx.add_norm(x[:, 0].flatten(1), None, weight, out=y, out_residual=h)
    assert torch.equal(y, a) and torch.equal(h, b)
    assert (wide[:, 0, :shift] == mark).all() and (wide[:, 0, shift + H * P:] == mark).all()
    mx.gated_norm(x[:, 0], weight.view(H, P), x[:, 1], out=y.unflatten(1, (H, P)))
    assert torch.equal(y.unflatten(1, (H, P)), mx.gated_norm(x[:, 0], weight.view(H, P), x[:, 1]))
    assert (wide[:, 0, :shift] == mark).all() and (wide[:, 0, shift + H * P:] == mark).all()
