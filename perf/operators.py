"""The operators around a recurrence, as cases that can be timed and checked.

Four operators that a linear-attention or state-space layer runs beside its
recurrent state:

  conv        short causal convolution over time with its activation, the L2
              normalisation of the query and key heads, and the carried inputs
  ssm         selective state space scan: per-head decay exp(dt A), input- and
              output maps B and C shared by the heads of a group, skip D
  gated_norm  norm of every head's output, gated
  add_norm    residual sum with its scale, and the norm before the next block

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with this package's kernels.  ``exact`` is the definition in
64 bits, one token after the other.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
CHUNK = 64          # tokens per chunk of the plain scan
L2_EPS, NORM_EPS = 1e-6, 1e-5


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # One decode token of one request with 4 heads of 64: q, k and v's convolution.
        dict(name="conv_step_1x768", op="conv", step=True, dtype="bf16", n=1, T=1, ragged=False,
             fresh=False, H=4, d=64, C=768, W=4, bias=False),
        # 16 contexts of 512 tokens, 32 heads of 128: the prompts of the chunked-prefill workload.
        dict(name="conv_prompt_16x512x12288", op="conv", step=False, dtype="bf16", n=16, T=512,
             ragged=False, fresh=True, H=32, d=128, C=12288, W=4, bias=False),
        # Packed continuations of 24 requests of up to 257 tokens, a channel count that no vector divides.
        dict(name="conv_ragged_24x257x5123", op="conv", step=False, dtype="fp16", n=24, T=257,
             ragged=True, fresh=False, H=0, d=0, C=5123, W=3, bias=True),
        # One decode token of one request, 4 heads.
        dict(name="ssm_step_1x4x64x64", op="ssm", step=True, dtype="bf16", n=1, T=1, ragged=False,
             fresh=False, H=4, G=1, P=64, N=64),
        # One decode token of 256 requests with 32 heads of 128 x 128 states: the serving batch.
        dict(name="ssm_step_256x32x128x128", op="ssm", step=True, dtype="bf16", n=256, T=1,
             ragged=False, fresh=False, H=32, G=4, P=128, N=128),
        # One context of 2048 tokens with 16 heads: few rows, a long axis.
        dict(name="ssm_prompt_1x2048x16", op="ssm", step=False, dtype="bf16", n=1, T=2048,
             ragged=False, fresh=True, H=16, G=1, P=64, N=128),
        # 16 contexts of 512 tokens with 32 heads of 128 x 128.
        dict(name="ssm_prompt_16x512x32", op="ssm", step=False, dtype="bf16", n=16, T=512,
             ragged=False, fresh=True, H=32, G=4, P=128, N=128),
        # Packed continuations in fp32 with odd sizes of head and state.
        dict(name="ssm_ragged_11x203x6_fp32", op="ssm", step=False, dtype="fp32", n=11, T=203,
             ragged=True, fresh=False, H=6, G=2, P=40, N=72),
        # The heads' norm and gate after a decode step of 256 requests.
        dict(name="gated_norm_256x32x128", op="gated_norm", dtype="bf16", rows=256, H=32, d=128,
             kind="rms", act="silu", gate_first=False, bias=False),
        # Per-head layer norm with bias and gate after 8192 prompt tokens of 40 heads of 64.
        dict(name="gated_norm_8192x40x64_layer", op="gated_norm", dtype="bf16", rows=8192, H=40,
             d=64, kind="layer", act="silu", gate_first=False, bias=True),
        # One token's residual sum and norm.
        dict(name="add_norm_1x4096", op="add_norm", dtype="bf16", rows=1, D=4096, kind="rms",
             res32=False, scale=False, post=False, bias=False),
        # 8192 prompt tokens, fp32 residual stream, norms on both sides and a channel-wise residual scale.
        dict(name="add_norm_8192x4096_both", op="add_norm", dtype="bf16", rows=8192, D=4096,
             kind="rms", res32=True, scale=True, post=True, bias=False),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    op = rng.choice(["conv", "ssm", "ssm", "gated_norm", "add_norm"])
    if op == "conv":
        step = rng.random() < 0.4
        heads = rng.random() < 0.5
        H, d = (rng.choice([1, 2, 4, 5, 7, 12, 24, 32]), rng.choice([64, 128])) if heads else (0, 0)
        C = 3 * H * d if heads else log_int(5, 12288)
        C += C == 3072
        T = 1 if step else log_int(2, 4096)
        n = max(1, min(log_int(1, 512), 16 * 512 * 12288 // (T * C)))
        return dict(op=op, step=step, dtype=dtype, n=n, T=T, ragged=not step and rng.random() < 0.5,
                    fresh=not step and rng.random() < 0.4, H=H, d=d, C=C, W=rng.choice([2, 3, 4]),
                    bias=rng.random() < 0.5)
    if op == "ssm":
        step = rng.random() < 0.4
        G = rng.choice([1, 1, 2, 4])
        H = G * rng.choice([1, 2, 3, 5, 8])
        P, N = rng.choice([16, 40, 64, 64, 128, 128]), rng.choice([16, 64, 64, 72, 128, 128])
        T = 1 if step else log_int(2, 4096)
        n = max(1, min(log_int(1, 256), 16 * 512 * 32 * 128 * 128 // (T * H * P * N), 16 * 512 * 32 // (T * H)))
        return dict(op=op, step=step, dtype=dtype, n=n, T=T, ragged=not step and rng.random() < 0.5,
                    fresh=not step and rng.random() < 0.4, H=H, G=G, P=P, N=N)
    kind, bias = rng.choice(["rms", "rms", "layer"]), rng.random() < 0.4
    if op == "gated_norm":
        H, d = rng.choice([1, 3, 8, 32, 40]), rng.choice([48, 64, 64, 128, 128, 200, 1024, 2048])
        rows = max(1, min(log_int(1, 8192), 8192 * 40 * 64 // (H * d)))
        return dict(op=op, dtype=dtype, rows=rows, H=H, d=d, kind=kind,
                    act=rng.choice(["silu", "sigmoid"]), gate_first=rng.random() < 0.3, bias=bias)
    D = log_int(33, 16384)
    D += D == 3072
    rows = max(1, min(log_int(1, 8192), 8192 * 4096 // D))
    return dict(op=op, dtype=dtype, rows=rows, D=D, kind=kind, res32=rng.random() < 0.5,
                scale=rng.random() < 0.5, post=rng.random() < 0.4, bias=bias)


def _lengths(case):
    """Tokens of every row: T, or spread over 0 .. T with the first row full."""
    n, T = case["n"], case["T"]
    if not case["ragged"]:
        return np.full(n, T, np.int32)
    return np.array([T if i == 0 else (i * 7919 + 13 * T) % (T + 1) for i in range(n)], np.int32)


# ------------------------------------------------------------------ inputs --
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    s = dict(case=case)
    if case["op"] in ("conv", "ssm"):
        n, T = case["n"], case["T"]
        lengths = _lengths(case)
        total = int(lengths.sum())
        # tokens: [n] for one token each, [T, n] token-major, or packed one after the other
        lead = (n,) if case["step"] else (total,) if case["ragged"] else (T, n)
        num_slots = n + n // 8 + 1
        slots = np.random.RandomState(int(seed) % (1 << 32)).permutation(num_slots)[:n].astype(np.int32)
        s.update(slots=slots, lengths=lengths, num_slots=num_slots,
                 slots_dev=torch.from_numpy(slots.astype(np.int64)).cuda(),
                 lens_dev=torch.from_numpy(lengths.astype(np.int64)).cuda())
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        # a projection's output, and filters that sum to about one
        s.update(x=randn(*lead, C).to(dt), weight=(randn(C, W) / W ** 0.5).to(dt),
                 bias=(0.1 * randn(C)).to(dt) if case["bias"] else None,
                 state=randn(num_slots, W - 1, C).to(dt))
    elif case["op"] == "ssm":
        H, G, P, N = case["H"], case["G"], case["P"], case["N"]
        silu = torch.nn.functional.silu
        # x, B and C as they leave the convolution; step sizes of 0.001 to 0.1, decays A of -1 to -16
        s.update(x=silu(randn(*lead, H, P)).to(dt), B=silu(randn(*lead, G, N)).to(dt),
                 C=silu(randn(*lead, G, N)).to(dt), dt=randn(*lead, H).to(dt),
                 dt_bias=torch.log(torch.expm1(torch.exp(np.log(1e-3) + np.log(100.0) * rand(H)))),
                 A=-(1.0 + 15.0 * rand(H)), D=1.0 + 0.1 * randn(H),
                 state=0.1 * randn(num_slots, H, P, N))
    elif case["op"] == "gated_norm":
        shape = (case["rows"], case["H"], case["d"])
        s.update(x=randn(*shape).to(dt), gate=randn(*shape).to(dt),
                 weight=(1 + 0.1 * randn(*shape[1:])).to(dt),
                 bias=(0.1 * randn(*shape[1:])).to(dt) if case["bias"] else None)
    else:
        rows, D = case["rows"], case["D"]
        s.update(x=randn(rows, D).to(dt),
                 residual=(3 * randn(rows, D)).to(torch.float32 if case["res32"] else dt),
                 weight=(1 + 0.1 * randn(D)).to(dt),
                 bias=(0.1 * randn(D)).to(dt) if case["bias"] else None,
                 scale=(0.5 + 0.1 * randn(D)).to(dt) if case["scale"] else None,
                 post=(1 + 0.1 * randn(D)).to(dt) if case["post"] else None)
    return s


# -------------------------------------------------------------- plain forms --
def _padded(s, x):
    """Tokens as [n, T, ...] in 32 bits, zero past each row's length."""
    case = s["case"]
    if case["step"]:
        return x.float().unsqueeze(1)
    if not case["ragged"]:
        return x.float().transpose(0, 1)
    lens = s["lens_dev"]
    t = torch.arange(case["T"], device="cuda")
    live = t < lens[:, None]
    idx = torch.where(live, (lens.cumsum(0) - lens)[:, None] + t, 0)
    return x[idx].float() * live.view(live.shape + (1,) * (x.dim() - 1))


def _unpadded(s, y):
    """[n, T, ...] back in the tokens' own layout."""
    case = s["case"]
    if case["step"]:
        return y[:, 0]
    if not case["ragged"]:
        return y.transpose(0, 1).contiguous()
    return y[torch.arange(case["T"], device="cuda") < s["lens_dev"][:, None]]


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_conv(s):
    case, W = s["case"], s["case"]["W"]
    x, dt = _padded(s, s["x"]), s["x"].dtype
    carried = s["state"][s["slots_dev"]].float()
    full = torch.cat([torch.zeros_like(carried) if case["fresh"] else carried, x], 1)
    T, w = x.shape[1], s["weight"].float()
    y = sum(full[:, j:j + T] * w[:, j] for j in range(W))
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = y / (1 + torch.exp(-y))
    last = s["lens_dev"][:, None] + torch.arange(W - 1, device="cuda")
    s["state"][s["slots_dev"]] = torch.gather(
        full, 1, last[:, :, None].expand(-1, -1, full.shape[2])).to(dt)
    if not case["H"]:
        return dict(y=_unpadded(s, y.to(dt)), state=s["state"])
    hd = case["H"] * case["d"]
    qk = y[..., :2 * hd].unflatten(-1, (2 * case["H"], case["d"]))
    qk = (qk / torch.sqrt((qk * qk).sum(-1, keepdim=True) + L2_EPS)).flatten(-2)
    return dict(q=_unpadded(s, qk[..., :hd].to(dt)), k=_unpadded(s, qk[..., hd:].to(dt)),
                v=_unpadded(s, y[..., 2 * hd:].to(dt)), state=s["state"])


def _plain_ssm(s):
    case = s["case"]
    H, G, N, dtype = case["H"], case["G"], case["N"], s["x"].dtype
    x, B, C = (_padded(s, s[k]) for k in ("x", "B", "C"))
    T = x.shape[1]
    live = torch.arange(T, device="cuda") < s["lens_dev"][:, None]
    dt = _softplus(_padded(s, s["dt"]) + s["dt_bias"]) * live[:, :, None]
    S0 = s["state"][s["slots_dev"]]
    if case["fresh"]:
        S0 = torch.zeros_like(S0)
    Q = min(CHUNK, T)
    pad = -T % Q
    grow = lambda v: torch.nn.functional.pad(v, (0, 0) * (v.dim() - 2) + (0, pad)).unflatten(1, (-1, Q))  # noqa: E731
    xc, Bc, Cc, dtc = grow(x), grow(B), grow(C), grow(dt)                 # [b, c, Q, ...]
    cum = (dtc.double() * s["A"].double()).cumsum(2)                      # [b, c, Q, H]
    # inside a chunk: pairs i >= j
    diff = (cum[:, :, :, None] - cum[:, :, None]).float()                 # [b, c, i, j, H]
    tri = torch.ones(Q, Q, device="cuda", dtype=torch.bool).tril()
    pair = torch.exp(diff.masked_fill(~tri[:, :, None], float("-inf"))) * dtc[:, :, None]
    scores = torch.einsum("bcign,bcjgn->bcijg", Cc, Bc).repeat_interleave(H // G, -1)
    y = torch.einsum("bcijh,bcjhp->bcihp", scores * pair, xc)
    # what each chunk adds to the state, and the states at the chunks' starts
    Bh = Bc.repeat_interleave(H // G, 3)
    Ch = Cc.repeat_interleave(H // G, 3)
    tail = torch.exp((cum[:, :, -1:] - cum).float()) * dtc
    adds = torch.einsum("bcjhp,bcjhn->bchpn", xc * tail[..., None], Bh)
    steps = torch.nn.functional.pad(cum[:, :, -1].cumsum(1), (0, 0, 1, 0))  # [b, c + 1, H]
    far = steps[:, :, None] - steps[:, None]                               # from start z to start c
    low = torch.ones(far.shape[1], far.shape[1], device="cuda", dtype=torch.bool).tril()
    carry = torch.exp(far.float().masked_fill(~low[:, :, None], float("-inf")))
    starts = torch.einsum("bczh,bzhpn->bchpn", carry, torch.cat([S0[:, None], adds], 1))
    y = y + torch.exp(cum.float())[..., None] * torch.einsum("bcihn,bchpn->bcihp", Ch, starts[:, :-1])
    y = y.flatten(1, 2)[:, :T] + s["D"][:, None] * x
    s["state"][s["slots_dev"]] = starts[:, -1]
    return dict(y=_unpadded(s, y.to(dtype)), state=s["state"])


def _norm(x, kind):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + NORM_EPS)


def _act(z, act):
    sig = 1 / (1 + torch.exp(-z))
    return z * sig if act == "silu" else sig


def _plain_gated_norm(s):
    case, x = s["case"], s["x"].float()
    gate = _act(s["gate"].float(), case["act"])
    y = _norm(x * gate if case["gate_first"] else x, case["kind"]) * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return dict(y=(y if case["gate_first"] else y * gate).to(s["x"].dtype))


def _plain_add_norm(s):
    case, x = s["case"], s["x"].float()
    if s["post"] is not None:
        x = _norm(x, case["kind"]) * s["post"].float()
    if s["scale"] is not None:
        x = x * s["scale"].float()
    h = s["residual"].float() + x
    y = _norm(h, case["kind"]) * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return dict(y=y.to(s["x"].dtype), residual=h.to(s["residual"].dtype))


# ------------------------------------------------------------ own kernels ----
def _own(s):
    from linear_attention_recurrent_gdn_gb300 import mixer
    case, op = s["case"], s["case"]["op"]
    if op == "conv":
        more = {}
        if case["H"]:
            hd = case["H"] * case["d"]
            more = dict(l2_channels=2 * hd, head_dim=case["d"], eps=L2_EPS, split=(hd, hd, hd))
        if case["step"]:
            y = mixer.conv_step(s["x"], s["weight"], s["bias"], slots=s["slots"], state=s["state"], **more)
        else:
            y = mixer.conv(s["x"], s["weight"], s["bias"], slots=s["slots"], state=s["state"],
                           lengths=s["lengths"] if case["ragged"] else None, fresh=case["fresh"], **more)
        if case["H"]:
            return dict(q=y[0], k=y[1], v=y[2], state=s["state"])
        return dict(y=y, state=s["state"])
    if op == "ssm":
        args = (s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"])
        if case["step"]:
            y = mixer.ssm_step(*args, dt_bias=s["dt_bias"], slots=s["slots"], state=s["state"])
        else:
            y = mixer.ssm(*args, dt_bias=s["dt_bias"], slots=s["slots"], state=s["state"],
                          lengths=s["lengths"] if case["ragged"] else None, fresh=case["fresh"])
        return dict(y=y, state=s["state"])
    if op == "gated_norm":
        return dict(y=mixer.gated_norm(s["x"], s["weight"], s["gate"], bias=s["bias"], kind=case["kind"],
                                       activation=case["act"], gate_first=case["gate_first"], eps=NORM_EPS))
    y, h = mixer.add_norm(s["x"], s["residual"], s["weight"], bias=s["bias"], scale=s["scale"],
                          post_weight=s["post"], kind=case["kind"], eps=NORM_EPS)
    return dict(y=y, residual=h)


def run(s):
    if own:
        return _own(s)
    plain = dict(conv=_plain_conv, ssm=_plain_ssm, gated_norm=_plain_gated_norm, add_norm=_plain_add_norm)
    return plain[s["case"]["op"]](s)


# -------------------------------------------------------------------- work --
def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] in ("conv", "ssm"):
        tokens, rows = int(_lengths(case).sum()), case["n"]
        passes = 1 if case["fresh"] else 2        # the carried state is written, and read unless fresh
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        return dict(bytes=e * (2 * tokens * C + C * (W + case["bias"]) + passes * rows * (W - 1) * C),
                    flops=tokens * C * (2 * W + 4))
    if case["op"] == "ssm":
        H, G, P, N = case["H"], case["G"], case["P"], case["N"]
        return dict(bytes=e * tokens * (2 * H * P + 2 * G * N + H) + 12 * H + 4 * passes * rows * H * P * N,
                    flops=4 * tokens * H * P * N)
    if case["op"] == "gated_norm":
        size = case["rows"] * case["H"] * case["d"]
        return dict(bytes=e * (3 * size + (1 + case["bias"]) * case["H"] * case["d"]), flops=10 * size)
    size, r = case["rows"] * case["D"], 4 if case["res32"] else e
    weights = 1 + case["bias"] + case["scale"] + case["post"]
    return dict(bytes=2 * size * (e + r) + e * weights * case["D"], flops=8 * size)


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda v: None if v is None else v.to(torch.float64)  # noqa: E731

    def normalised(v, scale, shift):
        mean = v.mean(-1, keepdim=True) if case["kind"] == "layer" else 0.0
        var = ((v - mean) ** 2).mean(-1, keepdim=True)
        out = (v - mean) * torch.rsqrt(var + NORM_EPS) * scale
        return out if shift is None else out + shift

    if case["op"] == "gated_norm":
        z = f64(s["gate"])
        g = torch.sigmoid(z) * (z if case["act"] == "silu" else 1.0)
        x, w, b = f64(s["x"]), f64(s["weight"]), f64(s["bias"])
        return dict(y=normalised(x * g, w, b) if case["gate_first"] else normalised(x, w, b) * g)
    if case["op"] == "add_norm":
        x = f64(s["x"])
        if case["post"]:
            x = normalised(x, f64(s["post"]), None)
        h = f64(s["residual"]) + (x * f64(s["scale"]) if case["scale"] else x)
        return dict(y=normalised(h, f64(s["weight"]), f64(s["bias"])), residual=h)

    # Token by token; rows that have ended keep their state.
    lengths, slots = _lengths(case), s["slots_dev"]
    begins = np.concatenate([[0], np.cumsum(lengths)[:-1]])

    def tokens_at(t):
        """(rows that have a token t, where those tokens are)"""
        rows = np.nonzero(lengths > t)[0]
        if case["step"]:
            at = rows
        else:
            at = begins[rows] + t if case["ragged"] else t * case["n"] + rows
        return torch.from_numpy(rows).cuda(), torch.from_numpy(np.asarray(at)).cuda()

    flat = lambda v: v if case["step"] or case["ragged"] else v.flatten(0, 1)  # noqa: E731
    pool = f64(s["state"])
    S = pool[slots] * (0.0 if case["fresh"] else 1.0)
    if case["op"] == "conv":
        x, w, b = flat(s["x"]), f64(s["weight"]), f64(s["bias"])
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for t in range(case["T"]):
            rows, at = tokens_at(t)
            window = torch.cat([S[rows], f64(x[at])[:, None]], 1)
            v = torch.einsum("rwc,cw->rc", window, w)
            v = v if b is None else v + b
            y[at] = v * torch.sigmoid(v)
            S[rows] = window[:, 1:]
        pool[slots] = S
        y = y.view(s["x"].shape)
        if not case["H"]:
            return dict(y=y, state=pool)
        parts = y.unflatten(-1, (3, case["H"], case["d"])).unbind(-3)
        unit = lambda v: (v * torch.rsqrt(v.square().sum(-1, keepdim=True) + L2_EPS)).flatten(-2)  # noqa: E731
        return dict(q=unit(parts[0]), k=unit(parts[1]), v=parts[2].flatten(-2), state=pool)
    x, B, C, raw = (flat(s[k]) for k in ("x", "B", "C", "dt"))
    A, D, bias, per = f64(s["A"]), f64(s["D"]), f64(s["dt_bias"]), case["H"] // case["G"]
    y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for t in range(case["T"]):
        rows, at = tokens_at(t)
        whole = len(rows) == case["n"]
        step = torch.logaddexp(f64(raw[at]) + bias, torch.zeros_like(bias))
        xt, Bt, Ct = f64(x[at]), f64(B[at]).repeat_interleave(per, 1), f64(C[at]).repeat_interleave(per, 1)
        St = S if whole else S[rows]
        St.mul_(torch.exp(step * A)[:, :, None, None])
        St.add_((step[:, :, None] * xt)[..., None] * Bt[:, :, None])
        y[at] = torch.matmul(St, Ct[..., None])[..., 0] + D[:, None] * xt
        if not whole:
            S[rows] = St
    pool[slots] = S
    return dict(y=y.view(s["x"].shape), state=pool)
