"""The layer operators around the recurrence, as workloads: the root-mean-square
norm before a layer, the short causal convolution behind its projections, and
the selective state space scan, each for prompts, for single tokens and for
training.

``run`` computes a case in plain torch operations, or, with ``own`` set, through
the entry points of ``chunked_gated_delta_prepare_amd``.  ``exact`` is the same
operator from its definition in 64 bits.

    norm   s = x + residual (kept in the residual's type), y = s r w with
           r = 1 / sqrt(mean(s^2) + eps); y in the io type or in e4m3 with one
           scale per row or per 128 columns
    conv   y_t = silu(b + sum_j w_{W-1-j} x_{t-j}), over at most W tokens of one
           sequence; the state is the last W - 1 inputs
    ssm    h_t = e^{dt_t A} h_{t-1} + dt_t B_t x_t^T,  y_t = h_t^T C_t + D x_t,
           dt = softplus(raw + bias); B and C are shared by the heads of a group
"""
import math

import torch

own = False

EPS = 1e-6
W = 4                      # taps of the convolution
E4M3_MAX = 448.0
TINY = 2.0 ** -126         # the least scale: a group of zeros has this one
QCHUNK = 128               # tokens per block of the plain scan
FP8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one decode step of 32 sequences: latency
        dict(name="norm_decode", op="norm", mode="infer", rows=32, D=4096, io="bf16", res="bf16", out="fp8", group=0),
        # a long prompt of a wide model, the rows feeding an 8-bit projection
        dict(name="norm_prompt", op="norm", mode="infer", rows=16384, D=8192, io="bf16", res="bf16", out="fp8", group=128),
        # a training step, 16-bit residual stream
        dict(name="norm_train", op="norm", mode="train", rows=16384, D=4096, io="bf16", res="bf16", out="io", group=0),
        # a training step with a 32-bit residual stream and a width that is no multiple of anything
        dict(name="norm_odd", op="norm", mode="train", rows=1003, D=2050, io="bf16", res="fp32", out="io", group=0),
        # one decode step: the states of 64 of 80 slots move on, two rows are padding
        dict(name="conv_decode", op="conv", mode="step", B=64, slots=80, pad=2, D=10240, io="bf16"),
        # prompts packed behind each other, some empty or of one token, some with a state to go on from
        dict(name="conv_packed", op="conv", mode="packed", seqs=9, T=16384, D=10240, io="bf16"),
        # a training step on two sequences
        dict(name="conv_train", op="conv", mode="train", B=2, T=8192, D=6144, io="bf16"),
        # one decode step over states of 64 KB a head
        dict(name="ssm_decode", op="ssm", mode="step", B=64, slots=80, pad=2, H=64, P=128, N=128, G=8, io="bf16", dt="bf16"),
        # the shortest prompts
        dict(name="ssm_short", op="ssm", mode="prompt", B=1, T=37, H=32, P=64, N=64, G=1, io="bf16", dt="bf16", h0=False),
        # one long sequence, the longest that this repository times
        dict(name="ssm_long", op="ssm", mode="prompt", B=1, T=65536, H=64, P=128, N=128, G=8, io="bf16", dt="bf16", h0=True),
        # packed prompts of ragged lengths going on from states
        dict(name="ssm_packed", op="ssm", mode="packed", seqs=9, T=16384, H=80, P=64, N=128, G=1, io="bf16", dt="bf16", h0=True),
        # a training step: every gradient
        dict(name="ssm_train", op="ssm", mode="train", B=2, T=8192, H=32, P=128, N=128, G=4, io="bf16", dt="bf16", h0=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "conv", "ssm"))
    io = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    if op == "norm":
        D = _log_int(rng, 64, 8192)
        D = D // 128 * 128 + 128 if rng.random() < 0.5 else D
        rows = _log_int(rng, 1, min(16384, (1 << 26) // D))
        if rng.random() < 0.5:
            return dict(op=op, mode="train", rows=rows, D=D, io=io, res=rng.choice((io, "fp32")), out="io", group=0)
        return dict(op=op, mode="infer", rows=rows, D=D, io=io, res=rng.choice((io, "fp32", "none")),
                    out=rng.choice(("io", "fp8", "fp8")), group=rng.choice((0, 128)))
    if op == "conv":
        mode = rng.choice(("step", "packed", "train"))
        D = _log_int(rng, 64, 10240)
        D = D // 64 * 64 + 64 if rng.random() < 0.7 else D
        if mode == "step":
            B = _log_int(rng, 1, 256)
            return dict(op=op, mode=mode, B=B, slots=B + rng.randrange(20), pad=rng.randrange(min(B, 3)), D=D, io=io)
        if mode == "packed":
            seqs = rng.randrange(1, 13)
            return dict(op=op, mode=mode, seqs=seqs, T=_log_int(rng, 16, min(16384, (1 << 26) // D)), D=D, io=io)
        B = rng.randrange(1, 4)
        return dict(op=op, mode=mode, B=B, T=_log_int(rng, 1, min(8192, (1 << 25) // (D * B))), D=D, io=io)
    mode = rng.choice(("step", "prompt", "packed", "train"))
    G = rng.choice((1, 2, 4))
    H, P, N = G * rng.randrange(1, 64 // G + 1), rng.choice((64, 128)), rng.choice((64, 128))
    dt = rng.choice((io, "fp32"))
    if mode == "step":
        B = _log_int(rng, 1, 96)
        return dict(op=op, mode=mode, B=B, slots=B + rng.randrange(20), pad=rng.randrange(min(B, 3)), H=H, P=P, N=N, G=G, io=io, dt=dt)
    room = (1 << 25) // (H * P)
    if mode == "packed":
        return dict(op=op, mode=mode, seqs=rng.randrange(1, 13), T=_log_int(rng, 16, min(8192, room)), H=H, P=P, N=N, G=G, io=io, dt=dt, h0=rng.random() < 0.5)
    B = rng.randrange(1, 4)
    return dict(op=op, mode=mode, B=B, T=_log_int(rng, 1, min(8192, room // B)), H=H, P=P, N=N, G=G, io=io, dt=dt, h0=rng.random() < 0.5)


def _lengths(n, T):
    """n lengths that sum to T: ragged, with an empty and a one-token sequence where there are enough."""
    share = [((7 * i + 3) % 11 + 1) ** 2 for i in range(n)]
    if n >= 4:
        share[1] = 0
        share[2] = 0
    out = [T * s // sum(share) for s in share]
    if n >= 4 and T >= 16:
        out[2] = 1
    out[-1] += T - sum(out)
    return out


def _size(c):
    return 2 if c["io"] == "bf16" else 4


def work(case):
    c, e = case, 2 if case["io"] == "bf16" else 4
    if c["op"] == "norm":
        n, D, r = c["rows"] * c["D"], c["D"], {"bf16": 2, "fp32": 4, "none": 0}[c["res"]]
        if c["mode"] == "infer":
            q = (1 if c["out"] == "fp8" else e) * n
            s = 4 * c["rows"] * (-(-D // c["group"]) if c["group"] else 1) if c["out"] == "fp8" else 0
            return dict(bytes=n * (e + 2 * r) + q + s + e * D, flops=6 * n)
        # in: x, residual, dy, dres, w; out: y, s, the gradients of x and of the residual, dw
        return dict(bytes=n * (2 * e + 2 * r) + n * (e + 2 * r + (e if c["res"] != c["io"] else 0)) + (e + 4) * D, flops=20 * n)
    if c["op"] == "conv":
        D = c["D"]
        if c["mode"] == "step":
            live = c["B"] - c["pad"]
            return dict(bytes=e * D * (2 * c["B"] + 2 * (W - 1) * live + W + 1), flops=(2 * W + 6) * D * live)
        if c["mode"] == "packed":
            return dict(bytes=e * D * (2 * c["T"] + 2 * (W - 1) * c["seqs"] + W + 1), flops=(2 * W + 6) * D * c["T"])
        n = c["B"] * c["T"] * D
        return dict(bytes=4 * e * n + D * (W + 1) * (e + 4), flops=(8 * W + 20) * n)
    H, P, N, G, d = c["H"], c["P"], c["N"], c["G"], 2 if c["dt"] == "bf16" else 4
    tok = e * (2 * H * P + 2 * G * N) + d * H
    if c["mode"] == "step":
        live = c["B"] - c["pad"]
        return dict(bytes=c["B"] * tok + 8 * live * H * P * N, flops=6 * live * H * P * N)
    T = c["T"] * c.get("B", 1)
    states = 4 * c.get("B", c.get("seqs", 1)) * H * P * N * (2 if c["h0"] else 1)
    # the recurrence's own products: the state's update and its read-out
    if c["mode"] != "train":
        return dict(bytes=T * tok + states, flops=4 * T * H * P * N)
    return dict(bytes=T * (2 * tok - d * H + e * H * P + d * H) + states * 2, flops=12 * T * H * P * N)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else torch.device("cpu")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    io = DT[c["io"]]

    def normal(*shape, scale=1.0, dtype=io):
        return (torch.randn(*shape, device=dev, generator=g) * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, device=dev, generator=g) * (hi - lo) + lo

    def slots_of(n, pool, pad):
        # the rows' places in the pool; a row of padding has none
        idx = torch.randperm(pool, device=dev, generator=g)[:n].to(torch.int32)
        if pad:
            idx[n - pad:] = -1
        return idx

    s = {"case": c}
    if c["op"] == "norm":
        R, D = c["rows"], c["D"]
        s["x"] = normal(R, D)
        s["residual"] = None if c["res"] == "none" else normal(R, D, scale=3.0, dtype=DT[c["res"]])
        s["weight"] = (1.0 + 0.1 * torch.randn(D, device=dev, generator=g)).to(io)
        if c["mode"] == "train":
            s["dy"] = normal(R, D)
            s["dres"] = normal(R, D, dtype=DT[c["res"]])
        return s
    if c["op"] == "conv":
        D = c["D"]
        s["weight"] = normal(D, W, scale=0.5)
        s["bias"] = normal(D, scale=0.1)
        if c["mode"] == "step":
            s["x"] = normal(c["B"], D)
            s["state"] = normal(c["slots"], W - 1, D)
            s["slots"] = slots_of(c["B"], c["slots"], c["pad"])
        elif c["mode"] == "packed":
            s["x"] = normal(1, c["T"], D)
            s["state"] = normal(c["seqs"], W - 1, D)
            s["cu"] = torch.tensor([0] + _lengths(c["seqs"], c["T"]), device=dev).cumsum(0).to(torch.int32)
        else:
            s["x"] = normal(c["B"], c["T"], D)
            s["dy"] = normal(c["B"], c["T"], D)
        return s
    H, P, N, G = c["H"], c["P"], c["N"], c["G"]
    s["A"] = -uniform(H, lo=1.0, hi=16.0)
    s["D"] = 1.0 + 0.1 * torch.randn(H, device=dev, generator=g)
    # softplus(bias) spread evenly over the logarithm of [0.001, 0.1]
    dt0 = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))
    lead = (c["B"],) if c["mode"] == "step" else (c.get("B", 1), c["T"])
    # x, B and C leave the convolution in one buffer, side by side
    xbc = torch.nn.functional.silu(torch.randn(*lead, H * P + 2 * G * N, device=dev, generator=g)).to(io)
    s["x"] = xbc[..., :H * P].unflatten(-1, (H, P))
    s["B"] = xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N))
    s["C"] = xbc[..., H * P + G * N:].unflatten(-1, (G, N))
    s["dt"] = normal(*lead, H, dtype=DT[c["dt"]])
    if c["mode"] == "step":
        s["state"] = normal(c["slots"], H, N, P, scale=0.1, dtype=torch.float32)
        s["slots"] = slots_of(c["B"], c["slots"], c["pad"])
        return s
    n = c["seqs"] if c["mode"] == "packed" else c["B"]
    s["h0"] = normal(n, H, N, P, scale=0.1, dtype=torch.float32) if c["h0"] else None
    if c["mode"] == "packed":
        s["cu"] = torch.tensor([0] + _lengths(n, c["T"]), device=dev).cumsum(0).to(torch.int32)
    if c["mode"] == "train":
        s["dy"] = normal(c["B"], c["T"], H, P)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _norm_plain(x, residual, weight, out, group):
    s = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    f = s.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * weight.float()
    if out == "io":
        return y.to(x.dtype), s, None
    R, D = y.shape
    g = group or D
    pad = -D % g
    blocks = torch.nn.functional.pad(y, (0, pad)).view(R, -1, g)
    scale = (blocks.abs().amax(-1) / E4M3_MAX).clamp(min=TINY)
    q = (blocks / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(FP8)
    return q.view(R, -1)[:, :D], s, scale


def _norm_grad_plain(dy, s, weight, dres):
    f, w, d = s.float(), weight.float(), dy.float()
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    u = d * w
    ds = dres.float() + r * (u - f * r.square() * (u * f).mean(-1, keepdim=True))
    return ds, (d * f * r).double().sum(0).float()


def _positions(cu, T):
    """Of every packed token: its sequence, and its place in it."""
    n = torch.diff(cu).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=cu.device), n, output_size=T)
    return seq, torch.arange(T, device=cu.device) - cu.long()[seq]


def _conv_rows(x, state, cu):
    """Every token's W inputs, newest first, from x [T, D] and the states [n, W-1, D]."""
    T, n = x.shape[0], state.shape[0]
    seq, pos = _positions(cu, T)
    j = torch.arange(W, device=x.device)
    p = pos[:, None] - j
    rows = torch.where(p >= 0, n * (W - 1) + torch.arange(T, device=x.device)[:, None] - j, (seq * (W - 1) + W - 1)[:, None] + p)
    both = torch.cat([state.reshape(-1, x.shape[1]), x])
    return both, rows, seq, pos


def _silu_grad(v):
    g = torch.sigmoid(v)
    return g * (1 + v * (1 - g))


def _conv_plain(x, weight, bias, state, cu):
    both, rows, _, _ = _conv_rows(x, state, cu)
    v = (both[rows].float() * weight.float().flip(1).T).sum(1) + bias.float()
    y = (v * torch.sigmoid(v)).to(x.dtype)
    i = torch.arange(W - 1, device=x.device)
    n = torch.diff(cu).long()[:, None]
    p = n + i - (W - 1)
    first = torch.arange(state.shape[0], device=x.device)[:, None] * (W - 1)
    at = torch.where(p >= 0, state.shape[0] * (W - 1) + cu[:-1].long()[:, None] + p, first + (W - 1) + p)
    return y, both[at], v


def _conv_grad_plain(dy, x, weight, bias, cu):
    T, D = x.shape
    state = x.new_zeros(cu.numel() - 1, W - 1, D)
    both, rows, seq, pos = _conv_rows(x, state, cu)
    taps = both[rows].float()
    v = (taps * weight.float().flip(1).T).sum(1) + bias.float()
    dv = dy.float() * _silu_grad(v)
    j = torch.arange(W, device=x.device)
    t = torch.arange(T, device=x.device)[:, None] + j
    inside = pos[:, None] + j < torch.diff(cu).long()[seq][:, None]
    after = dv[t.clamp(max=max(T - 1, 0))] * inside[..., None]
    dx = (after * weight.float().flip(1).T).sum(1)
    dw = (dv[:, None] * taps).double().sum(0).float().flip(0).T
    return dx.to(x.dtype), dw, dv.double().sum(0).float()


def _heads(v, H):
    """[..., G, N] for every one of H heads."""
    return v.repeat_interleave(H // v.shape[-2], -2)


def _decays(g):
    """e^(sum of g over (s, t]) for s <= t, else 0, from g [..., n] in 64 bits."""
    cum = g.cumsum(-1)
    n = g.shape[-1]
    keep = torch.ones(n, n, dtype=torch.bool, device=g.device).tril()
    return torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~keep, -math.inf)).float()


def _ssm_plain(x, dt, A, B, C, D, bias, h0):
    """y [b, T, H, P] in 32 bits and the last state, by blocks of QCHUNK tokens."""
    b, T, H, P = x.shape
    N, pad = B.shape[-1], -T % QCHUNK
    dt = torch.nn.functional.softplus(dt.float() + bias)
    fill = lambda v: torch.nn.functional.pad(v, (0, 0) * (v.dim() - 2) + (0, pad)).unflatten(1, (-1, QCHUNK))  # noqa: E731
    xs, dts, Bs, Cs = fill(x.float()), fill(dt), fill(B.float()), fill(C.float())
    g = (dts.double() * A.double()).permute(0, 1, 3, 2)                      # [b, n, H, Q]
    cum = g.cumsum(-1)
    dtx = xs * dts[..., None]
    scores = torch.matmul(Cs.transpose(2, 3), Bs.permute(0, 1, 3, 4, 2).contiguous()).repeat_interleave(H // B.shape[-2], 2)
    dtx_h = dtx.transpose(2, 3).contiguous()                                 # [b, n, H, Q, P]
    y = torch.matmul(scores * _decays(g), dtx_h)
    Bh = _heads(Bs, H).permute(0, 1, 3, 4, 2)                                # [b, n, H, N, Q]
    ends = torch.matmul((Bh * torch.exp(cum[..., -1:] - cum).float()[..., None, :]).contiguous(), dtx_h)
    start = torch.zeros_like(ends[:, :1]) if h0 is None else h0[:, None]
    ends = torch.cat([start, ends], 1)
    total = torch.nn.functional.pad(cum[..., -1].transpose(1, 2), (1, 0))    # [b, H, n + 1]
    states = torch.matmul(_decays(total), ends.transpose(1, 2).flatten(3)).unflatten(3, (N, P)).transpose(1, 2)
    Ch = _heads(Cs, H).transpose(2, 3) * torch.exp(cum).float()[..., None]
    y = y + torch.matmul(Ch.contiguous(), states[:, :-1].contiguous())
    y = y.transpose(2, 3).reshape(b, T + pad, H, P)[:, :T] + x.float() * D[:, None]
    return y, states[:, -1]


def _pad_packed(v, cu, longest, fill=0.0):
    """[1, T, ...] packed -> [n, longest, ...]."""
    seq, pos = _positions(cu, v.shape[1])
    out = v.new_full((cu.numel() - 1, longest) + v.shape[2:], fill)
    out[seq, pos] = v[0]
    return out, seq, pos


def _ssm_packed_plain(s, c):
    longest = max(_lengths(c["seqs"], c["T"]))
    x, seq, pos = _pad_packed(s["x"], s["cu"], longest)
    # softplus(-inf) = 0: a padded token neither decays the state nor adds to it
    dt, B, C = (_pad_packed(s[k], s["cu"], longest, f)[0] for k, f in (("dt", -math.inf), ("B", 0.0), ("C", 0.0)))
    y, hT = _ssm_plain(x, dt, s["A"], B, C, s["D"], s["dt_bias"], s["h0"])
    return y[seq, pos][None].to(s["x"].dtype), hT


def _ssm_train_plain(s):
    leaves = [s[k].float().requires_grad_() for k in ("x", "dt", "A", "B", "C", "D", "dt_bias")]
    h0 = None if s["h0"] is None else s["h0"].clone().requires_grad_()
    with torch.enable_grad():
        y, hT = _ssm_plain(*leaves, h0)
        grads = torch.autograd.grad(y, leaves + ([h0] if h0 is not None else []), s["dy"].float())
    kinds = [s[k].dtype for k in ("x", "dt", "A", "B", "C", "D", "dt_bias")] + [torch.float32]
    return [y.detach().to(s["x"].dtype), hT.detach()] + [v.to(t) for v, t in zip(grads, kinds)]


def _live(slots):
    """The rows that have a slot, and the slots: a row of padding is sent to a slot behind the pool."""
    return slots >= 0


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        y, kept, scale = _norm_plain(s["x"], s["residual"], s["weight"], c["out"], c["group"])
        if c["mode"] == "infer":
            return {"y": y, "s": None if s["residual"] is None else kept, "scale": scale}
        ds, dw = _norm_grad_plain(s["dy"], kept, s["weight"], s["dres"])
        return {"y": y, "s": kept, "ds": ds.to(kept.dtype), "dx": ds.to(s["x"].dtype), "dw": dw}
    if c["op"] == "conv":
        x = s["x"]
        if c["mode"] == "step":
            live = _live(s["slots"])
            at = s["slots"].long().clamp(min=0)
            taps = torch.cat([s["state"][at], x[:, None]], 1)
            v = (taps.float() * s["weight"].float().T).sum(1) + s["bias"].float()
            y = ((v * torch.sigmoid(v)) * live[:, None]).to(x.dtype)
            s["state"][at[live]] = taps[live, 1:]
            return {"y": y, "state": s["state"]}
        if c["mode"] == "packed":
            y, last, _ = _conv_plain(x[0], s["weight"], s["bias"], s["state"], s["cu"])
            return {"y": y[None], "last": last}
        B, T, D = x.shape
        cu = torch.arange(B + 1, device=x.device) * T
        state = x.new_zeros(B, W - 1, D)
        y, last, _ = _conv_plain(x.flatten(0, 1), s["weight"], s["bias"], state, cu)
        dx, dw, db = _conv_grad_plain(s["dy"].flatten(0, 1), x.flatten(0, 1), s["weight"], s["bias"], cu)
        return {"y": y.view_as(x), "last": last, "dx": dx.view_as(x), "dw": dw, "db": db}
    if c["mode"] == "step":
        live = _live(s["slots"])
        at = s["slots"].long().clamp(min=0)
        dt = torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"])
        B, C = (_heads(s[k].float(), c["H"]) for k in ("B", "C"))
        xf = s["x"].float()
        h = s["state"][at] * torch.exp(dt * s["A"])[..., None, None] + B[..., None] * (dt[..., None] * xf)[..., None, :]
        y = ((h * C[..., None]).sum(-2) + s["D"][:, None] * xf) * live[:, None, None]
        s["state"][at[live]] = h[live]
        return {"y": y.to(s["x"].dtype), "state": s["state"]}
    if c["mode"] == "packed":
        y, hT = _ssm_packed_plain(s, c)
        return {"y": y, "hT": hT}
    if c["mode"] == "prompt":
        y, hT = _ssm_plain(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dt_bias"], s["h0"])
        return {"y": y.to(s["x"].dtype), "hT": hT}
    return _ssm_train_plain(s)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import chunked_gated_delta_prepare_amd as gdn
    c = s["case"]
    if c["op"] == "norm":
        out = FP8 if c["out"] == "fp8" else None
        y, kept, scale = gdn.norm_forward(s["x"], s["weight"], s["residual"], eps=EPS, out_dtype=out, group=c["group"])
        if c["mode"] == "infer":
            return {"y": y, "s": kept, "scale": scale}
        ds, dx, dw = gdn.norm_backward(s["dy"], kept, s["weight"], s["dres"], eps=EPS, x_dtype=s["x"].dtype)
        return {"y": y, "s": kept, "ds": ds, "dx": dx, "dw": dw}
    if c["op"] == "conv":
        if c["mode"] == "step":
            return {"y": gdn.conv_step(s["x"], s["state"], s["weight"], s["bias"], activation="silu", slots=s["slots"]), "state": s["state"]}
        if c["mode"] == "packed":
            y, last = gdn.conv_forward(s["x"], s["weight"], s["bias"], activation="silu", initial_state=s["state"], cu_seqlens=s["cu"])
            return {"y": y, "last": last}
        y, last = gdn.conv_forward(s["x"], s["weight"], s["bias"], activation="silu")
        dx, dw, db, _ = gdn.conv_backward(s["dy"], s["x"], s["weight"], s["bias"], activation="silu")
        return {"y": y, "last": last, "dx": dx, "dw": dw, "db": db}
    if c["mode"] == "step":
        y = gdn.ssm_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], s["D"], s["dt_bias"], dt_softplus=True, slots=s["slots"])
        return {"y": y, "state": s["state"]}
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dt_bias"], s["h0"])
    y, hT = gdn.ssm_forward(*args, dt_softplus=True, cu_seqlens=s.get("cu"))
    if c["mode"] != "train":
        return {"y": y, "hT": hT}
    dx, ddt, dA, dB, dC, dD, dbias, dh0 = gdn.ssm_backward(s["dy"], *args, dt_softplus=True)
    return [y, hT, dx, ddt, dA, dB, dC, dD, dbias] + ([dh0] if s["h0"] is not None else [])


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(s, c):
    x, w = s["x"].double(), s["weight"].double()
    # the norm is taken of the row as it is kept
    kept = x if s["residual"] is None else (x + s["residual"].double()).to(s["residual"].dtype).double()
    if s["residual"] is not None and s["residual"].dtype == torch.bfloat16:
        # through 32 bits, as a sum of two bf16 numbers is rounded
        kept = (x + s["residual"].double()).float().to(torch.bfloat16).double()
    rms = torch.sqrt((kept * kept).sum(-1) / c["D"] + EPS)
    y = kept / rms[:, None] * w
    if c["mode"] == "infer":
        scale = None
        if c["out"] == "fp8":
            g = c["group"] or c["D"]
            cols = [y[:, k:k + g] for k in range(0, c["D"], g)]
            scale = torch.stack([(v.abs().max(1).values / E4M3_MAX).clamp(min=TINY) for v in cols], 1)
            y = torch.cat([v / scale[:, k:k + 1] for k, v in enumerate(cols)], 1)
        return {"y": y, "s": None if s["residual"] is None else kept, "scale": scale}
    dy, dres = s["dy"].double(), s["dres"].double()
    hat = kept / rms[:, None]
    inner = (dy * w * hat).sum(-1, keepdim=True) / c["D"]
    ds = dres + (dy * w - hat * inner) / rms[:, None]
    return {"y": y, "s": kept, "ds": ds, "dx": ds, "dw": (dy * hat).sum(0)}


def _exact_conv(s, c):
    w, b, x = s["weight"].double(), s["bias"].double(), s["x"].double()
    if c["mode"] == "step":
        pool, y = s["state"].double(), torch.zeros_like(x)
        for row, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                line = torch.cat([pool[slot], x[row:row + 1]])
                v = b + sum(w[:, j] * line[j] for j in range(W))
                y[row] = v / (1 + torch.exp(-v))
                pool[slot] = line[1:]
        return {"y": y, "state": pool}
    train = c["mode"] == "train"
    lens = [c["T"]] * c["B"] if train else _lengths(c["seqs"], c["T"])
    flat, at, ys, last = x.flatten(0, 1), 0, [], []
    dxs, dw, db = [], torch.zeros_like(w), torch.zeros_like(b)
    for k, n in enumerate(lens):
        before = torch.zeros(W - 1, c["D"], dtype=w.dtype, device=w.device) if train else s["state"][k].double()
        line = torch.cat([before, flat[at:at + n]])
        v = b + sum(w[:, j] * line[j:j + n] for j in range(W))
        ys.append(v / (1 + torch.exp(-v)))
        last.append(line[n:])
        if train:
            sg = 1 / (1 + torch.exp(-v))
            dv = s["dy"].double()[k] * (sg + v * sg * (1 - sg))
            dline = torch.zeros_like(line)
            for j in range(W):
                dline[j:j + n] += w[:, j] * dv
                dw[:, j] += (dv * line[j:j + n]).sum(0)
            db += dv.sum(0)
            dxs.append(dline[W - 1:])
        at += n
    y = torch.cat(ys).view_as(x)
    if not train:
        return {"y": y, "last": torch.stack(last)}
    return {"y": y, "last": torch.stack(last), "dx": torch.stack(dxs), "dw": dw, "db": db}


def _exact_ssm(s, c):
    H, G, P, N = c["H"], c["G"], c["P"], c["N"]
    A, D = s["A"].double(), s["D"].double()
    raw = s["dt"].double() + s["dt_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    x, B, C = s["x"].double(), s["B"].double(), s["C"].double()
    group = torch.arange(H, device=A.device) // (H // G)

    def token(h, i):
        """One step of every stream: i indexes x and the rest down to [streams, H, .]."""
        h = h * torch.exp(dt[i] * A)[..., None, None] + B[i][..., group, :, None] * (x[i] * dt[i][..., None])[..., None, :]
        return h, torch.matmul(C[i][..., group, None, :], h)[..., 0, :] + D[:, None] * x[i]

    if c["mode"] == "step":
        live = (s["slots"] >= 0).nonzero()[:, 0]
        pool, y = s["state"].double(), torch.zeros_like(x)
        at = s["slots"].long()[live]
        pool[at], y[live] = token(pool[at], live)
        return {"y": y, "state": pool}
    y = torch.zeros_like(x)
    if c["mode"] == "packed":
        lens = _lengths(c["seqs"], c["T"])
        h = torch.zeros(c["seqs"], H, N, P, dtype=A.dtype, device=A.device) if s["h0"] is None else s["h0"].double()
        first = s["cu"][:-1].long()
        order = sorted(range(len(lens)), key=lambda k: -lens[k])
        perm = torch.tensor(order, device=A.device)
        count = [sum(n > t for n in lens) for t in range(max(lens))]
        h, first = h[perm], first[perm]
        for t, k in enumerate(count):
            i = (0, first[:k] + t)
            h[:k], y[i] = token(h[:k], i)
        out = torch.empty_like(h)
        out[perm] = h
        return {"y": y, "hT": out}
    T = c["T"]
    h = torch.zeros(c["B"], H, N, P, dtype=A.dtype, device=A.device) if s["h0"] is None else s["h0"].double()
    keep, every = [], 64
    for t in range(T):
        if c["mode"] == "train" and t % every == 0:
            keep.append(h)
        h, y[:, t] = token(h, (slice(None), t))
    if c["mode"] == "prompt":
        return {"y": y, "hT": h}
    dy = s["dy"].double()
    dx, dB, dC = dy * D[:, None], torch.zeros_like(B), torch.zeros_like(C)
    ddt, dA = torch.zeros_like(dt), torch.zeros_like(A)
    dh = torch.zeros_like(h)
    sum_groups = lambda v: v.unflatten(1, (G, H // G)).sum(2)  # noqa: E731
    for blk in reversed(range(len(keep))):
        hs = [keep[blk]]
        for t in range(blk * every, min(T, blk * every + every)):
            hs.append(token(hs[-1], (slice(None), t))[0])
        for t in reversed(range(blk * every, min(T, blk * every + every))):
            k = t - blk * every
            dC[:, t] = sum_groups(torch.matmul(hs[k + 1], dy[:, t, :, :, None])[..., 0])
            dh = dh + C[:, t][:, group, :, None] * dy[:, t][..., None, :]
            du = torch.matmul(B[:, t][:, group, None, :], dh)[..., 0, :]
            dx[:, t] += du * dt[:, t][..., None]
            dB[:, t] = sum_groups(torch.matmul(dh, (x[:, t] * dt[:, t][..., None])[..., None])[..., 0])
            decay = torch.exp(dt[:, t] * A)
            dg = (dh * hs[k]).flatten(2).sum(-1) * decay
            ddt[:, t] = (du * x[:, t]).sum(-1) + dg * A
            dA += (dg * dt[:, t]).sum(0)
            dh = dh * decay[..., None, None]
    draw_ = ddt * torch.sigmoid(raw)
    out = [y, h, dx, draw_, dA, dB, dC, (dy * x).sum((0, 1, 3)), draw_.sum((0, 1))]
    return out + ([dh] if s["h0"] is not None else [])


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "ssm": _exact_ssm}[case["op"]](s, s["case"])
