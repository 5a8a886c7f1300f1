"""More operators of a layer around the recurrence, as workloads: layer norm,
the gated norm behind a recurrence's heads, and the gated linear recurrence of
single channels, each for prompts, for single tokens and for training.

``run`` computes a case in plain torch operations, or, with ``own`` set, through
the entry points of ``chunked_gated_delta_prepare_amd``.  ``exact`` is the same
operator from its definition in 64 bits.

    ln     s = x + residual (kept in the residual's type), y = (s - m) r w + b with
           m = mean(s), r = 1 / sqrt(mean((s - m)^2) + eps); y in the io type or in
           e4m3 with one scale per row or per 128 columns
    gn     rows of one head (or one group of channels): y = n(x) act(z), or, with the
           gate first, y = n(x act(z)); n(s) = s r w with r = 1 / sqrt(mean(s^2) + eps),
           or centred, (s - m) r w + b; w and b of one row, or of each of H
    glr    h_t = a_t h_{t-1} + c_t x_t per channel, y_t = h_t;
           log a = gate ("log"), a = sigmoid(gate + bias) ("sigmoid") or
           log a = -rate sigmoid(gate + bias) ("rate");
           c = 1, 1 - a ("complement") or sqrt(1 - a^2) ("norm")
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126         # the least scale: a group of zeros has this one
FP8 = torch.float8_e4m3fn
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one decode step of 32 sequences: latency
        dict(name="ln_decode", op="ln", mode="infer", rows=32, D=4096, io="bf16", res="bf16", bias=True, out="io", group=0),
        # a long prompt of a wide model, the rows feeding an 8-bit projection
        dict(name="ln_prompt", op="ln", mode="infer", rows=16384, D=8192, io="bf16", res="bf16", bias=True, out="fp8", group=128),
        # a training step, 16-bit residual stream
        dict(name="ln_train", op="ln", mode="train", rows=16384, D=4096, io="bf16", res="bf16", bias=True, out="io", group=0),
        # a training step with a 32-bit residual stream and a width that is no multiple of anything
        dict(name="ln_odd", op="ln", mode="train", rows=1003, D=2050, io="bf16", res="fp32", bias=True, out="io", group=0),
        # one decode step of 64 sequences behind a gated delta layer of 64 heads
        dict(name="gn_decode", op="gn", mode="infer", T=64, H=64, D=128, io="bf16", first=False, center=False, act="silu", each=False),
        # a long prompt behind the same layer, the gate a part of the projection's rows
        dict(name="gn_prompt", op="gn", mode="infer", T=16384, H=64, D=128, io="bf16", first=False, center=False, act="silu", each=False),
        # a training step behind a state space layer: gate first, four groups of channels with weights of their own
        dict(name="gn_train", op="gn", mode="train", T=16384, H=4, D=1024, io="bf16", first=True, center=False, act="silu", each=True),
        # one decode step: the states of 64 of 80 slots move on, two rows are padding
        dict(name="glr_decode", op="glr", mode="step", B=64, slots=80, pad=2, D=4096, io="bf16", gate="bf16", form="rate", scale="norm"),
        # a short prompt in 32 bits from given log decays, a width that is no multiple of anything
        dict(name="glr_short", op="glr", mode="prompt", B=1, T=37, seqs=0, D=1030, io="fp32", gate="fp32", form="log", scale="none", h0=True),
        # one long sequence, the longest that this repository times
        dict(name="glr_long", op="glr", mode="prompt", B=1, T=65536, seqs=0, D=4096, io="bf16", gate="bf16", form="sigmoid", scale="complement", h0=True),
        # packed prompts of ragged lengths going on from states
        dict(name="glr_packed", op="glr", mode="prompt", B=1, T=16384, seqs=9, D=4096, io="bf16", gate="bf16", form="rate", scale="norm", h0=True),
        # a training step: every gradient
        dict(name="glr_train", op="glr", mode="train", B=2, T=8192, seqs=0, D=4096, io="bf16", gate="bf16", form="rate", scale="norm", h0=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("ln", "gn", "glr"))
    io = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    if op == "ln":
        D = _log_int(rng, 64, 8192)
        D = D // 128 * 128 + 128 if rng.random() < 0.5 else D
        rows = _log_int(rng, 1, min(16384, (1 << 26) // D))
        bias = rng.random() < 0.7
        if rng.random() < 0.5:
            return dict(op=op, mode="train", rows=rows, D=D, io=io, res=rng.choice((io, "fp32")), bias=bias, out="io", group=0)
        return dict(op=op, mode="infer", rows=rows, D=D, io=io, res=rng.choice((io, "fp32", "none")), bias=bias,
                    out=rng.choice(("io", "io", "fp8")), group=rng.choice((0, 128)))
    if op == "gn":
        D = _log_int(rng, 32, 4096)
        D = D // 32 * 32 + 32 if rng.random() < 0.7 else D
        H = _log_int(rng, 1, max(1, min(64, 8192 // D)))
        T = _log_int(rng, 1, min(16384, (1 << 25) // (D * H)))
        return dict(op=op, mode=rng.choice(("infer", "train")), T=T, H=H, D=D, io=io, first=rng.random() < 0.4,
                    center=rng.random() < 0.3, act=rng.choice(("silu", "silu", "sigmoid")), each=rng.random() < 0.4)
    mode = rng.choice(("step", "prompt", "prompt", "train"))
    D = _log_int(rng, 64, 8192)
    D = D // 64 * 64 + 64 if rng.random() < 0.7 else D
    form, scale, gate = rng.choice(("log", "sigmoid", "rate")), rng.choice(("none", "complement", "norm")), rng.choice((io, "fp32"))
    if mode == "step":
        B = _log_int(rng, 1, 256)
        return dict(op=op, mode=mode, B=B, slots=B + rng.randrange(20), pad=rng.randrange(min(B, 3)), D=D, io=io, gate=gate, form=form, scale=scale)
    seqs = rng.choice((0, rng.randrange(1, 13)))
    B = 1 if seqs else rng.randrange(1, 4)
    T = _log_int(rng, 16 if seqs else 1, min(16384, (1 << 25) // (D * B)))
    return dict(op=op, mode=mode, B=B, T=T, seqs=seqs, D=D, io=io, gate=gate, form=form, scale=scale, h0=rng.random() < 0.5)


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


def work(case):
    c, e = case, 2 if case["io"] == "bf16" else 4
    D = c["D"]
    if c["op"] == "ln":
        n, r = c["rows"] * D, {"bf16": 2, "fp32": 4, "none": 0}[c["res"]]
        par = (2 if c["bias"] else 1) * D
        if c["mode"] == "infer":
            q = (1 if c["out"] == "fp8" else e) * n
            s = 4 * c["rows"] * (-(-D // c["group"]) if c["group"] else 1) if c["out"] == "fp8" else 0
            return dict(bytes=n * (e + 2 * r) + q + s + e * par, flops=9 * n)
        # in: x, residual, dy, dres, weights; out: y, s, the gradients of x and of the residual, those of the weights
        return dict(bytes=n * (2 * e + 2 * r) + n * (e + 2 * r + (e if c["res"] != c["io"] else 0)) + (e + 4) * par, flops=25 * n)
    if c["op"] == "gn":
        n = c["T"] * c["H"] * D
        par = D * (c["H"] if c["each"] else 1) * (2 if c["center"] else 1)
        if c["mode"] == "infer":
            return dict(bytes=3 * n * e + e * par, flops=12 * n)
        # in: x, z, dy, weights; out: y, the gradients
        return dict(bytes=6 * n * e + (e + 4) * par, flops=40 * n)
    g = 2 if c["gate"] == "bf16" else 4
    par = 4 * D * {"log": 0, "sigmoid": 1, "rate": 2}[c["form"]]
    if c["mode"] == "step":
        live = c["B"] - c["pad"]
        return dict(bytes=c["B"] * D * (2 * e + g) + 8 * live * D + par, flops=12 * live * D)
    n, states = c["B"] * c["T"] * D, (c["seqs"] or c["B"]) * 4 * D * (2 if c["h0"] else 1)
    if c["mode"] != "train":
        return dict(bytes=n * (2 * e + g) + states + par, flops=12 * n)
    return dict(bytes=n * (4 * e + 2 * g) + 2 * states + 2 * par, flops=40 * n)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else torch.device("cpu")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    io, D = DT[c["io"]], c["D"]

    def normal(*shape, scale=1.0, dtype=io):
        return (torch.randn(*shape, device=dev, generator=g) * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, device=dev, generator=g) * (hi - lo) + lo

    s = {"case": c}
    if c["op"] == "ln":
        R = c["rows"]
        s["x"] = normal(R, D)
        s["residual"] = None if c["res"] == "none" else (3.0 * torch.randn(R, D, device=dev, generator=g) + 0.5).to(DT[c["res"]])
        s["weight"] = (1.0 + 0.1 * torch.randn(D, device=dev, generator=g)).to(io)
        s["bias"] = normal(D, scale=0.1) if c["bias"] else None
        if c["mode"] == "train":
            s["dy"] = normal(R, D)
            s["dres"] = normal(R, D, dtype=DT[c["res"]])
        return s
    if c["op"] == "gn":
        T, H = c["T"], c["H"]
        s["x"] = normal(T, H, D, scale=0.5)
        # the gate leaves the projection beside other things
        s["z"] = normal(T, (H + 1) * D)[:, D:].unflatten(-1, (H, D))
        shape = (H, D) if c["each"] else (D,)
        s["weight"] = (1.0 + 0.1 * torch.randn(*shape, device=dev, generator=g)).to(io)
        s["bias"] = normal(*shape, scale=0.1) if c["center"] else None
        if c["mode"] == "train":
            s["dy"] = normal(T, H, D)
        return s
    lead = (c["B"],) if c["mode"] == "step" else (c["B"], c["T"])
    s["bias"] = s["rate"] = None
    if c["form"] == "log":
        # of a projection z: log sigmoid(z) / 16, as memories of some tens of tokens have it
        raw = torch.nn.functional.logsigmoid(torch.randn(*lead, D, device=dev, generator=g)) / 16
    else:
        raw = torch.randn(*lead, D, device=dev, generator=g)
        s["bias"] = uniform(D, lo=1.0, hi=5.0) if c["form"] == "sigmoid" else 0.1 * torch.randn(D, device=dev, generator=g)
    if c["form"] == "rate":
        # e^-rate spread over [0.9, 0.999]
        s["rate"] = -torch.log(uniform(D, lo=0.9, hi=0.999))
    if c["gate"] == c["io"]:
        # x and the gate leave the projection in one buffer, side by side
        both = torch.empty(*lead, 2 * D, device=dev, dtype=io)
        s["x"], s["gate"] = both[..., :D], both[..., D:]
        s["x"].copy_(normal(*lead, D))
        s["gate"].copy_(raw)
    else:
        s["x"], s["gate"] = normal(*lead, D), raw
    if c["mode"] == "step":
        s["state"] = normal(c["slots"], D, dtype=torch.float32)
        # the rows' places in the pool; a row of padding has none
        idx = torch.randperm(c["slots"], device=dev, generator=g)[:c["B"]].to(torch.int32)
        if c["pad"]:
            idx[c["B"] - c["pad"]:] = -1
        s["slots"] = idx
        return s
    n = c["seqs"] or c["B"]
    s["h0"] = normal(n, D, dtype=torch.float32) if c["h0"] else None
    s["cu"] = torch.tensor([0] + _lengths(n, c["T"]), device=dev).cumsum(0).to(torch.int32) if c["seqs"] else None
    if c["mode"] == "train":
        s["dy"] = normal(*lead, D)
        s["dhT"] = normal(n, D, dtype=torch.float32) if c["h0"] else None
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _eight_bits(y, group):
    R, D = y.shape
    g = group or D
    pad = -D % g
    blocks = torch.nn.functional.pad(y, (0, pad)).view(R, -1, g)
    scale = (blocks.abs().amax(-1) / E4M3_MAX).clamp(min=TINY)
    q = (blocks / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(FP8)
    return q.view(R, -1)[:, :D], scale


def _moments(s, center):
    """(s - mean or s, 1 / its root mean square) over the last dimension."""
    if center:
        s = s - s.mean(-1, keepdim=True)
    return s, torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS)


def _norm_grad(u, v, r, center):
    """The gradient of s for that of v r, u, where v = s or s - mean."""
    hat = v * r
    du = u - hat * (u * hat).mean(-1, keepdim=True)
    if center:
        du = du - u.mean(-1, keepdim=True)
    return r * du


def _plain_ln(s):
    c, x, res, w, b = s["case"], s["x"], s["residual"], s["weight"].float(), s["bias"]
    kept = x if res is None else (x.float() + res.float()).to(res.dtype)
    v, r = _moments(kept.float(), True)
    y = v * r * w
    if b is not None:
        y = y + b.float()
    if c["mode"] == "infer":
        scale = None
        if c["out"] == "fp8":
            y, scale = _eight_bits(y, c["group"])
        else:
            y = y.to(x.dtype)
        return {"y": y, "s": None if res is None else kept, "scale": scale}
    d = s["dy"].float()
    ds = s["dres"].float() + _norm_grad(d * w, v, r, True)
    out = {"y": y.to(x.dtype), "s": kept, "ds": ds.to(kept.dtype), "dx": ds.to(x.dtype), "dw": (d * v * r).double().sum(0).float()}
    if b is not None:
        out["db"] = d.double().sum(0).float()
    return out


def _plain_gn(s):
    c, x, z, w = s["case"], s["x"].float(), s["z"].float(), s["weight"].float()
    io = s["x"].dtype
    sg = torch.sigmoid(z)
    act, slope = (z * sg, sg * (1 + z * (1 - sg))) if c["act"] == "silu" else (sg, sg * (1 - sg))
    v, r = _moments(x * act if c["first"] else x, c["center"])
    n = v * r * w
    if c["center"]:
        n = n + s["bias"].float()
    y = n if c["first"] else n * act
    if c["mode"] == "infer":
        return {"y": y.to(io)}
    d = s["dy"].float()
    dn = d if c["first"] else d * act
    ds = _norm_grad(dn * w, v, r, c["center"])
    dx, dz = (ds * act, ds * x * slope) if c["first"] else (ds, d * n * slope)
    rows = 0 if c["each"] else (0, 1)
    out = {"y": y.to(io), "dx": dx.to(io), "dz": dz.to(io), "dw": (dn * v * r).double().sum(rows).float()}
    if c["center"]:
        out["db"] = dn.double().sum(rows).float()
    return out


def _decay(s):
    """a, 1 - a, d(log a) / d(gate) and sigmoid(gate + bias) of every token and channel."""
    form, z = s["case"]["form"], s["gate"].float()
    if form == "log":
        return torch.exp(z), -torch.expm1(z), torch.ones_like(z), None
    z = z + s["bias"]
    sg, other = torch.sigmoid(z), torch.sigmoid(-z)
    if form == "sigmoid":
        return sg, other, other, sg
    la = -s["rate"] * sg
    return torch.exp(la), -torch.expm1(la), la * other, sg


def _input_scale(kind, a, c):
    """c_t of the input, and its derivative by log a."""
    if kind == "none":
        return torch.ones_like(a), torch.zeros_like(a)
    if kind == "complement":
        return c, -a
    k = torch.sqrt(c * (1 + a))
    return k, -a * a / k


def _scan(less, u):
    """h_t = (1 - less_t) h_{t-1} + u_t along dimension 1, by doubling.  (Products of decays
    near 1, rounded to 32 bits, would lose a digit over long memories; what they lack to 1 does not.)"""
    k = 1
    while k < u.shape[1]:
        last, some = u[:, :-k], less[:, :-k]
        u = torch.cat([u[:, :k], u[:, k:] + (last - less[:, k:] * last)], 1)
        less = torch.cat([less[:, :k], less[:, k:] + (some - less[:, k:] * some)], 1)
        k *= 2
    return u


def _bounds(s):
    """Every sequence's first row and length, the rows counted through the batch."""
    c, dev = s["case"], s["x"].device
    if s["cu"] is not None:
        cu = s["cu"].long()
        return cu[:-1], torch.diff(cu)
    first = torch.arange(c["B"], device=dev) * c["T"]
    return first, torch.full_like(first, c["T"])


def _plain_glr(s):
    c, io = s["case"], s["x"].dtype
    a, comp, slope, sg = _decay(s)
    k, dk = _input_scale(c["scale"], a, comp)
    if c["mode"] == "step":
        live = s["slots"] >= 0
        at = s["slots"].long().clamp(min=0)
        h = a * s["state"][at] + k * s["x"].float()
        s["state"][at[live]] = h[live]
        return {"y": (h * live[:, None]).to(io), "state": s["state"]}
    B, T, D = s["x"].shape
    x = s["x"].float()
    first, n = _bounds(s)
    some = n > 0
    head, tail = first[some], (first + n - 1)[some]
    # the chain of tokens is cut in front of every sequence, whose first token takes the state given to it
    chain, u = comp.clone(), k * x
    if s["h0"] is not None:
        u.view(-1, D)[head] += a.view(-1, D)[head] * s["h0"][some]
    chain.view(-1, D)[head] = 1
    h = _scan(chain, u)
    hT = torch.zeros(n.numel(), D, device=x.device) if s["h0"] is None else s["h0"].clone()
    hT[some] = h.view(-1, D)[tail]
    if c["mode"] != "train":
        return {"y": h.to(io), "hT": hT}
    dh = s["dy"].float()
    if s["dhT"] is not None:
        dh = dh.clone()
        dh.view(-1, D)[tail] += s["dhT"][some]
    back = torch.cat([chain[:, 1:], torch.ones_like(chain[:, :1])], 1)
    dh = _scan(back.flip(1), dh.flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    start = torch.zeros_like(hT) if s["h0"] is None else s["h0"]
    before.view(-1, D)[head] = start[some]
    da = a * dh * before + dh * x * dk                  # of log a
    out = {"y": h.to(io), "hT": hT, "dx": (dh * k).to(io), "dgate": (da * slope).to(s["gate"].dtype)}
    if s["bias"] is not None:
        out["dbias"] = (da * slope).double().sum((0, 1)).float()
    if s["rate"] is not None:
        out["drate"] = -(da * sg).double().sum((0, 1)).float()
    if s["h0"] is not None:
        dh0 = s["dhT"].clone()
        dh0[some] = (a * dh).view(-1, D)[head]
        out["dh0"] = dh0
    return out


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import chunked_gated_delta_prepare_amd as gdn
    c = s["case"]
    if c["op"] == "ln":
        out = FP8 if c["out"] == "fp8" else None
        y, kept, scale = gdn.layer_norm_forward(s["x"], s["weight"], s["bias"], s["residual"], eps=EPS, out_dtype=out, group=c["group"])
        if c["mode"] == "infer":
            return {"y": y, "s": kept, "scale": scale}
        ds, dx, dw, db = gdn.layer_norm_backward(s["dy"], kept, s["weight"], s["bias"], s["dres"], eps=EPS, x_dtype=s["x"].dtype)
        return {"y": y, "s": kept, "ds": ds, "dx": dx, "dw": dw} | ({} if db is None else {"db": db})
    if c["op"] == "gn":
        form = dict(eps=EPS, activation=c["act"], gate_first=c["first"], center=c["center"])
        y = gdn.gate_norm_forward(s["x"], s["z"], s["weight"], s["bias"], **form)
        if c["mode"] == "infer":
            return {"y": y}
        dx, dz, dw, db = gdn.gate_norm_backward(s["dy"], s["x"], s["z"], s["weight"], s["bias"], **form)
        return {"y": y, "dx": dx, "dz": dz, "dw": dw} | ({} if db is None else {"db": db})
    form = dict(gate_bias=s["bias"], rate=s["rate"], form=c["form"], scale=None if c["scale"] == "none" else c["scale"])
    if c["mode"] == "step":
        return {"y": gdn.glr_step(s["x"], s["gate"], s["state"], slots=s["slots"], **form), "state": s["state"]}
    y, hT = gdn.glr_forward(s["x"], s["gate"], s["h0"], cu_seqlens=s["cu"], **form)
    if c["mode"] != "train":
        return {"y": y, "hT": hT}
    dx, dgate, dbias, drate, dh0 = gdn.glr_backward(s["dy"], s["x"], s["gate"], s["h0"], s["dhT"], cu_seqlens=s["cu"], **form)
    more = {"dbias": dbias, "drate": drate, "dh0": dh0}
    return {"y": y, "hT": hT, "dx": dx, "dgate": dgate} | {k: v for k, v in more.items() if v is not None}


def run(state):
    if own:
        return _run_own(state)
    return {"ln": _plain_ln, "gn": _plain_gn, "glr": _plain_glr}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_ln(s, c):
    x, w, b = s["x"].double(), s["weight"].double(), 0.0 if s["bias"] is None else s["bias"].double()
    # the norm is taken of the row as it is kept
    kept = x if s["residual"] is None else x + s["residual"].double()
    if s["residual"] is not None and s["residual"].dtype == torch.bfloat16:
        # through 32 bits, as a sum of two bf16 numbers is rounded
        kept = kept.float().to(torch.bfloat16).double()
    elif s["residual"] is not None:
        kept = kept.float().double()
    D = c["D"]
    mean = kept.sum(-1, keepdim=True) / D
    dev = torch.sqrt(((kept - mean) ** 2).sum(-1, keepdim=True) / D + EPS)
    hat = (kept - mean) / dev
    y = hat * w + b
    if c["mode"] == "infer":
        scale = None
        if c["out"] == "fp8":
            g = c["group"] or D
            cols = [y[:, k:k + g] for k in range(0, D, g)]
            scale = torch.stack([(v.abs().max(1).values / E4M3_MAX).clamp(min=TINY) for v in cols], 1)
            y = torch.cat([v / scale[:, k:k + 1] for k, v in enumerate(cols)], 1)
        return {"y": y, "s": None if s["residual"] is None else kept, "scale": scale}
    dy = s["dy"].double()
    dhat = dy * w
    # through hat = (s - mean) / dev: the share of each row that its mean and its deviation take
    inner, total = (dhat * hat).sum(-1, keepdim=True), dhat.sum(-1, keepdim=True)
    ds = s["dres"].double() + (dhat - total / D - hat * inner / D) / dev
    out = {"y": y, "s": kept, "ds": ds, "dx": ds, "dw": (dy * hat).sum(0)}
    if s["bias"] is not None:
        out["db"] = dy.sum(0)
    return out


def _exact_gn(s, c):
    x, z, w = (s[k].double() for k in ("x", "z", "weight"))
    b = s["bias"].double() if c["center"] else 0.0
    e = 1 / (1 + torch.exp(-z))
    gate = z * e if c["act"] == "silu" else e
    dgate = e + z * e * (1 - e) if c["act"] == "silu" else e * (1 - e)
    row = x * gate if c["first"] else x
    mean = row.sum(-1, keepdim=True) / c["D"] if c["center"] else torch.zeros_like(row[..., :1])
    dev = torch.sqrt(((row - mean) ** 2).sum(-1, keepdim=True) / c["D"] + EPS)
    hat = (row - mean) / dev
    normed = hat * w + b
    y = normed if c["first"] else normed * gate
    if c["mode"] == "infer":
        return {"y": y}
    dy = s["dy"].double()
    dn = dy if c["first"] else dy * gate
    dhat = dn * w
    drow = (dhat - hat * ((dhat * hat).sum(-1, keepdim=True) / c["D"])) / dev
    if c["center"]:
        drow = drow - dhat.sum(-1, keepdim=True) / c["D"] / dev
    out = {"y": y, "dx": drow * gate if c["first"] else drow, "dz": (drow * x if c["first"] else dy * normed) * dgate}
    dw, db = (dn * hat).sum(0), dn.sum(0)
    out["dw"] = dw if c["each"] else dw.sum(0)
    if c["center"]:
        out["db"] = db if c["each"] else db.sum(0)
    return out


def _exact_gates(s, c, z):
    """(a, c, d c / d a, d a / d gate, d a / d rate) for raw gates z in 64 bits."""
    if c["form"] == "log":
        a, less = torch.exp(z), -torch.expm1(z)
        dgate, drate = a, None
    else:
        z = z + s["bias"].double()
        e, f = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))
        if c["form"] == "sigmoid":
            a, less, dgate, drate = e, f, e * f, None
        else:
            rate = s["rate"].double()
            a, less = torch.exp(-rate * e), -torch.expm1(-rate * e)
            dgate, drate = -a * rate * e * f, -a * e
    if c["scale"] == "none":
        return a, torch.ones_like(a), torch.zeros_like(a), dgate, drate
    if c["scale"] == "complement":
        return a, less, -torch.ones_like(a), dgate, drate
    k = torch.sqrt(less * (2 - less))
    return a, k, -a / k, dgate, drate


def _exact_glr(s, c):
    if c["mode"] == "step":
        pool, y = s["state"].double(), torch.zeros(c["B"], c["D"], device=s["x"].device, dtype=torch.float64)
        a, k, _, _, _ = _exact_gates(s, c, s["gate"].double())
        for row, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                pool[slot] = y[row] = a[row] * pool[slot] + k[row] * s["x"][row].double()
        return {"y": y, "state": pool}
    B, T, D = s["x"].shape
    dev, train = s["x"].device, c["mode"] == "train"
    x = s["x"].double()
    a, k, dk, dgate_, drate_ = _exact_gates(s, c, s["gate"].double())
    if not train:
        del dk, dgate_, drate_
    lens = _lengths(c["seqs"], T) if c["seqs"] else [T]
    first = [sum(lens[:i]) for i in range(len(lens))]
    starts = {at: i for i, (at, n) in enumerate(zip(first, lens)) if n}
    ends = {at + n - 1: i for i, (at, n) in enumerate(zip(first, lens)) if n}
    N = c["seqs"] or B
    # packed: a state per sequence; a batch: row b's state is that of sequence b
    init = torch.zeros(N, D, dtype=torch.float64, device=dev) if s["h0"] is None else s["h0"].double()
    pick = (lambda v, i: v[i:i + 1]) if c["seqs"] else (lambda v, i: v)
    hT, y = init.clone(), torch.empty(B, T, D, dtype=torch.float64, device=dev)
    prev = torch.empty_like(y) if train else None
    for t in range(T):
        if t in starts:
            h = pick(init, starts[t])
        if train:
            prev[:, t] = h
        h = a[:, t] * h + k[:, t] * x[:, t]
        y[:, t] = h
        if t in ends:
            if c["seqs"]:
                hT[ends[t]] = h[0]
            else:
                hT = h
    if not train:
        return {"y": y, "hT": hT}
    dy, dlast = s["dy"].double(), torch.zeros_like(init) if s["dhT"] is None else s["dhT"].double()
    dx, da = torch.empty_like(y), torch.empty_like(y)
    dh0 = dlast.clone()
    for t in reversed(range(T)):
        if t in ends:
            dh = pick(dlast, ends[t])
        dh = dh + dy[:, t]
        dx[:, t] = dh * k[:, t]
        da[:, t] = dh * (prev[:, t] + x[:, t] * dk[:, t])
        dh = dh * a[:, t]
        if t in starts:
            if c["seqs"]:
                dh0[starts[t]] = dh[0]
            else:
                dh0 = dh
    out = {"y": y, "hT": hT, "dx": dx, "dgate": da * dgate_}
    if s["bias"] is not None:
        out["dbias"] = out["dgate"].sum((0, 1))
    if s["rate"] is not None:
        out["drate"] = (da * drate_).sum((0, 1))
    if s["h0"] is not None:
        out["dh0"] = dh0
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"ln": _exact_ln, "gn": _exact_gn, "glr": _exact_glr}[case["op"]](s, s["case"])
